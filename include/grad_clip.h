/*
 * grad_clip.h — C ABI of the global gradient norm over many tensors and clipping
 * on MI355X (gfx950) (libconvfwd.so; status codes and element types of conv.h).
 *
 *   norm = (sum over all tensors and elements of |g|^p)^(1/p), p = 1 or 2, or the
 *          largest |g| (infinity norm);
 *   c    = min(1, max_norm / (norm + eps)), rounded to float32, NaN if the quotient
 *          is (the norm NaN, 0 / 0 or infinity / infinity);
 *   out  = c * g in float32, rounded to the tensor's type.
 *
 * The sums run in float64 over exact squares (the square of a float32 has at most
 * 48 significant bits and its exponent fits), in an order that depends on the
 * lengths and types alone: no atomics, reruns are bit-identical.  An infinite element gives
 * an infinite norm and c = 0, so finite elements become 0 and infinite ones NaN;
 * a NaN makes the norm and every element NaN (for every p).
 *
 * Ownership, errors and threading as in conv.h: grad_clip only enqueues on the
 * stream, never allocates or synchronises.  The table of tensors is host memory,
 * read during the call only (its contents travel as kernel arguments).
 */
#ifndef CONVFWD_GRAD_CLIP_H
#define CONVFWD_GRAD_CLIP_H

#include <stdint.h>

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GRAD_NORM_1 = 1, GRAD_NORM_2 = 2, GRAD_NORM_INF = 3 } grad_norm_kind;

/* One gradient: elems contiguous elements of the given type.  out may equal g
 * exactly (clipping in place); NULL with every other out NULL too asks for the
 * norm alone.  Different tensors must not overlap (not checked). */
typedef struct grad_tensor {
    const void* g;
    void* out;
    int64_t elems;      /* >= 0 */
    int32_t dtype;      /* conv_dtype, may differ from tensor to tensor */
    int32_t reserved;   /* 0 */
} grad_tensor;

typedef struct grad_clip_problem {
    const grad_tensor* tensors;   /* host array */
    int64_t count;                /* 0 .. 65536 */
    int32_t kind;                 /* grad_norm_kind */
    float max_norm;               /* >= 0 */
    float eps;                    /* >= 0, usually 1e-6 */
    int32_t reserved;             /* 0 */
} grad_clip_problem;

/* Scratch in bytes; a function of the tensors' lengths alone. */
int grad_clip_scratch_size(const grad_clip_problem* p, uint64_t* bytes);

/* The status grad_clip would return before enqueueing (host only). */
int grad_clip_check(const grad_clip_problem* p, const void* norm, const void* scratch,
                    uint64_t scratch_bytes);

/* Enqueue the norm (norm: one float32 on the device, the norm before clipping)
 * and the clipping.  scratch must be 256-byte aligned.  Errors: CONV_ERR_ARG (null
 * pointer, bad enum, negative or NaN max_norm or eps, some out NULL and some not,
 * a tensor or scratch misaligned to its elements), CONV_ERR_SHAPE (count or a
 * length out of range), CONV_ERR_OVERLAP (an out that partly overlaps its g, or
 * scratch or norm overlapping a tensor), CONV_ERR_SCRATCH before anything is
 * enqueued; CONV_ERR_DEVICE if the runtime refuses a launch. */
int grad_clip(const grad_clip_problem* p, float* norm, void* scratch, uint64_t scratch_bytes,
              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_GRAD_CLIP_H */
