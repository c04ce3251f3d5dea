/*
 * layer_norm.h — C ABI of the layer norm over the rows of a matrix on MI355X
 * (gfx950), forward and backward, with the dropout and the residual addition that
 * go before it in a training step (libconvfwd.so; status codes and element types of
 * conv.h, the mask of dropout.h).
 *
 *   forward    s = r + drop(x)                        (drop and r are optional)
 *              mean = sum(s) / n,  rstd = 1 / sqrt(sum((s - mean)^2) / n + eps)
 *              y = (s - mean) * rstd * w + b          (w and b are optional)
 *   backward   u = (s - mean) * rstd,  g = dy * w
 *              d = rstd * (g - sum(g) / n - u * sum(g u) / n) [+ ds]
 *              dr = d,  dx = drop'(d)  (d scaled where x was kept, 0 elsewhere)
 *              dw = sum over rows of dy * u,  db = sum over rows of dy
 *
 * Without a dropout and a residual s is x, and dx is d.
 *
 * Layouts (row-major; rows ld elements apart, ld = 0 meaning dense):
 *   x, r, y, s, dy, ds, dx, dr  [m, n];  w, b, dw, db [n]: one element type for all
 *   mean, rstd [m] float32, dense
 * Everything between loads and stores is float32: s is not rounded before it is
 * normalised, the variance is the mean of squared distances from the mean (never a
 * difference of squares), and every output is rounded once.  The backward pass
 * reads s as the forward stored it.  A row with an infinity or a NaN is NaN; a row of
 * equal values is b up to the rounding of its mean (times 1 / sqrt(eps); NaN with
 * eps = 0 and a mean without rounding).  The sums have float32's range: a row whose
 * sum passes it is NaN, one whose sum of squared distances does (all of them 2^64 /
 * sqrt(n), say) has rstd 0 and is b.
 *
 * Any m >= 0 is valid: with m = 0 the forward writes nothing, the backward writes
 * zeros to dw and db, and operands of m rows may be NULL.  n and the row strides
 * are at most 2^20, m at most 2^31-1; operands may pass 2^31 elements.
 *
 * Ownership, errors and threading as in linear.h: device buffers are the caller's;
 * the calls only enqueue on the stream, never allocate or synchronise; every check
 * runs on the host before anything is enqueued; calls are reentrant, each with a
 * scratch of its own.  No atomics, sums in an order that depends on the problem
 * alone: reruns are bit-identical.
 */
#ifndef CONVFWD_LAYER_NORM_H
#define CONVFWD_LAYER_NORM_H

#include <stdint.h>

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row strides are in elements, 0 = dense.  Element offsets are added to the
 * pointers of the same name (arena-style placement). */
typedef struct layer_norm_problem {
    int64_t m, n;
    int64_t ldx, ldr, ldy, lds;           /* forward operands; ldy is dy's stride too */
    int64_t ldds, lddx, lddr;             /* gradients */
    int64_t x_off, r_off, w_off, b_off, y_off, s_off;
    int64_t dy_off, ds_off, dx_off, dr_off, dw_off, db_off;
    uint64_t seed, offset;                /* the mask's (dropout.h) */
    float eps;                            /* >= 0, usually 1e-5 */
    float drop;                           /* probability of a zero, 0 .. 1; 0 = no dropout */
    int32_t has_weight, has_bias, has_residual;  /* 0/1 */
    int32_t reserved;                     /* 0 */
} layer_norm_problem;

/* Scratch in bytes (0 = none needed).  Shape-only: never queries the HIP runtime,
 * the same on every device.  A call's scratch must be 256-byte aligned. */
int layer_norm_scratch_size(const layer_norm_problem* p, int dtype, uint64_t* bytes);
int layer_norm_backward_scratch_size(const layer_norm_problem* p, int dtype, uint64_t* bytes);

/* Name of the kernel plan, e.g. "layer_norm.bf16.rows256x2" (rows held by 256 threads,
 * up to 2 runs of 8 elements each), "layer_norm.f32.split13" (rows cut into 13 parts),
 * "layer_norm_backward.f16.rows64x2.once" (dw and db beside the rows, in one pass).
 * CONV_ERR_ARG when len is too small, or the validation status of the problem. */
int layer_norm_describe_variant(const layer_norm_problem* p, int dtype, char* buf, uint64_t len);
int layer_norm_backward_describe_variant(const layer_norm_problem* p, int dtype, char* buf,
                                         uint64_t len);

/* Pre-flight: the status the call of the same arguments would return before it
 * enqueues anything.  Pointers are compared, never read. */
int layer_norm_check(const layer_norm_problem* p, int dtype, const void* x, const void* r,
                     const void* w, const void* b, const void* y, const void* s, const void* mean,
                     const void* rstd, const void* step, const void* scratch,
                     uint64_t scratch_bytes);
int layer_norm_backward_check(const layer_norm_problem* p, int dtype, const void* s, const void* w,
                              const void* mean, const void* rstd, const void* dy, const void* ds,
                              const void* dx, const void* dr, const void* dw, const void* db,
                              const void* step, const void* scratch, uint64_t scratch_bytes);

/* Forward.  x and y are required; r, w, b where the problem says so (others are not
 * read).  s, and mean with rstd, are written where not NULL: what the backward pass
 * reads.  step: dropout.h.  y and s may each equal x or r exactly; every other overlap
 * of an output is CONV_ERR_OVERLAP.  Errors: CONV_ERR_ARG (null required pointer,
 * mean without rstd, bad flag or probability, operands off their elements, misaligned
 * scratch), CONV_ERR_SHAPE (m < 0, n < 1, a stride below its row, a size beyond the
 * limits above), CONV_ERR_OVERLAP, CONV_ERR_SCRATCH before anything is enqueued;
 * CONV_ERR_DEVICE if the runtime refuses a launch. */
int layer_norm_forward(const layer_norm_problem* p, int dtype, const void* x, const void* r,
                       const void* w, const void* b, void* y, void* s, void* mean, void* rstd,
                       const void* step, void* scratch, uint64_t scratch_bytes, void* stream);

/* Backward.  s is what the forward stored, or x where the problem has neither a
 * dropout nor a residual.  ds (optional): the gradient that reaches s by other ways.
 * Each of dx, dr, dw, db is computed if not NULL (one at least; dr, dw and db only for
 * a problem with a residual, a weight, a bias).  With the same seed, offset and step
 * as the forward the mask is the same.  dx and dr may each equal dy or ds exactly. */
int layer_norm_backward(const layer_norm_problem* p, int dtype, const void* s, const void* w,
                        const void* mean, const void* rstd, const void* dy, const void* ds,
                        void* dx, void* dr, void* dw, void* db, const void* step, void* scratch,
                        uint64_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_LAYER_NORM_H */
