/*
 * dropout.h — C ABI of dropout with a mask that is never stored, forward and
 * backward, on MI355X (gfx950) (libconvfwd.so; status codes and element types of
 * conv.h).
 *
 *   forward    y = drop(x) [+ r],   drop(x) = scale * x where x is kept, 0 elsewhere
 *   backward   dx = scale * dy where x was kept, 0 elsewhere  (the residual's is dy)
 *
 * The mask is a function of an element's place and the call's numbers alone, so
 * the backward pass makes it again.  Element (row, col) takes 16 bits u of the
 * counter-based generator Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
 * random numbers: as easy as 1, 2, 3", 2011):
 *
 *   key      the two 32-bit halves of seed, low half first
 *   counter  (col / 8, row, low half, high half of offset + *step), modulo 2^64
 *   u        of the four words w, bits 16 (col % 2) .. 16 (col % 2) + 15 of w[col % 8 / 2]
 *
 * and is kept where u >= t, t = drop * 2^16 rounded to the nearest whole number (to
 * even at a half).  So probabilities are multiples of 2^-16 (below 2^-17 nothing is
 * dropped), and scale = 2^16 / (2^16 - t), rounded to float32: the mean of drop(x) over
 * masks is x.  A dropped element is 0 whatever x holds; with drop = 1 all are.
 * Strides, pointers and the element type do not enter, so a row's mask is the same
 * in a wider buffer, and layer_norm.h's calls make the same one.
 *
 * step: optional device pointer to one uint64_t that is added to offset when the
 * call runs (NULL: 0).  A captured call draws a new mask on every replay if the
 * graph, or the program between replays, moves the number on; the backward pass
 * has to see the number that the forward saw.
 *
 * Layouts (row-major; rows ld elements apart, ld = 0 meaning dense): x, r, y, dy, dx
 * [m, n], one element type; float32 between loads and stores, one rounding.
 * n and the strides are at most 2^20, m at most 2^31-1; m = 0 writes nothing.
 * Ownership, errors and threading as in linear.h; no scratch.
 */
#ifndef CONVFWD_DROPOUT_H
#define CONVFWD_DROPOUT_H

#include <stdint.h>

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dropout_problem {
    int64_t m, n;
    int64_t ldx, ldr, ldy;                /* ldx is dx's stride too, ldy dy's */
    int64_t x_off, r_off, y_off;          /* element offsets; x_off is dx's too, y_off dy's */
    uint64_t seed, offset;
    float drop;                           /* probability of a zero, 0 .. 1 */
    int32_t has_residual;                 /* 0/1 */
    int32_t reserved;                     /* 0 */
} dropout_problem;

/* Name of the kernel plan ("dropout.f32.runs2": 2 runs of 8 elements a thread).
 * Shape-only. */
int dropout_describe_variant(const dropout_problem* p, int dtype, char* buf, uint64_t len);

/* Pre-flight: the status the call of the same arguments would return before it
 * enqueues anything.  Pointers are compared, never read. */
int dropout_check(const dropout_problem* p, int dtype, const void* x, const void* r, const void* y,
                  const void* step);
int dropout_backward_check(const dropout_problem* p, int dtype, const void* dy, const void* dx,
                           const void* step);

/* Forward.  x and y are required (r where has_residual); y may equal x or r
 * exactly, every other overlap is CONV_ERR_OVERLAP.  Errors: CONV_ERR_ARG (null
 * pointer, bad flag or probability, operands off their elements, step off 8 bytes),
 * CONV_ERR_SHAPE, CONV_ERR_OVERLAP before anything is enqueued; CONV_ERR_DEVICE if the
 * runtime refuses a launch. */
int dropout_forward(const dropout_problem* p, int dtype, const void* x, const void* r, void* y,
                    const void* step, void* stream);

/* Backward.  dx may equal dy exactly. */
int dropout_backward(const dropout_problem* p, int dtype, const void* dy, void* dx,
                     const void* step, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_DROPOUT_H */
