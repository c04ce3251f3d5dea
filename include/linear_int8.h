/*
 * linear_int8.h — C ABI of the linear layer in 8-bit integers with a scale for
 * each token and each channel, and of the quantization of rows that feeds it, on
 * MI355X (gfx950) (libconvfwd.so; status codes and element types of conv.h,
 * activations and residuals of linear.h).
 *
 *   quantize_rows  a = max |x| of the row,  scale = fl(a / 127),
 *                  q = x * fl(127 / a) rounded to float32, then to the nearest whole
 *                  number (to even at a half): -127 .. 127
 *   linear_int8    z = fl( fl( (sum_k x w) * (xs * ws) + b ) + r )  residual before the
 *                  activation, y = act(z); or z without r, y = fl( act(z) + r )
 *
 * A row whose largest |x| is below 2^-100 has scale 0 and q 0 (fl(127 / a) may not be
 * finite there); a row with an infinity or a NaN has scale NaN and q 0, so that z of
 * that row is NaN, and y with it but for relu: as in linear.h, relu(NaN) is 0, so such a
 * token comes out as zeros (or as r, with the residual after), and only its scale tells.
 * The sum over k is exact (int32), rounded once to float32; the product of the two scales,
 * the product with the sum and every step after it are float32, and y is rounded once to
 * its type.
 *
 * Layouts (row-major; rows ld elements apart, ld = 0 meaning dense):
 *   quantize_rows  x [m, n] of the call's element type, q [m, n] int8, scale [m] float32
 *   linear_int8    x [m, k], w [n, k] int8;  xs [m], ws [n] float32, dense;
 *                  b [n], r, y [m, n] of the call's element type
 * Any int8 value is valid, -128 too.  k is at most 131071, so that every sum fits
 * int32; n and the strides at most 2^20, m 2^31-1.  m = 0 writes nothing (and scales
 * nothing), and operands of m rows may then be NULL.
 *
 * Ownership, errors and threading as in linear.h.  Integer sums: the results depend on
 * the arguments alone, whatever the plan.
 */
#ifndef CONVFWD_LINEAR_INT8_H
#define CONVFWD_LINEAR_INT8_H

#include <stdint.h>

#include "conv.h"
#include "linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strides and offsets in elements of each operand's own type, stride 0 = dense. */
typedef struct quantize_problem {
    int64_t m, n;
    int64_t ldx, ldq;
    int64_t x_off, q_off, scale_off;
    int32_t reserved;                     /* 0 */
} quantize_problem;

typedef struct linear_int8_problem {
    int64_t m, n, k;
    int64_t ldx, ldw, ldr, ldy;
    int64_t x_off, xs_off, w_off, ws_off, b_off, r_off, y_off;
    int32_t activation;                   /* conv_activation or LINEAR_ACT_* */
    float act_alpha, act_beta;            /* as in conv_problem */
    int32_t has_bias, has_residual;       /* 0/1; LINEAR_RES_* */
    int32_t reserved;                     /* 0 */
} linear_int8_problem;

/* The status quantize_rows would return before enqueueing (host only). */
int quantize_check(const quantize_problem* p, int dtype, const void* x, const void* q,
                   const void* scale);

/* Rows of x (dtype: CONV_F32, CONV_F16, CONV_BF16) to 8 bits.  Errors: CONV_ERR_ARG (null
 * pointer, bad enum, operands off their elements), CONV_ERR_SHAPE (m < 0, n < 1, a
 * stride below its row, a size beyond the limits above), CONV_ERR_OVERLAP (any operands
 * overlap) before anything is enqueued; CONV_ERR_DEVICE if the runtime refuses a launch. */
int quantize_rows(const quantize_problem* p, int dtype, const void* x, void* q, void* scale,
                  void* stream);

/* Scratch in bytes (0 = none needed); shape-only.  256-byte aligned. */
int linear_int8_scratch_size(const linear_int8_problem* p, int dtype, uint64_t* bytes);

/* Name of the kernel plan, e.g. "linear_int8.bf16.tile256x256" (the type is that of
 * b, r and y), as in linear.h; ".cut": the tiles of the last round are cut in two. */
int linear_int8_describe_variant(const linear_int8_problem* p, int dtype, char* buf, uint64_t len);

/* The status linear_int8_forward would return before enqueueing (host only). */
int linear_int8_check(const linear_int8_problem* p, int dtype, const void* x, const void* xs,
                      const void* w, const void* ws, const void* b, const void* r, const void* y,
                      const void* scratch, uint64_t scratch_bytes);

/* dtype: of b, r and y.  x, xs, w, ws and y are required; b and r are read when
 * has_bias / has_residual say so.  y may equal r exactly; every other overlap of y or
 * the scratch is CONV_ERR_OVERLAP.  Errors as in linear_forward. */
int linear_int8_forward(const linear_int8_problem* p, int dtype, const void* x, const void* xs,
                        const void* w, const void* ws, const void* b, const void* r, void* y,
                        void* scratch, uint64_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_LINEAR_INT8_H */
