/*
 * linear.h — C ABI of the linear layer and the gated feed-forward projection on
 * MI355X (gfx950), forward and backward (libconvfwd.so, beside the convolution
 * of conv.h, whose status codes, element types and activations it shares): what
 * follows the last pool of a convolutional network, and its gradients.
 *
 * Operations (row = one token, or one pooled image):
 *
 *   linear          z = fl( fl( x W^T + b ) + r )      residual before the activation
 *                   y = act(z)                         (the convolution epilogue's order), or
 *                   z = fl( x W^T + b ),  y = fl( act(z) + r )   residual after it
 *   linear_backward dz = dy * act'(z)
 *                   dx = dz W,  dw = dz^T x,  db = sum over rows of dz,
 *                   dr = dz (residual before) or dy (after)
 *   gated           pg = fl( x Wg^T + bg ),  pu = fl( x Wu^T + bu ),  h = act(pg) * pu
 *   gated_backward  dg = dh * pu * act'(pg),  du = dh * act(pg)
 *                   dx = dg Wg + du Wu,  dwg = dg^T x,  dwu = du^T x,
 *                   dbg, dbu = sums over rows of dg and du
 *
 * Layouts (row-major; rows ld elements apart, ld = 0 meaning dense):
 *   x, dx     [m, k]
 *   w, dw     [n, k], or [k, n] with w_layout = LINEAR_W_KN (ONNX MatMul's order)
 *   y, z, r, dy, dr  [m, n];  b, db [n]
 *   gated: wg, wu, dwg, dwu [f, k];  h, dh, pg, pu [m, f];  bg, bu, dbg, dbu [f]
 * Element types CONV_F32, CONV_F16, CONV_BF16, one for every operand of a call.
 * Products of 16-bit operands are exact in float32 and every sum is held in
 * float32; z, pg and pu are rounded only where they are stored.  Activations and
 * their slopes are evaluated to within 16 float32 ulps of argument and value (below
 * 2^-119 in size they may come out as 0).  The backward
 * passes round dz, dg and du once to the element type (they are operands of
 * matrix products) unless the type is float32; db, dbg and dbu sum the
 * unrounded values.
 *
 * Any m >= 0 is valid: with m = 0 the forward calls write nothing, the backward
 * calls write zero weight and bias gradients, and operands of m rows may be NULL.  m, n, f, k and the row
 * strides are at most 2^20 for the contiguous extents (n, f, k and strides) and
 * 2^31-1 for m; operands may pass 2^31 elements.
 *
 * Ownership, errors and threading as in conv.h: device buffers are the caller's;
 * the calls only enqueue on the stream, never allocate or synchronise; every
 * check runs on the host before anything is enqueued; calls are reentrant.  A
 * call that needs scratch may run beside others if each has its own.  Results
 * do not depend on anything but the arguments: no atomics, sums in a fixed
 * order, so reruns are bit-identical.
 */
#ifndef CONVFWD_LINEAR_H
#define CONVFWD_LINEAR_H

#include <stdint.h>

#include "conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations beyond conv_activation's, accepted by the calls of this header:
 * gelu v * Phi(v) with the normal distribution function (erf form), and its
 * tanh approximation v/2 * (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))).
 * Derivatives at corners are the flat side's (relu at 0, the ends of clip,
 * hard_sigmoid and hard_swish); leaky_relu's at 0 is 1.  A NaN sum stays NaN, but
 * for relu, whose comparison fails and gives 0; the slopes that are picked by
 * comparisons are at NaN 0 (relu, clip, hard_sigmoid) and act_alpha (leaky_relu). */
enum { LINEAR_ACT_GELU = 9, LINEAR_ACT_GELU_TANH = 10 };

enum { LINEAR_W_NK = 0, LINEAR_W_KN = 1 };
enum { LINEAR_RES_NONE = 0, LINEAR_RES_BEFORE = 1, LINEAR_RES_AFTER = 2 };

/* Row strides are in elements, 0 = dense.  Element offsets are added to the
 * pointers of the same name (arena-style placement). */
typedef struct linear_problem {
    int64_t m, n, k;
    int64_t ldx, ldw, ldr, ldy, ldz;      /* forward operands; ldy is dy's stride too */
    int64_t lddx, lddw, lddr;             /* gradients */
    int64_t x_off, w_off, b_off, r_off, y_off, z_off;
    int64_t dy_off, dx_off, dw_off, db_off, dr_off;
    int32_t activation;                   /* conv_activation or LINEAR_ACT_* */
    float act_alpha, act_beta;            /* as in conv_problem */
    int32_t has_bias, has_residual;       /* 0/1; LINEAR_RES_* */
    int32_t save_z;                       /* forward: 1 = also store z */
    int32_t w_layout;                     /* LINEAR_W_* */
    int32_t reserved;                     /* 0 */
} linear_problem;

typedef struct gated_problem {
    int64_t m, f, k;
    int64_t ldx, ldw, ldh, ldp;           /* ldw: wg and wu; ldh: h and dh; ldp: pg and pu */
    int64_t lddx, lddw;                   /* lddw: dwg and dwu */
    int64_t x_off, wg_off, wu_off, bg_off, bu_off, h_off, pg_off, pu_off;
    int64_t dh_off, dx_off, dwg_off, dwu_off, dbg_off, dbu_off;
    int32_t activation;
    float act_alpha, act_beta;
    int32_t has_bias;
    int32_t save_p;                       /* forward: 1 = also store pg and pu */
    int32_t reserved;                     /* 0 */
} gated_problem;

/* Scratch in bytes (0 = none needed).  Shape-only: never queries the HIP
 * runtime, the same on every device.  A call's scratch must be 256-byte aligned. */
int linear_scratch_size(const linear_problem* p, int dtype, uint64_t* bytes);
int linear_backward_scratch_size(const linear_problem* p, int dtype, uint64_t* bytes);
int gated_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes);
int gated_backward_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes);

/* Name of the kernel plan, e.g. "linear.bf16.tile256x256" or
 * "gated.f16.stream16.r8" (streamed, for up to 16 rows, 8 weight rows a workgroup);
 * for the backward calls, of both products, in one launch or in two:
 * "linear_backward.bf16.both.tile256x128",
 * "linear_backward.f32.dx.tile64x64.split4.dw.tile64x64.split4.both",
 * "linear_backward.f32.dx.tile128x128.split2.dw.tile64x64".  CONV_ERR_ARG when
 * len is too small, or the validation status of the problem. */
int linear_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len);
int linear_backward_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len);
int gated_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len);
int gated_backward_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len);

/* Pre-flight: the status the call of the same arguments would return before it
 * enqueues anything.  Pointers are compared, never read. */
int linear_check(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                 const void* r, const void* y, const void* z, const void* scratch,
                 uint64_t scratch_bytes);
int linear_backward_check(const linear_problem* p, int dtype, const void* x, const void* w,
                          const void* z, const void* dy, const void* dx, const void* dw,
                          const void* db, const void* dr, const void* scratch,
                          uint64_t scratch_bytes);
int gated_check(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                const void* bg, const void* bu, const void* h, const void* pg, const void* pu,
                const void* scratch, uint64_t scratch_bytes);
int gated_backward_check(const gated_problem* p, int dtype, const void* x, const void* wg,
                         const void* wu, const void* pg, const void* pu, const void* dh,
                         const void* dx, const void* dwg, const void* dwu, const void* dbg,
                         const void* dbu, const void* scratch, uint64_t scratch_bytes);

/* Linear forward.  x, w, y are required; b and r are read when has_bias /
 * has_residual say so, z is written when save_z is set (then they are required).
 * y may alias r exactly; every other overlap of an output is CONV_ERR_OVERLAP.
 * Errors: CONV_ERR_ARG (null required pointer, bad enum, misaligned scratch),
 * CONV_ERR_SHAPE (n or k < 1, m < 0, a stride below its row, a size beyond the
 * limits above), CONV_ERR_OVERLAP, CONV_ERR_SCRATCH before anything is enqueued;
 * CONV_ERR_DEVICE if the runtime refuses a launch. */
int linear_forward(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                   const void* r, void* y, void* z, void* scratch, uint64_t scratch_bytes,
                   void* stream);

/* Linear backward.  Each of dx, dw, db, dr is computed if it is not NULL (one at
 * least; dr only for a problem with a residual).  x is required for dw, w for
 * dx, z (as the forward stored it) where the activation is not the identity and
 * dx, dw, db or a dr = dz is wanted.  dr may alias dy exactly. */
int linear_backward(const linear_problem* p, int dtype, const void* x, const void* w, const void* z,
                    const void* dy, void* dx, void* dw, void* db, void* dr, void* scratch,
                    uint64_t scratch_bytes, void* stream);

/* Gated forward: both projections, the activation and the product in one pass
 * over x.  pg and pu are written when save_p is set; they may be the two halves
 * of the rows of one [m, 2f] buffer. */
int gated_forward(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                  const void* bg, const void* bu, void* h, void* pg, void* pu, void* scratch,
                  uint64_t scratch_bytes, void* stream);

/* Gated backward from the stored pg and pu.  dx, dwg and dwu, dbg and dbu are
 * computed if not NULL (the weight gradients in pairs, and the bias gradients). */
int gated_backward(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                   const void* pg, const void* pu, const void* dh, void* dx, void* dwg, void* dwu,
                   void* dbg, void* dbu, void* scratch, uint64_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVFWD_LINEAR_H */
