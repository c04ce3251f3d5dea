// Tiled products of 8-bit operands, and the launch half of linear_int8_forward
// (include/linear_int8.h): the kernels of the linear layer with int32 sums, an output
// type of their own and the scales in the epilogue.
//
// 8192 x 11008 x 4096 to bfloat16 in 256 x 256 tiles: 314 us with relu, 335 with gelu_tanh
// (2.2 to 2.35 POP/s; the library's product alone, int32 out, 354).  A step of 128 k takes
// 1.46 us at the clock that the card's power allows; a round of tiles 9.4 us more, of
// which writing 33 MB of outputs at one time is 7, and gelu_tanh 20 us of a call.  Few
// rows are the weights' way from memory: one row by 32000 x 4096 25 us (5.2 TB/s), 16 rows
// by 2048 x 5632 7.5.  Rows at odd bytes go through registers in 64 x 64 tiles, 16 misaligned
// bytes a load: 777 x 1001 x 1531 12.6 us (aligned words joined instead: 17; two steps
// ahead in place of one: 12.0).
#include <algorithm>

#include "linear_int8_plan.h"
#include "linear_launch.h"
#include "linear_launch_tile.h"

namespace convfwd {

namespace {

template <typename O>
hipError_t run(const linear_int8_problem* p, const Int8Geo& g, const LinearPlan& pl, const void* x,
               const void* xs, const void* w, const void* ws, const void* b, const void* r, void* y,
               void* scratch, hipStream_t s) {
  const void* src[2] = {at(x, p->x_off, 1), at(w, p->w_off, 1)};
  int64_t ld[2] = {g.ldx, g.ldw};
  PackArgs pack{};
  if (fill_pack(pl.pack, 1, src, ld, scratch, &pack)) {
    const hipError_t e = launch_pack<signed char>(pack, s);
    if (e != hipSuccess) return e;
  }
  ProductArgs a{};
  a.P[0] = src[1];
  a.Q[0] = src[0];
  a.ldp = ld[1]; a.ldq = ld[0];
  LinEpilogue& e = a.e;
  e.xs = static_cast<const float*>(xs) + p->xs_off;
  e.ws = static_cast<const float*>(ws) + p->ws_off;
  e.bias[0] = p->has_bias ? at(b, p->b_off, g.es) : nullptr;
  e.res = p->has_residual ? at(r, p->r_off, g.es) : nullptr;
  e.res_mode = p->has_residual;
  e.out[0] = at(y, p->y_off, g.es);
  e.ldo = g.ldy; e.ldres = g.ldr;
  e.act = p->activation; e.alpha = p->act_alpha; e.beta = p->act_beta;
  const ProductShape& shape = pl.product;
  const ProductPlan& plan = pl.run;
  set_plan(shape, plan, scratch, &a);
  const bool dma = direct(shape, a, 1, pl.pack.on, pl.pack.on);
  if (plan.tile == TILE_STREAM) return launch_int8_stream<O>(a, plan.stream_t, plan.stream_rows, dma, s);
  const int64_t rows = launch_rows(shape, plan.splits);
  hipError_t st = hipSuccess;
  for (int64_t c = 0; c < shape.C && st == hipSuccess; c += rows) {
    ProductArgs q = a;  // rows c .. c + rows alone
    q.C = (int)std::min(rows, shape.C - c);
    q.Q[0] = at(a.Q[0], c * a.ldq, 1);
    q.e.xs = e.xs + c;
    q.e.out[0] = at(e.out[0], c * e.ldo, g.es);
    q.e.res = at(e.res, c * e.ldres, g.es);
    st = launch_int8_product<O>(q, plan.tile, dma, s);
  }
  if (st != hipSuccess || plan.splits == 1) return st;
  return launch_int8_join<O>(join_of(shape, a), s);
}

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" int linear_int8_forward(const linear_int8_problem* p, int dtype, const void* x,
                                   const void* xs, const void* w, const void* ws, const void* b,
                                   const void* r, void* y, void* scratch, uint64_t scratch_bytes,
                                   void* stream) {
  Int8Geo g;
  LinearPlan pl;
  const int st = linear_int8_checked(p, dtype, x, xs, w, ws, b, r, y, scratch, scratch_bytes, &g, &pl);
  if (st || g.m == 0) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (dtype == CONV_F16) e = run<_Float16>(p, g, pl, x, xs, w, ws, b, r, y, scratch, s);
  else if (dtype == CONV_BF16) e = run<__bf16>(p, g, pl, x, xs, w, ws, b, r, y, scratch, s);
  else e = run<float>(p, g, pl, x, xs, w, ws, b, r, y, scratch, s);
  return e == hipSuccess ? CONV_OK : CONV_ERR_DEVICE;
}
