// Dropout with a mask made in place (include/dropout.h), forward and backward: one
// kernel, since the backward pass is the forward without a residual.
//
// Bound by memory: an element is read (with its residual) and written once; bfloat16
// 8192 x 11008 61 us, 5.9 TB/s, 4096 x 5632 float16 16 us.  The mask is next:
// 40 operations for 8 elements, of which the 20 products take four times an addition's
// time (with two operations for each three-way exclusive or, 64 to 68 us).
#include "row_ops.h"
#include "rows_plan.h"

namespace convfwd {

namespace {

template <typename E>
struct DropoutArgs {
  const E *x, *r;
  E* y;
  long long ldx, ldr, ldy;
  unsigned row0;      // of this launch
  unsigned runs_all;  // runs of 8 of this launch's rows
  int runs;           // of a row
  Magic mg;           // division by runs
  int n;
  DropArgs d;
};

// A workgroup takes 256 R runs in order, a thread R of them 256 apart: their loads are
// in flight together.  R = 1 but for large float32 matrices (rows_plan.cpp).
template <typename E, int R, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(const DropoutArgs<E> a) {
  const unsigned i0 = blockIdx.x * (256 * R) + threadIdx.x;
  Eight<E> x[R] = {}, r[R] = {};
  unsigned row[R], run[R];
  int left[R];  // elements to the end of the row, 0 where there is no run
  auto fetch = [](const E* p, int n, Eight<E>& q) {
    if (n >= 8) q = *reinterpret_cast<const Eight<E>*>(p);
    else if (n > 0) fetch_tail(p, n, q);
  };
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const unsigned i = i0 + 256 * k;
    row[k] = mdiv(i, a.mg);
    run[k] = i - row[k] * a.runs;
    left[k] = i < a.runs_all ? a.n - (int)run[k] * 8 : 0;
    fetch(a.x + row[k] * a.ldx + run[k] * 8, left[k], x[k]);
    if constexpr (RES) fetch(a.r + row[k] * a.ldr + run[k] * 8, left[k], r[k]);
  }
  const DropCounter c = drop_counter(a.d);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float v[8];
    unpack(x[k], v);
    drop8(a.d, c, run[k], a.row0 + row[k], left[k], v);
    if constexpr (RES) {
      float t[8];
      unpack(r[k], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    E* y = a.y + row[k] * a.ldy + run[k] * 8;
    if (left[k] >= 8) store8(y, 8, v);
    else if (left[k] > 0) store_tail(y, left[k], v);
  }
}

template <typename E>
int dropout(const DropGeo& g, const void* x, const void* r, void* y, const DropArgs& d,
            int64_t ldx, int64_t ldy, hipStream_t s) {
  const int64_t runs = ceil_div(g.n, 8);
  // row and run come from one 32-bit index
  const int64_t most = 0x7fff0000LL / runs;
  for (int64_t at = 0; at < g.m; at += most) {
    const int64_t rows = g.m - at < most ? g.m - at : most;
    DropoutArgs<E> a{};
    a.x = static_cast<const E*>(x) + at * ldx;
    a.r = r ? static_cast<const E*>(r) + at * g.ldr : nullptr;
    a.y = static_cast<E*>(y) + at * ldy;
    a.ldx = ldx; a.ldr = g.ldr; a.ldy = ldy;
    a.row0 = (unsigned)at;
    a.runs_all = (unsigned)(rows * runs);
    a.runs = (int)runs;
    a.mg = make_magic((unsigned)runs);
    a.n = (int)g.n;
    a.d = d;
    const dim3 grid((unsigned)ceil_div(rows * runs, 256 * g.runs)), block(256);
    if (g.runs == 2) {
      if (r) hipLaunchKernelGGL((dropout_kernel<E, 2, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((dropout_kernel<E, 2, false>), grid, block, 0, s, a);
    } else {
      if (r) hipLaunchKernelGGL((dropout_kernel<E, 1, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((dropout_kernel<E, 1, false>), grid, block, 0, s, a);
    }
    if (hipGetLastError() != hipSuccess) return CONV_ERR_DEVICE;
  }
  return CONV_OK;
}

template <typename E>
int run(const dropout_problem* p, const DropGeo& g, const void* x, const void* r, void* y,
        bool back, const void* step, void* stream) {
  const DropArgs d = drop_args(drop_threshold(p->drop), p->seed, p->offset, step);
  return dropout<E>(g, elements<E>(x, back ? p->y_off : p->x_off), elements<E>(r, p->r_off),
                    elements<E>(y, back ? p->x_off : p->y_off), d, back ? g.ldy : g.ldx,
                    back ? g.ldx : g.ldy, static_cast<hipStream_t>(stream));
}

int run_type(const dropout_problem* p, int dtype, const DropGeo& g, const void* x, const void* r,
             void* y, bool back, const void* step, void* stream) {
  if (dtype == CONV_F16) return run<_Float16>(p, g, x, r, y, back, step, stream);
  if (dtype == CONV_BF16) return run<__bf16>(p, g, x, r, y, back, step, stream);
  return run<float>(p, g, x, r, y, back, step, stream);
}

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" {

int dropout_forward(const dropout_problem* p, int dtype, const void* x, const void* r, void* y,
                    const void* step, void* stream) {
  DropGeo g;
  const int st = dropout_checked(p, dtype, x, r, y, step, &g);
  if (st) return st;
  return run_type(p, dtype, g, x, p->has_residual ? r : nullptr, y, false, step, stream);
}

int dropout_backward(const dropout_problem* p, int dtype, const void* dy, void* dx,
                     const void* step, void* stream) {
  DropGeo g;
  const int st = dropout_backward_checked(p, dtype, dy, dx, step, &g);
  if (st) return st;
  return run_type(p, dtype, g, dy, nullptr, dx, true, step, stream);
}

}  // extern "C"
