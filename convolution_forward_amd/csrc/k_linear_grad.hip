// Elementwise half of the backward passes (include/linear.h):
//   linear  dz = dy act'(z)
//   gated   dg = dh pu act'(pg),  du = dh act(pg)   (side by side in one buffer)
// and the column sums that are the bias gradients, in one pass over the operands.
// Bound by memory: dy, z (dh, pg, pu) are read once, dz written once.  The buffer
// holds the element type (it is an operand of the two matrix products after it)
// and its rows are padded with zeros to whole 8-element runs; the column sums take
// the unrounded float32 values: each thread 8 columns of every 8th row of a chunk,
// the 8 row groups joined in order through LDS, one float32 row per chunk, and the
// chunks joined in order by a second kernel.
#include "linear_epilogue.h"

namespace convfwd {

namespace {

template <typename E, bool GATED>
__global__ __launch_bounds__(256) void linear_dz_kernel(const DzArgs a) {
  constexpr int KINDS = GATED ? 2 : 1;
  __shared__ float red[8][KINDS][256];
  const int tid = threadIdx.x, cl = tid & 31, rg = tid >> 5;
  const int col = (blockIdx.x * 32 + cl) * 8;
  const int nv = min(8, a.n - col);
  const long long m0 = (long long)blockIdx.y * a.rows, m1 = min(a.m, m0 + a.rows);
  float sum[KINDS][8];
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[d][i] = 0.0f;
  if (nv > 0) {
    for (long long m = m0 + rg; m < m1; m += 8) {
      float dy[8], z[8], t[8];
      load8(static_cast<const E*>(a.dy) + m * a.ldy + col, nv, a.vec, dy);
      if constexpr (GATED) {
        float pu[8];
        load8(static_cast<const E*>(a.z[0]) + m * a.ldz + col, nv, a.vec, z);
        load8(static_cast<const E*>(a.z[1]) + m * a.ldz + col, nv, a.vec, pu);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, d;
          act_and_slope(z[i], a.act, a.alpha, a.beta, &f, &d);
          t[i] = i < nv ? dy[i] * f : 0.0f;           // du
          z[i] = i < nv ? dy[i] * pu[i] * d : 0.0f;   // dg
          sum[0][i] += z[i];
          sum[KINDS - 1][i] += t[i];
        }
        E* o = static_cast<E*>(a.dz) + m * a.lddz + col;
        store8(o, 8, true, z);
        store8(o + a.np, 8, true, t);
      } else {
        if (a.act != 0) {
          load8(static_cast<const E*>(a.z[0]) + m * a.ldz + col, nv, a.vec, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float f, d;
            act_and_slope(z[i], a.act, a.alpha, a.beta, &f, &d);
            t[i] = i < nv ? dy[i] * d : 0.0f;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = dy[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0][i] += t[i];
        if (a.dz) store8(static_cast<E*>(a.dz) + m * a.lddz + col, 8, true, t);
        if (a.dr)
          store8(static_cast<E*>(a.dr) + m * a.lddr + col, nv, a.vec, a.dr_is_dy ? dy : t);
      }
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[rg][d][cl * 8 + i] = sum[d][i];
  __syncthreads();
  const int c = blockIdx.x * 256 + tid;
  if (c < a.np) {
#pragma unroll
    for (int d = 0; d < KINDS; ++d) {
      float s = red[0][d][tid];
#pragma unroll
      for (int g = 1; g < 8; ++g) s += red[g][d][tid];
      a.sums[((long long)blockIdx.y * KINDS + d) * a.np + c] = s;
    }
  }
}

template <typename E>
__global__ __launch_bounds__(64) void linear_sums_kernel(const SumsArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x, d = blockIdx.y;
  if (c >= a.n) return;
  const float* p = a.sums + (long long)d * a.np + c;
  const long long step = (long long)a.parts * a.np;
  float s = 0.0f;
  for (int i = 0; i < a.chunks; ++i) s += p[i * step];
  static_cast<E*>(a.db[d])[c] = (E)s;
}

}  // namespace

template <typename E>
hipError_t launch_dz(const DzArgs& a, bool gated, int chunks, hipStream_t s) {
  const dim3 grid((a.np + 255) / 256, chunks);
  if (gated) hipLaunchKernelGGL((linear_dz_kernel<E, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear_dz_kernel<E, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sums(const SumsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_sums_kernel<E>), dim3((a.n + 63) / 64, a.parts), dim3(64), 0, s, a);
  return hipGetLastError();
}

#define CONVFWD_INST(E)                                                          \
  template hipError_t launch_dz<E>(const DzArgs&, bool, int, hipStream_t);      \
  template hipError_t launch_sums<E>(const SumsArgs&, hipStream_t);
CONVFWD_INST(_Float16)
CONVFWD_INST(__bf16)
CONVFWD_INST(float)
#undef CONVFWD_INST

}  // namespace convfwd
