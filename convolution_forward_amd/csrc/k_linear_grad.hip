// Elementwise half of the backward passes (include/linear.h):
//   linear  dz = dy act'(z)
//   gated   dg = dh pu act'(pg),  du = dh act(pg)   (side by side in one buffer)
// and the column sums that are the bias gradients, in one pass over the operands.
// Bound by memory: dy, z (dh, pg, pu) are read once, dz written once: 4096 x 4096 bf16
// with GELU in 22 us (4.5 TB/s), gated 4096 x 5632 in 53 (4.3 TB/s).  The buffer
// holds the element type (it is an operand of the two matrix products after it)
// and its rows are padded with zeros to whole 8-element runs; the column sums take
// the unrounded float32 values: each thread 8 columns of every 8th row of a chunk,
// the 8 row groups joined in order through LDS, one float32 row per chunk, and the
// chunks joined in order by a second kernel.
#include "linear_tile.h"

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
    constexpr bool FX = sizeof(E) == 2;
    const E* gy = static_cast<const E*>(a.dy) + col;
    const E* gz = static_cast<const E*>(a.z[0]) + col;
    const E* gu = GATED ? static_cast<const E*>(a.z[1]) + col : nullptr;
    // two rows at a time: their loads are in flight together
    for (long long m = m0 + rg; m < m1; m += 16) {
      const bool two = m + 8 < m1;
      float dy[2][8], z[2][8], t[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k == 1 && !two) break;
        const long long row = m + 8 * k;
        load8(gy + row * a.ldy, nv, dy[k]);
        if (GATED || a.act != 0) load8(gz + row * a.ldz, nv, z[k]);
        if constexpr (GATED) load8(gu + row * a.ldz, nv, t[k]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k == 1 && !two) break;
        const long long row = m + 8 * k;
        float f[8];
        if constexpr (GATED) {
          acts_and_slopes<FX>(z[k], f, a.act, a.alpha, a.beta);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[k][i] = i < nv ? dy[k][i] * t[k][i] * z[k][i] : 0.0f;  // dg
            t[k][i] = i < nv ? dy[k][i] * f[i] : 0.0f;               // du
            sum[0][i] += z[k][i];
            sum[KINDS - 1][i] += t[k][i];
          }
          E* o = static_cast<E*>(a.dz) + row * a.lddz + col;
          store8(o, 8, z[k]);
          store8(o + a.np, 8, t[k]);
        } else {
          if (a.act != 0) {
            acts_and_slopes<FX>(z[k], f, a.act, a.alpha, a.beta);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] = i < nv ? dy[k][i] * z[k][i] : 0.0f;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[k][i] = dy[k][i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0][i] += t[k][i];
          if (a.dz) store8(static_cast<E*>(a.dz) + row * a.lddz + col, 8, t[k]);
          if (a.dr)
            store8(static_cast<E*>(a.dr) + row * a.lddr + col, nv, a.dr_is_dy ? dy[k] : t[k]);
        }
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

// 32 columns a workgroup; each of 8 groups of lanes adds an eighth of the chunks in
// order, then the groups in order.
template <typename E>
__global__ __launch_bounds__(256) void linear_sums_kernel(const SumsArgs a) {
  __shared__ float red[8][32];
  const int cl = threadIdx.x & 31, g = threadIdx.x >> 5, d = blockIdx.y;
  const int c = blockIdx.x * 32 + cl;
  const int per = (a.chunks + 7) / 8, i1 = min(a.chunks, (g + 1) * per);
  float s = 0.0f;
  if (c < a.n) {
    const float* p = a.sums + (long long)d * a.np + c;
    const long long step = (long long)a.parts * a.np;
#pragma unroll 8
    for (int i = g * per; i < i1; ++i) s += p[i * step];
  }
  red[g][cl] = s;
  __syncthreads();
  if (g == 0 && c < a.n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][cl];
    static_cast<E*>(a.db[d])[c] = (E)s;
  }
}

// Operands with odd rows, copied so that the products can load them to LDS directly:
// a thread moves 16-byte pieces, the last one of a row loaded from further back and
// shifted.  Bound by memory: every element is read and written once (two operands of
// 1531 x 1001 and 777 x 1531 f16 in 5.7 us, most of it the launch).
template <typename E>
__global__ __launch_bounds__(256) void linear_pack_kernel(const PackArgs a) {
  constexpr int EPC = 16 / (int)sizeof(E), PER = 4;
  using R = lin::Ragged<E, false>;
  int q = 0;
  while (q + 1 < a.n && (int)blockIdx.x >= a.first[q + 1]) ++q;
  const int cols = a.cols[q], ppr = (int)(a.packed_ld[q] / EPC);
  const long long at = (long long)((int)blockIdx.x - a.first[q]) * 256 * PER + threadIdx.x;
  lin::i32x4 v[PER];
  int piece[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const long long id = min(at + i * 256, a.pieces[q] - 1);
    const long long row = a.pieces[q] < (1LL << 31) ? (unsigned)id / (unsigned)ppr : id / ppr;
    piece[i] = (int)(id - row * ppr);
    const E* p = static_cast<const E*>(a.src[q]) + row * a.ld[q];
    if (cols >= EPC)
      v[i] = lin::load_piece<E>(reinterpret_cast<const char*>(p),
                                min(piece[i] * EPC, cols - EPC) * (int)sizeof(E));
    else
      v[i] = R::raw(p, 0, 0, 0, 1, cols, true);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (at + i * 256 < a.pieces[q])
      static_cast<lin::i32x4*>(a.dst[q])[at + i * 256] =
          cols >= EPC ? R::shift(v[i], piece[i], cols) : v[i];
}

}  // namespace

template <typename E>
hipError_t launch_pack(const PackArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_pack_kernel<E>), dim3(a.first[a.n]), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_dz(const DzArgs& a, bool gated, int chunks, hipStream_t s) {
  const dim3 grid((a.np + 255) / 256, chunks);
  if (gated) hipLaunchKernelGGL((linear_dz_kernel<E, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear_dz_kernel<E, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sums(const SumsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_sums_kernel<E>), dim3((a.n + 31) / 32, a.parts), dim3(256), 0, s, a);
  return hipGetLastError();
}

#define CONVFWD_INST(E)                                                          \
  template hipError_t launch_dz<E>(const DzArgs&, bool, int, hipStream_t);      \
  template hipError_t launch_sums<E>(const SumsArgs&, hipStream_t);             \
  template hipError_t launch_pack<E>(const PackArgs&, hipStream_t);
CONVFWD_INST(_Float16)
CONVFWD_INST(__bf16)
CONVFWD_INST(float)
#undef CONVFWD_INST

}  // namespace convfwd
