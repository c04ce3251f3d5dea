// Linear and gated products of few rows (single tokens, small batches): the
// weights are streamed from memory once, straight into MFMA operands.
//
// out[c][r] = sum_k P(r, k) Q(c, k) with at most 32 rows c: 2 C flops per weight
// byte, far below the card's ratio, so the bound is the weights' stream.  A
// workgroup owns 16 weight rows and all of Q; its waves split k.  Lane (l, g)
// loads 16 bytes of weight row l at piece g of each 64-byte unit of k, which is
// the MFMA A operand as it lies: no LDS, no shuffles.  Q (a few KB to a few
// hundred) comes from L2 the same way.  The waves' sums are added in wave order
// through LDS, then the epilogue runs on runs of 8 outputs.
#include "linear_tile.h"

namespace convfwd {

namespace {

template <typename E, int TC, bool GATED, bool VEC>
__global__ __launch_bounds__(512) void linear_stream_kernel(const ProductArgs a) {
  using namespace lin;
  constexpr int EB = (int)sizeof(E), EPC = 16 / EB, UE = 64 / EB;
  constexpr int WAVES = 8, KINDS = GATED ? 2 : 1;
  constexpr int U = TC * KINDS >= 4 ? 4 : 8;  // units in flight per wave
  typedef std::conditional_t<EB == 2, s16x8, f32x4> Frag;
  __shared__ __attribute__((aligned(16))) float red[WAVES][KINDS * TC][16][16];

  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = blockIdx.x * 16;
  const int nr = min(16, a.R - r0);
  const int nu = (a.K + UE - 1) / UE;
  const int upw = (nu + WAVES - 1) / WAVES;
  const int u0 = wave * upw, u1 = min(nu, u0 + upw);

  const E* pb[KINDS];
  __amdgpu_buffer_rsrc_t pr[KINDS], qr;
#pragma unroll
  for (int d = 0; d < KINDS; ++d) {
    pb[d] = static_cast<const E*>(a.P[d]) + (long long)r0 * a.ldp;
    pr[d] = __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(pb[d]), 0,
                                              (int)(((nr - 1) * a.ldp + a.K) * EB), 0x00020000);
  }
  const E* qb = static_cast<const E*>(a.Q[0]);
  qr = __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(qb), 0,
                                         (int)(((a.C - 1) * a.ldq + a.K) * EB), 0x00020000);
  const int poff = (int)(l * a.ldp * EB) + g * 16;
  int qoff[TC];
#pragma unroll
  for (int t = 0; t < TC; ++t) qoff[t] = (int)((t * 16 + l) * a.ldq * EB) + g * 16;

  mfma_f32x4 acc[KINDS][TC];
#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int t = 0; t < TC; ++t) acc[d][t] = mfma_f32x4{0, 0, 0, 0};

  for (int u = u0; u < u1; u += U) {
    Frag p[KINDS][U], q[TC][U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      // a piece past k or past this wave's units reads zeros
      const bool in = u + i < u1 && (u + i) * UE + g * EPC < a.K;
      const int ko = (u + i) * 64;
      if constexpr (VEC) {
#pragma unroll
        for (int d = 0; d < KINDS; ++d)
          p[d][i] = __builtin_bit_cast(
              Frag, __builtin_amdgcn_raw_buffer_load_b128(pr[d], in ? poff + ko : kOob, 0, 0));
#pragma unroll
        for (int t = 0; t < TC; ++t)
          q[t][i] = __builtin_bit_cast(
              Frag, __builtin_amdgcn_raw_buffer_load_b128(qr, in ? qoff[t] + ko : kOob, 0, 0));
      } else {
        const int piece = in ? (u + i) * 4 + g : 0;
        const int k = in ? a.K : 0;
#pragma unroll
        for (int d = 0; d < KINDS; ++d)
          p[d][i] = __builtin_bit_cast(Frag, gather<E, false>(pb[d], a.ldp, l, piece, nr, k));
#pragma unroll
        for (int t = 0; t < TC; ++t)
          q[t][i] = __builtin_bit_cast(Frag,
                                       gather<E, false>(qb, a.ldq, t * 16 + l, piece, a.C, k));
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int d = 0; d < KINDS; ++d)
#pragma unroll
        for (int t = 0; t < TC; ++t) acc[d][t] = multiply<E>(p[d][i], q[t][i], acc[d][t]);
  }

#pragma unroll
  for (int d = 0; d < KINDS; ++d)
#pragma unroll
    for (int t = 0; t < TC; ++t)
      *reinterpret_cast<mfma_f32x4*>(&red[wave][d * TC + t][l][g * 4]) = acc[d][t];
  __syncthreads();
  for (int i = tid; i < KINDS * TC * 256; i += 512) {
    float* f = &red[0][0][0][0] + i;
    float s = f[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += f[w * KINDS * TC * 256];
    f[0] = s;
  }
  __syncthreads();
  if (tid < TC * 32) {
    const int c = tid >> 1, r = r0 + (tid & 1) * 8;
    if (c < a.C && r < a.R) {
      float v[8], w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = red[0][c >> 4][c & 15][(tid & 1) * 8 + q];
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = red[0][TC + (c >> 4)][c & 15][(tid & 1) * 8 + q];
        finish_gated<E>(a.e, c, r, v, w);
      } else {
        finish_linear<E>(a.e, 0, c, r, v);
      }
    }
  }
}

// Joins the planes of a split contraction in split order: 8 outputs a thread.
template <typename E, bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(const JoinArgs a) {
  const int per_row = (int)(a.plane_ld / 8);
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = id / per_row;  // z * C + c
  if (row >= (long long)a.nz * a.C) return;
  const int r = (int)(id - row * per_row) * 8;
  const int z = (int)(row / a.C);
  const long long c = row - (long long)z * a.C;
  const float* s = a.planes + row * a.plane_ld + r;
  float v[8], u[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = u[q] = 0.0f;
  for (int i = 0; i < a.splits; ++i) {
    const lin::f32x4 lo = *reinterpret_cast<const lin::f32x4*>(s);
    const lin::f32x4 hi = *reinterpret_cast<const lin::f32x4*>(s + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) { v[q] += lo[q]; v[4 + q] += hi[q]; }
    if constexpr (GATED) {
      const float* t = s + (long long)a.C * a.plane_ld;
      const lin::f32x4 tl = *reinterpret_cast<const lin::f32x4*>(t);
      const lin::f32x4 th = *reinterpret_cast<const lin::f32x4*>(t + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) { u[q] += tl[q]; u[4 + q] += th[q]; }
    }
    s += a.plane_stride;
  }
  if (r >= a.e.R) return;
  if constexpr (GATED) finish_gated<E>(a.e, c, r, v, u);
  else finish_linear<E>(a.e, z, c, r, v);
}

template <typename E, int TC, bool GATED>
hipError_t stream_t(const ProductArgs& a, bool vec, hipStream_t s) {
  const dim3 grid((a.R + 15) / 16), block(512);
  if (vec) hipLaunchKernelGGL((linear_stream_kernel<E, TC, GATED, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((linear_stream_kernel<E, TC, GATED, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

template <typename E>
hipError_t launch_stream(const ProductArgs& a, int blocks16, bool gated, bool vec, hipStream_t s) {
  if (gated) return blocks16 == 1 ? stream_t<E, 1, true>(a, vec, s) : stream_t<E, 2, true>(a, vec, s);
  return blocks16 == 1 ? stream_t<E, 1, false>(a, vec, s) : stream_t<E, 2, false>(a, vec, s);
}

template <typename E>
hipError_t launch_join(const JoinArgs& a, bool gated, hipStream_t s) {
  const long long items = (long long)a.nz * a.C * (a.plane_ld / 8);
  const dim3 grid((unsigned)((items + 255) / 256));
  if (gated) hipLaunchKernelGGL((linear_join_kernel<E, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear_join_kernel<E, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

#define CONVFWD_INST(E)                                                                      \
  template hipError_t launch_stream<E>(const ProductArgs&, int, bool, bool, hipStream_t);   \
  template hipError_t launch_join<E>(const JoinArgs&, bool, hipStream_t);
CONVFWD_INST(_Float16)
CONVFWD_INST(__bf16)
CONVFWD_INST(float)
#undef CONVFWD_INST

}  // namespace convfwd
