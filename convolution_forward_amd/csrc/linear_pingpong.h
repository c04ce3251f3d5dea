// The large tile of the linear and gated products on 16-bit operands (see
// linear_tile.h for operands, layouts in LDS and the epilogue's idea): 256 outputs
// r by BC = 256 or 128 outputs c for 8 waves, two waves on each SIMD.
//
//  * Both operands are cut into halves (128 rows of P, BC / 2 of Q).  A wave owns
//    64 rows of each half of P and BC / 8 of each half of Q: four quadrants of the
//    accumulators, one for each pair of halves, taken one a phase.
//  * The waves form two groups of four, one wave of each on every SIMD, half a
//    phase apart: while one group multiplies a quadrant, the other reads its next
//    fragments from LDS and issues global loads, and the SIMD's matrix core is fed
//    by one or the other all the time.
//  * Quadrants go round: P0 Qf, P0 Qs, P1 Qs, P1 Qf, where f and s change places
//    every step, so that each phase reads one half and no half is read twice.
//  * Half tiles live in two LDS buffers.  The half that a phase has read for the
//    last time is overwritten from the next phase on by the half of two steps
//    later; seven phases pass between a half's load and its use, so six halves (96
//    KB) are in flight at any time and no phase waits for memory in steady state.
//  * Gated products: half 0 of P is gate rows, half 1 the same rows of up, and a
//    wave holds both sums of its outputs.
#pragma once

#include "linear_tile.h"

namespace convfwd {

namespace lin {

__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

template <typename E, bool PT, bool QT, int BC, bool GATED>
struct PingPong {
  static_assert(sizeof(E) == 2 && (BC == 256 || BC == 128), "16-bit operands");
  static constexpr int NT = 512, HR = 128, HC = BC / 2;
  static constexpr int NI = 4, NJ = BC / 128;  // 16-row blocks of a quadrant
  using TP = Tile<E, HR, PT, NT>;
  using TQ = Tile<E, HC, QT, NT>;
  static constexpr int BUF = 2 * (TP::BYTES + TQ::BYTES);
  static constexpr int EPLD = 64 + 4;
  static constexpr int EPW = 16 * EPLD * 4 * (GATED ? 2 : 1);
  static constexpr int SMEM = 2 * BUF > 8 * EPW ? 2 * BUF : 8 * EPW;
  static constexpr int FLIGHT = 3 * (TP::ITEMS + TQ::ITEMS);  // six halves

  // id: index of this workgroup among the product's own, after xcd_logical
  static __device__ __forceinline__ void run(const ProductArgs& a, int id, char* smem) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave & 1, wc = wave >> 1;

    const int per = a.ntr * a.ntc;
    const int batch = id / per;  // split * nz + z
    const int z = batch % a.nz, split = batch / a.nz;
    const int idx = id - batch * per;
    const int band = idx / (8 * a.ntr), bw = min(8, a.ntc - 8 * band);
    const int in = idx - band * 8 * a.ntr;
    const int tr = in / bw, tc = 8 * band + in - tr * bw;
    const int r0 = tr * (GATED ? HR : 2 * HR);
    const long long c0 = (long long)tc * BC;
    const long long nr = a.R - r0, nc = a.C - c0;

    const int t_all = a.ktiles * a.nseg;
    const int t0 = split * a.per_split, t1 = min(t0 + a.per_split, t_all);

    mfma_f32x4 acc[2][2][NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[0][0][i][j] = acc[0][1][i][j] = acc[1][0][i][j] = acc[1][1][i][j] = mfma_f32x4{0, 0, 0, 0};

    // byte offsets of this thread's pieces in a half; the piece's k, alike for all
    int poff[TP::ITEMS], qoff[TQ::ITEMS], pk, qk;
#pragma unroll
    for (int i = TP::ITEMS - 1; i >= 0; --i) {
      int row, piece;
      TP::item(i, tid, &row, &piece);
      poff[i] = (int)(row * a.ldp * TP::EB) + piece * 16;
      pk = piece * TP::EPC;
    }
#pragma unroll
    for (int i = TQ::ITEMS - 1; i >= 0; --i) {
      int row, piece;
      TQ::item(i, tid, &row, &piece);
      qoff[i] = (int)(row * a.ldq * TQ::EB) + piece * 16;
      qk = piece * TQ::EPC;
    }
    const unsigned lds0 = lds_addr(smem) + wave * 1024;

    // The half at row `row` of an operand, step t: rows run along k, or are of
    // constant k (T).  The descriptor ends with the last valid row (T: with the last
    // valid k), so that everything past an end reads as zeros; it is empty past the
    // last step and past the operand's rows.
    auto issue = [&](auto transposed, const char* m0, const char* m1, long long ld, long long row,
                     long long rows, int most, const int* off, int items, int kpiece, int t,
                     unsigned lds) {
      constexpr bool T = decltype(transposed)::value;
      const int seg = t >= a.ktiles ? 1 : 0;
      const int k0 = (t - (seg ? a.ktiles : 0)) * 64;
      const int kk = min(a.K - k0, 64), ldb = (int)ld * 2;
      const int n = (int)min(rows, (long long)most);
      int bytes = T ? (kk - 1) * ldb + ((n + 7) & ~7) * 2 : (n - 1) * ldb + ((kk + 7) & ~7) * 2;
      bytes = n <= 0 || t >= t1 ? 0 : bytes;
      const char* p = (seg ? m1 : m0) + (T ? k0 * ld + row : row * ld + k0) * 2;
      const i32x4 rs = make_rsrc(p, bytes);
#pragma unroll
      for (int i = 0; i < items; ++i)
        dma16(rs, !T && kpiece >= kk ? kOob : off[i], lds + i * NT * 16);
    };
    const char* const P0 = static_cast<const char*>(a.P[0]);
    const char* const P1 = static_cast<const char*>(a.P[1]);
    const char* const Q0 = static_cast<const char*>(a.Q[z]);
    const char* const Q1 = static_cast<const char*>(a.Q[1]);
    auto issue_p = [&](int t, int half, int buf) {
      const char* m = GATED && half ? P1 : P0;
      const int h = GATED ? 0 : half * HR;
      issue(std::integral_constant<bool, PT>(), m, GATED ? m : P1, a.ldp, r0 + h, nr - h, HR, poff,
            TP::ITEMS, pk, t, lds0 + buf * BUF + half * TP::BYTES);
    };
    auto issue_q = [&](int t, int half, int buf) {
      issue(std::integral_constant<bool, QT>(), Q0, Q1, a.ldq, c0 + half * HC, nc - half * HC, HC,
            qoff, TQ::ITEMS, qk, t, lds0 + buf * BUF + 2 * TP::BYTES + half * TQ::BYTES);
    };

    typename TP::Frag p[NI][2];
    typename TQ::Frag q[2][NJ][2];
    auto read_p = [&](int half, int buf) {
      const char* b = smem + buf * BUF + half * TP::BYTES;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) p[i][j2] = TP::frag(b, wr * 64 + i * 16, j2, lane);
    };
    auto read_q = [&](int half, int buf) {
      const char* b = smem + buf * BUF + 2 * TP::BYTES + half * TQ::BYTES;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) q[half][j][j2] = TQ::frag(b, wc * (HC / 4) + j * 16, j2, lane);
    };
    // end of a phase's reads: they are in registers, and the half that the next
    // phase reads has arrived for every wave behind the barrier
    auto turn = [&] {
      lds_wait();
      vm_wait<FLIGHT>();
      fence();
      barrier();
      fence();
    };
    auto multiply_all = [&](int hp, int hq) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j2 = 0; j2 < 2; ++j2)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[hp][hq][i][j] = multiply<E>(p[i][j2], q[hq][j][j2], acc[hp][hq][i][j]);
      __builtin_amdgcn_s_setprio(0);
      fence();
      barrier();
      fence();
    };
    // one contraction step in buffer F (its parity): halves f = F, s = 1 - F of Q
    auto step = [&](int t, auto parity) {
      constexpr int F = decltype(parity)::value, S = 1 - F;
      read_p(0, F);
      issue_q(t + 2, F, F);
      turn();
      multiply_all(0, F);
      read_q(S, F);
      issue_p(t + 2, 0, F);
      turn();
      multiply_all(0, S);
      read_p(1, F);
      issue_q(t + 2, S, F);
      turn();
      multiply_all(1, S);
      read_q(S, S);  // the next step's first half
      issue_p(t + 2, 1, F);
      turn();
      multiply_all(1, F);
    };

    issue_q(t0, 0, 0);
    issue_p(t0, 0, 0);
    issue_q(t0, 1, 0);
    issue_p(t0, 1, 0);
    issue_q(t0 + 1, 1, 1);
    issue_p(t0 + 1, 0, 1);
    issue_q(t0 + 1, 0, 1);
    issue_p(t0 + 1, 1, 1);
    vm_wait<FLIGHT>();
    barrier();
    read_q(0, 0);
    lds_wait();
    fence();
    barrier();
    const bool late = wave >= 4;
    if (late) barrier();
    fence();
    for (int t = t0; t < t1; t += 2) {  // an odd count ends with a step of zeros
      step(t, std::integral_constant<int, 0>());
      step(t + 1, std::integral_constant<int, 1>());
    }
    if (!late) barrier();
    vm_wait<0>();  // loads past the end (zeros) land before the LDS is reused
    fence();
    barrier();

    // epilogue: each wave alone in its part of the LDS, 16 rows c at a time
    float* ep = reinterpret_cast<float*>(smem + wave * EPW);
    const int l = lane & 15, g = lane >> 4;
    const int er = (lane & 7) * 8, ec = lane >> 3;
#pragma unroll
    for (int hq = 0; hq < 2; ++hq)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int hp = 0; hp < (GATED ? 1 : 2); ++hp) {
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            float* d = ep + l * EPLD + i * 16 + g * 4;
            *reinterpret_cast<mfma_f32x4*>(d) = acc[hp][hq][i][j];
            if constexpr (GATED) *reinterpret_cast<mfma_f32x4*>(d + 16 * EPLD) = acc[1][hq][i][j];
          }
          lds_wait();
          __builtin_amdgcn_wave_barrier();
          const int r = r0 + hp * HR + wr * 64 + er;
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            const int row = pass * 8 + ec;
            const long long c = c0 + hq * HC + wc * (HC / 4) + j * 16 + row;
            const float* s = ep + row * EPLD + er;
            if (r < a.R && c < a.C) {
              float v[8], u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = s[e];
              if constexpr (GATED) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = s[16 * EPLD + e];
              }
              if (a.splits > 1) {
                constexpr int KINDS = GATED ? 2 : 1;
                float* d = a.planes + (((long long)split * a.nz + z) * KINDS * a.C + c) * a.plane_ld + r;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = v[e];  // rows padded to 8 floats
                if constexpr (GATED) {
                  d += (long long)a.C * a.plane_ld;
#pragma unroll
                  for (int e = 0; e < 8; ++e) d[e] = u[e];
                }
              } else if constexpr (GATED) {
                finish_gated<E>(a.e, c, r, v, u);
              } else {
                finish_linear<E>(a.e, z, c, r, v);
              }
            }
          }
          lds_wait();
          __builtin_amdgcn_wave_barrier();
        }
  }
};

}  // namespace lin

template <typename E, bool PT, bool QT, int BC, bool GATED>
__global__ __launch_bounds__(512) void linear_pingpong_kernel(const ProductArgs a) {
  using K = lin::PingPong<E, PT, QT, BC, GATED>;
  __shared__ __attribute__((aligned(1024))) char smem[K::SMEM];
  K::run(a, xcd_logical(blockIdx.x, gridDim.x), smem);
}

}  // namespace convfwd
