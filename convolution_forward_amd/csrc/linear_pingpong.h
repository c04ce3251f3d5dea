// The large tile of the linear and gated products on 16-bit operands (see
// linear_tile.h for operands, layouts in LDS and the epilogue's idea): 256 outputs
// r by BC = 256 or 128 outputs c for 8 waves, two waves on each SIMD.
//
//  * Both operands are cut into halves (128 rows of P, BC / 2 of Q).  A wave owns a
//    part of each half (2 x 4 waves share 256 x 256, 4 x 2 share 256 x 128, so that
//    parts stay near square) and takes a step in two phases, a half of P each.
//  * The waves form two groups of four, one wave of each on every SIMD, half a
//    phase apart: while one group multiplies, the other reads its next fragments
//    from LDS and issues global loads, and the SIMD's matrix core is fed by one or
//    the other all the time.
//  * Half tiles live in two LDS buffers.  A half that was read for the last time in
//    a phase is overwritten from the next one on by the half of two steps later;
//    three phases pass between a half's load and its use, and the loads of a whole
//    step (64 or 48 KB) are in flight at every turn.
//  * Gated products: half 0 of P is gate rows, half 1 the same rows of up, and a
//    wave holds both sums of its outputs.
//  * The epilogue takes the sums from registers (runs_of_8): 9500 cycles a tile with
//    no activation, 24000 with GELU, beside which nothing multiplies (6 and 14% of a
//    tile with k = 4096).  A trip through LDS, 16 rows at a time, took 21000 (as much
//    as 9 steps), with erff's GELU 70000.
//
// What bounds it: a step of 256 x 256 has 2048 cycles of products on each SIMD and
// takes 2360 (the turns between the groups); 256 x 128 takes 1500 for 1024, so it is
// chosen where 256 x 256 would leave units idle.  With the start (3800 cycles) and the
// epilogue the matrix cores are busy for 73% of a tile of k = 4096 with GELU, 80%
// without.  With the whole card at work the clock falls to 1.8 GHz (2.2 with zeros as
// operands): 8192 x 4096 x 4096 bf16 194 to 201 us (1370 to 1420 TFLOP/s), with GELU 207
// to 216; 4096 x 4096 x 4096 97 us.  Measured and not taken:
// four phases a step (1 to 3% slower), one (256 x 128, transposed operands 10%
// slower), v_mfma 32x32x16 (2 to 5%), four waves of 128 x 128 (2730 cycles a step: one
// wave a SIMD cannot hide its own scalar code).
#pragma once

#include "linear_tile.h"

namespace convfwd {

namespace lin {

__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

template <typename E, bool PT, bool QT, int BC, bool GATED, bool PLAIN = false>
struct PingPong {
  static_assert(sizeof(E) == 2 && (BC == 256 || BC == 128), "16-bit operands");
  static constexpr int NT = 512, HR = 128, HC = BC / 2;
  static constexpr int WVR = BC == 256 ? 2 : 4, WVC = 8 / WVR;  // waves along r and c
  static constexpr int WR = HR / WVR, WC = HC / WVC;  // a wave's part of a half
  static constexpr int NI = WR / 16, NJ = WC / 16;
  using TP = Tile<E, HR, PT, NT>;
  using TQ = Tile<E, HC, QT, NT>;
  static constexpr int SMEM = 4 * (TP::BYTES + TQ::BYTES);
  // an operand's four half tiles lie side by side, within an LDS instruction's
  // 64 KB offset of one address
  static constexpr int p_at(int half, int buf) { return (2 * buf + half) * TP::BYTES; }
  static constexpr int q_at(int half, int buf) {
    return 4 * TP::BYTES + (2 * buf + half) * TQ::BYTES;
  }
  static constexpr int LOADS = 2 * (TP::ITEMS + TQ::ITEMS);  // of a step, per wave

  // id: index of this workgroup among the product's own, after xcd_logical
  static __device__ __forceinline__ void run(const ProductArgs& a, int id, char* smem) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave % WVR, wc = wave / WVR;

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

    // What the loads of a step need, moved on from step to step in small pieces
    // between a phase's products: scalar code costs a wave 4 cycles an instruction,
    // and the reading side of a turn has none to spare.  A descriptor ends with the
    // last valid row (transposed: the last valid k), so that everything past an end
    // reads as zeros; it is empty past the last step and past the operand's rows.
    constexpr int kNone = -(1 << 30);
    const int ldpb = (int)a.ldp * 2, ldqb = (int)a.ldq * 2;
    const int seg0 = t0 >= a.ktiles ? 1 : 0, kt0 = t0 - (seg0 ? a.ktiles : 0);
    const long long pstep = PT ? 64LL * ldpb : 128, qstep = QT ? 64LL * ldqb : 128;
    const char *pb[2], *qb[2], *pseg[2], *qseg[2];  // present, and of the second segment
    int pspan[2], qspan[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long pr = r0 + (GATED ? 0 : h * HR), qr = c0 + h * HC;
      const long long po = PT ? pr * 2 : pr * ldpb, qo = QT ? qr * 2 : qr * ldqb;
      pseg[h] = static_cast<const char*>(a.P[1]) + po;
      qseg[h] = static_cast<const char*>(a.Q[1]) + qo;
      pb[h] = (GATED ? h : seg0) ? pseg[h] : static_cast<const char*>(a.P[0]) + po;
      qb[h] = seg0 ? qseg[h] : static_cast<const char*>(a.Q[z]) + qo;
      pb[h] += kt0 * pstep;
      qb[h] += kt0 * qstep;
      const int np = (int)min(a.R - pr, (long long)HR), nq = (int)min(a.C - qr, (long long)HC);
      pspan[h] = np <= 0 ? kNone : PT ? ((np + 7) & ~7) * 2 : (np - 1) * ldpb;
      qspan[h] = nq <= 0 ? kNone : QT ? ((nq + 7) & ~7) * 2 : (nq - 1) * ldqb;
    }
    int count = t0, left = a.K - kt0 * 64, kk, pbytes, qbytes;
    const int ktail = a.K - (a.K - 1) / 64 * 64;  // k of a segment's last step
    const bool ptail = PT || pk < ktail, qtail = QT || qk < ktail;
    bool turn = false;
    auto stage = [&](int n) {
      if (n == 0) {
        ++count;
        turn = !GATED && count == a.ktiles;
        left = turn ? a.K : left - 64;
      } else if (n == 1) {
        kk = count < t1 ? min(left, 64) : kNone;
      } else if (n == 2) {
        pbytes = kk < 0 ? kNone : PT ? (kk - 1) * ldpb : ((kk + 7) & ~7) * 2;
      } else if (n == 3) {
        qbytes = kk < 0 ? kNone : QT ? (kk - 1) * ldqb : ((kk + 7) & ~7) * 2;
      } else if (n < 6) {
        pb[n - 4] = turn ? pseg[n - 4] : pb[n - 4] + pstep;
      } else {
        qb[n - 6] = turn ? qseg[n - 6] : qb[n - 6] + qstep;
      }
    };
    auto issue_p = [&](int half, int buf) {
      const i32x4 rs = make_rsrc(pb[half], max(pspan[half] + pbytes, 0));
      const bool all = kk >= 64 || ptail;
#pragma unroll
      for (int i = 0; i < TP::ITEMS; ++i)
        dma16(rs, all ? poff[i] : kOob, lds0 + p_at(half, buf) + i * NT * 16);
    };
    auto issue_q = [&](int half, int buf) {
      const i32x4 rs = make_rsrc(qb[half], max(qspan[half] + qbytes, 0));
      const bool all = kk >= 64 || qtail;
#pragma unroll
      for (int i = 0; i < TQ::ITEMS; ++i)
        dma16(rs, all ? qoff[i] : kOob, lds0 + q_at(half, buf) + i * NT * 16);
    };

    typename TP::Frag p[NI][2];
    typename TQ::Frag q[2][NJ][2];
    auto read_p = [&](int half, int buf) {
      const char* b = smem + p_at(half, buf);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2)
          p[i][j2] = TP::frag(b, wr * WR + i * 16, j2, lane);
    };
    auto read_q = [&](int buf) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int j2 = 0; j2 < 2; ++j2)
            q[h][j][j2] = TQ::frag(smem + q_at(h, buf), wc * WC + j * 16, j2, lane);
    };
    // end of a phase's reads: they are in registers, and what the next phase reads has
    // arrived for every wave behind the barrier
    auto turn_over = [&] {
      lds_wait();
      vm_wait<LOADS>();
      fence();
      barrier();
      fence();
    };
    // the products of a half of P; with MOVE the state of the loads moves on between
    // them
    auto multiply_half = [&](int hp, auto move) {
      constexpr bool MOVE = decltype(move)::value;
      constexpr int N = 4 * NI * NJ, EACH = N / 8;
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int j2 = n / (2 * NI * NJ), h = n / (NI * NJ) % 2, i = n / NJ % NI, j = n % NJ;
        acc[hp][h][i][j] = multiply<E>(p[i][j2], q[h][j][j2], acc[hp][h][i][j]);
        if (MOVE && n % EACH == EACH - 1) {
          fence();
          stage(n / EACH);
          fence();
        }
      }
      __builtin_amdgcn_s_setprio(0);
      fence();
      barrier();
      fence();
    };
    constexpr std::integral_constant<bool, false> stay;
    constexpr std::integral_constant<bool, true> move;
    auto issue_first = [&](int buf) {  // what the first phase reads
      issue_q(0, buf);
      issue_q(1, buf);
      issue_p(0, buf);
    };

#pragma unroll
    for (int n = 1; n < 4; ++n) {
      if (n == 1) kk = min(left, 64);
      else stage(n);
    }
    issue_first(0);
    issue_p(1, 0);
#pragma unroll
    for (int n = 0; n < 8; ++n) stage(n);
    issue_first(1);
    // the first phase's part of the first step has arrived
    vm_wait<LOADS>();
    barrier();
    const bool late = wave >= 4;
    if (late) barrier();
    fence();
    auto step = [&](int b) {
      read_q(b);
      read_p(0, b);
      issue_p(1, b ^ 1);  // the next step's
      turn_over();
      multiply_half(0, move);
      read_p(1, b);
      issue_first(b);  // of two steps later
      turn_over();
      multiply_half(1, stay);
    };
    for (int t = t0; t < t1; t += 2) {  // an odd count ends with a step of zeros
      step(0);
      step(1);
    }
    if (!late) barrier();
    vm_wait<0>();  // loads past the end (zeros) land before the workgroup's LDS is given up

    // epilogue: 16 rows c at a time, one a lane, its outputs in runs of 8
    constexpr int NR = GATED ? NI / 2 : NI;
    auto off = [](int n) { return n % (NI / 2) * 32 + n / (NI / 2) * HR; };
    const int rl = r0 + wr * WR + run_offset(lane);
    const bool whole = nr >= (GATED ? HR : 2 * HR);
#pragma unroll 1
    for (int round = 0; round < 2 * NJ; ++round) {
      float v[NR * 8], u[GATED ? NR * 8 : 1];
#pragma unroll
      for (int n = 0; n < 2 * NJ; ++n)
        if (n == round) {
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const int h = GATED ? 0 : i / (NI / 2), b = i % (NI / 2) * 2;
            runs_of_8(acc[h][n / NJ][b][n % NJ], acc[h][n / NJ][b + 1][n % NJ], v + i * 8);
            if constexpr (GATED)
              runs_of_8(acc[1][n / NJ][b][n % NJ], acc[1][n / NJ][b + 1][n % NJ], u + i * 8);
          }
        }
      const long long c = c0 + round / NJ * HC + wc * WC + round % NJ * 16 + (lane & 15);
      const bool in = c < a.C;
      if (!PLAIN && a.splits > 1) {
        constexpr int KINDS = GATED ? 2 : 1;
        float* d = a.planes + (((long long)split * a.nz + z) * KINDS * a.C + c) * a.plane_ld + rl;
#pragma unroll
        for (int n = 0; n < NR; ++n)
          if (in && rl + off(n) < a.R) {  // rows padded to 8 floats
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              d[off(n) + e] = v[n * 8 + e];
              if constexpr (GATED) d[(long long)a.C * a.plane_ld + off(n) + e] = u[n * 8 + e];
            }
          }
      } else if constexpr (PLAIN) {
        if (in) finish_plain_runs<E, NR>(a.e, z, c, rl, off, whole, v);
      } else if constexpr (GATED) {
        finish_gated_runs<E, NR>(a.e, c, in, rl, off, whole, v, u);
      } else {
        finish_linear_runs<E, NR>(a.e, z, c, in, rl, off, whole, v);
      }
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

// The two products of a backward pass in one launch, the one with the longer
// contraction first: dx = dz w (DT: w transposed in the sense of linear_tile.h) and
// dw = dz^T x.  Each alone often fills part of the card's last round of workgroups
// only; together they fill one another's.  4096 x 4096 x 1024 bf16: 61 us (1120
// TFLOP/s) with 256 x 128 tiles, 107 in two launches; a gated block of 4096 x 5632 x
// 2048: 277 us (1360 TFLOP/s), 375 in two.
template <typename E, bool DT, int BC>
__global__ __launch_bounds__(512) void linear_pair_kernel(const PairArgs a) {
  using DX = lin::PingPong<E, DT, false, BC, false, true>;
  using DW = lin::PingPong<E, true, true, BC, false, true>;
  static_assert(DX::SMEM == DW::SMEM, "one buffer for both");
  __shared__ __attribute__((aligned(1024))) char smem[DX::SMEM];
  const bool second = (int)blockIdx.x >= a.first;
  const int id = second ? xcd_logical(blockIdx.x - a.first, gridDim.x - a.first)
                        : xcd_logical(blockIdx.x, a.first);
  if (second != a.dw_first) DW::run(a.dw, id, smem);
  else DX::run(a.dx, id, smem);
}

}  // namespace convfwd
