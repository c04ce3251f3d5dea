// Linear and gated products of few rows (single tokens, small batches): the
// weights are streamed from memory once, straight into MFMA operands.
//
// out[c][r] = sum_k P(r, k) Q(c, k) with at most 32 rows c: 2 C flops per weight
// byte, far below the card's ratio, so the bound is the weights' stream, and for
// the smallest calls its latency.  A workgroup owns 16 M / G weight rows and all of
// Q; its 8 waves take turns along k, so that together they read runs of 4 KB of
// each row.  Lane (l, g) loads 16 bytes of weight row l mod 16 / G at piece g of a
// 64-byte unit of k, which is the MFMA A operand as it lies: no LDS, no shuffles.
//  * G > 1 (few weight rows): the operand's G row groups hold the same rows at G
//    neighbouring units; G products, one with each unit's Q, give one valid group
//    each.  Few rows then still occupy every compute unit, at the price of G times
//    the (idle) matrix work.
//  * M = 2 (many weight rows, more than 16 rows c): two blocks of weight rows share
//    the loads of Q, which comes from L2.
// The next loads are in flight during the products of the present ones.  The
// partial sums are added in wave and group order through LDS, then the epilogue runs.
//
// Measured, weights from memory: one row, bf16 4096 x 4096 8.5 us (4.0 TB/s), 8192 x 4096
// 13.5 (5.0), 32000 x 4096 43 (6.1); a gated block of 5632 x 2048 10.1 (4.6 TB/s); 32 rows,
// 8192 x 4096 22 (3.0 TB/s, bound by Q from L2; 64 x 64 tiles in 4 splits take 19); one row,
// 1000 x 2048 f16 4.2 (a launch).  Waves that each stream their own
// range of k were 10 to 35% slower, 16 waves a workgroup slower still.
//
// The gated kernel of 17 to 32 rows c with 4 weight rows holds 16 pieces of Q twice over
// and spills (60 registers of aligned 16-bit operands, 382 of odd ones, 69 and 135 of
// float32).  24 rows, f 1024: k 2048 f16 7.5 us for 8.1 with 8 weight rows, but k 2047 24
// for 10, and float32 24 for 16: the plan does not know of that.
#include "linear_tile.h"

namespace convfwd {

namespace {

constexpr int kStreamWaves = 8;

// VEC: rows of whole aligned 16-byte pieces; otherwise rows start anywhere and the
// last pieces of a row are loaded from further back and shifted.
// O: the outputs' type (8-bit operands have int32 sums).
template <typename E, int TC, bool GATED, bool VEC, int G, int M, typename O = E>
__global__ __launch_bounds__(kStreamWaves * 64) void linear_stream_kernel(const ProductArgs a) {
  using namespace lin;
  constexpr int EB = (int)sizeof(E), EPC = 16 / EB, UE = 64 / EB, WAVES = kStreamWaves;
  constexpr int KINDS = GATED ? 2 : 1, RG = 16 / G, RB = RG * M;
  // weight loads of a batch, each of G units
  constexpr int N = G > 1 || M > 1 || TC * KINDS >= 4 ? 2 : 4;
  constexpr int BU = N * G;  // units of a batch
  using Frag = typename Tile<E, 16, false, 64>::Frag;
  using R = Ragged<E, false>;
  typedef std::conditional_t<EB == 1, int, float> S;
  constexpr int PARTS = WAVES * G;
  __shared__ __attribute__((aligned(16))) S red[PARTS][KINDS * TC][16][RB];

  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = blockIdx.x * RB;
  const int nr = min(RB, a.R - r0);
  const int nu = (a.K + UE - 1) / UE;
  const int pu = l / RG;  // this lane's unit within a weight load

  const char* pb[KINDS];
  __amdgpu_buffer_rsrc_t pr[KINDS], qr;
#pragma unroll
  for (int d = 0; d < KINDS; ++d) {
    pb[d] = static_cast<const char*>(a.P[d]) + (long long)r0 * a.ldp * EB;
    pr[d] = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(pb[d]), 0,
                                              (int)(((nr - 1) * a.ldp + a.K) * EB), 0x00020000);
  }
  const char* qb = static_cast<const char*>(a.Q[0]);
  qr = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(qb), 0,
                                         (int)(((a.C - 1) * a.ldq + a.K) * EB), 0x00020000);
  // row offsets in bytes; without VEC of the last row where there is no such row
  int prow[M], qrow[TC];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int row = m * RG + l % RG;
    prow[m] = (int)((VEC ? row : min(row, nr - 1)) * a.ldp * EB);
  }
#pragma unroll
  for (int t = 0; t < TC; ++t)
    qrow[t] = (int)((VEC ? t * 16 + l : min(t * 16 + l, a.C - 1)) * a.ldq * EB);
  const int last = (a.K - EPC) * EB;  // of a row's last whole piece

  Sums<E> acc[M][KINDS][TC][G];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int d = 0; d < KINDS; ++d)
#pragma unroll
      for (int t = 0; t < TC; ++t)
#pragma unroll
        for (int j = 0; j < G; ++j) acc[m][d][t][j] = Sums<E>{0, 0, 0, 0};

  struct Batch {
    Frag p[M][KINDS][N], q[TC][BU];
  };
  // a piece of the row at byte offset `row`, at byte offset ko of k (16-byte steps);
  // zeros past k
  auto piece = [&](const __amdgpu_buffer_rsrc_t& rs, const char* base, int row, int ko) {
    if constexpr (VEC)
      return __builtin_amdgcn_raw_buffer_load_b128(rs, ko < a.K * EB ? row + ko : kOob, 0, 0);
    else
      return load_piece<E>(base, row + min(ko, last));
  };
  auto fetch = [&](int u, Batch& b) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int d = 0; d < KINDS; ++d)
          b.p[m][d][i] = __builtin_bit_cast(
              Frag, piece(pr[d], pb[d], prow[m], (u + i * G + pu) * 64 + g * 16));
#pragma unroll
    for (int i = 0; i < BU; ++i)
#pragma unroll
      for (int t = 0; t < TC; ++t)
        b.q[t][i] = __builtin_bit_cast(Frag, piece(qr, qb, qrow[t], (u + i) * 64 + g * 16));
    if constexpr (!VEC) {
      if ((u + BU) * UE > a.K) {  // the row's end lies in this batch
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int d = 0; d < KINDS; ++d)
              b.p[m][d][i] = R::shift(b.p[m][d][i], (u + i * G + pu) * 4 + g, a.K);
#pragma unroll
        for (int i = 0; i < BU; ++i)
#pragma unroll
          for (int t = 0; t < TC; ++t) b.q[t][i] = R::shift(b.q[t][i], (u + i) * 4 + g, a.K);
      }
    }
  };
  auto products = [&](const Batch& b) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int d = 0; d < KINDS; ++d)
#pragma unroll
            for (int t = 0; t < TC; ++t)
              acc[m][d][t][j] = multiply<E>(b.p[m][d][i], b.q[t][i * G + j], acc[m][d][t][j]);
  };
  Batch b0, b1;
  int u = wave * BU;
  if (u < nu) fetch(u, b0);
  while (u < nu) {
    u += WAVES * BU;
    if (u < nu) fetch(u, b1);
    products(b0);
    if (u >= nu) break;
    u += WAVES * BU;
    if (u < nu) fetch(u, b0);
    products(b1);
  }

  // lane (l, g) holds rows 4g .. 4g + 3 of column l: row group 4g / RG of the sums
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int d = 0; d < KINDS; ++d)
#pragma unroll
      for (int t = 0; t < TC; ++t) {
        Sums<E> v = acc[m][d][t][0];
#pragma unroll
        for (int j = 1; j < G; ++j)
          if (g * 4 / RG == j) v = acc[m][d][t][j];
        *reinterpret_cast<Sums<E>*>(
            &red[wave * G + g * 4 / RG][d * TC + t][l][m * RG + g * 4 % RG]) = v;
      }
  __syncthreads();
  constexpr int ALL = KINDS * TC * 16 * RB;
  for (int i = tid; i < ALL; i += WAVES * 64) {
    S* f = &red[0][0][0][0] + i;
    S s = f[0];
#pragma unroll
    for (int w = 1; w < PARTS; ++w) s += f[w * ALL];
    f[0] = s;
  }
  __syncthreads();
  constexpr int RUNS = (RB + 7) / 8;
  if (tid < TC * 16 * RUNS) {
    const int c = tid / RUNS, rr = tid % RUNS * 8, r = r0 + rr;
    if (c < a.C && r < a.R) {
      LinEpilogue e = a.e;
      e.R = min(e.R, r0 + RB);
      float v[8], w[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < RB ? (float)red[0][c >> 4][c & 15][rr + q % RB] : 0.0f;
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = q < RB ? red[0][TC + (c >> 4)][c & 15][rr + q % RB] : 0.0f;
        finish_gated<E>(e, c, r, v, w);
      } else {
        if constexpr (EB == 1) finish_scaled<O>(e, c, r, v);
        else finish_linear<O>(e, 0, c, r, v);
      }
    }
  }
}

// Joins the planes of a split contraction in split order: 8 outputs a thread, 8
// planes' loads in flight: a round trip to planes that other XCDs wrote takes about a
// us, which bounds this.
template <typename E, bool GATED, typename S = float>
__device__ __forceinline__ void join(const JoinArgs& a, long long block) {
  constexpr int KINDS = GATED ? 2 : 1, B = GATED ? 4 : 8;
  const int per_row = (int)(a.plane_ld / 8);
  const long long id = block * 256 + threadIdx.x;
  const long long row = id / per_row;  // z * C + c
  if (row >= (long long)a.nz * a.C) return;
  const int r = (int)(id - row * per_row) * 8;
  const int z = (int)(row / a.C);
  const long long c = row - (long long)z * a.C;
  const float* s = a.planes + row * a.plane_ld + r;
  S v[8], u[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = u[q] = 0;
  typedef S V __attribute__((ext_vector_type(4)));
  for (int i = 0; i < a.splits; i += B) {
    V lo[KINDS][B], hi[KINDS][B];
#pragma unroll
    for (int p = 0; p < B; ++p)
#pragma unroll
      for (int d = 0; d < KINDS; ++d) {  // past the last plane: the last one again, not added
        const float* f = s + min(i + p, a.splits - 1) * a.plane_stride + d * (long long)a.C * a.plane_ld;
        lo[d][p] = *reinterpret_cast<const V*>(f);
        hi[d][p] = *reinterpret_cast<const V*>(f + 4);
      }
#pragma unroll
    for (int p = 0; p < B; ++p)
      if (i + p < a.splits) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] += lo[0][p][q];
          v[4 + q] += hi[0][p][q];
          u[q] += lo[KINDS - 1][p][q];
          u[4 + q] += hi[KINDS - 1][p][q];
        }
      }
  }
  if (r >= a.e.R) return;
  if constexpr (GATED) {
    finish_gated<E>(a.e, c, r, v, u);
  } else if constexpr (std::is_same_v<S, float>) {
    finish_linear<E>(a.e, z, c, r, v);
  } else {
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = (float)v[q];
    finish_scaled<E>(a.e, c, r, f);
  }
}

template <typename E, bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(const JoinArgs a) {
  join<E, GATED>(a, blockIdx.x);
}

// Planes of int32 sums (8-bit operands).
template <typename O>
__global__ __launch_bounds__(256) void linear_int8_join_kernel(const JoinArgs a) {
  join<O, false, int>(a, blockIdx.x);
}

template <typename E>
__global__ __launch_bounds__(256) void linear_join_pair_kernel(const JoinArgs a, const JoinArgs b,
                                                               int first) {
  if ((int)blockIdx.x < first) join<E, false>(a, blockIdx.x);
  else join<E, false>(b, (int)blockIdx.x - first);
}

unsigned join_blocks(const JoinArgs& a) {
  const long long items = (long long)a.nz * a.C * (a.plane_ld / 8);
  return (unsigned)((items + 255) / 256);
}

template <typename E, int TC, bool GATED, int G, int M, typename O>
hipError_t stream_g(const ProductArgs& a, bool vec, hipStream_t s) {
  const int rb = 16 * M / G;
  const dim3 grid((a.R + rb - 1) / rb), block(kStreamWaves * 64);
  if (vec) hipLaunchKernelGGL((linear_stream_kernel<E, TC, GATED, true, G, M, O>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((linear_stream_kernel<E, TC, GATED, false, G, M, O>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename E, int TC, bool GATED, typename O = E>
hipError_t stream_t(const ProductArgs& a, int rows, bool vec, hipStream_t s) {
  if constexpr (TC == 2)  // 32 weight rows share Q's loads, which 16 rows c do not need
    if (rows == 32) return stream_g<E, TC, GATED, 1, 2, O>(a, vec, s);
  if (rows == 16) return stream_g<E, TC, GATED, 1, 1, O>(a, vec, s);
  if (rows == 8) return stream_g<E, TC, GATED, 2, 1, O>(a, vec, s);
  return stream_g<E, TC, GATED, 4, 1, O>(a, vec, s);
}

}  // namespace

template <typename E>
hipError_t launch_stream(const ProductArgs& a, int blocks16, int rows, bool gated, bool vec,
                         hipStream_t s) {
  if (gated)
    return blocks16 == 1 ? stream_t<E, 1, true>(a, rows, vec, s)
                         : stream_t<E, 2, true>(a, rows, vec, s);
  return blocks16 == 1 ? stream_t<E, 1, false>(a, rows, vec, s)
                       : stream_t<E, 2, false>(a, rows, vec, s);
}

template <typename E>
hipError_t launch_join(const JoinArgs& a, bool gated, hipStream_t s) {
  const dim3 grid(join_blocks(a));
  if (gated) hipLaunchKernelGGL((linear_join_kernel<E, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((linear_join_kernel<E, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename O>
hipError_t launch_int8_stream(const ProductArgs& a, int blocks16, int rows, bool vec, hipStream_t s) {
  return blocks16 == 1 ? stream_t<signed char, 1, false, O>(a, rows, vec, s)
                       : stream_t<signed char, 2, false, O>(a, rows, vec, s);
}

template <typename O>
hipError_t launch_int8_join(const JoinArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((linear_int8_join_kernel<O>), dim3(join_blocks(a)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_join_pair(const JoinArgs& a, const JoinArgs& b, hipStream_t s) {
  const unsigned first = join_blocks(a);
  hipLaunchKernelGGL((linear_join_pair_kernel<E>), dim3(first + join_blocks(b)), dim3(256), 0, s, a, b,
                     (int)first);
  return hipGetLastError();
}

#define CONVFWD_INST(E)                                                                      \
  template hipError_t launch_stream<E>(const ProductArgs&, int, int, bool, bool, hipStream_t); \
  template hipError_t launch_join<E>(const JoinArgs&, bool, hipStream_t);                   \
  template hipError_t launch_join_pair<E>(const JoinArgs&, const JoinArgs&, hipStream_t);    \
  template hipError_t launch_int8_stream<E>(const ProductArgs&, int, int, bool, hipStream_t); \
  template hipError_t launch_int8_join<E>(const JoinArgs&, hipStream_t);
CONVFWD_INST(_Float16)
CONVFWD_INST(__bf16)
CONVFWD_INST(float)
#undef CONVFWD_INST

}  // namespace convfwd
