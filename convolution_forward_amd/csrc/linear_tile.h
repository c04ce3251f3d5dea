// Tiled matrix product on MFMA for gfx950: out[c][r] = sum_k P(r, k) Q(c, k),
// float32 sums, with the epilogue of linear_epilogue.h.  One kernel template for
// the linear layer, the gated projections and every gradient: each operand is
// k-major (rows run along the contraction) or transposed (rows of constant k).
//
//  * A workgroup owns BR x BC outputs; P rows feed MFMA's A operand and Q rows
//    its B operand, so a lane ends with 4 consecutive r of one c.
//  * Contraction step: 128 bytes of k (64 halves, 32 floats, 128 elements of 8 bits;
//    those are k-major only, with int32 sums and outputs of another type O).  Both operands are
//    staged in LDS, in two buffers (small tiles: three); the next step (two) is in
//    flight while one is multiplied.
//  * DMA: global to LDS directly (16 bytes a lane, no registers), for rows of
//    whole 16-byte pieces at multiples of 4 bytes; descriptor range checks give
//    zeros past the last row and, per lane, past the end of k.  Otherwise (odd
//    strides, sizes or bases) the pieces come through registers (Ragged).
//  * k-major image in LDS: 128-byte rows, 16-byte piece p of row i kept at slot
//    p ^ (i & 7): the 16 rows of a fragment read hit all banks.  Transposed
//    image: one row per k, kept as it lies, in 32-byte units (16 halves) moved to
//    unit u ^ h(k); fragments come out transposed by the LDS transpose read
//    (16-bit), or are read element by element (float32, 64-byte units).
//  * Epilogue from registers: 16 rows c at a time, one a lane, each lane's sums
//    exchanged into runs of 8 consecutive r (runs_of_8), so that loads and stores
//    are 16-byte pieces of rows.
//
// What bounds it: 128 x 128 the LDS (a wave's 64 x 64 reads 16 KB for 256 cycles of
// products), 64 x 64 the barrier and the loads' way, float32 the matrix cores.
// 2048 x 1024 x 1024 bf16 in 64 x 64: 11 us; 4096 x 4096 x 4096 float32 in 128 x 128:
// 986 us (139 TFLOP/s of the 157 that the card has), 4095 x 4097 x 4095 in 64 x 64,
// through registers, 1198.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_epilogue.h"
#include "mfma16.h"

namespace convfwd {

namespace lin {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kOob = (int)0x80000000;  // byte offset past every descriptor's range

__device__ __forceinline__ unsigned lds_addr(const void* p) {
  return (unsigned)(unsigned long long)(lds_char*)const_cast<void*>(p);
}

// Raw buffer descriptor over [p, p + bytes), wave-uniform.
__device__ __forceinline__ i32x4 make_rsrc(const char* p, long long bytes) {
  const unsigned long long v = reinterpret_cast<unsigned long long>(p);
  const int n = (int)min(max(bytes, 0LL), 0x7fffffffLL);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)v);
  r[1] = __builtin_amdgcn_readfirstlane((int)(v >> 32) & 0xffff);
  r[2] = __builtin_amdgcn_readfirstlane(n);
  r[3] = 0x00020000;
  return r;
}

// 16 bytes per lane from rsrc + voff to LDS at lds + 16 * lane (out of range:
// zeros).  Nothing is returned to registers; wait with vm_wait before reading.  The
// descriptor comes from scalar code: after a vector instruction that writes one of its
// registers the load would need five wait states, which the compiler does not know of.
__device__ __forceinline__ void dma16(i32x4 rsrc, int voff, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void vm_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
__device__ __forceinline__ void lds_wait() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Unit rotation h of the transposed image (see above): the rows 8g + i, i = 0 .. 3, of
// two lane groups g are read together, 32 bytes each, and should hit all banks.  Rows
// of 4 units start in either half of the banks by their parity.
template <typename E, int UNITS>
__device__ __forceinline__ int unit_xor(int k) {
  if constexpr (sizeof(E) == 4) return (k >> 2) & 3 & (UNITS - 1);
  if constexpr (UNITS == 4) return ((k >> 1) & 1) | ((k >> 2) & 2);
  return ((k & 3) | (((k >> 3) & 3) << 2)) & (UNITS - 1);
}

// One operand's tile: ROWS rows (r or c) x 128 bytes of k.
template <typename E, int ROWS, bool T, int NT>
struct Tile {
  static constexpr int EB = (int)sizeof(E);
  static constexpr int EPC = 16 / EB;              // elements per 16-byte piece
  static constexpr int BKE = 128 / EB;             // k per step
  static constexpr int ITEMS = ROWS * 8 / NT;      // pieces per thread
  static constexpr int ROWB = T ? ROWS * EB : 128; // bytes of an LDS row
  static constexpr int CPR = ROWB / 16;            // pieces per LDS row
  static constexpr int UNIT = EB == 2 ? 2 : 4;     // pieces per unit (transposed)
  static constexpr int UNITS = CPR / UNIT;
  static constexpr int BYTES = ROWS * 128;
  static_assert(ROWS * 8 % NT == 0, "whole pieces per thread");

  // LDS row and global piece (within the row) of item i
  static __device__ __forceinline__ void item(int i, int tid, int* row, int* piece) {
    const int q = i * NT + tid;
    const int lr = q / CPR, slot = q % CPR;
    *row = lr;
    if constexpr (T)
      *piece = (((slot / UNIT) ^ unit_xor<E, UNITS>(lr)) * UNIT) | (slot % UNIT);
    else
      *piece = slot ^ (lr & 7);
  }

  // A 16-row fragment at row0 (a multiple of 16), 64 bytes of k (16-bit: 32 k,
  // float32: 16 k; lane group g holds k 8g.. or 4g..; 8-bit: 64 k, 16g..), step half j.
  typedef std::conditional_t<EB == 1, i32x4, std::conditional_t<EB == 2, s16x8, f32x4>> Frag;
  static __device__ __forceinline__ Frag frag(const char* base, int row0, int j, int lane) {
    const int l = lane & 15, g = lane >> 4;
    if constexpr (!T) {
      return *reinterpret_cast<const Frag*>(base + (row0 + l) * 128 + (((4 * j + g) ^ (l & 7)) << 4));
    } else if constexpr (EB == 2) {
      const int i = l >> 2;
      const int u = (row0 / 16) ^ unit_xor<E, UNITS>(8 * g + i);
      const char* p = base + (32 * j + 8 * g + i) * ROWB + u * 32 + (l & 3) * 8;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)const_cast<char*>(p));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)const_cast<char*>(p + 4 * ROWB));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      Frag f;
      const int u = (row0 / 16) ^ (g & (UNITS - 1));
#pragma unroll
      for (int s = 0; s < 4; ++s)
        f[s] = *reinterpret_cast<const float*>(base + (16 * j + 4 * g + s) * ROWB + u * 64 + l * 4);
      return f;
    }
  }
};

// Sums of a 16 x 16 block: four a lane.
template <typename E>
using Sums = std::conditional_t<sizeof(E) == 1, i32x4, mfma_f32x4>;

template <typename E, typename F>
__device__ __forceinline__ Sums<E> multiply(const F& p, const F& q, Sums<E> c) {
  if constexpr (sizeof(E) == 1) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(p, q, c, 0, 0, 0);
  } else if constexpr (sizeof(E) == 2) {
    return mfma_16x16x32<E>(p, q, c);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(p[s], q[s], c, 0, 0, 0);
    return c;
  }
}

// Sums as floats for runs_of_8: integer sums by their values, or, raw, by their bits.
template <typename E>
__device__ __forceinline__ mfma_f32x4 as_floats(const Sums<E>& s, bool raw) {
  if constexpr (sizeof(E) == 1) {
    mfma_f32x4 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = s[i];
      f[i] = raw ? __builtin_bit_cast(float, v) : (float)v;
    }
    return f;
  } else {
    return s;
  }
}

// 16 bytes at base + off, aligned to their elements.  The card reads 16 bytes at a
// multiple of 4 at full speed, elsewhere at less than half: those come as the five
// words around them (a word that holds an element is on its page).  8 bits, streamed:
// 1 x 5632 x 2047 6.4 us (misaligned loads 9.0), 16 x 2048 x 5631 9.9 (17.5), 2 x 11008 x 4097
// 22.4 (32.2).  The 64 x 64 tiles measured the other way round and load as it lies (777 x
// 1001 x 1531 12.6 us, joined words 17).
template <typename E>
__device__ __forceinline__ i32x4 load_piece(const char* base, int off) {
  typedef i32x4 A4 __attribute__((aligned(4)));
  if constexpr (sizeof(E) == 4) {
    return *reinterpret_cast<const A4*>(base + off);
  } else {
    constexpr int PAST = 4 - (int)sizeof(E);  // largest distance from a multiple of 4
    const int odd = ((int)reinterpret_cast<unsigned long long>(base) + off) & PAST;
    const i32x4 v = *reinterpret_cast<const A4*>(base + (off - odd));
    const int last = sizeof(E) == 2 ? off + odd + 12 : off - odd + (odd ? 16 : 12);
    const int w = *reinterpret_cast<const int*>(base + last);
    i32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = (int)__builtin_amdgcn_alignbyte((unsigned)(i < 3 ? v[i < 3 ? i + 1 : 3] : w), (unsigned)v[i], odd);
    return o;
  }
}

// Pieces of operands whose rows start anywhere (odd strides, sizes or bases), loaded
// into registers.  raw: the 16 bytes at the piece, moved back where it would pass the
// end of its row and to the last row where there is no such row, so that every load
// is inside the operand and none waits for a branch.  fix: those bytes as the piece:
// elements past an end are zeros.  (A row past the last r or c is whatever raw gave:
// its outputs are not stored.)  Rows shorter than a piece go element by element.
template <typename E, bool T>
struct Ragged {
  static constexpr int EPC = 16 / (int)sizeof(E);
  struct __attribute__((packed, aligned(sizeof(E)))) P { i32x4 v; };

  // The byte offset of a piece's load where the step has all its k.
  static __device__ __forceinline__ int at(long long ld, int row, int piece, long long nrow) {
    const int r = T ? row : (int)min((long long)row, nrow - 1);
    const int c = T ? (int)min((long long)piece * EPC, nrow - EPC) : piece * EPC;
    return (int)(r * ld + c) * (int)sizeof(E);
  }
  static __device__ __forceinline__ i32x4 raw(const E* base, long long ld, int row, int piece,
                                              long long nrow, long long nk, bool tiny) {
    const int len = (int)min(T ? nrow : nk, 1LL << 20), rows = (int)min(T ? nk : nrow, 256LL);
    const int at = piece * EPC;
    const E* p = base + (long long)min(row, rows - 1) * ld;
    if (!tiny) return reinterpret_cast<const P*>(p + min(at, len - EPC))->v;
    union { E e[EPC]; i32x4 v; } u;
#pragma unroll
    for (int i = 0; i < EPC; ++i) u.e[i] = at + i < len ? p[at + i] : (E)0.0f;
    return u.v;
  }
  // The elements of a piece that lies partly past len, loaded so that it ends there.
  template <typename V>
  static __device__ __forceinline__ V shift(V v, int piece, int len) {
    const int past = min(max(piece * EPC + EPC - len, 0), EPC), s = past * (int)sizeof(E) * 8;
    typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
    const u64x2 u = __builtin_bit_cast(u64x2, v);
    const unsigned long long a = u[0], b = u[1];
    u64x2 o;
    o[0] = s == 0 ? a : s < 64 ? (a >> s) | (b << (64 - s)) : s < 128 ? b >> (s - 64) : 0;
    o[1] = s < 64 ? b >> s : 0;
    return __builtin_bit_cast(V, o);
  }
  static __device__ __forceinline__ i32x4 fix(i32x4 v, int row, int piece, long long nrow,
                                              long long nk, bool tiny) {
    if (!tiny) v = shift(v, piece, (int)min(T ? nrow : nk, 1LL << 20));
    return T && row >= nk ? i32x4{0, 0, 0, 0} : v;
  }
};

}  // namespace lin

// WVR x WVC waves; GATED: P's rows are gate and up rows, side by side within
// each wave's share.  O: the outputs' type.
template <typename E, bool PT, bool QT, int BR, int BC, int WVR, int WVC, bool DMA, bool GATED,
          typename O = E>
struct LinearTile {
  static constexpr int NT = WVR * WVC * 64;
  static constexpr int STAGE = lin::Tile<E, BR, PT, NT>::BYTES + lin::Tile<E, BC, QT, NT>::BYTES;
  // small tiles: buffers for two steps ahead (a step's products are shorter than a
  // load's way); large ones: two buffers, so that two workgroups fit on a compute unit
  static constexpr int STAGES = DMA && BR * BC <= 64 * 64 ? 3 : 2;
  static constexpr int SMEM = STAGES * STAGE;

// id: index of this workgroup among the product's own, after xcd_logical
static __device__ __forceinline__ void run(const ProductArgs& a, const int id, char* smem) {
  using namespace lin;
  constexpr int WR = BR / WVR, WC = BC / WVC, NI = WR / 16, NJ = WC / 16;
  constexpr int HW = WR / 2;  // gated: rows of each kind per wave
  using TP = Tile<E, BR, PT, NT>;
  using TQ = Tile<E, BC, QT, NT>;
  static_assert(!GATED || (!PT && !QT), "gated weights are k-major");
  static_assert(sizeof(E) > 1 || (!GATED && !PT && !QT), "8-bit operands are k-major");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave % WVR, wc = wave / WVR;

  // tile of this workgroup: bands of 8 tiles along c, so that the tiles an XCD
  // runs at one time share few rows of P and Q
  const int per = a.ntr * a.ntc;
  const int batch = id / per;  // split * nz + z
  const int z = batch % a.nz, split = batch / a.nz;
  const int idx = id - batch * per;
  const int band = idx / (8 * a.ntr), bw = min(8, a.ntc - 8 * band);
  const int in = idx - band * 8 * a.ntr;
  const int tr = in / bw, tc = 8 * band + in - tr * bw;
  const int r0 = tr * (GATED ? BR / 2 : BR);
  const long long c0 = (long long)tc * BC;
  const long long nr = a.R - r0, nc = a.C - c0;  // rows left

  const int t_all = a.ktiles * a.nseg;
  const int t0 = split * a.per_split, t1 = min(t0 + a.per_split, t_all);

  Sums<E> acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = Sums<E>{0, 0, 0, 0};

  // byte offsets of this thread's pieces, constant over the contraction; the piece's
  // k, alike for all
  int poff[TP::ITEMS], qoff[TQ::ITEMS], pk, qk;
#pragma unroll
  for (int i = TP::ITEMS - 1; i >= 0; --i) {
    int row, piece;
    TP::item(i, tid, &row, &piece);
    if constexpr (GATED) row = (row / WR) * HW + row % HW;
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
  const unsigned lds0 = lds_addr(smem);

  auto bases = [&](int t, const char** p0, const char** p1, const char** q, int* kk) {
    const int seg = t >= a.ktiles ? 1 : 0;
    const int k0 = (t - seg * a.ktiles) * TP::BKE;
    const long long po = PT ? k0 * a.ldp + r0 : r0 * a.ldp + k0;
    const long long qo = QT ? k0 * a.ldq + c0 : c0 * a.ldq + k0;
    *p0 = static_cast<const char*>(a.P[GATED ? 0 : seg]) + po * TP::EB;
    *p1 = GATED ? static_cast<const char*>(a.P[1]) + po * TP::EB : *p0;
    *q = static_cast<const char*>(a.Q[seg | z]) + qo * TP::EB;
    *kk = a.K - k0;  // k left in this segment
  };

  auto compute = [&](const char* buf) {
    const char* pb = buf;
    const char* qb = buf + TP::BYTES;
#pragma unroll
    for (int j2 = 0; j2 < 2; ++j2) {
      typename TP::Frag p[NI];
      typename TQ::Frag q[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) q[j] = TQ::frag(qb, wc * WC + j * 16, j2, lane);
#pragma unroll
      for (int i = 0; i < NI; ++i) p[i] = TP::frag(pb, wr * WR + i * 16, j2, lane);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = multiply<E>(p[i], q[j], acc[i][j]);
    }
  };

  if constexpr (DMA) {
    // What the next step's loads need, moved on by additions after each.  A descriptor
    // ends with the last valid row (transposed: the last valid k; a padded operand's
    // last piece is filled with zeros), so that everything past an end reads as zeros.
    constexpr int EB = TP::EB, EPC = TP::EPC, BKE = TP::BKE;
    const int ldpb = (int)a.ldp * EB, ldqb = (int)a.ldq * EB;
    const long long pstep = PT ? (long long)BKE * ldpb : 128, qstep = QT ? (long long)BKE * ldqb : 128;
    auto up = [](int n) { return (n + EPC - 1) / EPC * EPC * EB; };
    const int np = (int)min(nr, (long long)(GATED ? BR / 2 : BR)), nq = (int)min(nc, (long long)BC);
    const int pspan = PT ? up(np) : (np - 1) * ldpb, qspan = QT ? up(nq) : (nq - 1) * ldqb;
    const char *pp, *pu, *qq;
    int left;
    auto start = [&](int t) {
      bases(t, &pp, &pu, &qq, &left);
    };
    int at = t0;
    start(t0);
    const int ktail = a.K - (a.K - 1) / BKE * BKE;  // k of a segment's last step
    const bool ptail = PT || pk < ktail, qtail = QT || qk < ktail;
    auto issue = [&](int b) {
      const int kv = min(left, BKE);
      const i32x4 rp0 = make_rsrc(pp, pspan + (PT ? (kv - 1) * ldpb : up(kv)));
      const i32x4 rp1 = GATED ? make_rsrc(pu, pspan + up(kv)) : rp0;
      const i32x4 rq = make_rsrc(qq, qspan + (QT ? (kv - 1) * ldqb : up(kv)));
      const unsigned lp = lds0 + b * STAGE + wave * 1024, lq = lp + TP::BYTES;
      const bool pall = left >= BKE || ptail, qall = left >= BKE || qtail;
#pragma unroll
      for (int i = 0; i < TP::ITEMS; ++i) {
        const bool up_row = GATED && ((i * (NT / 8) + wave * 8) % WR) >= HW;
        dma16(up_row ? rp1 : rp0, pall ? poff[i] : kOob, lp + i * NT * 16);
      }
#pragma unroll
      for (int i = 0; i < TQ::ITEMS; ++i) dma16(rq, qall ? qoff[i] : kOob, lq + i * NT * 16);
      ++at;
      pp += pstep;
      pu += pstep;
      qq += qstep;
      left -= BKE;
      if (a.nseg > 1 && at == a.ktiles) start(at);  // the second segment
    };
    constexpr int LOADS = TP::ITEMS + TQ::ITEMS;
    if constexpr (STAGES > 2) {
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i)
        if (t0 + i < t1) issue(i);
      int b = 0;
      for (int t = t0; t < t1; ++t) {
        if (t + STAGES - 2 < t1) vm_wait<(STAGES - 2) * LOADS>();
        else vm_wait<0>();
        lds_wait();
        barrier();  // step t is staged, and every wave is done with step t - 1's buffer
        if (t + STAGES - 1 < t1) issue(b == 0 ? STAGES - 1 : b - 1);
        compute(smem + b * STAGE);
        b = b == STAGES - 1 ? 0 : b + 1;
      }
    } else {
      int b = 0;
      if (t0 < t1) issue(0);
      for (int t = t0; t < t1; ++t) {
        if (t + 1 < t1) {
          issue(b ^ 1);
          vm_wait<LOADS>();
        } else {
          vm_wait<0>();
        }
        barrier();
        compute(smem + b * STAGE);
        lds_wait();
        barrier();
        b ^= 1;
      }
    }
  } else {
    i32x4 pv[TP::ITEMS], qv[TQ::ITEMS];
    using RP = Ragged<E, PT>;
    using RQ = Ragged<E, QT>;
    const bool ptiny = (PT ? a.R : a.K) < TP::EPC, qtiny = (QT ? a.C : a.K) < TQ::EPC;
    // byte offsets from a step's first element, alike for all steps of whole k
    int pat[TP::ITEMS], qat[TQ::ITEMS];
#pragma unroll
    for (int i = 0; i < TP::ITEMS; ++i) {
      int row, piece;
      TP::item(i, tid, &row, &piece);
      if constexpr (GATED) row = (row / WR) * HW + row % HW;
      pat[i] = RP::at(a.ldp, row, piece, nr);
    }
#pragma unroll
    for (int i = 0; i < TQ::ITEMS; ++i) {
      int row, piece;
      TQ::item(i, tid, &row, &piece);
      qat[i] = RQ::at(a.ldq, row, piece, nc);
    }
    auto fetch = [&](int t) {
      const char *p0, *p1, *q;
      int kk;
      bases(t, &p0, &p1, &q, &kk);
      if (kk >= TP::BKE && !ptiny && !qtiny) {
#pragma unroll
        for (int i = 0; i < TP::ITEMS; ++i) {
          const bool up = GATED && ((i * (NT / 8) + wave * 8) % WR) >= HW;
          pv[i] = reinterpret_cast<const typename RP::P*>((up ? p1 : p0) + pat[i])->v;
        }
#pragma unroll
        for (int i = 0; i < TQ::ITEMS; ++i)
          qv[i] = reinterpret_cast<const typename RQ::P*>(q + qat[i])->v;
        return;
      }
#pragma unroll
      for (int i = 0; i < TP::ITEMS; ++i) {
        int row, piece;
        TP::item(i, tid, &row, &piece);
        const char* base = p0;
        if constexpr (GATED) {
          if (row % WR >= HW) base = p1;
          row = (row / WR) * HW + row % HW;
        }
        pv[i] = RP::raw(reinterpret_cast<const E*>(base), a.ldp, row, piece, nr, kk, ptiny);
      }
#pragma unroll
      for (int i = 0; i < TQ::ITEMS; ++i) {
        int row, piece;
        TQ::item(i, tid, &row, &piece);
        qv[i] = RQ::raw(reinterpret_cast<const E*>(q), a.ldq, row, piece, nc, kk, qtiny);
      }
    };
    auto put = [&](int t, int b) {
      const int kk = a.K - (t - (t >= a.ktiles ? a.ktiles : 0)) * TP::BKE;
      if (kk < TP::BKE || (PT && nr < BR)) {
#pragma unroll
        for (int i = 0; i < TP::ITEMS; ++i) {
          int row, piece;
          TP::item(i, tid, &row, &piece);
          pv[i] = RP::fix(pv[i], row, piece, nr, kk, ptiny);
        }
      }
      if (kk < TP::BKE || (QT && nc < BC)) {
#pragma unroll
        for (int i = 0; i < TQ::ITEMS; ++i) {
          int row, piece;
          TQ::item(i, tid, &row, &piece);
          qv[i] = RQ::fix(qv[i], row, piece, nc, kk, qtiny);
        }
      }
      char* d = smem + b * STAGE;
#pragma unroll
      for (int i = 0; i < TP::ITEMS; ++i) *reinterpret_cast<i32x4*>(d + (i * NT + tid) * 16) = pv[i];
#pragma unroll
      for (int i = 0; i < TQ::ITEMS; ++i)
        *reinterpret_cast<i32x4*>(d + TP::BYTES + (i * NT + tid) * 16) = qv[i];
    };
    int b = 0;
    if (t0 < t1) {
      fetch(t0);
      put(t0, 0);
    }
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) fetch(t + 1);
      lds_wait();
      barrier();  // step t is staged; buffer b ^ 1 was last read before this
      compute(smem + b * STAGE);
      if (t + 1 < t1) put(t + 1, b ^ 1);
      b ^= 1;
    }
  }

  // epilogue: 16 rows c at a time, one a lane, its outputs in runs of 8
  constexpr int RUN = GATED ? HW : WR;  // outputs of a wave's row and kind
  constexpr int NR = RUN / 32;
  auto off = [](int n) { return n * 32; };
  const int rl = r0 + wr * RUN + run_offset(lane);
  const bool whole = nr >= WVR * RUN;
  ScaledColumns<O, sizeof(E) == 1 ? NR : 1> cols;
  if constexpr (sizeof(E) == 1)
    if (a.splits == 1) cols.load(a.e, rl, off, whole);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    float v[NR * 8], u[GATED ? NR * 8 : 1];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      runs_of_8(as_floats<E>(acc[2 * i][j], a.splits > 1),
                as_floats<E>(acc[2 * i + 1][j], a.splits > 1), v + i * 8);
      if constexpr (GATED) runs_of_8(acc[NI / 2 + 2 * i][j], acc[NI / 2 + 2 * i + 1][j], u + i * 8);
    }
    const long long c = c0 + wc * WC + j * 16 + (lane & 15);
    const bool in = c < a.C;
    if (a.splits > 1) {
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
    } else if constexpr (GATED) {
      finish_gated_runs<E, NR>(a.e, c, in, rl, off, whole, v, u);
    } else if constexpr (sizeof(E) == 1) {
      finish_scaled_runs<O, NR>(a.e, cols, in ? a.e.xs[c] : 0.0f, c, in, rl, off, whole, v);
    } else {
      finish_linear_runs<O, NR>(a.e, z, c, in, rl, off, whole, v);
    }
  }
}
};

template <typename E, bool PT, bool QT, int BR, int BC, int WVR, int WVC, bool DMA, bool GATED,
          typename O = E>
__global__ __launch_bounds__(WVR * WVC * 64) void linear_tile_kernel(const ProductArgs a) {
  using K = LinearTile<E, PT, QT, BR, BC, WVR, WVC, DMA, GATED, O>;
  __shared__ __attribute__((aligned(1024))) char smem[K::SMEM];
  K::run(a, xcd_logical(blockIdx.x, gridDim.x), smem);
}

// Both products of a small backward pass in one launch (see linear_pair_kernel), each
// with its own splits.
template <typename E, bool DT>
__global__ __launch_bounds__(256) void linear_tile_pair_kernel(const PairArgs a) {
  using DX = LinearTile<E, DT, false, 64, 64, 2, 2, true, false>;
  using DW = LinearTile<E, true, true, 64, 64, 2, 2, true, false>;
  static_assert(DX::SMEM == DW::SMEM, "one buffer for both");
  __shared__ __attribute__((aligned(1024))) char smem[DX::SMEM];
  const bool second = (int)blockIdx.x >= a.first;
  const int id = second ? xcd_logical(blockIdx.x - a.first, gridDim.x - a.first)
                        : xcd_logical(blockIdx.x, a.first);
  if (second != a.dw_first) DW::run(a.dw, id, smem);
  else DX::run(a.dx, id, smem);
}

}  // namespace convfwd
