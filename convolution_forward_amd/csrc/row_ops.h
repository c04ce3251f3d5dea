// Device pieces shared by the row operators: sums over the threads of a row, and the
// dropout mask (include/dropout.h).  A row is cut into runs of 8 consecutive elements;
// run i of a row belongs to thread i mod T of the T threads that hold it.
#pragma once

#include <hip/hip_runtime.h>

#include "linear_epilogue.h"

namespace convfwd {

// v joined over the T = 8, 16, 32 or 64 neighbouring lanes of a row by f, the same in all
// of them: lanes paired by 1, 2, and mirrored halves and rows of 16, then lane swaps
// between rows of 16; no LDS.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               0xf, 0xf, true));
}
template <int T, typename F>
__device__ __forceinline__ float lanes_join(float v, F f) {
  static_assert(T == 8 || T == 16 || T == 32 || T == 64, "lanes of a row");
  v = f(v, dpp<0xB1>(v));   // lane ^ 1
  v = f(v, dpp<0x4E>(v));   // lane ^ 2
  v = f(v, dpp<0x141>(v));  // mirrored within 8
  if constexpr (T >= 16) v = f(v, dpp<0x140>(v));  // mirrored within 16
  if constexpr (T >= 32) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned a0 = a[0], a1 = a[1];
    v = f(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
  }
  if constexpr (T >= 64) {
    const unsigned w = __builtin_bit_cast(unsigned, v);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const unsigned b0 = b[0], b1 = b[1];
    v = f(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
  }
  return v;
}
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_join<T>(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }

// Sum over the T threads that hold a row (T <= 64: lanes of a wave, no barrier; more: a
// whole workgroup).  Two calls in turn need two arrays: a wave may be a call ahead,
// never two.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  if constexpr (T <= 64) {
    return lanes_sum<T>(v);
  } else {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += lds[i];
    return v;
  }
}

// Which of a workgroup's rows a thread works on; the same in a wave where it can be.
template <int T>
__device__ __forceinline__ int team_of() {
  const int team = threadIdx.x / T;
  return T >= 64 ? __builtin_amdgcn_readfirstlane(team) : team;
}
constexpr int teams_of(int threads) { return threads >= 256 ? 1 : 256 / threads; }
constexpr int waves_of(int threads) { return threads > 64 ? threads / 64 : 1; }

// The numbers of a mask, see include/dropout.h.
struct DropArgs {
  unsigned threshold;  // 0: no dropout
  float scale;
  unsigned key0, key1;
  unsigned long long offset;
  const unsigned long long* step;
};

struct DropCounter {
  unsigned lo, hi;
};
__device__ __forceinline__ DropCounter drop_counter(const DropArgs& a) {
  const unsigned long long c = a.offset + (a.step ? *a.step : 0);
  return {(unsigned)c, (unsigned)(c >> 32)};
}

__device__ __forceinline__ unsigned xor3(unsigned a, unsigned b, unsigned c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Philox4x32-10: 8 numbers of 16 bits for run `run` of row `row`.  20 products of 32
// bits (low and high half from one instruction) and 20 logic operations for 8 elements.
struct DropBits {
  unsigned w[4];
};
__device__ __forceinline__ DropBits drop_bits(const DropArgs& a, DropCounter c, unsigned run,
                                              unsigned row) {
  unsigned x0 = run, x1 = row, x2 = c.lo, x3 = c.hi, k0 = a.key0, k1 = a.key1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long p = (unsigned long long)x0 * 0xD2511F53u;
    const unsigned long long q = (unsigned long long)x2 * 0xCD9E8D57u;
    x0 = xor3((unsigned)(q >> 32), x1, k0);
    x1 = (unsigned)q;
    x2 = xor3((unsigned)(p >> 32), x3, k1);
    x3 = (unsigned)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{x0, x1, x2, x3}};
}

__device__ __forceinline__ bool drop_keeps(const DropBits& b, int e, unsigned threshold) {
  const unsigned u = e & 1 ? b.w[e >> 1] >> 16 : b.w[e >> 1] & 0xffffu;
  return u >= threshold;
}

// left: elements of the row from the run on; below 8 they lie in a partial run's slots.
__device__ __forceinline__ void drop8(const DropArgs& a, DropCounter c, unsigned run, unsigned row,
                                      int left, float (&v)[8]) {
  DropBits b = drop_bits(a, c, run, row);
  if (left < 8) {
    const unsigned w0 = b.w[0], w1 = b.w[1], w2 = b.w[2], w3 = b.w[3];
    b.w[2] = left & 4 ? w2 : w0;
    b.w[3] = left & 4 ? (left & 2 ? w3 : w2) : left & 2 ? w1 : w0;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = drop_keeps(b, e, a.threshold) ? v[e] * a.scale : 0.0f;
}

// Host side: the numbers of a problem.
inline DropArgs drop_args(int threshold, uint64_t seed, uint64_t offset, const void* step) {
  DropArgs a;
  a.threshold = (unsigned)threshold;
  a.scale = threshold < 65536 ? (float)(65536.0 / (65536 - threshold)) : 0.0f;
  a.key0 = (unsigned)seed;
  a.key1 = (unsigned)(seed >> 32);
  a.offset = offset;
  a.step = static_cast<const unsigned long long*>(step);
  return a;
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// A run of 8 elements in memory as it is held: two pieces of 16 bytes of float32, one of
// 16 bits, from any element's address on.
template <typename E>
__device__ __forceinline__ void unpack(const Eight<E>& q, float (&v)[8]) {
  constexpr int W = 16 / (int)sizeof(E);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)q.q[e / W][e % W];
}

// A few elements at any element's address.
template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Few {
  typedef E vec __attribute__((ext_vector_type(N)));
  vec v;
};

// The last, partial run of a row, 1 <= left <= 7 elements at p, in pieces of 4, 2 and 1
// (nothing past the end is touched).  The pieces have slots of their own among a run's 8:
// 0 .. 3, 4 and 5, and 6; slots without an element hold zeros.  Nothing that is done to a
// row depends on where in the run an element lies, but for the mask (drop8).
template <typename E>
__device__ __forceinline__ void fetch_tail(const E* p, int left, Eight<E>& q) {
  constexpr int W = 16 / (int)sizeof(E);
  if (left & 4) {
    const auto f = reinterpret_cast<const Few<E, 4>*>(p)->v;
#pragma unroll
    for (int e = 0; e < 4; ++e) q.q[0][e] = f[e];
  }
  if (left & 2) {
    const auto f = reinterpret_cast<const Few<E, 2>*>(p + (left & 4))->v;
    q.q[4 / W][4 % W] = f[0];
    q.q[5 / W][5 % W] = f[1];
  }
  if (left & 1) {
    if constexpr (sizeof(E) == 2) {  // a word of its own: nothing to join before it is used
      u32x4 w = __builtin_bit_cast(u32x4, q);
      w[3] = *reinterpret_cast<const unsigned short*>(p + (left & 6));
      q = __builtin_bit_cast(Eight<E>, w);
    } else {
      q.q[6 / W][6 % W] = p[left & 6];
    }
  }
}
// Whether slot e of a partial run holds an element.
__device__ __forceinline__ bool in_tail(int e, int left) {
  return e < 4 ? left & 4 : e < 6 ? left & 2 : e == 6 ? left & 1 : false;
}
template <typename E>
__device__ __forceinline__ void store_tail(E* p, int left, const float (&v)[8]) {
  if (left & 4) {
    typename Few<E, 4>::vec f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (E)v[e];
    reinterpret_cast<Few<E, 4>*>(p)->v = f;
  }
  if (left & 2) {
    typename Few<E, 2>::vec f;
    f[0] = (E)v[4];
    f[1] = (E)v[5];
    reinterpret_cast<Few<E, 2>*>(p + (left & 4))->v = f;
  }
  if (left & 1) p[left & 6] = (E)v[6];
}

// Runs run0, run0 + T, .. of a row of n elements, as they lie in memory: fetched ahead of
// their use.  Runs past the end stay as they were made: zeros.  (16-bit rows at odd
// elements are loaded as they lie, which costs: bfloat16 16384 x 2047 forward 39 us, backward
// 68, where 2046 takes 30 and 48, 2048 27 and 47.  Aligned words and a lane exchange in their
// place took 49 and 54.)
template <typename E, int T, int U>
struct Runs {
  Eight<E> q[U];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = Eight<E>{};
  }
  __device__ __forceinline__ void fetch(const E* p, int n, int run0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (run0 + u * T < (n >> 3)) q[u] = *reinterpret_cast<const Eight<E>*>(p + (run0 + u * T) * 8);
    if (n & 7) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (run0 + u * T == (n >> 3)) fetch_tail(p + (n & ~7), n & 7, q[u]);
    }
  }
  __device__ __forceinline__ void get(float (&v)[U][8]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) unpack(q[u], v[u]);
  }
};
template <int T, int U, typename E>
__device__ __forceinline__ void load_runs(const E* p, int n, int run0, float (&v)[U][8]) {
  Runs<E, T, U> r;
  r.clear();
  r.fetch(p, n, run0);
  r.get(v);
}
template <int T, int U, typename E>
__device__ __forceinline__ void store_runs(E* p, int n, int run0, const float (&v)[U][8]) {
  const int whole = n >> 3;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (run0 + u * T < whole) store8(p + (run0 + u * T) * 8, 8, v[u]);
  if (n & 7) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (run0 + u * T == whole) store_tail(p + whole * 8, n & 7, v[u]);
  }
}

template <typename E>
inline const E* elements(const void* p, int64_t off) {
  return p ? static_cast<const E*>(p) + off : nullptr;
}
template <typename E>
inline E* elements(void* p, int64_t off) {
  return p ? static_cast<E*>(p) + off : nullptr;
}

}  // namespace convfwd
