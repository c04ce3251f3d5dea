// Epilogue of the linear and gated products (include/linear.h): 8 consecutive
// outputs of one row at a time, from float32 sums, each step in float32 and one
// rounding where a value is stored.
#pragma once

#include <hip/hip_runtime.h>

#include "epilogue.h"
#include "linear_args.h"

namespace convfwd {

// Eight elements at p, whatever its alignment (the card reads and writes 16 bytes at
// any element's address): two pieces of float32, one of 16 bits.  The last run of a
// row, nv < 8 of them, goes element by element.
template <typename E>
struct __attribute__((packed, aligned(sizeof(E)))) Eight {
  typedef E piece __attribute__((ext_vector_type(16 / sizeof(E))));
  piece q[sizeof(E) / 2];
};

template <typename E>
__device__ __forceinline__ void load8(const E* p, int nv, float (&v)[8]) {
  constexpr int W = 16 / (int)sizeof(E);
  if (nv >= 8) {
    const Eight<E> u = *reinterpret_cast<const Eight<E>*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)u.q[e / W][e % W];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < nv ? (float)p[e] : 0.0f;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, int nv, const float (&v)[8]) {
  constexpr int W = 16 / (int)sizeof(E);
  if (nv >= 8) {
    Eight<E> u;
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) {
      typename Eight<E>::piece q;
#pragma unroll
      for (int e = 0; e < W; ++e) q[e] = (E)v[i * W + e];
      u.q[i] = q;
    }
    *reinterpret_cast<Eight<E>*>(p) = u;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nv) p[e] = (E)v[e];
  }
}

// Phi(-|v|), the normal distribution function's tail, from erfc(x) = e^(-x^2) t P(t)
// with t = 1 / (1 + 0.38 x), x = |v| / sqrt 2; P's coefficients are a fit of least
// relative error (1.04e-6 for x in [0, 13], far into the tail), halved.  Together
// with the hardware's exp2 and reciprocal within 2e-6 of the value up to |v| = 4 and,
// by the rounding of the exponent, 4e-6 at 6 and 8e-6 at 13: below a 16-bit output's
// rounding.  14 operations for erff's 40 and more.
__device__ __forceinline__ float normal_tail_fast(float v) {
  const float a = fabsf(v), t = __builtin_amdgcn_rcpf(fmaf(0.26870058f, a, 1.0f));
  float p = -0.0627085285f;
  p = fmaf(p, t, 0.1680174795f);
  p = fmaf(p, t, -0.03495600065f);
  p = fmaf(p, t, 0.123917023f);
  p = fmaf(p, t, 0.0902971255f);
  p = fmaf(p, t, 0.1082887315f);
  p = fmaf(p, t, 0.107143653f);
  return p * t * __builtin_amdgcn_exp2f(-0.72134752f * a * a);
}

// The normal distribution function, from erfc: 1 + erf would cancel on the negative side
// (4% off at -5, 0 from -5.6 on).
__device__ __forceinline__ float normal_cdf(float v) {
  return 0.5f * erfcf(v * -0.70710678118654752f);
}

// GELU, erf form: v Phi(v); inf at infinity and, as the product says, NaN at -infinity.
template <bool FX>
__device__ __forceinline__ float gelu_erf(float v) {
  if constexpr (FX) {
    const float h = normal_tail_fast(v);
    return v < 0.0f ? v * h : v - fminf(v, 1e4f) * h;
  }
  return v * normal_cdf(v);
}

// tanh from the hardware's exp2 and reciprocal, by its series (to x^9) below 0.35
// where 1 - e^-2x would cancel: within 4e-7 of the value.
__device__ __forceinline__ float tanh_fast(float v) {
  const float a = fabsf(v), q = v * v;
  const float e = __builtin_amdgcn_exp2f(-2.885390082f * a);
  const float big = copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), v);
  float p = 0.0218694885f;
  p = fmaf(p, q, -0.0539682540f);
  p = fmaf(p, q, 0.1333333333f);
  p = fmaf(p, q, -0.3333333333f);
  return a < 0.35f ? fmaf(p * q, v, v) : big;
}

// GELU, tanh form: v/2 (1 + tanh u) = v / (1 + e^-2u), which keeps the relative
// accuracy of the negative side that 1 + tanh u loses by cancellation.
template <bool FX>
__device__ __forceinline__ float gelu_tanh(float v) {
  const float u2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);  // 2 sqrt(2/pi) (..)
  if constexpr (FX) return v * logistic_fast(u2);
  return v / (1.0f + expf(-u2));
}

// v between lo and hi; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float bounded(float v, float lo, float hi) {
  const float t = v < lo ? lo : v;
  return t > hi ? hi : t;
}

// Every activation of include/linear.h over a batch: one uniform branch, then 8
// values at a time (more of them side by side would cost registers).
template <bool FX, int N>
__device__ __forceinline__ void lin_act(float (&v)[N], int act, float alpha, float beta) {
  auto each = [&](auto f) {
#pragma unroll
    for (int n = 0; n < N; n += 8) {
#pragma unroll
      for (int i = n; i < n + 8; ++i) v[i] = f(v[i]);
      if (N > 8) __builtin_amdgcn_sched_barrier(0);
    }
  };
  switch (act) {
    case 1: each([&](float q) { return act_t<1, FX>(q, alpha, beta); }); break;
    case 2: each([&](float q) { return FX ? tanh_fast(q) : tanhf(q); }); break;
    case 3: each([&](float q) { return act_t<3, FX>(q, alpha, beta); }); break;
    case 4: each([&](float q) { return act_t<4, FX>(q, alpha, beta); }); break;
    case 5: each([&](float q) { return bounded(alpha * q + beta, 0.0f, 1.0f); }); break;
    case 6: each([&](float q) { return act_t<6, FX>(q, alpha, beta); }); break;
    case 7: each([&](float q) { return bounded(q, alpha, beta); }); break;
    case 8: each([&](float q) { return act_t<8, FX>(q, alpha, beta); }); break;
    case 9: each([&](float q) { return gelu_erf<FX>(q); }); break;
    case 10: each([&](float q) { return gelu_tanh<FX>(q); }); break;
    default: break;
  }
}

// Activation and its derivative at v, for the backward passes.  FX (16-bit
// gradients): the logistic function's two sides from one exponential of -|v| and one
// reciprocal, each to a few ulps of its own size, and normal_tail_fast.
template <bool FX>
__device__ __forceinline__ void logistic_sides(float v, float* q, float* c) {
  if constexpr (FX) {
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(v));
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    *q = v < 0.0f ? small : big;
    *c = v < 0.0f ? big : small;
  } else {
    *q = 1.0f / (1.0f + expf(-v));
    *c = 1.0f / (1.0f + expf(v));
  }
}

template <int ACT, bool FX>
__device__ __forceinline__ void act_and_slope(float v, float alpha, float beta, float* a, float* d) {
  if constexpr (ACT == 1) {
    *a = v > 0.0f ? v : 0.0f;
    *d = v > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == 2) {
    // 1 - tanh^2 as 4 sigmoid(2v) sigmoid(-2v): the difference cancels in float32, 3% of
    // its value at 7.5 and nearly all of it at 9
    float q, c;
    logistic_sides<FX>(2.0f * v, &q, &c);
    *a = FX ? tanh_fast(v) : tanhf(v);
    *d = 4.0f * q * c;
  } else if constexpr (ACT == 3) {
    float q, c;
    logistic_sides<FX>(v, &q, &c);
    *a = q;
    *d = q * c;
  } else if constexpr (ACT == 4) {
    float q, c;
    logistic_sides<FX>(v, &q, &c);
    *a = v * q;
    *d = q * (1.0f + v * c);
  } else if constexpr (ACT == 5) {
    const float u = alpha * v + beta;
    *a = bounded(u, 0.0f, 1.0f);
    *d = u > 0.0f && u < 1.0f ? alpha : 0.0f;
  } else if constexpr (ACT == 6) {
    *a = v * fminf(fmaxf(v * (1.0f / 6.0f) + 0.5f, 0.0f), 1.0f);
    *d = v >= 3.0f ? 1.0f : v <= -3.0f ? 0.0f : v * (1.0f / 3.0f) + 0.5f;
  } else if constexpr (ACT == 7) {
    *a = bounded(v, alpha, beta);
    *d = v > alpha && v < beta ? 1.0f : 0.0f;
  } else if constexpr (ACT == 8) {
    *a = v >= 0.0f ? v : alpha * v;
    *d = v >= 0.0f ? 1.0f : alpha;
  } else if constexpr (ACT == 9) {
    const float pdf = 0.39894228040143268f *
                      (FX ? __builtin_amdgcn_exp2f(-0.72134752f * v * v) : expf(-0.5f * v * v));
    float cdf;
    if constexpr (FX) {
      const float h = normal_tail_fast(v);
      cdf = v < 0.0f ? h : 1.0f - h;
    } else {
      cdf = normal_cdf(v);
    }
    *a = v * cdf;
    *d = cdf + v * pdf;
  } else if constexpr (ACT == 10) {
    // with q = sigmoid(2u): gelu = v q, derivative q + v q (1 - q) 2u'
    // (q (1 - q) is 0 long before v^2 overflows: the bound keeps 0 times it from NaN)
    float q, c;
    logistic_sides<FX>(1.5957691216057308f * (v + 0.044715f * v * v * v), &q, &c);
    *a = v * q;
    *d = q + v * (q * c) * 1.5957691216057308f * (1.0f + 0.134145f * fminf(v * v, 1e30f));
  } else {
    *a = v;
    *d = 1.0f;
  }
}

// Eight values behind one uniform branch: z becomes the derivative, f the activation.
template <bool FX>
__device__ __forceinline__ void acts_and_slopes(float (&z)[8], float (&f)[8], int act, float alpha,
                                                float beta) {
  switch (act) {
#define CONVFWD_CASE(A)                                                              \
  case A:                                                                            \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) {                                  \
      float d;                                                                       \
      act_and_slope<A, FX>(z[i], alpha, beta, &f[i], &d);                            \
      z[i] = d;                                                                      \
    }                                                                                \
    break;
    CONVFWD_CASE(0)
    CONVFWD_CASE(1)
    CONVFWD_CASE(2)
    CONVFWD_CASE(3)
    CONVFWD_CASE(4)
    CONVFWD_CASE(5)
    CONVFWD_CASE(6)
    CONVFWD_CASE(7)
    CONVFWD_CASE(8)
    CONVFWD_CASE(9)
    CONVFWD_CASE(10)
#undef CONVFWD_CASE
    default: break;
  }
}

// Two blocks of 16 r as the matrix cores leave them (lane (l, g): r = 4g .. 4g + 3 of
// column l) into runs of 8 consecutive r: lane (l, g) gets block g & 1 from r =
// 8 (g >> 1) on.  The odd quarter of the lanes of a changes places with the even
// quarter of b: four swaps between registers in place of a trip through LDS.
template <typename V>
__device__ __forceinline__ void runs_of_8(const V& a, const V& b, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float ai = a[i], bi = b[i];
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, ai),
                                                    __builtin_bit_cast(unsigned, bi), false, false);
    const unsigned lo = s[0], hi = s[1];
    v[i] = __builtin_bit_cast(float, lo);
    v[4 + i] = __builtin_bit_cast(float, hi);
  }
}
// The offset of a lane's run from the first block's first row.
__device__ __forceinline__ int run_offset(int lane) {
  return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
}

// Linear: v holds the sums of one row c, NR runs of 8 outputs at r + off(n).  whole
// (uniform): every run is inside; in: c is a row.  The runs' loads are in flight
// together and one branch picks the activation for all.
template <typename E, int NR, typename Off>
__device__ __forceinline__ void finish_linear_runs(const LinEpilogue& e, int z, long long c,
                                                   bool in, int r, Off off, bool whole,
                                                   float (&v)[NR * 8]) {
  auto add = [&](const void* from, long long at) {
    const E* p = static_cast<const E*>(from) + at + r;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float t[8];
      load8(p + off(n), whole ? 8 : e.R - r - off(n), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[n * 8 + i] += t[i];
    }
  };
  auto store = [&](void* to, long long at) {
    E* p = static_cast<E*>(to) + at + r;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[n * 8 + i];
      store8(p + off(n), whole ? 8 : e.R - r - off(n), t);
    }
  };
  if (e.bias[0]) add(e.bias[0], 0);
  if (e.res_mode == 1 && in) add(e.res, c * e.ldres);
  if (e.save[0] && in) store(e.save[0], c * e.ldsave);
  lin_act<sizeof(E) == 2>(v, e.act, e.alpha, e.beta);
  if (in) {
    if (e.res_mode == 2) add(e.res, c * e.ldres);
    store(e.out[z], c * e.ldo);
  }
}

// The sums as they are (gradients).
template <typename E, int NR, typename Off>
__device__ __forceinline__ void finish_plain_runs(const LinEpilogue& e, int z, long long c, int r,
                                                  Off off, bool whole, const float (&v)[NR * 8]) {
  E* p = static_cast<E*>(e.out[z]) + c * e.ldo + r;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[n * 8 + i];
    store8(p + off(n), whole ? 8 : e.R - r - off(n), t);
  }
}

template <typename E>
__device__ __forceinline__ void finish_linear(const LinEpilogue& e, int z, long long c, int r,
                                              float (&v)[8]) {
  finish_linear_runs<E, 1>(e, z, c, true, r, [](int) { return 0; }, false, v);
}

// Gated: g and u hold both projections' sums.
template <typename E, int NR, typename Off>
__device__ __forceinline__ void finish_gated_runs(const LinEpilogue& e, long long c, bool in, int r,
                                                  Off off, bool whole, float (&g)[NR * 8],
                                                  float (&u)[NR * 8]) {
  auto add = [&](const E* p, float (&v)[NR * 8]) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float t[8];
      load8(p + r + off(n), whole ? 8 : e.R - r - off(n), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[n * 8 + i] += t[i];
    }
  };
  auto store = [&](void* out, long long ld, const float (&v)[NR * 8]) {
    E* p = static_cast<E*>(out) + c * ld;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[n * 8 + i];
      store8(p + r + off(n), whole ? 8 : e.R - r - off(n), t);
    }
  };
  if (e.bias[0]) {
    add(static_cast<const E*>(e.bias[0]), g);
    add(static_cast<const E*>(e.bias[1]), u);
  }
  if (e.save[0] && in) {
    store(e.save[0], e.ldsave, g);
    store(e.save[1], e.ldsave, u);
  }
  lin_act<sizeof(E) == 2>(g, e.act, e.alpha, e.beta);
#pragma unroll
  for (int i = 0; i < NR * 8; ++i) g[i] *= u[i];
  if (in) store(e.out[0], e.ldo, g);
}

template <typename E>
__device__ __forceinline__ void finish_gated(const LinEpilogue& e, long long c, int r,
                                             float (&g)[8], float (&u)[8]) {
  finish_gated_runs<E, 1>(e, c, true, r, [](int) { return 0; }, false, g, u);
}

}  // namespace convfwd
