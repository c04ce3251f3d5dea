// Epilogue of the linear and gated products (include/linear.h): 8 consecutive
// outputs of one row at a time, from float32 sums, each step in float32 and one
// rounding where a value is stored.
#pragma once

#include <hip/hip_runtime.h>

#include "epilogue.h"
#include "linear_args.h"

namespace convfwd {

template <typename E>
struct Vec8 {
  static constexpr int N = (int)sizeof(E) / 2;  // 16-byte pieces
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  typedef E piece __attribute__((ext_vector_type(16 / sizeof(E))));
  static constexpr int W = 16 / (int)sizeof(E);
};

// Eight elements at p: two 16-byte pieces of float32, one of 16 bits.
template <typename E>
__device__ __forceinline__ void load8(const E* p, int nv, bool vec, float (&v)[8]) {
  using V = Vec8<E>;
  if (vec && nv == 8) {
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      const typename V::piece q = *reinterpret_cast<const typename V::piece*>(p + i * V::W);
#pragma unroll
      for (int e = 0; e < V::W; ++e) v[i * V::W + e] = (float)q[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < nv ? (float)p[e] : 0.0f;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, int nv, bool vec, const float (&v)[8]) {
  using V = Vec8<E>;
  if (vec && nv == 8) {
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
      typename V::piece q;
#pragma unroll
      for (int e = 0; e < V::W; ++e) q[e] = (E)v[i * V::W + e];
      *reinterpret_cast<typename V::piece*>(p + i * V::W) = q;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nv) p[e] = (E)v[e];
  }
}

// GELU, erf form.
__device__ __forceinline__ float gelu_erf(float v) {
  return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
}

// GELU, tanh form: v/2 (1 + tanh u) = v / (1 + e^-2u), which keeps the relative
// accuracy of the negative side that 1 + tanh u loses by cancellation.
template <bool FX>
__device__ __forceinline__ float gelu_tanh(float v) {
  const float u2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);  // 2 sqrt(2/pi) (..)
  if constexpr (FX) return v * logistic_fast(u2);
  return v / (1.0f + expf(-u2));
}

// Every activation of include/linear.h over a batch, one uniform branch.
template <bool FX, int N>
__device__ __forceinline__ void lin_act(float (&v)[N], int act, float alpha, float beta) {
  if (act < 9) {
    act_array<FX>(v, act, alpha, beta);
  } else if (act == 9) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu_erf(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu_tanh<FX>(v[i]);
  }
}

// Activation and its derivative at v (for the backward passes, 16-bit or float32).
__device__ __forceinline__ void act_and_slope(float v, int act, float alpha, float beta, float* a,
                                              float* d) {
  switch (act) {
    case 1: *a = v > 0.0f ? v : 0.0f; *d = v > 0.0f ? 1.0f : 0.0f; return;
    case 2: { const float t = tanhf(v); *a = t; *d = 1.0f - t * t; return; }
    case 3: { const float q = 1.0f / (1.0f + expf(-v)); *a = q; *d = q / (1.0f + expf(v)); return; }
    case 4: {
      const float q = 1.0f / (1.0f + expf(-v)), c = 1.0f / (1.0f + expf(v));
      *a = v * q; *d = q * (1.0f + v * c); return;
    }
    case 5: {
      const float u = alpha * v + beta;
      *a = fminf(fmaxf(u, 0.0f), 1.0f); *d = u > 0.0f && u < 1.0f ? alpha : 0.0f; return;
    }
    case 6:
      *a = v * fminf(fmaxf(v * (1.0f / 6.0f) + 0.5f, 0.0f), 1.0f);
      *d = v >= 3.0f ? 1.0f : v <= -3.0f ? 0.0f : v * (1.0f / 3.0f) + 0.5f;
      return;
    case 7: *a = fminf(fmaxf(v, alpha), beta); *d = v > alpha && v < beta ? 1.0f : 0.0f; return;
    case 8: *a = v >= 0.0f ? v : alpha * v; *d = v >= 0.0f ? 1.0f : alpha; return;
    case 9: {
      const float cdf = 0.5f * (1.0f + erff(v * 0.70710678118654752f));
      *a = v * cdf; *d = cdf + v * 0.39894228040143268f * expf(-0.5f * v * v); return;
    }
    case 10: {
      // with s = sigmoid(2u): gelu = v s, derivative s + v s (1 - s) 2u'
      const float u2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);
      const float s = 1.0f / (1.0f + expf(-u2)), c = 1.0f / (1.0f + expf(u2));
      *a = v * s;
      *d = s + v * s * c * 1.5957691216057308f * (1.0f + 0.134145f * v * v);
      return;
    }
    default: *a = v; *d = 1.0f;
  }
}

// Linear: v holds the sums of outputs (c, r .. r + nv - 1).
template <typename E>
__device__ __forceinline__ void finish_linear(const LinEpilogue& e, int z, long long c, int r,
                                              float (&v)[8]) {
  const int nv = min(8, e.R - r);
  const bool vec = e.vec;
  float t[8];
  if (e.bias[0]) {
    load8(static_cast<const E*>(e.bias[0]) + r, nv, vec, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
  if (e.res_mode != 0) load8(static_cast<const E*>(e.res) + c * e.ldres + r, nv, vec, t);
  if (e.res_mode == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
  if (e.save[0]) store8(static_cast<E*>(e.save[0]) + c * e.ldsave + r, nv, vec, v);
  lin_act<sizeof(E) == 2>(v, e.act, e.alpha, e.beta);
  if (e.res_mode == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
  store8(static_cast<E*>(e.out[z]) + c * e.ldo + r, nv, vec, v);
}

// Gated: g and u hold both projections' sums.
template <typename E>
__device__ __forceinline__ void finish_gated(const LinEpilogue& e, long long c, int r,
                                             float (&g)[8], float (&u)[8]) {
  const int nv = min(8, e.R - r);
  const bool vec = e.vec;
  if (e.bias[0]) {
    float t[8];
    load8(static_cast<const E*>(e.bias[0]) + r, nv, vec, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += t[i];
    load8(static_cast<const E*>(e.bias[1]) + r, nv, vec, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] += t[i];
  }
  if (e.save[0]) {
    store8(static_cast<E*>(e.save[0]) + c * e.ldsave + r, nv, vec, g);
    store8(static_cast<E*>(e.save[1]) + c * e.ldsave + r, nv, vec, u);
  }
  lin_act<sizeof(E) == 2>(g, e.act, e.alpha, e.beta);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= u[i];
  store8(static_cast<E*>(e.out[0]) + c * e.ldo + r, nv, vec, g);
}

}  // namespace convfwd
