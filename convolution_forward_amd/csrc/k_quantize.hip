// Rows to 8 bits with a scale each (quantize_rows of include/linear_int8.h).
//
// The largest |x| of a row is found on its bits (the bits of finite values order as the
// values do; infinities and NaNs are above all of them and stay visible), then every
// element is scaled and rounded.  Rows up to 32768 elements are held in registers
// between the two (T threads, U runs of 8 each); longer ones are read twice.  Bound by
// memory: 2 or 4 bytes read and one written for an element; bfloat16 8192 x 11008 48 us,
// 5.6 TB/s, 8192 x 4096 20.  Rows at odd bytes cost: 8192 x 11007 66 us.  Short rows take
// 8 lanes: 4000000 x 9 104 us, where a wave a row took 903.
#include <algorithm>

#include "row_ops.h"
#include "rows_plan.h"

namespace convfwd {

namespace {

template <typename E>
struct QuantArgs {
  const E* x;
  signed char* q;
  float* scale;
  long long ldx, ldq;
  long long row0, m;
  int n;
};

template <int U>
__device__ __forceinline__ unsigned largest(const float (&v)[U][8]) {
  unsigned top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(unsigned, v[u][e]) & 0x7fffffffu);
  return top;
}

template <int T>
__device__ __forceinline__ unsigned row_max(unsigned v, unsigned* lds) {
  v = __builtin_bit_cast(unsigned, lanes_join<T < 64 ? T : 64>(__builtin_bit_cast(float, v), [](float a, float b) {
        return __builtin_bit_cast(float, max(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b)));
      }));
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v = max(v, lds[i]);
  }
  return v;
}

struct __attribute__((packed, aligned(1))) EightBytes {
  unsigned lo, hi;
};
struct __attribute__((packed, aligned(1))) FourBytes {
  unsigned v;
};
struct __attribute__((packed, aligned(1))) TwoBytes {
  unsigned short v;
};

template <int T, int U>
__device__ __forceinline__ void store_quantized(signed char* q, int n, int run0, float inv,
                                                const float (&v)[U][8]) {
  const int whole = n >> 3;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int run = run0 + u * T;
    unsigned w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      unsigned b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = (unsigned)(int)rintf(v[u][4 * h + e] * inv) & 0xffu;
      w[h] = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    }
    if (run < whole) {
      *reinterpret_cast<EightBytes*>(q + run * 8) = {w[0], w[1]};
    } else if (run == whole) {  // the pieces of a partial run
      const int left = n & 7;
      signed char* p = q + run * 8;
      if (left & 4) reinterpret_cast<FourBytes*>(p)->v = w[0];
      if (left & 2) reinterpret_cast<TwoBytes*>(p + (left & 4))->v = (unsigned short)w[1];
      if (left & 1) p[left & 6] = (signed char)(w[1] >> 16);
    }
  }
}

// The row's scale and the factor to whole numbers, from the bits of its largest |x|.
__device__ __forceinline__ void scales(unsigned top, float* scale, float* inv) {
  const float a = __builtin_bit_cast(float, top);
  if (top >= 0x7f800000u) {  // an infinity or a NaN
    *scale = __builtin_nanf("");
    *inv = 0.0f;
  } else if (a < 0x1p-100f) {
    *scale = *inv = 0.0f;
  } else {
    *scale = a / 127.0f;
    *inv = 127.0f / a;
  }
}

template <typename E, int T, int U, bool LONG>
__global__ __launch_bounds__(T* teams_of(T)) void quantize_kernel(const QuantArgs<E> a) {
  __shared__ unsigned lds[waves_of(T)];
  const int t = threadIdx.x % T;
  const long long row = a.row0 + (long long)blockIdx.x * teams_of(T) + team_of<T>();
  if (row >= a.m) return;
  const E* x = a.x + row * a.ldx;
  signed char* q = a.q + row * a.ldq;
  float v[U][8], scale, inv;
  load_runs<T>(x, a.n, t, v);
  unsigned top = largest(v);
  if constexpr (LONG) {
    for (int at = T * U; at * 8 < a.n; at += T * U) {
      load_runs<T>(x, a.n, at + t, v);
      top = max(top, largest(v));
    }
  }
  scales(row_max<T>(top, lds), &scale, &inv);
  if (t == 0) a.scale[row] = scale;
  // 0 times an infinity or a NaN would be a NaN: those rows are all 0
  const bool zero = inv == 0.0f;
  auto put = [&](int run0) {
    if (zero) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
    }
    store_quantized<T>(q, a.n, run0, inv, v);
  };
  if constexpr (LONG) {
    for (int at = 0; at * 8 < a.n; at += T * U) {
      load_runs<T>(x, a.n, at + t, v);
      put(at + t);
    }
  } else {
    put(t);
  }
}

template <typename E, int T, int U, bool LONG>
hipError_t launch(QuantArgs<E> a, hipStream_t s) {
  constexpr int TEAMS = teams_of(T);
  const long long most = rows_of_launch(T, TEAMS);
  for (long long at = 0; at < a.m; at += most) {
    a.row0 = at;
    const long long rows = std::min(most, a.m - at);
    hipLaunchKernelGGL((quantize_kernel<E, T, U, LONG>), dim3((unsigned)((rows + TEAMS - 1) / TEAMS)),
                       dim3(T * TEAMS), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename E>
int run(const quantize_problem* p, const QuantGeo& g, const void* x, void* q, void* scale,
        void* stream) {
  QuantArgs<E> a{};
  a.x = elements<E>(x, p->x_off);
  a.q = elements<signed char>(q, p->q_off);
  a.scale = elements<float>(scale, p->scale_off);
  a.ldx = g.ldx; a.ldq = g.ldq;
  a.m = g.m;
  a.n = (int)g.n;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const RowPlan& r = g.row;
  hipError_t e;
  if (r.threads == 8) e = launch<E, 8, 1, false>(a, s);
  else if (r.threads == 16) e = launch<E, 16, 1, false>(a, s);
  else if (r.threads == 32) e = launch<E, 32, 1, false>(a, s);
  else if (r.threads == 64) e = r.runs == 1 ? launch<E, 64, 1, false>(a, s) : launch<E, 64, 2, false>(a, s);
  else if (r.threads == 256) e = r.runs == 1 ? launch<E, 256, 1, false>(a, s) : launch<E, 256, 2, false>(a, s);
  else if (r.parts) e = launch<E, 1024, 4, true>(a, s);
  else if (r.runs == 1) e = launch<E, 1024, 1, false>(a, s);
  else if (r.runs == 2) e = launch<E, 1024, 2, false>(a, s);
  else e = launch<E, 1024, 4, false>(a, s);
  return e == hipSuccess ? CONV_OK : CONV_ERR_DEVICE;
}

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" int quantize_rows(const quantize_problem* p, int dtype, const void* x, void* q,
                             void* scale, void* stream) {
  QuantGeo g;
  const int st = quantize_checked(p, dtype, x, q, scale, &g);
  if (st) return st;
  if (dtype == CONV_F16) return run<_Float16>(p, g, x, q, scale, stream);
  if (dtype == CONV_BF16) return run<__bf16>(p, g, x, q, scale, stream);
  return run<float>(p, g, x, q, scale, stream);
}
