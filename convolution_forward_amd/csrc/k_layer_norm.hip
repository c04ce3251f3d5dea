// Layer norm forward (include/layer_norm.h), with the dropout and the residual before
// it: one read of x and r, one write of y and s.
//
// Rows up to 32768 elements are held in registers by T threads, U runs of 8 each, so
// that mean and variance are two sums over registers (the second of squared distances,
// which does not cancel).  Short rows take 8 to 64 lanes of a wave, several to a
// workgroup, with no barrier.  Longer rows go in two launches: a mean and a sum of
// squared distances for each part of 4096 elements, then every part joins those of its
// row (Chan, Golub and LeVeque's formula for the variance of joined samples) and
// normalises.
//
// Bound by memory where there are many rows: bfloat16 8192 x 4096 with dropout, residual
// and s 49 us, 5.5 TB/s (52 when a row's loads were not all in flight first), alone 26 us;
// 65536 x 512 and 2048 x 16384 the same within 7%.  Odd 16-bit rows are loaded and stored
// off their words: 16384 x 2047 39 us for 27.  Rows in parts are read twice, the second
// time from the caches where they fit: float32 32 x 50176 8.8 us (parts of 8192: 10),
// 512 x 50176 55.
#include <algorithm>
#include <type_traits>

#include "row_ops.h"
#include "rows_plan.h"

namespace convfwd {

namespace {

template <typename E>
struct NormArgs {
  const E *x, *r, *w, *b;
  E *y, *s;
  float *mean, *rstd;
  long long ldx, ldr, ldy, lds;
  long long row0, m;  // first row of this launch, rows of all
  int n;
  float eps;
  DropArgs d;
  float2* parts;  // [m][nparts]: mean, sum of squared distances
  int nparts;
};

// Everything that a thread reads for its runs run0, run0 + T, .. of a row, all in flight
// before the first is used; w and b only where there are registers to spare (HOLD).
template <typename E, int T, int U>
struct Loads {
  static constexpr bool HOLD = T * U <= 1024 && U < 4;
  Runs<E, T, U> x, r, w, b;
  __device__ __forceinline__ void fetch(const NormArgs<E>& a, long long row, int run0, bool params) {
    x.clear();
    x.fetch(a.x + row * a.ldx, a.n, run0);
    if (a.r) {
      r.clear();
      r.fetch(a.r + row * a.ldr, a.n, run0);
    }
    if (HOLD && params && a.w) {
      w.clear();
      w.fetch(a.w, a.n, run0);
    }
    if (HOLD && params && a.b) {
      b.clear();
      b.fetch(a.b, a.n, run0);
    }
  }
};

// s = r + drop(x); elements past n are 0 (with or without the mask).
template <typename E, int T, int U, bool DROP>
__device__ __forceinline__ void join_row(const NormArgs<E>& a, const Loads<E, T, U>& l,
                                         DropCounter c, long long row, int run0, float (&v)[U][8]) {
  l.x.get(v);
  if constexpr (DROP) {
#pragma unroll
    for (int u = 0; u < U; ++u) drop8(a.d, c, run0 + u * T, (unsigned)row, a.n - (run0 + u * T) * 8, v[u]);
  }
  if (a.r) {
    float t[U][8];
    l.r.get(t);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] += t[u][e];
  }
}

template <typename E, int T, int U>
__device__ __forceinline__ void store_row(const NormArgs<E>& a, const Loads<E, T, U>& l,
                                          long long row, int run0, float mean, float rstd,
                                          float (&v)[U][8]) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[u][e] = (v[u][e] - mean) * rstd;
  float t[U][8];
  if (a.w) {
    if constexpr (Loads<E, T, U>::HOLD) l.w.get(t);
    else load_runs<T>(a.w, a.n, run0, t);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] *= t[u][e];
  }
  if (a.b) {
    if constexpr (Loads<E, T, U>::HOLD) l.b.get(t);
    else load_runs<T>(a.b, a.n, run0, t);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] += t[u][e];
  }
  store_runs<T>(a.y + row * a.ldy, a.n, run0, v);
}

// Sum of squared distances from mean of a thread's elements before n.
template <int T, int U>
__device__ __forceinline__ float spread(const float (&v)[U][8], int run0, int n, float mean) {
  const int whole = n >> 3;
  float q = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = v[u][e] - mean;
      s = fmaf(d, d, s);
    }
    if (run0 + u * T < whole) q += s;
  }
  if (n & 7) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (run0 + u * T == whole) {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
          const float d = v[u][e] - mean;
          if (in_tail(e, n & 7)) q = fmaf(d, d, q);
        }
      }
  }
  return q;
}

template <int U>
__device__ __forceinline__ float total(const float (&v)[U][8]) {
  float t = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) t += v[u][e];
  return t;
}

template <typename E, int T, int U, bool DROP>
__global__ __launch_bounds__(T* teams_of(T)) void layer_norm_rows_kernel(const NormArgs<E> a) {
  __shared__ float lds[2][waves_of(T)];
  const int t = threadIdx.x % T;
  const long long row = a.row0 + (long long)blockIdx.x * teams_of(T) + team_of<T>();
  if (row >= a.m) return;
  Loads<E, T, U> l;
  l.fetch(a, row, t, true);
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  float v[U][8];
  join_row<E, T, U, DROP>(a, l, c, row, t, v);
  if (a.s) store_runs<T>(a.s + row * a.lds, a.n, t, v);
  // quotients, not products with 1 / n: a row of equal values has its value as mean
  const float mean = row_sum<T>(total(v), lds[0]) / (float)a.n;
  const float var = row_sum<T>(spread<T>(v, t, a.n, mean), lds[1]) / (float)a.n;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (a.mean && t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  store_row<E, T, U>(a, l, row, t, mean, rstd, v);
}

constexpr int kPartRuns = 2, kPart = 256 * 8 * kPartRuns;  // elements of a part: 256 threads, 2 runs each

// A workgroup takes one part of one row.
template <typename E, bool DROP>
__global__ __launch_bounds__(256) void layer_norm_parts_kernel(const NormArgs<E> a) {
  __shared__ float lds[2][4];
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  const int local = blockIdx.x / a.nparts, part = blockIdx.x - local * a.nparts;
  const long long row = a.row0 + local;
  const int run0 = part * (kPart / 8) + threadIdx.x, count = min(kPart, a.n - part * kPart);
  float v[kPartRuns][8];
  Loads<E, 256, kPartRuns> l;
  l.fetch(a, row, run0, false);
  join_row<E, 256, kPartRuns, DROP>(a, l, c, row, run0, v);
  const float mean = row_sum<256>(total(v), lds[0]) / (float)count;
  const float q = row_sum<256>(spread<256>(v, run0, a.n, mean), lds[1]);
  if (threadIdx.x == 0) a.parts[row * a.nparts + part] = make_float2(mean, q);
}

template <typename E, bool DROP>
__global__ __launch_bounds__(256) void layer_norm_joined_kernel(const NormArgs<E> a) {
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  const int lane = threadIdx.x & 63;
  const int local = blockIdx.x / a.nparts, part = blockIdx.x - local * a.nparts;
  const long long row = a.row0 + local;
  const int run0 = part * (kPart / 8) + threadIdx.x;
  float v[kPartRuns][8];
  Loads<E, 256, kPartRuns> l;
  l.fetch(a, row, run0, true);
  // every wave joins the row's parts (256 at most, four a lane)
  const float2* p = a.parts + row * a.nparts;
  float2 q[4];
  float count[4], s = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = lane + 64 * k;
    q[k] = at < a.nparts ? p[at] : make_float2(0.0f, 0.0f);
    count[k] = at < a.nparts ? (float)min(kPart, a.n - at * kPart) : 0.0f;
    s += count[k] * q[k].x;
  }
  const float mean = wave_sum(s) / (float)a.n;
  float far = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float d = q[k].x - mean;
    far += q[k].y + (count[k] > 0.0f ? count[k] * d * d : 0.0f);
  }
  const float rstd = 1.0f / sqrtf(wave_sum(far) / (float)a.n + a.eps);
  if (a.mean && part == 0 && threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  join_row<E, 256, kPartRuns, DROP>(a, l, c, row, run0, v);
  if (a.s) store_runs<256>(a.s + row * a.lds, a.n, run0, v);
  store_row<E, 256, kPartRuns>(a, l, row, run0, mean, rstd, v);
}

// f(args, rows) for the rows of every launch, `each` work-items a row, `teams` rows a workgroup.
template <typename E, typename F>
hipError_t by_rows(NormArgs<E> a, long long each, int teams, F f) {
  const long long most = rows_of_launch(each, teams);
  for (long long at = 0; at < a.m; at += most) {
    a.row0 = at;
    f(a, (unsigned)std::min(most, a.m - at));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// f(DROP) as a constant.
template <typename E, typename F>
void with_drop(const NormArgs<E>& a, F f) {
  if (a.d.threshold) f(std::true_type());
  else f(std::false_type());
}

template <typename E, int T, int U>
hipError_t launch_rows(const NormArgs<E>& args, hipStream_t s) {
  constexpr int TEAMS = teams_of(T);
  return by_rows(args, T, TEAMS, [&](const NormArgs<E>& a, unsigned rows) {
    const dim3 grid((rows + TEAMS - 1) / TEAMS), block(T * TEAMS);
    with_drop(a, [&](auto drop) {
      hipLaunchKernelGGL((layer_norm_rows_kernel<E, T, U, drop.value>), grid, block, 0, s, a);
    });
  });
}

template <typename E>
hipError_t launch_parts(const NormArgs<E>& args, hipStream_t s) {
  const hipError_t e = by_rows(args, 256 * args.nparts, 1, [&](const NormArgs<E>& a, unsigned rows) {
    const dim3 grid(rows * a.nparts), block(256);
    with_drop(a, [&](auto drop) {
      hipLaunchKernelGGL((layer_norm_parts_kernel<E, drop.value>), grid, block, 0, s, a);
    });
  });
  if (e != hipSuccess) return e;
  return by_rows(args, 256 * args.nparts, 1, [&](const NormArgs<E>& a, unsigned rows) {
    const dim3 grid(rows * a.nparts), block(256);
    with_drop(a, [&](auto drop) {
      hipLaunchKernelGGL((layer_norm_joined_kernel<E, drop.value>), grid, block, 0, s, a);
    });
  });
}

template <typename E>
hipError_t norm(const NormArgs<E>& a, const RowPlan& pl, hipStream_t s) {
  if (pl.parts) return launch_parts(a, s);
  switch (pl.threads) {
    case 8: return launch_rows<E, 8, 1>(a, s);
    case 16: return launch_rows<E, 16, 1>(a, s);
    case 32: return launch_rows<E, 32, 1>(a, s);
    case 64: return pl.runs == 1 ? launch_rows<E, 64, 1>(a, s) : launch_rows<E, 64, 2>(a, s);
    case 256: return pl.runs == 1 ? launch_rows<E, 256, 1>(a, s) : launch_rows<E, 256, 2>(a, s);
    default:
      return pl.runs == 1   ? launch_rows<E, 1024, 1>(a, s)
             : pl.runs == 2 ? launch_rows<E, 1024, 2>(a, s)
                            : launch_rows<E, 1024, 4>(a, s);
  }
}

template <typename E>
int run(const layer_norm_problem* p, const NormGeo& g, const NormPlan& pl, const void* x,
        const void* r, const void* w, const void* b, void* y, void* s, void* mean, void* rstd,
        const void* step, void* scratch, void* stream) {
  NormArgs<E> a{};
  a.x = elements<E>(x, p->x_off);
  a.r = p->has_residual ? elements<E>(r, p->r_off) : nullptr;
  a.w = p->has_weight ? elements<E>(w, p->w_off) : nullptr;
  a.b = p->has_bias ? elements<E>(b, p->b_off) : nullptr;
  a.y = elements<E>(y, p->y_off);
  a.s = elements<E>(s, p->s_off);
  a.mean = static_cast<float*>(mean);
  a.rstd = static_cast<float*>(rstd);
  a.ldx = g.ldx; a.ldr = g.ldr; a.ldy = g.ldy; a.lds = g.lds;
  a.m = g.m;
  a.n = (int)g.n;
  a.eps = p->eps;
  a.d = drop_args(drop_threshold(p->drop), p->seed, p->offset, step);
  a.parts = static_cast<float2*>(scratch);
  a.nparts = (int)pl.row.parts;
  return norm<E>(a, pl.row, static_cast<hipStream_t>(stream)) == hipSuccess ? CONV_OK
                                                                             : CONV_ERR_DEVICE;
}

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" int layer_norm_forward(const layer_norm_problem* p, int dtype, const void* x,
                                  const void* r, const void* w, const void* b, void* y, void* s,
                                  void* mean, void* rstd, const void* step, void* scratch,
                                  uint64_t scratch_bytes, void* stream) {
  NormGeo g;
  NormPlan pl;
  const int st = layer_norm_checked(p, dtype, x, r, w, b, y, s, mean, rstd, step, scratch,
                                    scratch_bytes, &g, &pl);
  if (st || g.m == 0) return st;
  if (dtype == CONV_F16)
    return run<_Float16>(p, g, pl, x, r, w, b, y, s, mean, rstd, step, scratch, stream);
  if (dtype == CONV_BF16)
    return run<__bf16>(p, g, pl, x, r, w, b, y, s, mean, rstd, step, scratch, stream);
  return run<float>(p, g, pl, x, r, w, b, y, s, mean, rstd, step, scratch, stream);
}
