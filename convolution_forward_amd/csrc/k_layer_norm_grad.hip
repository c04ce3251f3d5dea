// Layer norm backward (include/layer_norm.h): one read of s, dy (and ds), one write of
// dx (and dr), and the column sums dw and db on the way.
//
// A workgroup walks over rows and keeps, for the columns that its threads hold, the
// sums of dy u and of dy in registers; at the end it writes one partial row of each,
// and a second kernel adds the partial rows in order.  So no atomics, and dy and s are
// read once for both the row's gradient and the columns' sums.  A row needs two sums
// (of g and of g u) before its first gradient: one exchange through LDS and one barrier
// a row, none where lanes of a wave hold it.  Few rows take one launch in which some
// workgroups sum columns and the others take rows.  Rows of more than 8192 elements go
// in parts of 2048, in two launches: the parts' sums (and, of few rows, the columns'),
// then the gradients.
//
// bfloat16 8192 x 4096 with dropout, residual and ds: 72 us (4.6 TB/s), of which the join
// 5; without them 46.  The loop is bound by memory, and two workgroups on a unit ask for
// about as much of it as there is: the 16-bit kernels' 140 to 150 registers allow a third,
// but 768 groups, with half as many partial rows again, take 75 and 49 us (8192 x 3000: 60
// and 39 for 61 and 42).  float32's 204 to 212 registers allow two.  In parts, 2048 x 16384:
// 95 us (one workgroup of 1024 threads by 2 runs spilled: 193).
#include <algorithm>
#include <type_traits>

#include "linear_tile.h"
#include "row_ops.h"
#include "rows_plan.h"

namespace convfwd {

namespace {

template <typename E>
struct GradArgs {
  const E *s, *w, *dy, *ds;
  const float *mean, *rstd;
  E *dx, *dr;        // either may be null
  float* partials;   // [group][2][np] of dw and db; null: neither is wanted
  float2* sums;      // [m][parts]: sums of g u and of g
  long long lds, lddy, ldds, lddx, lddr;
  long long row0, m;  // row0: first row of this launch (parts' sums)
  int n, np, parts;
  int cols;           // workgroups at the front that sum columns (one launch)
  E *dw, *db;         // theirs; either may be null
  float inv_n;
  DropArgs d;
};

// u = (s - mean) rstd of a thread's elements.  Past the row's end s is 0, and mean counts as 0
// too: its product with rstd may pass float32's range, and times a g of 0 would make the
// row's sums NaN.  A partial run's elements lie in pieces (fetch_tail), so four choices of
// a mean serve its 8 slots.  For mean everywhere: bfloat16 8192 x 4096 and 16384 x 2047 the
// same within 1%, 16384 x 1001 46.9 us for 46.4, float32 400000 x 33 with dropout 74.8 for 69.7.
template <int T, int U>
__device__ __forceinline__ void normalise(float (&u)[U][8], int run0, int n, float mean, float rstd) {
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int left = n - (run0 + k * T) * 8;
    float mu[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) mu[e] = left >= 8 || (left > 0 && in_tail(e, left)) ? mean : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[k][e] = (u[k][e] - mu[e]) * rstd;
  }
}

// The gradient of s from u, g and the row's two means (and ds), and its stores.
template <typename E, int T, int U, bool DROP>
__device__ __forceinline__ void finish_row(const GradArgs<E>& a, DropCounter c, long long row,
                                           int run0, float rstd, float along, float level,
                                           const float (&u)[U][8], float (&g)[U][8],
                                           const Runs<E, T, U>& ds) {
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) g[k][e] = rstd * (g[k][e] - level - u[k][e] * along);
  if (a.ds) {
    float t[U][8];
    ds.get(t);
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) g[k][e] += t[k][e];
  }
  if (a.dr) store_runs<T>(a.dr + row * a.lddr, a.n, run0, g);
  if (a.dx) {
    if constexpr (DROP) {
#pragma unroll
      for (int k = 0; k < U; ++k) drop8(a.d, c, run0 + k * T, (unsigned)row, a.n - (run0 + k * T) * 8, g[k]);
    }
    store_runs<T>(a.dx + row * a.lddx, a.n, run0, g);
  }
}

// The sums of a run's columns to p, from the slots of a partial run where it is one.
__device__ __forceinline__ void store_columns(float* p, int left, const float (&v)[8]) {
  if (left >= 8) store8(p, 8, v);
  else store_tail(p, left, v);
}

// T threads a row, U runs each; TEAMS rows at a time.  The next row's loads are in
// flight from before the present one's sums are exchanged (8192 x 4096 bf16: 73 us with
// it, 108 without).
template <typename E, int T, int U, int TEAMS, bool DROP>
__global__ __launch_bounds__(T* TEAMS) void layer_norm_grad_kernel(const GradArgs<E> a) {
  constexpr int WAVES = waves_of(T);
  __shared__ float2 red[2][TEAMS * WAVES];
  __shared__ alignas(16) float columns[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? T * 8 : 1];
  const int t = threadIdx.x % T, team = team_of<T>();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  float w[U][8], dw[U][8], db[U][8];
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[k][e] = 1.0f;
      dw[k][e] = db[k][e] = 0.0f;
    }
  if (a.w) load_runs<T>(a.w, a.n, t, w);
  const long long stride = (long long)gridDim.x * TEAMS, first = (long long)blockIdx.x * TEAMS;
  long long row = first + team;
  Runs<E, T, U> s, dy, ds, ds_next;
  s.clear();
  dy.clear();
  ds_next.clear();
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](long long at) {
    s.fetch(a.s + at * a.lds, a.n, t);
    dy.fetch(a.dy + at * a.lddy, a.n, t);
    if (a.ds) ds_next.fetch(a.ds + at * a.ldds, a.n, t);
    mean = a.mean[at];
    rstd = a.rstd[at];
  };
  if (row < a.m) fetch(row);
  int buf = 0;
  for (long long base = first; base < a.m; base += stride, row += stride) {
    const bool in = row < a.m;  // every wave reaches the barrier
    float u[U][8], g[U][8], along = 0.0f, level = 0.0f;
    const float r = rstd;
    if (in) {
      s.get(u);
      dy.get(g);
      const float mu = mean;
      ds = ds_next;
      if (row + stride < a.m) fetch(row + stride);
      normalise<T>(u, t, a.n, mu, r);
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[k][e] = fmaf(g[k][e], u[k][e], dw[k][e]);
          db[k][e] += g[k][e];
          g[k][e] *= w[k][e];
          along = fmaf(g[k][e], u[k][e], along);
          level += g[k][e];
        }
      along = lanes_sum<T < 64 ? T : 64>(along);
      level = lanes_sum<T < 64 ? T : 64>(level);
    }
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) red[buf][wave] = make_float2(along, level);
      __syncthreads();  // a wave may be one row ahead, hence two buffers
      along = level = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        along += red[buf][team * WAVES + i].x;
        level += red[buf][team * WAVES + i].y;
      }
      buf ^= 1;
    }
    if (in) finish_row<E, T, U, DROP>(a, c, row, t, r, along * a.inv_n, level * a.inv_n, u, g, ds);
  }
  if (!a.partials) return;
  float* p = a.partials + (long long)blockIdx.x * 2 * a.np;
  if constexpr (TEAMS == 1) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int at = (t + k * T) * 8;
      if (at < a.n) {
        store_columns(p + at, a.n - at, dw[k]);
        store_columns(p + a.np + at, a.n - at, db[k]);
      }
    }
  } else {
    // the teams' sums joined in order, T runs at a time
#pragma unroll
    for (int k = 0; k < 2 * U; ++k) {
      store_columns(&columns[team][t * 8], a.n - (t + k % U * T) * 8, k < U ? dw[k % U] : db[k % U]);
      __syncthreads();
      for (int i = threadIdx.x; i < T * 8; i += T * TEAMS) {
        const int at = k % U * T * 8 + i;
        if (at < a.n) {
          float q = columns[0][i];
#pragma unroll
          for (int j = 1; j < TEAMS; ++j) q += columns[j][i];
          p[(k < U ? 0 : a.np) + at] = q;
        }
      }
      __syncthreads();
    }
  }
}

constexpr int kColumns = 32;  // of a workgroup that sums columns

struct ColumnLds {
  float2 stats[kOnceRows];  // mean and 1 / deviation of every row
  float sums[2][32][kColumns];
};

// dw and db of 32 columns over all rows: 8 lanes of 4 columns a row, 32 rows at a time
// (the first 256 threads), then these in order.  The last piece of a row that has no 4
// columns left lies further to the left, over its neighbour's.
template <typename E>
__device__ __forceinline__ void sum_columns(const GradArgs<E>& a, int threads, ColumnLds& lds) {
  constexpr int SLOTS = 32, B = 32 / (int)sizeof(E), Q = 4;  // B loads of each in flight
  const int m = (int)a.m;
  for (int i = threadIdx.x; i < m; i += threads) lds.stats[i] = make_float2(a.mean[i], a.rstd[i]);
  const int lane = threadIdx.x & 7, slot = threadIdx.x >> 3, first = blockIdx.x * kColumns;
  const int want = first + lane * 4, at = a.n < 4 ? 0 : want < a.n - 4 ? want : a.n - 4;
  float dw[4] = {0, 0, 0, 0}, db[4] = {0, 0, 0, 0};
  __syncthreads();
  if (slot < SLOTS) {
    for (int base = 0; base < m; base += SLOTS * B) {
      Few<E, 4> s[B], dy[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (base + k / Q * Q * SLOTS >= m) break;  // the same in all threads
        const int row = base + k * SLOTS + slot;
        const long long i = row < m ? row : m - 1;
        const E *ps = a.s + i * a.lds + at, *pd = a.dy + i * a.lddy + at;
        if (a.n < 4) {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (e < a.n) {
              s[k].v[e] = ps[e];
              dy[k].v[e] = pd[e];
            }
        } else {
          s[k] = *reinterpret_cast<const Few<E, 4>*>(ps);
          dy[k] = *reinterpret_cast<const Few<E, 4>*>(pd);
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (base + k / Q * Q * SLOTS >= m) break;
        const int row = base + k * SLOTS + slot;
        const float2 q = lds.stats[row < m ? row : m - 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = ((float)s[k].v[e] - q.x) * q.y, g = (float)dy[k].v[e];
          dw[e] = row < m ? fmaf(g, u, dw[e]) : dw[e];
          db[e] += row < m ? g : 0.0f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (at + e >= want && at + e < a.n) {
        lds.sums[0][slot][at + e - first] = dw[e];
        lds.sums[1][slot][at + e - first] = db[e];
      }
  }
  __syncthreads();
  const int which = threadIdx.x / kColumns, c = threadIdx.x % kColumns;
  E* out = which == 0 ? a.dw : a.db;
  if (which < 2 && first + c < a.n && out) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) t += lds.sums[which][i][c];
    out[first + c] = (E)t;
  }
}

// Few rows: one launch, a row a team, and dw and db by workgroups of their own that read
// s and dy once more.  These come first and take longest: a unit gets a line of memory
// in about 4 ns, two lines a row (float16 777 x 1001: kernels 8.5 us, as long as the two
// launches', a call 9.1 for 11.8; 64 x 4096 kernels 2.8 us for 7.2).  More loads in flight (24
// for 16 of 16 bits) changed nothing.  The sums' exchange at the end has several slots of
// a wave in the same banks, once a workgroup (192 cycles of conflicts).
template <typename E, int T, int U, int TEAMS, bool DROP>
__global__ __launch_bounds__(T* TEAMS) void layer_norm_grad_once_kernel(const GradArgs<E> a) {
  __shared__ ColumnLds lds;
  if ((int)blockIdx.x < a.cols) {
    sum_columns(a, T * TEAMS, lds);
    return;
  }
  const int t = threadIdx.x % T;
  const long long row = (long long)(blockIdx.x - a.cols) * TEAMS + team_of<T>();
  if (row >= a.m) return;  // whole teams; a row of more than a wave has the workgroup to itself
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  Runs<E, T, U> s, dy, ds;
  s.clear();
  dy.clear();
  ds.clear();
  s.fetch(a.s + row * a.lds, a.n, t);
  dy.fetch(a.dy + row * a.lddy, a.n, t);
  if (a.ds) ds.fetch(a.ds + row * a.ldds, a.n, t);
  float u[U][8], g[U][8], w[U][8], along = 0.0f, level = 0.0f;
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[k][e] = 1.0f;
  if (a.w) load_runs<T>(a.w, a.n, t, w);
  const float mean = a.mean[row], rstd = a.rstd[row];
  s.get(u);
  dy.get(g);
  normalise<T>(u, t, a.n, mean, rstd);
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[k][e] *= w[k][e];
      along = fmaf(g[k][e], u[k][e], along);
      level += g[k][e];
    }
  along = row_sum<T>(along, lds.sums[0][0]);
  level = row_sum<T>(level, lds.sums[1][0]);
  finish_row<E, T, U, DROP>(a, c, row, t, rstd, along * a.inv_n, level * a.inv_n, u, g, ds);
}

constexpr int kPartRuns = 256;  // runs of a part, a thread each

// Sums of g u and g of one part of one row.  FEW rows: dw and db beside them, with the
// registers and LDS of that (many rows with them: 2048 x 16384 bfloat16 99 us for 96).
template <typename E, bool FEW>
__global__ __launch_bounds__(256) void layer_norm_grad_sums_kernel(const GradArgs<E> a) {
  if constexpr (FEW) {
    __shared__ ColumnLds columns;
    if ((int)blockIdx.x < a.cols) {
      sum_columns(a, 256, columns);
      return;
    }
  }
  __shared__ float lds[2][4];
  const int id = blockIdx.x - (FEW ? a.cols : 0), local = id / a.parts, part = id - local * a.parts;
  const long long row = a.row0 + local;
  const int run0 = part * kPartRuns + threadIdx.x;
  float u[1][8], g[1][8], along = 0.0f, level = 0.0f;
  load_runs<kPartRuns>(a.s + row * a.lds, a.n, run0, u);
  load_runs<kPartRuns>(a.dy + row * a.lddy, a.n, run0, g);
  if (a.w) {
    float w[1][8];
    load_runs<kPartRuns>(a.w, a.n, run0, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[0][e] *= w[0][e];
  }
  normalise<kPartRuns>(u, run0, a.n, a.mean[row], a.rstd[row]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    along = fmaf(g[0][e], u[0][e], along);
    level += g[0][e];
  }
  along = row_sum<256>(along, lds[0]);
  level = row_sum<256>(level, lds[1]);
  if (threadIdx.x == 0) a.sums[row * a.parts + part] = make_float2(along, level);
}

// Gradients of one part of every gridDim.x / parts-th row.
template <typename E, bool DROP>
__global__ __launch_bounds__(256) void layer_norm_grad_parts_kernel(const GradArgs<E> a) {
  const DropCounter c = DROP ? drop_counter(a.d) : DropCounter{0, 0};
  const int group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
  const int groups = gridDim.x / a.parts, lane = threadIdx.x & 63;
  const int run0 = part * kPartRuns + threadIdx.x;
  float w[1][8], dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[0][e] = 1.0f;
    dw[e] = db[e] = 0.0f;
  }
  if (a.w) load_runs<kPartRuns>(a.w, a.n, run0, w);
  // from the last row back: what the sums read last is what the last-level cache holds
  for (long long row = a.m - 1 - group; row >= 0; row -= groups) {
    float u[1][8], g[1][8], along = 0.0f, level = 0.0f;
    Runs<E, kPartRuns, 1> ds;
    ds.clear();
    if (a.ds) ds.fetch(a.ds + row * a.ldds, a.n, run0);
    load_runs<kPartRuns>(a.s + row * a.lds, a.n, run0, u);
    load_runs<kPartRuns>(a.dy + row * a.lddy, a.n, run0, g);
    for (int i = lane; i < a.parts; i += 64) {
      const float2 q = a.sums[row * a.parts + i];
      along += q.x;
      level += q.y;
    }
    along = wave_sum(along) * a.inv_n;
    level = wave_sum(level) * a.inv_n;
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u[0][e] = (u[0][e] - mean) * rstd;
      dw[e] = fmaf(g[0][e], u[0][e], dw[e]);
      db[e] += g[0][e];
      g[0][e] *= w[0][e];
    }
    finish_row<E, kPartRuns, 1, DROP>(a, c, row, run0, rstd, along, level, u, g, ds);
  }
  const int left = a.n - run0 * 8;
  if (!a.partials || left <= 0) return;
  float* p = a.partials + (long long)group * 2 * a.np + run0 * 8;
  store_columns(p, left, dw);
  store_columns(p + a.np, left, db);
}

// Adds the groups' partial rows: 32 columns of dw or db a workgroup (a line of memory; a
// unit takes lines at a rate of its own, so few columns to a workgroup), 128 rows at a
// time, 8 lanes of 4 columns a row, then the 128 sums in order.
template <typename E>
__global__ __launch_bounds__(1024) void layer_norm_grad_join_kernel(const float* partials, E* dw,
                                                                    E* db, int groups, int n,
                                                                    int np) {
  constexpr int SLOTS = 128, B = 8;
  __shared__ float lds[SLOTS][kColumns + 4], part[8][kColumns];
  const int slot = threadIdx.x >> 3, col = (threadIdx.x & 7) * 4, first = blockIdx.x * kColumns;
  const float* p = partials + (blockIdx.y ? np : 0) + first + col;
  lin::f32x4 s = {0, 0, 0, 0};
  if (first + col < np) {
    for (int i = slot; i < groups; i += SLOTS * B) {
      lin::f32x4 q[B];
#pragma unroll
      for (int k = 0; k < B; ++k)
        q[k] = i + SLOTS * k < groups
                   ? *reinterpret_cast<const lin::f32x4*>(p + (long long)(i + SLOTS * k) * 2 * np)
                   : lin::f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < B; ++k) s += q[k];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) lds[slot][col + e] = s[e];
  __syncthreads();
  const int c = threadIdx.x % kColumns, q = threadIdx.x / kColumns;
  if (q < 8) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS / 8; ++i) t += lds[q * (SLOTS / 8) + i][c];
    part[q][c] = t;
  }
  __syncthreads();
  E* out = blockIdx.y ? db : dw;
  if (q == 0 && first + c < n && out) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += part[i][c];
    out[first + c] = (E)t;
  }
}

// f(DROP) as a constant.
template <typename E, typename F>
void with_drop(const GradArgs<E>& a, F f) {
  if (a.d.threshold) f(std::true_type());
  else f(std::false_type());
}

// Workgroups that sum columns.
template <typename E>
int columns_of(const GradArgs<E>& a) {
  return a.dw || a.db ? (a.n + kColumns - 1) / kColumns : 0;
}

template <typename E, int T, int U>
void launch_grad(const GradArgs<E>& a, const NormBackwardPlan& pl, bool in_place, hipStream_t s) {
  constexpr int TEAMS = teams_of(T);
  const dim3 block(T * TEAMS);
  with_drop(a, [&](auto drop) {
    if (!pl.once) {
      const dim3 grid((unsigned)pl.groups);
      hipLaunchKernelGGL((layer_norm_grad_kernel<E, T, U, TEAMS, drop.value>), grid, block, 0, s, a);
      return;
    }
    GradArgs<E> q = a;
    q.cols = columns_of(a);
    unsigned rows = a.dx || a.dr ? (unsigned)pl.groups : 0;
    auto launch = [&](unsigned grid) {
      hipLaunchKernelGGL((layer_norm_grad_once_kernel<E, T, U, TEAMS, drop.value>), dim3(grid), block,
                         0, s, q);
    };
    if (in_place && q.cols && rows) {  // the columns' sums before the rows overwrite dy
      launch(q.cols);
      q.cols = 0;
    }
    launch(q.cols + rows);
  });
}

template <typename E>
void launch_parts(const GradArgs<E>& a, unsigned groups, hipStream_t s) {
  with_drop(a, [&](auto drop) {
    hipLaunchKernelGGL((layer_norm_grad_parts_kernel<E, drop.value>), dim3(groups * a.parts), dim3(256), 0,
                       s, a);
  });
}

template <typename E>
hipError_t grad(GradArgs<E>& a, const NormBackwardPlan& pl, bool in_place, hipStream_t s) {
  const unsigned groups = (unsigned)pl.groups;
  if (pl.row.parts && pl.once) {
    a.cols = columns_of(a);
    const bool rows = a.dx || a.dr;
    const dim3 grid((unsigned)(a.cols + (rows ? a.m * a.parts : 0)));
    hipLaunchKernelGGL((layer_norm_grad_sums_kernel<E, true>), grid, dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !rows) return e;
    launch_parts(a, groups, s);
  } else if (pl.row.parts) {
    const long long most = rows_of_launch(256 * a.parts, 1);
    for (long long at = 0; at < a.m; at += most) {
      a.row0 = at;
      const dim3 grid((unsigned)(std::min(most, a.m - at) * a.parts));
      hipLaunchKernelGGL((layer_norm_grad_sums_kernel<E, false>), grid, dim3(256), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    launch_parts(a, groups, s);
  } else if (pl.row.threads == 8) {
    launch_grad<E, 8, 1>(a, pl, in_place, s);
  } else if (pl.row.threads == 16) {
    launch_grad<E, 16, 1>(a, pl, in_place, s);
  } else if (pl.row.threads == 32) {
    launch_grad<E, 32, 1>(a, pl, in_place, s);
  } else if (pl.row.threads == 64) {
    if (pl.row.runs == 1) launch_grad<E, 64, 1>(a, pl, in_place, s);
    else launch_grad<E, 64, 2>(a, pl, in_place, s);
  } else if (pl.row.threads == 256) {
    if (pl.row.runs == 1) launch_grad<E, 256, 1>(a, pl, in_place, s);
    else launch_grad<E, 256, 2>(a, pl, in_place, s);
  } else {
    launch_grad<E, 1024, 1>(a, pl, in_place, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.once || !a.partials) return e;
  hipLaunchKernelGGL((layer_norm_grad_join_kernel<E>), dim3((a.np + kColumns - 1) / kColumns, 2),
                     dim3(1024), 0, s, a.partials, a.dw, a.db, (int)groups, a.n, a.np);
  return hipGetLastError();
}

template <typename E>
int run(const layer_norm_problem* p, const NormGeo& g, const NormBackwardPlan& pl, const void* s,
        const void* w, const void* mean, const void* rstd, const void* dy, const void* ds, void* dx,
        void* dr, void* dw, void* db, const void* step, void* scratch, void* stream) {
  GradArgs<E> a{};
  a.s = elements<E>(s, p->s_off);
  a.w = p->has_weight ? elements<E>(w, p->w_off) : nullptr;
  a.dy = elements<E>(dy, p->dy_off);
  a.ds = elements<E>(ds, p->ds_off);
  a.mean = static_cast<const float*>(mean);
  a.rstd = static_cast<const float*>(rstd);
  a.dx = elements<E>(dx, p->dx_off);
  a.dr = elements<E>(dr, p->dr_off);
  char* sc = static_cast<char*>(scratch);
  a.dw = elements<E>(dw, p->dw_off);
  a.db = elements<E>(db, p->db_off);
  a.partials = (dw || db) && !pl.once ? reinterpret_cast<float*>(sc + pl.partials) : nullptr;
  a.sums = reinterpret_cast<float2*>(sc + pl.sums);
  a.lds = g.lds; a.lddy = g.ldy; a.ldds = g.ldds; a.lddx = g.lddx; a.lddr = g.lddr;
  a.m = g.m;
  a.n = (int)g.n;
  a.np = (int)(ceil_div(g.n, 8) * 8);
  a.parts = (int)pl.row.parts;
  a.inv_n = 1.0f / (float)g.n;
  a.d = drop_args(drop_threshold(p->drop), p->seed, p->offset, step);
  const bool in_place = (dx && a.dx == a.dy) || (dr && a.dr == a.dy);
  const hipError_t e = grad<E>(a, pl, in_place, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? CONV_OK : CONV_ERR_DEVICE;
}

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" int layer_norm_backward(const layer_norm_problem* p, int dtype, const void* s,
                                   const void* w, const void* mean, const void* rstd,
                                   const void* dy, const void* ds, void* dx, void* dr, void* dw,
                                   void* db, const void* step, void* scratch,
                                   uint64_t scratch_bytes, void* stream) {
  NormGeo g;
  NormBackwardPlan pl;
  const int st = layer_norm_backward_checked(p, dtype, s, w, mean, rstd, dy, ds, dx, dr, dw, db,
                                             step, scratch, scratch_bytes, &g, &pl);
  if (st || (g.m == 0 && !dw && !db)) return st;
  if (dtype == CONV_F16)
    return run<_Float16>(p, g, pl, s, w, mean, rstd, dy, ds, dx, dr, dw, db, step, scratch, stream);
  if (dtype == CONV_BF16)
    return run<__bf16>(p, g, pl, s, w, mean, rstd, dy, ds, dx, dr, dw, db, step, scratch, stream);
  return run<float>(p, g, pl, s, w, mean, rstd, dy, ds, dx, dr, dw, db, step, scratch, stream);
}
