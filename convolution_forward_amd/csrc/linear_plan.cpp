// Host half of include/linear.h that never touches the device: validation,
// overlap rules, the shape-only plan of each matrix product, scratch layout,
// describe and check.
#include "linear_plan.h"

#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <cmath>

namespace convfwd {

namespace {

constexpr int64_t kLim = 2147483647LL;
constexpr int kCus = 256;  // gfx950

// rows x cols elements, rows ld apart, starting at p + off
struct Range {
  uintptr_t base;
  int64_t rows, cols, ld;
};

Range range_of(const void* p, int64_t off, int64_t rows, int64_t cols, int64_t ld, int es) {
  return {(uintptr_t)p + (uintptr_t)off * (uintptr_t)es, rows, cols, ld};
}

uintptr_t end_of(const Range& a, int es) {
  return a.base + (uintptr_t)((a.rows - 1) * a.ld + a.cols) * (uintptr_t)es;
}

// Whether two strided matrices share an element.  Matrices of one stride whose
// columns do not meet (two halves of the rows of one buffer) do not.
bool overlap(const Range& a, const Range& b, int es) {
  if (a.rows < 1 || b.rows < 1) return false;
  if (a.base >= end_of(b, es) || b.base >= end_of(a, es)) return false;
  if (a.ld == b.ld && (a.base > b.base ? a.base - b.base : b.base - a.base) % (uintptr_t)es == 0) {
    const Range &lo = a.base < b.base ? a : b, &hi = a.base < b.base ? b : a;
    const int64_t d = (int64_t)((hi.base - lo.base) / (uintptr_t)es) % a.ld;
    if (d >= lo.cols && d + hi.cols <= a.ld) return false;
  }
  return true;
}

bool same(const Range& a, const Range& b) {
  return a.base == b.base && a.rows == b.rows && a.cols == b.cols && (a.ld == b.ld || a.rows <= 1);
}

bool bytes_overlap(const Range& a, int es, const void* s, uint64_t bytes) {
  if (a.rows < 1 || bytes == 0) return false;
  const uintptr_t s0 = (uintptr_t)s;
  return a.base < s0 + bytes && s0 < end_of(a, es);
}

// ld of a matrix with rows of `cols` elements: 0 = dense; -1 if out of range
int64_t stride_of(int64_t ld, int64_t cols) {
  if (ld == 0) return cols;
  return ld >= cols && ld <= kLinMaxExtent ? ld : -1;
}

// the last element's byte offset stays in int64, and an operand below 2^40
// elements (beyond the card's memory), which also bounds every grid
bool offset_ok(int64_t off, int64_t rows, int64_t ld, int es) {
  int64_t e, b;
  if (off < 0) return false;
  if (__builtin_mul_overflow(rows < 1 ? 1 : rows, ld, &e) || e > (1LL << 40)) return false;
  return !__builtin_add_overflow(e, off, &e) && !__builtin_mul_overflow(e, (int64_t)es, &b);
}

bool dtype_ok(int dtype) { return dtype == CONV_F32 || dtype == CONV_F16 || dtype == CONV_BF16; }

bool act_ok(int a) { return a >= CONV_ACT_IDENTITY && a <= LINEAR_ACT_GELU_TANH; }

const char* dtype_name(int dtype) {
  return dtype == CONV_F16 ? "f16" : dtype == CONV_BF16 ? "bf16" : "f32";
}

bool vec16(int64_t elems, int es) { return elems * es % 16 == 0; }

}  // namespace

int linear_validate(const linear_problem* p, int dtype, LinearGeo* out) {
  if (!p || !dtype_ok(dtype)) return CONV_ERR_ARG;
  if (!act_ok(p->activation) || (p->has_bias != 0 && p->has_bias != 1) ||
      p->has_residual < LINEAR_RES_NONE || p->has_residual > LINEAR_RES_AFTER ||
      (p->save_z != 0 && p->save_z != 1) ||
      (p->w_layout != LINEAR_W_NK && p->w_layout != LINEAR_W_KN) || p->reserved != 0)
    return CONV_ERR_ARG;
  const int64_t offs[] = {p->x_off, p->w_off, p->b_off, p->r_off, p->y_off, p->z_off,
                          p->dy_off, p->dx_off, p->dw_off, p->db_off, p->dr_off};
  for (int64_t o : offs)
    if (o < 0) return CONV_ERR_ARG;
  LinearGeo g{};
  g.m = p->m; g.n = p->n; g.k = p->k;
  if (g.m < 0 || g.m > kLim || g.n < 1 || g.n > kLinMaxExtent || g.k < 1 || g.k > kLinMaxExtent)
    return CONV_ERR_SHAPE;
  g.es = (int)dtype_size(dtype);
  g.kn = p->w_layout == LINEAR_W_KN;
  const int64_t wr = g.kn ? g.k : g.n, wc = g.kn ? g.n : g.k;
  g.ldx = stride_of(p->ldx, g.k);
  g.ldw = stride_of(p->ldw, wc);
  g.ldr = stride_of(p->ldr, g.n);
  g.ldy = stride_of(p->ldy, g.n);
  g.ldz = stride_of(p->ldz, g.n);
  g.lddx = stride_of(p->lddx, g.k);
  g.lddw = stride_of(p->lddw, wc);
  g.lddr = stride_of(p->lddr, g.n);
  if (g.ldx < 0 || g.ldw < 0 || g.ldr < 0 || g.ldy < 0 || g.ldz < 0 || g.lddx < 0 || g.lddw < 0 ||
      g.lddr < 0)
    return CONV_ERR_SHAPE;
  if (!offset_ok(p->x_off, g.m, g.ldx, g.es) || !offset_ok(p->w_off, wr, g.ldw, g.es) ||
      !offset_ok(p->b_off, 1, g.n, g.es) || !offset_ok(p->r_off, g.m, g.ldr, g.es) ||
      !offset_ok(p->y_off, g.m, g.ldy, g.es) || !offset_ok(p->z_off, g.m, g.ldz, g.es) ||
      !offset_ok(p->dy_off, g.m, g.ldy, g.es) || !offset_ok(p->dx_off, g.m, g.lddx, g.es) ||
      !offset_ok(p->dw_off, wr, g.lddw, g.es) || !offset_ok(p->db_off, 1, g.n, g.es) ||
      !offset_ok(p->dr_off, g.m, g.lddr, g.es))
    return CONV_ERR_SHAPE;
  *out = g;
  return CONV_OK;
}

int gated_validate(const gated_problem* p, int dtype, GatedGeo* out) {
  if (!p || !dtype_ok(dtype)) return CONV_ERR_ARG;
  if (!act_ok(p->activation) || (p->has_bias != 0 && p->has_bias != 1) ||
      (p->save_p != 0 && p->save_p != 1) || p->reserved != 0)
    return CONV_ERR_ARG;
  const int64_t offs[] = {p->x_off, p->wg_off, p->wu_off, p->bg_off, p->bu_off, p->h_off,
                          p->pg_off, p->pu_off, p->dh_off, p->dx_off, p->dwg_off, p->dwu_off,
                          p->dbg_off, p->dbu_off};
  for (int64_t o : offs)
    if (o < 0) return CONV_ERR_ARG;
  GatedGeo g{};
  g.m = p->m; g.f = p->f; g.k = p->k;
  if (g.m < 0 || g.m > kLim || g.f < 1 || g.f > kLinMaxExtent || g.k < 1 || g.k > kLinMaxExtent)
    return CONV_ERR_SHAPE;
  g.es = (int)dtype_size(dtype);
  g.ldx = stride_of(p->ldx, g.k);
  g.ldw = stride_of(p->ldw, g.k);
  g.ldh = stride_of(p->ldh, g.f);
  g.ldp = stride_of(p->ldp, g.f);
  g.lddx = stride_of(p->lddx, g.k);
  g.lddw = stride_of(p->lddw, g.k);
  if (g.ldx < 0 || g.ldw < 0 || g.ldh < 0 || g.ldp < 0 || g.lddx < 0 || g.lddw < 0)
    return CONV_ERR_SHAPE;
  if (!offset_ok(p->x_off, g.m, g.ldx, g.es) || !offset_ok(p->wg_off, g.f, g.ldw, g.es) ||
      !offset_ok(p->wu_off, g.f, g.ldw, g.es) || !offset_ok(p->bg_off, 1, g.f, g.es) ||
      !offset_ok(p->bu_off, 1, g.f, g.es) || !offset_ok(p->h_off, g.m, g.ldh, g.es) ||
      !offset_ok(p->pg_off, g.m, g.ldp, g.es) || !offset_ok(p->pu_off, g.m, g.ldp, g.es) ||
      !offset_ok(p->dh_off, g.m, g.ldh, g.es) || !offset_ok(p->dx_off, g.m, g.lddx, g.es) ||
      !offset_ok(p->dwg_off, g.f, g.lddw, g.es) || !offset_ok(p->dwu_off, g.f, g.lddw, g.es) ||
      !offset_ok(p->dbg_off, 1, g.f, g.es) || !offset_ok(p->dbu_off, 1, g.f, g.es))
    return CONV_ERR_SHAPE;
  *out = g;
  return CONV_OK;
}

namespace {

// A tile's measured times, in us on the whole card: of a launch of one round
// without a step, of every further round's start and epilogue, and of a contraction
// step (128 bytes of k): step, plus busy by the share of the units at work (the card
// lowers its clock as they fill), plus more for every further workgroup on a unit,
// up to units of them.  Fitted to 1300 timings of m 48 .. 8192, n and k 256 .. 4096
// with 1 to 16 splits: off by 9% (root mean square), and the choice by it costs 1.6%
// more than the best on average, 15% at most.
struct Tiling {
  int tile, r, c, units;
  double fixed, round, step, busy, more;
};
const Tiling kTiles16[] = {{TILE_256, 256, 256, 1, 10.3, 7.3, 0.908, 0.314, 0.0},
                           {TILE_256X128, 256, 128, 1, 8.0, 3.3, 0.555, 0.231, 0.0},
                           {TILE_128, 128, 128, 2, 5.4, 0.7, 0.650, 0.114, 0.277},
                           {TILE_64, 64, 64, 4, 4.2, 1.6, 0.400, 0.011, 0.160}};
const Tiling kTiles16Gather[] = {{TILE_128, 128, 128, 2, 5.5, 0.0, 0.930, 0.166, 0.200},
                                 {TILE_64, 64, 64, 4, 3.8, 0.0, 0.489, 0.081, 0.251}};
const Tiling kTiles32[] = {{TILE_128, 128, 128, 2, 5.9, 0.0, 2.100, 0.294, 1.560},
                           {TILE_64, 64, 64, 4, 4.2, 0.0, 0.753, 0.059, 0.525}};
constexpr double kJoin = 3.6, kJoinByte = 3.4e-7;  // the second pass of a split: launch, plane bytes

int64_t tile_count(const ProductShape& s, const Tiling& t) {
  return ceil_div(s.gated ? 2 * s.R : s.R, t.r) * ceil_div(s.C, t.c) * s.nz;
}

double time_of(const Tiling& t, int64_t groups, int64_t steps) {
  const auto step = [&](double u) {
    return t.step + t.busy * std::min(u, 1.0) + t.more * std::max(u - 1.0, 0.0);
  };
  const int64_t slots = (int64_t)kCus * t.units, full = groups / slots, rest = groups % slots;
  double us = t.fixed;
  if (full) us += full * steps * step(t.units) + (full - 1) * t.round;
  if (rest) us += steps * step((double)rest / kCus) + (full ? t.round : 0.0);
  return us;
}

}  // namespace

ProductPlan plan_product(const ProductShape& s, int es) {
  ProductPlan pl{};
  const int64_t bk = 128 / es;  // elements of one contraction step
  pl.ktiles = ceil_div(s.K, bk);
  pl.splits = 1;
  const int64_t all = std::max<int64_t>(pl.ktiles * s.nseg, 1);  // no k: one step of zeros
  pl.per_split = all;
  if (!s.pt && !s.qt && s.nseg == 1 && s.nz == 1 && s.C <= 32) {
    pl.tile = TILE_STREAM;
    pl.stream_t = s.C <= 16 ? 1 : 2;
    pl.time = 0.0;
    return pl;
  }
  // the cheapest tile and split count by the model of the measured times
  const Tiling* table = es == 4 ? kTiles32 : s.aligned ? kTiles16 : kTiles16Gather;
  const int count = es == 2 && s.aligned ? 4 : 2;
  static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int64_t plane_ld = round_up(s.R, 8);
  const int64_t plane = plane_ld * s.C * 4 * (s.gated ? 2 : 1) * s.nz;  // bytes of one
  double best = 0.0;
  pl.tile = -1;
  for (int i = 0; i < count; ++i) {
    const int64_t tiles = tile_count(s, table[i]);
    for (int want : kSplits) {
      if (want > 1 && (all / want < 2 || tiles >= 2 * kCus || plane * want > (1LL << 30))) break;
      const int64_t per = ceil_div(all, want), n = ceil_div(all, per);
      double t = time_of(table[i], tiles * n, per);
      if (n > 1) t += kJoin + kJoinByte * (double)(plane * n);
      if (pl.tile < 0 || t < best) {
        best = t;
        pl.tile = table[i].tile;
        pl.splits = (int)n;
        pl.per_split = per;
      }
    }
  }
  pl.time = best;
  if (pl.splits > 1) {
    pl.plane_ld = plane_ld;
    pl.planes_bytes = plane * pl.splits;
  }
  return pl;
}

int plan_pair(const ProductShape& dx, const ProductShape& dw, int es) {
  if (es != 2 || !dx.aligned || !dw.aligned) return -1;
  const bool dw_first = dw.K * dw.nseg > dx.K * dx.nseg;
  const ProductShape &f = dw_first ? dw : dx, &l = dw_first ? dx : dw;
  double best = plan_product(dx, es).time + plan_product(dw, es).time;
  int tile = -1;
  for (int i = 0; i < 2; ++i) {
    const Tiling& t = kTiles16[i];
    const int64_t nf = tile_count(f, t), nl = tile_count(l, t);
    // one workgroup a compute unit; tiles of the first product, then of the last
    const double step = t.step + t.busy * std::min(1.0, (double)(nf + nl) / kCus);
    const double lf = ceil_div(f.K, 64) * f.nseg * step + t.round;
    const double ll = ceil_div(l.K, 64) * l.nseg * step + t.round;
    const int64_t full = nf / kCus, rest = nf % kCus;
    // the least time by which the units, rest of them busy for a round longer, have
    // taken every tile of the last product
    double lo = full * lf + (rest ? lf : 0.0), hi = (full + 1) * lf + (nl / kCus + 2) * ll;
    for (int k = 0; k < 40; ++k) {
      const double mid = 0.5 * (lo + hi);
      const double taken = (kCus - rest) * std::floor((mid - full * lf) / ll) +
                           rest * std::floor(std::max(0.0, mid - (full + 1) * lf) / ll);
      (taken >= (double)nl ? hi : lo) = mid;
    }
    if (t.fixed + hi < best) {
      best = t.fixed + hi;
      tile = t.tile;
    }
  }
  return tile;
}

ColsumPlan plan_colsum(int64_t m, int64_t n) {
  // one workgroup per chunk and 256 columns: about four per compute unit,
  // at least 32 rows each, at most 256 chunks to join
  const int64_t cols = ceil_div(n, 256);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(256, 4 * kCus / cols));
  ColsumPlan c;
  c.rows = std::max<int64_t>(32, round_up(ceil_div(std::max<int64_t>(m, 1), want), 8));
  c.chunks = ceil_div(std::max<int64_t>(m, 1), c.rows);
  return c;
}

ProductShape linear_product(const linear_problem* p, const LinearGeo& g) {
  ProductShape s{g.n, g.m, g.k, 1, 1, g.kn, false, false, false};
  s.aligned = vec16(g.k, g.es) && vec16(g.ldx, g.es) && vec16(p->x_off, g.es) &&
              vec16(g.ldw, g.es) && vec16(p->w_off, g.es) && (!g.kn || vec16(g.n, g.es));
  return s;
}

ProductShape linear_dx_product(const linear_problem* p, const LinearGeo& g) {
  // P = w with n contracted; Q = dz, whose rows the scratch pads with zeros
  ProductShape s{g.k, g.m, g.n, 1, 1, !g.kn, false, false, false};
  s.aligned = vec16(g.ldw, g.es) && vec16(p->w_off, g.es) && vec16(g.kn ? g.n : g.k, g.es);
  if (p->activation == CONV_ACT_IDENTITY)
    s.aligned = s.aligned && vec16(g.n, g.es) && vec16(g.ldy, g.es) && vec16(p->dy_off, g.es);
  return s;
}

ProductShape linear_dw_product(const linear_problem* p, const LinearGeo& g) {
  ProductShape s{g.kn ? g.n : g.k, g.kn ? g.k : g.n, g.m, 1, 1, true, true, false, false};
  s.aligned = vec16(g.k, g.es) && vec16(g.ldx, g.es) && vec16(p->x_off, g.es);
  if (p->activation == CONV_ACT_IDENTITY)
    s.aligned = s.aligned && vec16(g.n, g.es) && vec16(g.ldy, g.es) && vec16(p->dy_off, g.es);
  return s;
}

ProductShape gated_product(const gated_problem* p, const GatedGeo& g) {
  ProductShape s{g.f, g.m, g.k, 1, 1, false, false, true, false};
  s.aligned = vec16(g.k, g.es) && vec16(g.ldx, g.es) && vec16(p->x_off, g.es) &&
              vec16(g.ldw, g.es) && vec16(p->wg_off, g.es) && vec16(p->wu_off, g.es);
  return s;
}

ProductShape gated_dx_product(const gated_problem* p, const GatedGeo& g) {
  ProductShape s{g.k, g.m, g.f, 2, 1, true, false, false, false};
  s.aligned = vec16(g.k, g.es) && vec16(g.ldw, g.es) && vec16(p->wg_off, g.es) &&
              vec16(p->wu_off, g.es);
  return s;
}

ProductShape gated_dw_product(const gated_problem* p, const GatedGeo& g) {
  ProductShape s{g.k, g.f, g.m, 1, 2, true, true, false, false};
  s.aligned = vec16(g.k, g.es) && vec16(g.ldx, g.es) && vec16(p->x_off, g.es);
  return s;
}

BackwardScratch linear_backward_scratch(const linear_problem* p, const LinearGeo& g) {
  BackwardScratch b{};
  int64_t at = 0;
  b.dz = 0;
  b.dz_ld = round_up(g.n, 8);
  if (p->activation != CONV_ACT_IDENTITY) at += round_up(g.m * b.dz_ld * g.es, 256);
  b.sums = at;
  at += round_up(plan_colsum(g.m, g.n).chunks * round_up(g.n, 8) * 4, 256);
  b.planes = at;
  at += round_up(std::max(plan_product(linear_dx_product(p, g), g.es).planes_bytes,
                          plan_product(linear_dw_product(p, g), g.es).planes_bytes), 256);
  b.total = at;
  return b;
}

BackwardScratch gated_backward_scratch(const gated_problem* p, const GatedGeo& g) {
  BackwardScratch b{};
  int64_t at = 0;
  b.dz = 0;
  b.dz_ld = 2 * round_up(g.f, 8);
  at += round_up(g.m * b.dz_ld * g.es, 256);
  b.sums = at;
  at += round_up(plan_colsum(g.m, g.f).chunks * 2 * round_up(g.f, 8) * 4, 256);
  b.planes = at;
  at += round_up(std::max(plan_product(gated_dx_product(p, g), g.es).planes_bytes,
                          plan_product(gated_dw_product(p, g), g.es).planes_bytes), 256);
  b.total = at;
  return b;
}

namespace {

void product_name(const ProductPlan& pl, char* buf, size_t len) {
  if (pl.tile == TILE_STREAM) {
    snprintf(buf, len, "stream%d", 16 * pl.stream_t);
    return;
  }
  const char* tile = pl.tile == TILE_256       ? "tile256x256"
                     : pl.tile == TILE_256X128 ? "tile256x128"
                     : pl.tile == TILE_128     ? "tile128x128"
                                               : "tile64x64";
  if (pl.splits > 1)
    snprintf(buf, len, "%s.split%d", tile, pl.splits);
  else
    snprintf(buf, len, "%s", tile);
}

void backward_name(const char* call, int dtype, const ProductShape& sx, const ProductShape& sw,
                   int es, char* buf, size_t len) {
  const int tile = plan_pair(sx, sw, es);
  if (tile >= 0) {
    snprintf(buf, len, "%s.%s.both.tile256x%d", call, dtype_name(dtype), tile == TILE_256 ? 256 : 128);
    return;
  }
  char dx[48], dw[48];
  product_name(plan_product(sx, es), dx, sizeof dx);
  product_name(plan_product(sw, es), dw, sizeof dw);
  snprintf(buf, len, "%s.%s.dx.%s.dw.%s", call, dtype_name(dtype), dx, dw);
}

int put(const char* text, char* buf, uint64_t len) {
  const size_t need = strlen(text) + 1;
  if (!buf || len < need) return CONV_ERR_ARG;
  memcpy(buf, text, need);
  return CONV_OK;
}

int scratch_ok(const void* scratch, uint64_t bytes, int64_t need) {
  if (need == 0) return CONV_OK;
  if (bytes < (uint64_t)need) return CONV_ERR_SCRATCH;
  if (!scratch || (uintptr_t)scratch % 256 != 0) return CONV_ERR_ARG;
  return CONV_OK;
}

// every output against every input, the other outputs and the scratch; alias
// pairs (output i may equal input j exactly) are given as bit masks
int overlaps(const Range* outs, int no, const Range* ins, int ni, int alias_out, int alias_in,
             int es, const void* scratch, int64_t need) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j) {
      if (i == alias_out && j == alias_in && same(outs[i], ins[j])) continue;
      if (overlap(outs[i], ins[j], es)) return CONV_ERR_OVERLAP;
    }
    for (int j = i + 1; j < no; ++j)
      if (overlap(outs[i], outs[j], es)) return CONV_ERR_OVERLAP;
    if (bytes_overlap(outs[i], es, scratch, (uint64_t)need)) return CONV_ERR_OVERLAP;
  }
  for (int j = 0; j < ni; ++j)
    if (bytes_overlap(ins[j], es, scratch, (uint64_t)need)) return CONV_ERR_OVERLAP;
  return CONV_OK;
}

// operands aligned to their elements
bool elem_aligned(const void* p, int es) { return (uintptr_t)p % (uintptr_t)es == 0; }

}  // namespace

}  // namespace convfwd

using namespace convfwd;

extern "C" {

int linear_scratch_size(const linear_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)round_up(plan_product(linear_product(p, g), g.es).planes_bytes, 256);
  return CONV_OK;
}

int linear_backward_scratch_size(const linear_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)linear_backward_scratch(p, g).total;
  return CONV_OK;
}

int gated_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)round_up(plan_product(gated_product(p, g), g.es).planes_bytes, 256);
  return CONV_OK;
}

int gated_backward_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)gated_backward_scratch(p, g).total;
  return CONV_OK;
}

int linear_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len) {
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  char name[48], text[96];
  product_name(plan_product(linear_product(p, g), g.es), name, sizeof name);
  snprintf(text, sizeof text, "linear.%s.%s", dtype_name(dtype), name);
  return put(text, buf, len);
}

int linear_backward_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len) {
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  char text[160];
  backward_name("linear_backward", dtype, linear_dx_product(p, g), linear_dw_product(p, g), g.es,
                text, sizeof text);
  return put(text, buf, len);
}

int gated_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len) {
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  char name[48], text[96];
  product_name(plan_product(gated_product(p, g), g.es), name, sizeof name);
  snprintf(text, sizeof text, "gated.%s.%s", dtype_name(dtype), name);
  return put(text, buf, len);
}

int gated_backward_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len) {
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  char text[160];
  backward_name("gated_backward", dtype, gated_dx_product(p, g), gated_dw_product(p, g), g.es, text,
                sizeof text);
  return put(text, buf, len);
}

int linear_check(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                 const void* r, const void* y, const void* z, const void* scratch,
                 uint64_t scratch_bytes) {
  LinearGeo g;
  int st = linear_validate(p, dtype, &g);
  if (st) return st;
  if (!w || (p->has_bias && !b)) return CONV_ERR_ARG;
  // operands of m rows may be null where there is no row
  if (g.m > 0 && (!x || !y || (p->has_residual && !r) || (p->save_z && !z))) return CONV_ERR_ARG;
  Range ins[4], outs[2];
  int ni = 0, no = 0;
  const int res_at = p->has_residual ? 0 : -1;
  if (p->has_residual) ins[ni++] = range_of(r, p->r_off, g.m, g.n, g.ldr, g.es);
  ins[ni++] = range_of(x, p->x_off, g.m, g.k, g.ldx, g.es);
  ins[ni++] = range_of(w, p->w_off, g.kn ? g.k : g.n, g.kn ? g.n : g.k, g.ldw, g.es);
  if (p->has_bias) ins[ni++] = range_of(b, p->b_off, 1, g.n, g.n, g.es);
  outs[no++] = range_of(y, p->y_off, g.m, g.n, g.ldy, g.es);
  if (p->save_z) outs[no++] = range_of(z, p->z_off, g.m, g.n, g.ldz, g.es);
  for (int i = 0; i < ni; ++i)
    if (!elem_aligned((const void*)ins[i].base, g.es)) return CONV_ERR_ARG;
  for (int i = 0; i < no; ++i)
    if (!elem_aligned((const void*)outs[i].base, g.es)) return CONV_ERR_ARG;
  const int64_t need = plan_product(linear_product(p, g), g.es).planes_bytes;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, 0, res_at, g.es, scratch, need);
}

int linear_backward_check(const linear_problem* p, int dtype, const void* x, const void* w,
                          const void* z, const void* dy, const void* dx, const void* dw,
                          const void* db, const void* dr, const void* scratch,
                          uint64_t scratch_bytes) {
  LinearGeo g;
  int st = linear_validate(p, dtype, &g);
  if (st) return st;
  const bool rows = g.m > 0;  // operands of m rows may be null where there is no row
  if ((rows && !dy) || (rows && !dx && !dw && !db && !dr) || (dr && !p->has_residual) ||
      (dx && !w) || (rows && dw && !x))
    return CONV_ERR_ARG;
  const bool act = p->activation != CONV_ACT_IDENTITY;
  const bool need_z = act && (dx || dw || db || (dr && p->has_residual == LINEAR_RES_BEFORE));
  if (rows && need_z && !z) return CONV_ERR_ARG;
  Range ins[4], outs[4];
  int ni = 0, no = 0, dr_at = -1;
  const int64_t wr = g.kn ? g.k : g.n, wc = g.kn ? g.n : g.k;
  ins[ni++] = range_of(dy, p->dy_off, g.m, g.n, g.ldy, g.es);
  if (dw) ins[ni++] = range_of(x, p->x_off, g.m, g.k, g.ldx, g.es);
  if (dx) ins[ni++] = range_of(w, p->w_off, wr, wc, g.ldw, g.es);
  if (need_z) ins[ni++] = range_of(z, p->z_off, g.m, g.n, g.ldz, g.es);
  if (dx) outs[no++] = range_of(dx, p->dx_off, g.m, g.k, g.lddx, g.es);
  if (dw) outs[no++] = range_of(dw, p->dw_off, wr, wc, g.lddw, g.es);
  if (db) outs[no++] = range_of(db, p->db_off, 1, g.n, g.n, g.es);
  if (dr) {
    dr_at = no;
    outs[no++] = range_of(dr, p->dr_off, g.m, g.n, g.lddr, g.es);
  }
  for (int i = 0; i < ni; ++i)
    if (!elem_aligned((const void*)ins[i].base, g.es)) return CONV_ERR_ARG;
  for (int i = 0; i < no; ++i)
    if (!elem_aligned((const void*)outs[i].base, g.es)) return CONV_ERR_ARG;
  const int64_t need = linear_backward_scratch(p, g).total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  // dr = dy in place is exact only where every later reader has its own copy of
  // dz, or dy itself is unchanged: with dr = dz (activation, residual before)
  // the products read the scratch; otherwise dr holds dy's values
  return overlaps(outs, no, ins, ni, dr_at, 0, g.es, scratch, need);
}

int gated_check(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                const void* bg, const void* bu, const void* h, const void* pg, const void* pu,
                const void* scratch, uint64_t scratch_bytes) {
  GatedGeo g;
  int st = gated_validate(p, dtype, &g);
  if (st) return st;
  if (!wg || !wu || (p->has_bias && (!bg || !bu))) return CONV_ERR_ARG;
  if (g.m > 0 && (!x || !h || (p->save_p && (!pg || !pu)))) return CONV_ERR_ARG;
  Range ins[5], outs[3];
  int ni = 0, no = 0;
  ins[ni++] = range_of(x, p->x_off, g.m, g.k, g.ldx, g.es);
  ins[ni++] = range_of(wg, p->wg_off, g.f, g.k, g.ldw, g.es);
  ins[ni++] = range_of(wu, p->wu_off, g.f, g.k, g.ldw, g.es);
  if (p->has_bias) {
    ins[ni++] = range_of(bg, p->bg_off, 1, g.f, g.f, g.es);
    ins[ni++] = range_of(bu, p->bu_off, 1, g.f, g.f, g.es);
  }
  outs[no++] = range_of(h, p->h_off, g.m, g.f, g.ldh, g.es);
  if (p->save_p) {
    outs[no++] = range_of(pg, p->pg_off, g.m, g.f, g.ldp, g.es);
    outs[no++] = range_of(pu, p->pu_off, g.m, g.f, g.ldp, g.es);
  }
  for (int i = 0; i < ni; ++i)
    if (!elem_aligned((const void*)ins[i].base, g.es)) return CONV_ERR_ARG;
  for (int i = 0; i < no; ++i)
    if (!elem_aligned((const void*)outs[i].base, g.es)) return CONV_ERR_ARG;
  const int64_t need = plan_product(gated_product(p, g), g.es).planes_bytes;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, -1, -1, g.es, scratch, need);
}

int gated_backward_check(const gated_problem* p, int dtype, const void* x, const void* wg,
                         const void* wu, const void* pg, const void* pu, const void* dh,
                         const void* dx, const void* dwg, const void* dwu, const void* dbg,
                         const void* dbu, const void* scratch, uint64_t scratch_bytes) {
  GatedGeo g;
  int st = gated_validate(p, dtype, &g);
  if (st) return st;
  const bool rows = g.m > 0;
  if ((rows && (!pg || !pu || !dh)) || (rows && !dx && !dwg && !dbg) || !dwg != !dwu ||
      !dbg != !dbu || (dx && (!wg || !wu)) || (rows && dwg && !x))
    return CONV_ERR_ARG;
  Range ins[6], outs[5];
  int ni = 0, no = 0;
  ins[ni++] = range_of(pg, p->pg_off, g.m, g.f, g.ldp, g.es);
  ins[ni++] = range_of(pu, p->pu_off, g.m, g.f, g.ldp, g.es);
  ins[ni++] = range_of(dh, p->dh_off, g.m, g.f, g.ldh, g.es);
  if (dwg) ins[ni++] = range_of(x, p->x_off, g.m, g.k, g.ldx, g.es);
  if (dx) {
    ins[ni++] = range_of(wg, p->wg_off, g.f, g.k, g.ldw, g.es);
    ins[ni++] = range_of(wu, p->wu_off, g.f, g.k, g.ldw, g.es);
    outs[no++] = range_of(dx, p->dx_off, g.m, g.k, g.lddx, g.es);
  }
  if (dwg) {
    outs[no++] = range_of(dwg, p->dwg_off, g.f, g.k, g.lddw, g.es);
    outs[no++] = range_of(dwu, p->dwu_off, g.f, g.k, g.lddw, g.es);
  }
  if (dbg) {
    outs[no++] = range_of(dbg, p->dbg_off, 1, g.f, g.f, g.es);
    outs[no++] = range_of(dbu, p->dbu_off, 1, g.f, g.f, g.es);
  }
  for (int i = 0; i < ni; ++i)
    if (!elem_aligned((const void*)ins[i].base, g.es)) return CONV_ERR_ARG;
  for (int i = 0; i < no; ++i)
    if (!elem_aligned((const void*)outs[i].base, g.es)) return CONV_ERR_ARG;
  const int64_t need = gated_backward_scratch(p, g).total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, -1, -1, g.es, scratch, need);
}

}  // extern "C"
