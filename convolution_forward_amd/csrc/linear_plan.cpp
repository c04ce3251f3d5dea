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
// elements (beyond the card's memory)
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

// rows of cols elements (0: padded with zeros), ld apart from element off on, as
// whole 16-byte pieces at multiples of 4 bytes
bool whole_rows(int64_t cols, int64_t ld, int64_t off, int es) {
  return cols * es % 16 == 0 && ld * es % 4 == 0 && off * es % 4 == 0;
}

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
// up to units of them.  Fitted to timings of m 48 .. 8192, n and k 256 .. 4096 with 1 to
// 16 splits (of the two large tiles, before their steps had two phases).  Checked
// with 1300 timings of the present kernels at those sizes: the choice by it costs 1.1%
// more than the best of them on average, more than 10% at 6 of 135 sizes, 14% at most
// (4096 x 1024 x 256 bf16: 10.1 us for 8.8).
// It has no term for memory, and promises few rows with more weights than were fitted
// more than memory gives: one row, bf16 8192 x 4096 runs 64 x 64 tiles in 8 splits (19
// us) where the streamed kernel takes 13.5, gated 11008 x 4096 45 for 33; at 32 rows the
// tiles are the faster ones (19 for 22, 42 for 51).
struct Tiling {
  int tile, r, c, units;
  double fixed, round, step, busy, more;
};
const Tiling kTiles16[] = {{TILE_256, 256, 256, 1, 10.1, 7.3, 0.912, 0.317, 0.0},
                           {TILE_256X128, 256, 128, 1, 7.8, 3.1, 0.558, 0.227, 0.0},
                           {TILE_128, 128, 128, 2, 5.2, 0.5, 0.547, 0.096, 0.326},
                           {TILE_64, 64, 64, 4, 3.9, 2.1, 0.314, 0.0, 0.160}};
const Tiling kTiles16Gather[] = {{TILE_128, 128, 128, 2, 5.6, 0.0, 0.883, 0.123, 0.281},
                                 {TILE_64, 64, 64, 4, 3.8, 0.0, 0.465, 0.083, 0.250}};
const Tiling kTiles32[] = {{TILE_128, 128, 128, 2, 5.9, 0.0, 1.990, 0.284, 1.410},
                           {TILE_64, 64, 64, 4, 4.3, 0.0, 0.651, 0.048, 0.494}};
const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
constexpr double kJoin = 3.6, kJoinByte = 3.3e-7;  // the second pass of a split: launch, plane bytes

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
  // the cheapest tile and split count by the model of the measured times
  const Tiling* table = es == 4 ? kTiles32 : s.aligned ? kTiles16 : kTiles16Gather;
  const int count = es <= 2 && s.aligned ? 4 : 2;
  const int64_t plane_ld = round_up(s.R, 8);
  const int64_t plane = plane_ld * s.C * 4 * (s.gated ? 2 : 1) * s.nz;  // bytes of one
  double best = 0.0;
  pl.tile = -1;
  // fewer than two small tiles a compute unit: the large ones would leave most idle
  const int first = count == 4 && tile_count(s, table[3]) < 2 * kCus ? 2 : 0;
  for (int i = first; i < count; ++i) {
    const int64_t tiles = tile_count(s, table[i]);
    double before = 0.0;
    for (int want : kSplits) {
      if (want > 1 && (all / want < 2 || tiles >= 2 * kCus || plane * want > (1LL << 30))) break;
      const int64_t per = ceil_div(all, want), n = ceil_div(all, per);
      // a transposed operand that is gathered costs a third more (777 x 1001 x 1531, the
      // one size that was timed: 21 us for 16)
      const double slow = s.pt && es == 2 && !s.aligned ? 1.35 : 1.0;
      double t = slow * time_of(table[i], tiles * n, per);
      if (es == 1 && table[i].tile == TILE_256 && n == 1 && cut_tiles(tiles) > 0) {
        // the last round in halves
        const int64_t cut = cut_tiles(tiles);
        const Tiling& h = table[1];
        t = time_of(table[i], tiles - cut, per) + h.round +
            (double)per * (h.step + h.busy * (double)(2 * cut) / kCus);
      }
      if (n > 1) t += kJoin + kJoinByte * (double)(plane * n);
      // 8 bits: no less than the weights take from memory (one row, 32000 x 4096: 64 x 64
      // tiles 33 us, streamed 25)
      if (es == 1) t = std::max(t, 4.0 + (double)(s.R * s.K) / 4.4e6 + 0.01 * t);
      if (want > 2 && t > before) break;  // past the best count
      before = t;
      if (pl.tile < 0 || t < best) {
        best = t;
        pl.tile = table[i].tile;
        pl.splits = (int)n;
        pl.per_split = per;
      }
    }
  }
  if (!s.pt && !s.qt && s.nseg == 1 && s.nz == 1 && s.C <= 32 && s.K * es >= 16) {
    // the streamed kernel: on every compute unit the bytes of its weight rows, of Q
    // (from L2, 0.8 of a weight row's time) and a workgroup's start (4 rows' time), at
    // 30 KB a us (float32, bound by its products as well: 26; 16-bit rows from odd
    // elements on: 21).  Of 36 timings of bf16, 34 to 262 MB of weights, 14% below to
    // 21% above: it overrates what 16 and more rows of Q cost
    const double rate = es == 4 ? 26e3 : s.aligned ? 30e3 : 21e3;
    for (int rows = s.C > 16 ? 32 : 16; rows >= 4; rows /= 2) {
      const int64_t groups = ceil_div(s.R, rows);
      const double cost = (double)ceil_div(groups, kCus) *
                          ((s.gated ? 2 : 1) * rows + 0.8 * (double)s.C + 4.0);
      const double t = 3.0 + cost * (double)(s.K * es) / rate;
      if (t < best) {
        best = t;
        pl.tile = TILE_STREAM;
        pl.stream_t = s.C <= 16 ? 1 : 2;
        pl.stream_rows = rows;
        pl.splits = 1;
        pl.per_split = all;
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

// Counted in tiles of 64 x 64 and 256 threads each, up to 2^30 of them: larger tiles
// have no more work-items (by a quarter at most, where an odd half tile is left over), and
// the two products of one launch stay below 2^32 together.  Split products are small
// (fewer than 8 tiles a compute unit, 2^30 bytes of planes) and never cut.
int64_t launch_rows(const ProductShape& s, int splits) {
  const int64_t across = ceil_div(s.gated ? 2 * s.R : s.R, 64) * s.nz * splits;
  const int64_t rows = 64 * ((1LL << 30) / 256 / across) / 256 * 256;
  return std::min<int64_t>(std::max<int64_t>(rows, 256), 1LL << 30);
}

PairPlan plan_pair(const ProductShape& dx, const ProductShape& dw, int es) {
  const ProductPlan alone_x = plan_product(dx, es), alone_w = plan_product(dw, es);
  PairPlan out{-1, 0.0, alone_x, alone_w};
  out.time = out.dx.time + out.dw.time;
  if (!dx.aligned || !dw.aligned) return out;
  // small tiles: the contractions of both cut into pieces of one length
  const Tiling& small = es == 4 ? kTiles32[1] : kTiles16[3];
  const int64_t bk = 128 / es, ax = ceil_div(dx.K, bk) * dx.nseg, aw = ceil_div(dw.K, bk) * dw.nseg;
  const int64_t tx = tile_count(dx, small), tw = tile_count(dw, small);
  double before = 0.0;
  for (int want : kSplits) {
    const int64_t per = ceil_div(std::max(ax, aw), want);
    if (ax < 1 || aw < 1 || tx + tw >= 8 * kCus || (want > 1 && per < 2)) break;
    ProductPlan p[2] = {out.dx, out.dw};
    const ProductShape* shapes[2] = {&dx, &dw};
    const int64_t steps[2] = {ax, aw};
    int64_t bytes = 0;
    for (int i = 0; i < 2; ++i) {
      p[i].tile = TILE_64;
      p[i].ktiles = ceil_div(shapes[i]->K, bk);
      p[i].per_split = std::min(per, steps[i]);
      p[i].splits = (int)ceil_div(steps[i], per);
      p[i].plane_ld = p[i].planes_bytes = 0;
      if (p[i].splits > 1) {
        p[i].plane_ld = round_up(shapes[i]->R, 8);
        p[i].planes_bytes = p[i].plane_ld * shapes[i]->C * 4 * shapes[i]->nz * p[i].splits;
        bytes += p[i].planes_bytes;
      }
    }
    if (bytes > (1LL << 30)) break;
    double t = time_of(small, tx * p[0].splits + tw * p[1].splits, per);
    if (bytes > 0) t += kJoin + kJoinByte * (double)bytes;
    if (want > 2 && t > before) break;  // past the best count
    before = t;
    if (t < out.time) out = {TILE_64, t, p[0], p[1]};
  }
  if (es != 2) return out;
  const bool dw_first = dw.K * dw.nseg > dx.K * dx.nseg;
  const ProductShape &f = dw_first ? dw : dx, &l = dw_first ? dx : dw;
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
    for (int k = 0; k < 20; ++k) {
      const double mid = 0.5 * (lo + hi);
      const double taken = (kCus - rest) * std::floor((mid - full * lf) / ll) +
                           rest * std::floor(std::max(0.0, mid - (full + 1) * lf) / ll);
      (taken >= (double)nl ? hi : lo) = mid;
    }
    if (t.fixed + hi < out.time) out = {t.tile, t.fixed + hi, alone_x, alone_w};
  }
  return out;
}

ColsumPlan plan_colsum(int64_t m, int64_t n) {
  // one workgroup per chunk and 256 columns: about eight per compute unit,
  // at least 32 rows each, at most 256 chunks to join
  const int64_t cols = ceil_div(n, 256);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(256, 8 * kCus / cols));
  ColsumPlan c;
  c.rows = std::max<int64_t>(32, round_up(ceil_div(std::max<int64_t>(m, 1), want), 8));
  c.chunks = ceil_div(std::max<int64_t>(m, 1), c.rows);
  return c;
}

namespace {

PackItem item_of(int64_t rows, int64_t cols, int64_t ld, int64_t off, int es) {
  return {rows, cols, ld, !whole_rows(cols, ld, off, es), 0, 0};
}

// Lays the needed copies out from byte `at` on; returns their time, us.
double lay_out(Packing* k, int64_t at, int es) {
  double bytes = 0.0;
  k->bytes = 0;
  for (int i = 0; i < k->n; ++i) {
    PackItem& q = k->item[i];
    if (!q.need) continue;
    q.packed_ld = round_up(q.cols, 16 / es);
    q.off = at + k->bytes;
    k->bytes += round_up(q.rows * q.packed_ld * es, 256);
    bytes += 2.0 * (double)(q.rows * q.cols * es);
  }
  return 4.0 + bytes / 4e6;  // a launch, 4 TB/s
}

// Whether one launch can copy them: 2^33 pieces of 16 bytes are 2^31 work-items.
bool pack_fits(const Packing& k) { return k.bytes <= (1LL << 37); }

bool any_needed(const Packing& k) {
  for (int i = 0; i < k.n; ++i)
    if (k.item[i].need) return true;
  return false;
}

// One product: packs if that is estimated to pay; returns the planes' bytes.
int64_t settle(ProductShape* s, ProductPlan* run, Packing* k, int es, int64_t* total) {
  ProductPlan& pl = *run;
  pl = plan_product(*s, es);
  if (!s->aligned && s->C > 0 && pl.tile != TILE_STREAM) {
    ProductShape t = *s;
    t.aligned = true;
    const ProductPlan packed = plan_product(t, es);
    if (packed.tile != TILE_STREAM && packed.time + lay_out(k, 0, es) < pl.time && pack_fits(*k)) {
      k->on = true;
      *s = t;
      pl = packed;
    }
  }
  const int64_t planes = round_up(pl.planes_bytes, 256);
  if (k->on) lay_out(k, planes, es);
  *total = planes + (k->on ? k->bytes : 0);
  return planes;
}

// Both products of a backward pass, the same way.
void settle_backward(BackwardPlan* b, int es, int64_t at) {
  b->both = plan_pair(b->dx, b->dw, es);
  if (b->dx.C > 0 && (!b->dx.aligned || !b->dw.aligned)) {
    ProductShape x = b->dx, w = b->dw;
    x.aligned = w.aligned = true;
    const PairPlan packed = plan_pair(x, w, es);
    if (packed.time + lay_out(&b->pack, 0, es) < b->both.time && pack_fits(b->pack)) {
      b->pack.on = true;
      b->dx = x;
      b->dw = w;
      b->both = packed;
    }
  }
  b->scratch.planes = at;
  b->scratch.planes_dw = at;
  if (b->both.tile == TILE_64) {
    b->scratch.planes_dw += round_up(b->both.dx.planes_bytes, 256);
    at = b->scratch.planes_dw + round_up(b->both.dw.planes_bytes, 256);
  } else {
    at += round_up(std::max(b->both.dx.planes_bytes, b->both.dw.planes_bytes), 256);
  }
  b->scratch.pack = at;
  if (b->pack.on) {
    lay_out(&b->pack, at, es);
    at += b->pack.bytes;
  }
  b->scratch.total = at;
}

}  // namespace

LinearPlan plan_linear(const linear_problem* p, const LinearGeo& g) {
  LinearPlan o{};
  o.pack.n = 2;
  o.pack.item[0] = item_of(g.m, g.k, g.ldx, p->x_off, g.es);
  o.pack.item[1] = item_of(g.kn ? g.k : g.n, g.kn ? g.n : g.k, g.ldw, p->w_off, g.es);
  o.product = {g.n, g.m, g.k, 1, 1, g.kn, false, false, !any_needed(o.pack)};
  o.planes = settle(&o.product, &o.run, &o.pack, g.es, &o.total);
  return o;
}

LinearPlan plan_int8(int64_t m, int64_t n, int64_t k, int64_t ldx, int64_t ldw, int64_t x_off,
                     int64_t w_off) {
  LinearPlan o{};
  o.pack.n = 2;
  o.pack.item[0] = item_of(m, k, ldx, x_off, 1);
  o.pack.item[1] = item_of(n, k, ldw, w_off, 1);
  o.product = {n, m, k, 1, 1, false, false, false, !any_needed(o.pack)};
  o.planes = settle(&o.product, &o.run, &o.pack, 1, &o.total);
  return o;
}

GatedPlan plan_gated(const gated_problem* p, const GatedGeo& g) {
  GatedPlan o{};
  o.pack.n = 3;
  o.pack.item[0] = item_of(g.m, g.k, g.ldx, p->x_off, g.es);
  o.pack.item[1] = item_of(g.f, g.k, g.ldw, p->wg_off, g.es);
  o.pack.item[2] = item_of(g.f, g.k, g.ldw, p->wu_off, g.es);
  // both weights have one stride
  o.pack.item[1].need = o.pack.item[2].need = o.pack.item[1].need || o.pack.item[2].need;
  o.product = {g.f, g.m, g.k, 1, 1, false, false, true, !any_needed(o.pack)};
  o.planes = settle(&o.product, &o.run, &o.pack, g.es, &o.total);
  return o;
}

BackwardPlan plan_linear_backward(const linear_problem* p, const LinearGeo& g) {
  BackwardPlan o{};
  const bool act = p->activation != CONV_ACT_IDENTITY;
  o.pack.n = act ? 2 : 3;  // dz is laid out in scratch already
  o.pack.item[0] = item_of(g.m, g.k, g.ldx, p->x_off, g.es);
  o.pack.item[1] = item_of(g.kn ? g.k : g.n, g.kn ? g.n : g.k, g.ldw, p->w_off, g.es);
  if (!act) o.pack.item[2] = item_of(g.m, g.n, g.ldy, p->dy_off, g.es);
  const bool d = !act && o.pack.item[2].need;
  // dx: P = w with n contracted, Q = dz; dw: P and Q = x and dz, rows contracted
  o.dx = {g.k, g.m, g.n, 1, 1, !g.kn, false, false, !o.pack.item[1].need && !d};
  o.dw = {g.kn ? g.n : g.k, g.kn ? g.k : g.n, g.m, 1, 1, true, true, false, !o.pack.item[0].need && !d};
  BackwardScratch& b = o.scratch;
  int64_t at = 0;
  b.dz = 0;
  b.dz_ld = round_up(g.n, 8);
  if (act) at += round_up(g.m * b.dz_ld * g.es, 256);
  b.sums = at;
  at += round_up(plan_colsum(g.m, g.n).chunks * round_up(g.n, 8) * 4, 256);
  settle_backward(&o, g.es, at);
  return o;
}

BackwardPlan plan_gated_backward(const gated_problem* p, const GatedGeo& g) {
  BackwardPlan o{};
  o.pack.n = 3;
  o.pack.item[0] = item_of(g.m, g.k, g.ldx, p->x_off, g.es);
  o.pack.item[1] = item_of(g.f, g.k, g.ldw, p->wg_off, g.es);
  o.pack.item[2] = item_of(g.f, g.k, g.ldw, p->wu_off, g.es);
  o.pack.item[1].need = o.pack.item[2].need = o.pack.item[1].need || o.pack.item[2].need;
  o.dx = {g.k, g.m, g.f, 2, 1, true, false, false, !o.pack.item[1].need};
  o.dw = {g.k, g.f, g.m, 1, 2, true, true, false, !o.pack.item[0].need};
  BackwardScratch& b = o.scratch;
  int64_t at = 0;
  b.dz = 0;
  b.dz_ld = 2 * round_up(g.f, 8);
  at += round_up(g.m * b.dz_ld * g.es, 256);
  b.sums = at;
  at += round_up(plan_colsum(g.m, g.f).chunks * 2 * round_up(g.f, 8) * 4, 256);
  settle_backward(&o, g.es, at);
  return o;
}

void product_name(const ProductPlan& pl, char* buf, size_t len) {
  if (pl.tile == TILE_STREAM) {
    snprintf(buf, len, "stream%d.r%d", 16 * pl.stream_t, pl.stream_rows);
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

namespace {

void backward_name(const char* call, int dtype, const BackwardPlan& pl, char* buf, size_t len) {
  const char* pack = pl.pack.on ? ".pack" : "";
  const bool small = pl.both.tile == TILE_64;
  if (pl.both.tile >= 0 && !small) {
    snprintf(buf, len, "%s.%s.both.tile256x%d%s", call, dtype_name(dtype),
             pl.both.tile == TILE_256 ? 256 : 128, pack);
    return;
  }
  char dx[48], dw[48];
  product_name(pl.both.dx, dx, sizeof dx);
  product_name(pl.both.dw, dw, sizeof dw);
  snprintf(buf, len, "%s.%s.dx.%s.dw.%s%s%s", call, dtype_name(dtype), dx, dw, small ? ".both" : "",
           pack);
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
  *bytes = (uint64_t)plan_linear(p, g).total;
  return CONV_OK;
}

int linear_backward_scratch_size(const linear_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_linear_backward(p, g).scratch.total;
  return CONV_OK;
}

int gated_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_gated(p, g).total;
  return CONV_OK;
}

int gated_backward_scratch_size(const gated_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_gated_backward(p, g).scratch.total;
  return CONV_OK;
}

int linear_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len) {
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  char name[48], text[96];
  const LinearPlan pl = plan_linear(p, g);
  product_name(pl.run, name, sizeof name);
  snprintf(text, sizeof text, "linear.%s.%s%s", dtype_name(dtype), name, pl.pack.on ? ".pack" : "");
  return put(text, buf, len);
}

int linear_backward_describe_variant(const linear_problem* p, int dtype, char* buf, uint64_t len) {
  LinearGeo g;
  const int st = linear_validate(p, dtype, &g);
  if (st) return st;
  char text[160];
  backward_name("linear_backward", dtype, plan_linear_backward(p, g), text, sizeof text);
  return put(text, buf, len);
}

int gated_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len) {
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  char name[48], text[96];
  const GatedPlan pl = plan_gated(p, g);
  product_name(pl.run, name, sizeof name);
  snprintf(text, sizeof text, "gated.%s.%s%s", dtype_name(dtype), name, pl.pack.on ? ".pack" : "");
  return put(text, buf, len);
}

int gated_backward_describe_variant(const gated_problem* p, int dtype, char* buf, uint64_t len) {
  GatedGeo g;
  const int st = gated_validate(p, dtype, &g);
  if (st) return st;
  char text[160];
  backward_name("gated_backward", dtype, plan_gated_backward(p, g), text, sizeof text);
  return put(text, buf, len);
}

}  // extern "C"

namespace convfwd {

int linear_checked(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                   const void* r, const void* y, const void* z, const void* scratch,
                   uint64_t scratch_bytes,
                   LinearGeo* go, LinearPlan* plan) {
  LinearGeo& g = *go;
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
  *plan = plan_linear(p, g);
  const int64_t need = plan->total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, 0, res_at, g.es, scratch, need);
}

int linear_backward_checked(const linear_problem* p, int dtype, const void* x, const void* w,
                            const void* z, const void* dy, const void* dx, const void* dw,
                            const void* db, const void* dr, const void* scratch,
                            uint64_t scratch_bytes,
                            LinearGeo* go, BackwardPlan* plan) {
  LinearGeo& g = *go;
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
  *plan = plan_linear_backward(p, g);
  const int64_t need = plan->scratch.total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  // dr = dy in place is exact only where every later reader has its own copy of
  // dz, or dy itself is unchanged: with dr = dz (activation, residual before)
  // the products read the scratch; otherwise dr holds dy's values
  return overlaps(outs, no, ins, ni, dr_at, 0, g.es, scratch, need);
}

int gated_checked(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                  const void* bg, const void* bu, const void* h, const void* pg, const void* pu,
                  const void* scratch, uint64_t scratch_bytes,
                  GatedGeo* go, GatedPlan* plan) {
  GatedGeo& g = *go;
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
  *plan = plan_gated(p, g);
  const int64_t need = plan->total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, -1, -1, g.es, scratch, need);
}

int gated_backward_checked(const gated_problem* p, int dtype, const void* x, const void* wg,
                           const void* wu, const void* pg, const void* pu, const void* dh,
                           const void* dx, const void* dwg, const void* dwu, const void* dbg,
                           const void* dbu, const void* scratch, uint64_t scratch_bytes,
                           GatedGeo* go, BackwardPlan* plan) {
  GatedGeo& g = *go;
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
  *plan = plan_gated_backward(p, g);
  const int64_t need = plan->scratch.total;
  st = scratch_ok(scratch, scratch_bytes, need);
  if (st) return st;
  return overlaps(outs, no, ins, ni, -1, -1, g.es, scratch, need);
}

}  // namespace convfwd

extern "C" {

int linear_check(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                 const void* r, const void* y, const void* z, const void* scratch,
                 uint64_t scratch_bytes) {
  LinearGeo g;
  LinearPlan plan;
  return linear_checked(p, dtype, x, w, b, r, y, z, scratch, scratch_bytes, &g, &plan);
}

int linear_backward_check(const linear_problem* p, int dtype, const void* x, const void* w,
                          const void* z, const void* dy, const void* dx, const void* dw,
                          const void* db, const void* dr, const void* scratch,
                          uint64_t scratch_bytes) {
  LinearGeo g;
  BackwardPlan plan;
  return linear_backward_checked(p, dtype, x, w, z, dy, dx, dw, db, dr, scratch, scratch_bytes, &g, &plan);
}

int gated_check(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                const void* bg, const void* bu, const void* h, const void* pg, const void* pu,
                const void* scratch, uint64_t scratch_bytes) {
  GatedGeo g;
  GatedPlan plan;
  return gated_checked(p, dtype, x, wg, wu, bg, bu, h, pg, pu, scratch, scratch_bytes, &g, &plan);
}

int gated_backward_check(const gated_problem* p, int dtype, const void* x, const void* wg,
                         const void* wu, const void* pg, const void* pu, const void* dh,
                         const void* dx, const void* dwg, const void* dwu, const void* dbg,
                         const void* dbu, const void* scratch, uint64_t scratch_bytes) {
  GatedGeo g;
  BackwardPlan plan;
  return gated_backward_checked(p, dtype, x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu, scratch, scratch_bytes, &g, &plan);
}

}  // extern "C"
