// Host half of include/layer_norm.h, include/dropout.h and quantize_rows that never
// touches the device.
#include "rows_plan.h"

#include <math.h>
#include <stdio.h>

#include <algorithm>

namespace convfwd {

namespace {

constexpr int kCus = 256;  // gfx950

bool flag(int v) { return v == 0 || v == 1; }

bool probability(float p) { return p >= 0.0f && p <= 1.0f; }

bool off8(const void* p) { return (uintptr_t)p % 8 != 0; }

// Threads that hold a row of up to 32768 elements, one run of 8 each where that does
// not take too many: more runs a thread cost registers, and with them loads in flight
// (bf16 16384 x 2048: 64 threads of 4 runs 63 us, 256 of 1 53; 4096 x 8192: 256 of 4 63,
// 1024 of 1 54).  A row that does not fill its threads leaves some without loads, which
// weighs most just above 4096 (widths of 33.5 million elements in all, no dropout or residual:
// bfloat16 forward 5.2 TB/s at 4096, 3.1 at 4104, 3.5 at 5120, 4.2 at 7168, 4.4 at 8192; backward
// 4.4, 3.8, 4.1, 4.4, 4.4; float32 forward 5.1, 4.4, 4.6, 4.8, 5.0, backward 4.8 to 5.2 throughout).
RowPlan row_plan(int64_t runs) {
  if (runs <= 8) return {8, 1, 0};
  if (runs <= 16) return {16, 1, 0};
  if (runs <= 32) return {32, 1, 0};
  if (runs <= 128) return {64, runs <= 64 ? 1 : 2, 0};
  if (runs <= 512) return {256, runs <= 256 ? 1 : 2, 0};
  return {1024, runs <= 1024 ? 1 : runs <= 2048 ? 2 : 4, 0};
}

}  // namespace

int drop_threshold(float p) { return (int)nearbyint((double)p * 65536.0); }

// ------------------------------------------------------------------- layer norm

int layer_norm_validate(const layer_norm_problem* p, int dtype, NormGeo* out) {
  if (!p || !float_dtype(dtype)) return CONV_ERR_ARG;
  if (!flag(p->has_weight) || !flag(p->has_bias) || !flag(p->has_residual) || p->reserved != 0 ||
      !probability(p->drop) || !(p->eps >= 0.0f) || isinf(p->eps))
    return CONV_ERR_ARG;
  const int64_t offs[] = {p->x_off, p->r_off, p->w_off, p->b_off, p->y_off, p->s_off,
                          p->dy_off, p->ds_off, p->dx_off, p->dr_off, p->dw_off, p->db_off};
  for (int64_t o : offs)
    if (o < 0) return CONV_ERR_ARG;
  if (p->m < 0 || p->m > kRowsMax || p->n < 1 || p->n > kExtentMax) return CONV_ERR_SHAPE;
  NormGeo g{};
  g.m = p->m;
  g.n = p->n;
  g.es = (int)dtype_size(dtype);
  int64_t* lds[] = {&g.ldx, &g.ldr, &g.ldy, &g.lds, &g.ldds, &g.lddx, &g.lddr};
  const int64_t given[] = {p->ldx, p->ldr, p->ldy, p->lds, p->ldds, p->lddx, p->lddr};
  for (int i = 0; i < 7; ++i) {
    *lds[i] = row_stride(given[i], g.n);
    if (*lds[i] < 0) return CONV_ERR_SHAPE;
  }
  const int64_t off_ld[][2] = {{p->x_off, g.ldx},   {p->r_off, g.ldr},   {p->y_off, g.ldy},
                               {p->s_off, g.lds},   {p->dy_off, g.ldy},  {p->ds_off, g.ldds},
                               {p->dx_off, g.lddx}, {p->dr_off, g.lddr}};
  for (const auto& o : off_ld)
    if (!offset_fits(o[0], g.m, o[1], g.es)) return CONV_ERR_SHAPE;
  for (int64_t o : {p->w_off, p->b_off, p->dw_off, p->db_off})
    if (!offset_fits(o, 1, g.n, g.es)) return CONV_ERR_SHAPE;
  *out = g;
  return CONV_OK;
}

NormPlan plan_layer_norm(const NormGeo& g) {
  NormPlan o{};
  const int64_t runs = ceil_div(g.n, 8);
  if (runs <= 4096) {
    o.row = row_plan(runs);
  } else {
    o.row = {256, 2, ceil_div(runs, 256 * 2)};
    // a mean and a sum of squares for each part of each row
    o.scratch = ceil_div(g.m * o.row.parts * 8, 256) * 256;
  }
  return o;
}

NormBackwardPlan plan_layer_norm_backward(const NormGeo& g) {
  NormBackwardPlan o{};
  const int64_t runs = ceil_div(g.n, 8), np = runs * 8;
  int64_t at = 0;
  if (runs <= 1024) {
    o.row = row_plan(runs);
    o.teams = o.row.threads >= 256 ? 1 : 256 / o.row.threads;
  } else {
    o.row = {256, 1, ceil_div(runs, 256)};
    o.teams = 1;
    o.sums = at;
    at += ceil_div(g.m * o.row.parts * 8, 256) * 256;
  }
  // Workgroups that sum columns read s and dy once more, each at the rate of a unit, but
  // spare the partial rows and a launch.  Kernels, us for those of partial rows, float16
  // and float32: 512 x 4096 7.8 for 17 and 8.9 for 18, 1024 x 4096 14 for 19 and 15 for 18, 1024 x
  // 2048 11 for 13 and 12 for 14, 512 x 8192 14 for 18 and 18 for 18, 32 x 50176 11 for 23 and
  // 13 for 23, 256 x 16384 16 for 22 and 19 for 23.  Narrow rows near the limit lose some of
  // the kernels' time, 777 x 1001 8.5 for 8.5 and 9.5 for 9.0, 1024 x 1000 9.8 for 8.8 and 11 for
  // 9.2, 1000 x 240 7.0 for 5.6 and 6.9 for 5.7, and gain a launch where calls are not replayed
  // from a graph (float16 777 x 1001 9.1 for 11.8, 1024 x 63 8 for 11).  Beyond the limits,
  // float16: 2048 x 1001 19 for 14, 777 x 8192 24 for 20, 512 x 16384 29 for 26.
  o.once = g.m <= kOnceRows && g.m * g.n <= 1 << 22;
  if (o.once && !o.row.parts) {
    o.groups = ceil_div(g.m, o.teams);
    return o;
  }
  // Every group writes a partial row and the join reads it, too few leave loads unhidden:
  // eight rows each, within 512 groups and what the registers let run at once (float16
  // 2048 x 2048: 512 groups 17 us, 1024 20; 16384 x 1001: 1024 or 512 40, 256 54;
  // 8192 x 2048: 1024 35, 512 37).
  int64_t most = o.row.parts ? std::max<int64_t>(1, 4 * kCus / o.row.parts)
                 : o.row.threads == 1024 ? kCus : o.row.runs == 2 ? 2 * kCus : 4 * kCus;
  if (!o.row.parts) most = std::min(most, std::max<int64_t>(2 * kCus, ceil_div(g.m, 8 * o.teams)));
  o.groups = std::max<int64_t>(1, std::min<int64_t>(most, ceil_div(g.m, o.teams)));
  o.partials = at;
  if (!o.once) at += ceil_div(o.groups * 2 * np * 4, 256) * 256;
  o.scratch = at;
  return o;
}

namespace {

void row_name(const RowPlan& r, char* buf, size_t len) {
  if (r.parts)
    snprintf(buf, len, "split%lld", (long long)r.parts);
  else
    snprintf(buf, len, "rows%dx%d", r.threads, r.runs);
}

}  // namespace

int layer_norm_checked(const layer_norm_problem* p, int dtype, const void* x, const void* r,
                       const void* w, const void* b, const void* y, const void* s,
                       const void* mean, const void* rstd, const void* step, const void* scratch,
                       uint64_t scratch_bytes, NormGeo* go, NormPlan* plan) {
  NormGeo& g = *go;
  int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  if ((p->has_weight && !w) || (p->has_bias && !b) || !mean != !rstd || off8(step)) return CONV_ERR_ARG;
  // operands of m rows may be null where there is no row
  if (g.m > 0 && (!x || !y || (p->has_residual && !r))) return CONV_ERR_ARG;
  Operands o;
  int rows = o.read(operand(x, p->x_off, g.m, g.n, g.ldx, g.es));
  if (p->has_residual) rows |= o.read(operand(r, p->r_off, g.m, g.n, g.ldr, g.es));
  if (p->has_weight) o.read(operand(w, p->w_off, 1, g.n, g.n, g.es));
  if (p->has_bias) o.read(operand(b, p->b_off, 1, g.n, g.n, g.es));
  if (step && p->drop > 0.0f) o.read(operand(step, 0, 1, 1, 1, 8));
  o.write(operand(y, p->y_off, g.m, g.n, g.ldy, g.es), rows);
  if (s) o.write(operand(s, p->s_off, g.m, g.n, g.lds, g.es), rows);
  if (mean) {
    o.write(operand(mean, 0, g.m, 1, 1, 4));
    o.write(operand(rstd, 0, g.m, 1, 1, 4));
  }
  *plan = plan_layer_norm(g);
  st = scratch_fits(scratch, scratch_bytes, plan->scratch);
  if (st) return st;
  return o.check(scratch, plan->scratch);
}

int layer_norm_backward_checked(const layer_norm_problem* p, int dtype, const void* s,
                                const void* w, const void* mean, const void* rstd, const void* dy,
                                const void* ds, const void* dx, const void* dr, const void* dw,
                                const void* db, const void* step, const void* scratch,
                                uint64_t scratch_bytes, NormGeo* go, NormBackwardPlan* plan) {
  NormGeo& g = *go;
  int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  if ((p->has_weight && !w) || off8(step) || (dr && !p->has_residual) || (dw && !p->has_weight) ||
      (db && !p->has_bias))
    return CONV_ERR_ARG;
  if (g.m > 0 && (!s || !mean || !rstd || !dy || (!dx && !dr && !dw && !db))) return CONV_ERR_ARG;
  Operands o;
  int rows = o.read(operand(dy, p->dy_off, g.m, g.n, g.ldy, g.es));
  if (ds) rows |= o.read(operand(ds, p->ds_off, g.m, g.n, g.ldds, g.es));
  o.read(operand(s, p->s_off, g.m, g.n, g.lds, g.es));
  if (p->has_weight) o.read(operand(w, p->w_off, 1, g.n, g.n, g.es));
  o.read(operand(mean, 0, g.m, 1, 1, 4));
  o.read(operand(rstd, 0, g.m, 1, 1, 4));
  if (step && p->drop > 0.0f) o.read(operand(step, 0, 1, 1, 1, 8));
  if (dx) o.write(operand(dx, p->dx_off, g.m, g.n, g.lddx, g.es), rows);
  if (dr) o.write(operand(dr, p->dr_off, g.m, g.n, g.lddr, g.es), rows);
  if (dw) o.write(operand(dw, p->dw_off, 1, g.n, g.n, g.es));
  if (db) o.write(operand(db, p->db_off, 1, g.n, g.n, g.es));
  *plan = plan_layer_norm_backward(g);
  st = scratch_fits(scratch, scratch_bytes, plan->scratch);
  if (st) return st;
  return o.check(scratch, plan->scratch);
}

// ---------------------------------------------------------------------- dropout

namespace {

int dropout_validate(const dropout_problem* p, int dtype, DropGeo* out) {
  if (!p || !float_dtype(dtype)) return CONV_ERR_ARG;
  if (!flag(p->has_residual) || p->reserved != 0 || !probability(p->drop)) return CONV_ERR_ARG;
  if (p->x_off < 0 || p->r_off < 0 || p->y_off < 0) return CONV_ERR_ARG;
  if (p->m < 0 || p->m > kRowsMax || p->n < 1 || p->n > kExtentMax) return CONV_ERR_SHAPE;
  DropGeo g{};
  g.m = p->m;
  g.n = p->n;
  g.es = (int)dtype_size(dtype);
  g.ldx = row_stride(p->ldx, g.n);
  g.ldr = row_stride(p->ldr, g.n);
  g.ldy = row_stride(p->ldy, g.n);
  if (g.ldx < 0 || g.ldr < 0 || g.ldy < 0) return CONV_ERR_SHAPE;
  if (!offset_fits(p->x_off, g.m, g.ldx, g.es) || !offset_fits(p->r_off, g.m, g.ldr, g.es) ||
      !offset_fits(p->y_off, g.m, g.ldy, g.es))
    return CONV_ERR_SHAPE;
  // float32 4096 x 4096: one run a thread 28.0 us, two 26.8, four 27.2; 2048 x 1024 5.1, 5.2,
  // 5.4.  bfloat16 8192 x 11008 60.9, 62.9, 63.8, 32768 x 1001 26, 28, 33.
  g.runs = g.es == 4 && g.m * ceil_div(g.n, 8) >= 1 << 20 ? 2 : 1;
  *out = g;
  return CONV_OK;
}

}  // namespace

int dropout_checked(const dropout_problem* p, int dtype, const void* x, const void* r,
                    const void* y, const void* step, DropGeo* g) {
  const int st = dropout_validate(p, dtype, g);
  if (st) return st;
  if (off8(step)) return CONV_ERR_ARG;
  if (g->m > 0 && (!x || !y || (p->has_residual && !r))) return CONV_ERR_ARG;
  Operands o;
  int rows = o.read(operand(x, p->x_off, g->m, g->n, g->ldx, g->es));
  if (p->has_residual) rows |= o.read(operand(r, p->r_off, g->m, g->n, g->ldr, g->es));
  if (step) o.read(operand(step, 0, 1, 1, 1, 8));
  o.write(operand(y, p->y_off, g->m, g->n, g->ldy, g->es), rows);
  return o.check(nullptr, 0);
}

int dropout_backward_checked(const dropout_problem* p, int dtype, const void* dy, const void* dx,
                             const void* step, DropGeo* g) {
  const int st = dropout_validate(p, dtype, g);
  if (st) return st;
  if (off8(step) || (g->m > 0 && (!dy || !dx))) return CONV_ERR_ARG;
  Operands o;
  const int in = o.read(operand(dy, p->y_off, g->m, g->n, g->ldy, g->es));
  if (step) o.read(operand(step, 0, 1, 1, 1, 8));
  o.write(operand(dx, p->x_off, g->m, g->n, g->ldx, g->es), in);
  return o.check(nullptr, 0);
}

// --------------------------------------------------------------- rows to 8 bits

int quantize_checked(const quantize_problem* p, int dtype, const void* x, const void* q,
                     const void* scale, QuantGeo* out) {
  if (!p || !float_dtype(dtype)) return CONV_ERR_ARG;
  if (p->reserved != 0 || p->x_off < 0 || p->q_off < 0 || p->scale_off < 0) return CONV_ERR_ARG;
  if (p->m < 0 || p->m > kRowsMax || p->n < 1 || p->n > kExtentMax) return CONV_ERR_SHAPE;
  QuantGeo g{};
  g.m = p->m;
  g.n = p->n;
  g.es = (int)dtype_size(dtype);
  g.ldx = row_stride(p->ldx, g.n);
  g.ldq = row_stride(p->ldq, g.n);
  if (g.ldx < 0 || g.ldq < 0) return CONV_ERR_SHAPE;
  if (!offset_fits(p->x_off, g.m, g.ldx, g.es) || !offset_fits(p->q_off, g.m, g.ldq, 1) ||
      !offset_fits(p->scale_off, g.m, 1, 4))
    return CONV_ERR_SHAPE;
  if (g.m > 0 && (!x || !q || !scale)) return CONV_ERR_ARG;
  Operands o;
  o.read(operand(x, p->x_off, g.m, g.n, g.ldx, g.es));
  o.write(operand(q, p->q_off, g.m, g.n, g.ldq, 1));
  o.write(operand(scale, p->scale_off, g.m, 1, 1, 4));
  const int st = o.check(nullptr, 0);
  if (st) return st;
  const int64_t runs = ceil_div(g.n, 8);
  g.row = runs <= 4096 ? row_plan(runs) : RowPlan{1024, 4, ceil_div(runs, 4096)};
  *out = g;
  return CONV_OK;
}

}  // namespace convfwd

using namespace convfwd;

extern "C" {

int layer_norm_scratch_size(const layer_norm_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  NormGeo g;
  const int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_layer_norm(g).scratch;
  return CONV_OK;
}

int layer_norm_backward_scratch_size(const layer_norm_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  NormGeo g;
  const int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_layer_norm_backward(g).scratch;
  return CONV_OK;
}

int layer_norm_describe_variant(const layer_norm_problem* p, int dtype, char* buf, uint64_t len) {
  NormGeo g;
  const int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  char row[40], text[80];
  row_name(plan_layer_norm(g).row, row, sizeof row);
  snprintf(text, sizeof text, "layer_norm.%s.%s", float_dtype_name(dtype), row);
  return put_name(text, buf, len);
}

int layer_norm_backward_describe_variant(const layer_norm_problem* p, int dtype, char* buf,
                                         uint64_t len) {
  NormGeo g;
  const int st = layer_norm_validate(p, dtype, &g);
  if (st) return st;
  char row[40], text[80];
  const NormBackwardPlan plan = plan_layer_norm_backward(g);
  row_name(plan.row, row, sizeof row);
  snprintf(text, sizeof text, "layer_norm_backward.%s.%s%s", float_dtype_name(dtype), row,
           plan.once ? ".once" : "");
  return put_name(text, buf, len);
}

int layer_norm_check(const layer_norm_problem* p, int dtype, const void* x, const void* r,
                     const void* w, const void* b, const void* y, const void* s, const void* mean,
                     const void* rstd, const void* step, const void* scratch,
                     uint64_t scratch_bytes) {
  NormGeo g;
  NormPlan plan;
  return layer_norm_checked(p, dtype, x, r, w, b, y, s, mean, rstd, step, scratch, scratch_bytes,
                            &g, &plan);
}

int layer_norm_backward_check(const layer_norm_problem* p, int dtype, const void* s, const void* w,
                              const void* mean, const void* rstd, const void* dy, const void* ds,
                              const void* dx, const void* dr, const void* dw, const void* db,
                              const void* step, const void* scratch, uint64_t scratch_bytes) {
  NormGeo g;
  NormBackwardPlan plan;
  return layer_norm_backward_checked(p, dtype, s, w, mean, rstd, dy, ds, dx, dr, dw, db, step,
                                     scratch, scratch_bytes, &g, &plan);
}

int dropout_describe_variant(const dropout_problem* p, int dtype, char* buf, uint64_t len) {
  DropGeo g;
  const int st = dropout_validate(p, dtype, &g);
  if (st) return st;
  char text[64];
  snprintf(text, sizeof text, "dropout.%s.runs%d", float_dtype_name(dtype), g.runs);
  return put_name(text, buf, len);
}

int dropout_check(const dropout_problem* p, int dtype, const void* x, const void* r, const void* y,
                  const void* step) {
  DropGeo g;
  return dropout_checked(p, dtype, x, r, y, step, &g);
}

int dropout_backward_check(const dropout_problem* p, int dtype, const void* dy, const void* dx,
                           const void* step) {
  DropGeo g;
  return dropout_backward_checked(p, dtype, dy, dx, step, &g);
}

int quantize_check(const quantize_problem* p, int dtype, const void* x, const void* q,
                   const void* scale) {
  QuantGeo g;
  return quantize_checked(p, dtype, x, q, scale, &g);
}

}  // extern "C"
