// Host half of include/linear_int8.h's product that never touches the device.
#include "linear_int8_plan.h"

#include <stdio.h>

namespace convfwd {

int int8_validate(const linear_int8_problem* p, int dtype, Int8Geo* out) {
  if (!p || !float_dtype(dtype)) return CONV_ERR_ARG;
  if (p->activation < CONV_ACT_IDENTITY || p->activation > LINEAR_ACT_GELU_TANH ||
      (p->has_bias != 0 && p->has_bias != 1) || p->has_residual < LINEAR_RES_NONE ||
      p->has_residual > LINEAR_RES_AFTER || p->reserved != 0)
    return CONV_ERR_ARG;
  const int64_t offs[] = {p->x_off, p->xs_off, p->w_off, p->ws_off, p->b_off, p->r_off, p->y_off};
  for (int64_t o : offs)
    if (o < 0) return CONV_ERR_ARG;
  Int8Geo g{};
  g.m = p->m; g.n = p->n; g.k = p->k;
  if (g.m < 0 || g.m > kRowsMax || g.n < 1 || g.n > kExtentMax || g.k < 1 || g.k > kInt8MaxK)
    return CONV_ERR_SHAPE;
  g.es = (int)dtype_size(dtype);
  g.ldx = row_stride(p->ldx, g.k);
  g.ldw = row_stride(p->ldw, g.k);
  g.ldr = row_stride(p->ldr, g.n);
  g.ldy = row_stride(p->ldy, g.n);
  if (g.ldx < 0 || g.ldw < 0 || g.ldr < 0 || g.ldy < 0) return CONV_ERR_SHAPE;
  if (!offset_fits(p->x_off, g.m, g.ldx, 1) || !offset_fits(p->xs_off, g.m, 1, 4) ||
      !offset_fits(p->w_off, g.n, g.ldw, 1) || !offset_fits(p->ws_off, g.n, 1, 4) ||
      !offset_fits(p->b_off, 1, g.n, g.es) || !offset_fits(p->r_off, g.m, g.ldr, g.es) ||
      !offset_fits(p->y_off, g.m, g.ldy, g.es))
    return CONV_ERR_SHAPE;
  *out = g;
  return CONV_OK;
}

LinearPlan plan_linear_int8(const linear_int8_problem* p, const Int8Geo& g) {
  return plan_int8(g.m, g.n, g.k, g.ldx, g.ldw, p->x_off, p->w_off);
}

int linear_int8_checked(const linear_int8_problem* p, int dtype, const void* x, const void* xs,
                        const void* w, const void* ws, const void* b, const void* r, const void* y,
                        const void* scratch, uint64_t scratch_bytes, Int8Geo* go,
                        LinearPlan* plan) {
  Int8Geo& g = *go;
  int st = int8_validate(p, dtype, &g);
  if (st) return st;
  if (!w || !ws || (p->has_bias && !b)) return CONV_ERR_ARG;
  // operands of m rows may be null where there is no row
  if (g.m > 0 && (!x || !xs || !y || (p->has_residual && !r))) return CONV_ERR_ARG;
  Operands o;
  o.read(operand(x, p->x_off, g.m, g.k, g.ldx, 1));
  o.read(operand(xs, p->xs_off, 1, g.m, g.m, 4));
  o.read(operand(w, p->w_off, g.n, g.k, g.ldw, 1));
  o.read(operand(ws, p->ws_off, 1, g.n, g.n, 4));
  if (p->has_bias) o.read(operand(b, p->b_off, 1, g.n, g.n, g.es));
  const int res = p->has_residual ? o.read(operand(r, p->r_off, g.m, g.n, g.ldr, g.es)) : 0;
  o.write(operand(y, p->y_off, g.m, g.n, g.ldy, g.es), res);
  *plan = plan_linear_int8(p, g);
  st = scratch_fits(scratch, scratch_bytes, plan->total);
  if (st) return st;
  return o.check(scratch, plan->total);
}

}  // namespace convfwd

using namespace convfwd;

extern "C" {

int linear_int8_scratch_size(const linear_int8_problem* p, int dtype, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  Int8Geo g;
  const int st = int8_validate(p, dtype, &g);
  if (st) return st;
  *bytes = (uint64_t)plan_linear_int8(p, g).total;
  return CONV_OK;
}

int linear_int8_describe_variant(const linear_int8_problem* p, int dtype, char* buf, uint64_t len) {
  Int8Geo g;
  const int st = int8_validate(p, dtype, &g);
  if (st) return st;
  char name[48], text[112];
  const LinearPlan pl = plan_linear_int8(p, g);
  product_name(pl.run, name, sizeof name);
  const bool cut = pl.run.tile == TILE_256 && pl.run.splits == 1 &&
                   cut_tiles(ceil_div(g.n, 256) * ceil_div(g.m, 256)) > 0;
  snprintf(text, sizeof text, "linear_int8.%s.%s%s%s", float_dtype_name(dtype), name,
           cut ? ".cut" : "", pl.pack.on ? ".pack" : "");
  return put_name(text, buf, len);
}

int linear_int8_check(const linear_int8_problem* p, int dtype, const void* x, const void* xs,
                      const void* w, const void* ws, const void* b, const void* r, const void* y,
                      const void* scratch, uint64_t scratch_bytes) {
  Int8Geo g;
  LinearPlan plan;
  return linear_int8_checked(p, dtype, x, xs, w, ws, b, r, y, scratch, scratch_bytes, &g, &plan);
}

}  // extern "C"
