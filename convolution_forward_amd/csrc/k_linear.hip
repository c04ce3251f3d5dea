// Launch half of include/linear.h: runs the shape-only plans of linear_plan.cpp
// as gfx950 launches on the caller's stream.  Nothing here allocates, frees or
// synchronises.
#include <algorithm>

#include "linear_launch.h"

using namespace convfwd;

namespace {

hipError_t product(int dtype, const ProductArgs& a, int tile, int layout, bool gated, bool dma,
                   hipStream_t s) {
  if (dtype == CONV_F16) return launch_product<_Float16>(a, tile, layout, gated, dma, s);
  if (dtype == CONV_BF16) return launch_product<__bf16>(a, tile, layout, gated, dma, s);
  return launch_product<float>(a, tile, layout, gated, dma, s);
}

hipError_t stream_product(int dtype, const ProductArgs& a, int blocks16, int rows, bool gated,
                          bool vec, hipStream_t s) {
  if (dtype == CONV_F16) return launch_stream<_Float16>(a, blocks16, rows, gated, vec, s);
  if (dtype == CONV_BF16) return launch_stream<__bf16>(a, blocks16, rows, gated, vec, s);
  return launch_stream<float>(a, blocks16, rows, gated, vec, s);
}

hipError_t join(int dtype, const JoinArgs& a, bool gated, hipStream_t s) {
  if (dtype == CONV_F16) return launch_join<_Float16>(a, gated, s);
  if (dtype == CONV_BF16) return launch_join<__bf16>(a, gated, s);
  return launch_join<float>(a, gated, s);
}

hipError_t join_pair(int dtype, const JoinArgs& a, const JoinArgs& b, hipStream_t s) {
  if (dtype == CONV_F16) return launch_join_pair<_Float16>(a, b, s);
  if (dtype == CONV_BF16) return launch_join_pair<__bf16>(a, b, s);
  return launch_join_pair<float>(a, b, s);
}

hipError_t dz_pass(int dtype, const DzArgs& a, bool gated, int chunks, hipStream_t s) {
  if (dtype == CONV_F16) return launch_dz<_Float16>(a, gated, chunks, s);
  if (dtype == CONV_BF16) return launch_dz<__bf16>(a, gated, chunks, s);
  return launch_dz<float>(a, gated, chunks, s);
}

hipError_t sums_pass(int dtype, const SumsArgs& a, hipStream_t s) {
  if (dtype == CONV_F16) return launch_sums<_Float16>(a, s);
  if (dtype == CONV_BF16) return launch_sums<__bf16>(a, s);
  return launch_sums<float>(a, s);
}

// The product's rows c0 .. c0 + rows alone.
ProductArgs rows_from(const ProductShape& s, ProductArgs a, int64_t c0, int64_t rows, int es) {
  a.C = (int)std::min(rows, s.C - c0);
  if (c0 == 0) return a;
  LinEpilogue& e = a.e;
  for (int i = 0; i < 2; ++i) {
    a.Q[i] = at(a.Q[i], s.qt ? c0 : c0 * a.ldq, es);
    e.out[i] = at(e.out[i], c0 * e.ldo, es);
    e.save[i] = at(e.save[i], c0 * e.ldsave, es);
  }
  e.res = at(e.res, c0 * e.ldres, es);
  return a;
}

// Runs one planned product; a's operands and epilogue are set.
hipError_t run_product(const ProductShape& s, const ProductPlan& pl, int dtype, ProductArgs& a,
                       bool p_padded, bool q_padded, void* planes, hipStream_t st) {
  const int es = (int)dtype_size(dtype);
  set_plan(s, pl, planes, &a);
  const bool dma = direct(s, a, es, p_padded, q_padded);
  if (pl.tile == TILE_STREAM)
    return stream_product(dtype, a, pl.stream_t, pl.stream_rows, s.gated, dma, st);
  const int layout = s.pt ? (s.qt ? 2 : 1) : 0;
  const int64_t rows = launch_rows(s, pl.splits);
  hipError_t e = hipSuccess;
  for (int64_t c = 0; c < s.C && e == hipSuccess; c += rows)
    e = product(dtype, rows_from(s, a, c, rows, es), pl.tile, layout, s.gated, dma, st);
  if (e != hipSuccess || pl.splits == 1) return e;
  return join(dtype, join_of(s, a), s.gated, st);
}

hipError_t pair(int dtype, const PairArgs& a, int tile, bool dx_transposed, hipStream_t s) {
  if (dtype == CONV_F16) return launch_pair<_Float16>(a, tile, dx_transposed, s);
  if (dtype == CONV_BF16) return launch_pair<__bf16>(a, tile, dx_transposed, s);
  return launch_pair<float>(a, tile, dx_transposed, s);
}

// Both products of a backward pass: in one launch where the plan pairs them and the
// operands allow it, one after the other otherwise.
hipError_t run_both(const BackwardPlan& pl, int dtype, ProductArgs& dx, ProductArgs& dw,
                    bool dx_p_padded, bool dx_q_padded, bool dw_p_padded, bool dw_q_padded,
                    char* scratch, hipStream_t st) {
  const int es = (int)dtype_size(dtype);
  void *planes = scratch + pl.scratch.planes, *planes_dw = scratch + pl.scratch.planes_dw;
  if (pl.both.tile < 0 || !direct(pl.dx, dx, es, dx_p_padded, dx_q_padded) ||
      !direct(pl.dw, dw, es, dw_p_padded, dw_q_padded) ||
      launch_rows(pl.dx, pl.both.dx.splits) < pl.dx.C ||
      launch_rows(pl.dw, pl.both.dw.splits) < pl.dw.C) {
    const hipError_t e = run_product(pl.dx, pl.both.dx, dtype, dx, dx_p_padded, dx_q_padded, planes, st);
    if (e != hipSuccess) return e;
    return run_product(pl.dw, pl.both.dw, dtype, dw, dw_p_padded, dw_q_padded, planes_dw, st);
  }
  PairArgs a{};
  set_plan(pl.dx, pl.both.dx, planes, &dx);
  set_plan(pl.dw, pl.both.dw, planes_dw, &dw);
  if (pl.both.tile != TILE_64) {  // the large tiles' launch splits neither
    dx.splits = dw.splits = 1;
    dx.per_split = dx.ktiles * dx.nseg;
    dw.per_split = dw.ktiles * dw.nseg;
  }
  a.dx = dx;
  a.dw = dw;
  const hipError_t e = pair(dtype, a, pl.both.tile, pl.dx.pt, st);
  if (e != hipSuccess || (dx.splits == 1 && dw.splits == 1)) return e;
  if (dx.splits > 1 && dw.splits > 1)
    return join_pair(dtype, join_of(pl.dx, dx), join_of(pl.dw, dw), st);
  return dx.splits > 1 ? join(dtype, join_of(pl.dx, dx), false, st)
                       : join(dtype, join_of(pl.dw, dw), false, st);
}

hipError_t run_pack(const Packing& k, int dtype, const void** src, int64_t* ld, void* scratch,
                    hipStream_t s) {
  PackArgs a{};
  if (!fill_pack(k, (int)dtype_size(dtype), src, ld, scratch, &a)) return hipSuccess;
  if (dtype == CONV_F16) return launch_pack<_Float16>(a, s);
  if (dtype == CONV_BF16) return launch_pack<__bf16>(a, s);
  return launch_pack<float>(a, s);
}

int status(hipError_t e) { return e == hipSuccess ? CONV_OK : CONV_ERR_DEVICE; }

}  // namespace

extern "C" {

int linear_forward(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                   const void* r, void* y, void* z, void* scratch, uint64_t scratch_bytes,
                   void* stream) {
  LinearGeo g;
  LinearPlan pl;
  const int st = linear_checked(p, dtype, x, w, b, r, y, z, scratch, scratch_bytes, &g, &pl);
  if (st) return st;
  if (g.m == 0) return CONV_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const void* src[3] = {at(x, p->x_off, g.es), at(w, p->w_off, g.es)};
  int64_t ld[3] = {g.ldx, g.ldw};
  const hipError_t packed = run_pack(pl.pack, dtype, src, ld, scratch, s);
  if (packed != hipSuccess) return status(packed);
  ProductArgs a{};
  a.P[0] = src[1];
  a.Q[0] = src[0];
  a.ldp = ld[1]; a.ldq = ld[0];
  LinEpilogue& e = a.e;
  e.bias[0] = p->has_bias ? at(b, p->b_off, g.es) : nullptr;
  e.res = p->has_residual ? at(r, p->r_off, g.es) : nullptr;
  e.res_mode = p->has_residual;
  e.out[0] = at(y, p->y_off, g.es);
  e.save[0] = p->save_z ? at(z, p->z_off, g.es) : nullptr;
  e.ldo = g.ldy; e.ldres = g.ldr; e.ldsave = g.ldz;
  e.act = p->activation; e.alpha = p->act_alpha; e.beta = p->act_beta;
  return status(run_product(pl.product, pl.run, dtype, a, pl.pack.on, pl.pack.on, scratch, s));
}

int gated_forward(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                  const void* bg, const void* bu, void* h, void* pg, void* pu, void* scratch,
                  uint64_t scratch_bytes, void* stream) {
  GatedGeo g;
  GatedPlan pl;
  const int st = gated_checked(p, dtype, x, wg, wu, bg, bu, h, pg, pu,
                               scratch, scratch_bytes, &g, &pl);
  if (st) return st;
  if (g.m == 0) return CONV_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const void* src[3] = {at(x, p->x_off, g.es), at(wg, p->wg_off, g.es), at(wu, p->wu_off, g.es)};
  int64_t ld[3] = {g.ldx, g.ldw, g.ldw};
  const hipError_t packed = run_pack(pl.pack, dtype, src, ld, scratch, s);
  if (packed != hipSuccess) return status(packed);
  ProductArgs a{};
  a.P[0] = src[1];
  a.P[1] = src[2];
  a.Q[0] = src[0];
  a.ldp = ld[1]; a.ldq = ld[0];
  LinEpilogue& e = a.e;
  if (p->has_bias) {
    e.bias[0] = at(bg, p->bg_off, g.es);
    e.bias[1] = at(bu, p->bu_off, g.es);
  }
  e.out[0] = at(h, p->h_off, g.es);
  if (p->save_p) {
    e.save[0] = at(pg, p->pg_off, g.es);
    e.save[1] = at(pu, p->pu_off, g.es);
  }
  e.ldo = g.ldh; e.ldsave = g.ldp;
  e.act = p->activation; e.alpha = p->act_alpha; e.beta = p->act_beta;
  return status(run_product(pl.product, pl.run, dtype, a, pl.pack.on, pl.pack.on, scratch, s));
}

int linear_backward(const linear_problem* p, int dtype, const void* x, const void* w, const void* z,
                    const void* dy, void* dx, void* dw, void* db, void* dr, void* scratch,
                    uint64_t scratch_bytes, void* stream) {
  LinearGeo g;
  BackwardPlan pl;
  const int st = linear_backward_checked(p, dtype, x, w, z, dy, dx, dw, db, dr,
                                         scratch, scratch_bytes, &g, &pl);
  if (st) return st;
  const BackwardScratch& sc = pl.scratch;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* sb = static_cast<char*>(scratch);
  const bool act = p->activation != CONV_ACT_IDENTITY;
  const bool dr_is_dy = dr && (!act || p->has_residual == LINEAR_RES_AFTER);
  dy = at(dy, p->dy_off, g.es);
  dr = at(dr, p->dr_off, g.es);
  if (dr == dy && dr_is_dy) dr = nullptr;  // in place and unchanged
  const bool need_dz = act && (dx || dw);
  hipError_t e = hipSuccess;
  if (need_dz || db || dr) {
    const ColsumPlan cp = plan_colsum(g.m, g.n);
    DzArgs a{};
    a.dy = dy;
    a.z[0] = act && !(!need_dz && !db && dr_is_dy) ? at(z, p->z_off, g.es) : nullptr;
    a.act = a.z[0] ? p->activation : CONV_ACT_IDENTITY;
    a.dz = need_dz ? sb + sc.dz : nullptr;
    a.dr = dr;
    a.dr_is_dy = dr_is_dy;
    a.sums = db ? reinterpret_cast<float*>(sb + sc.sums) : nullptr;
    a.ldy = g.ldy; a.ldz = g.ldz; a.lddz = sc.dz_ld; a.lddr = g.lddr;
    a.m = g.m; a.rows = cp.rows;
    a.n = (int)g.n; a.np = (int)round_up(g.n, 8);
    a.alpha = p->act_alpha; a.beta = p->act_beta;
    e = dz_pass(dtype, a, false, (int)cp.chunks, s);
    if (e == hipSuccess && db) {
      SumsArgs q{};
      q.sums = a.sums;
      q.db[0] = at(db, p->db_off, g.es);
      q.chunks = (int)cp.chunks; q.n = a.n; q.np = a.np; q.parts = 1;
      e = sums_pass(dtype, q, s);
    }
  }
  const bool want_dx = dx && g.m > 0;
  const void* src[3] = {dw ? at(x, p->x_off, g.es) : nullptr,
                        want_dx ? at(w, p->w_off, g.es) : nullptr,
                        act ? static_cast<const void*>(sb + sc.dz) : dx || dw ? dy : nullptr};
  int64_t ld[3] = {g.ldx, g.ldw, act ? sc.dz_ld : g.ldy};
  if (e == hipSuccess) e = run_pack(pl.pack, dtype, src, ld, scratch, s);
  const bool on = pl.pack.on;
  ProductArgs ax{}, aw{};
  if (want_dx) {
    ax.P[0] = src[1];
    ax.Q[0] = src[2];
    ax.ldp = ld[1]; ax.ldq = ld[2];
    ax.e.out[0] = at(dx, p->dx_off, g.es);
    ax.e.ldo = g.lddx;
  }
  if (dw) {
    aw.P[0] = g.kn ? src[2] : src[0];
    aw.Q[0] = g.kn ? src[0] : src[2];
    aw.ldp = g.kn ? ld[2] : ld[0];
    aw.ldq = g.kn ? ld[0] : ld[2];
    aw.e.out[0] = at(dw, p->dw_off, g.es);
    aw.e.ldo = g.lddw;
  }
  // rows padded with zeros: packed ones, and dz
  const bool dpad = on || act, wp = g.kn ? dpad : on, wq = g.kn ? on : dpad;
  if (e == hipSuccess && want_dx && dw)
    e = run_both(pl, dtype, ax, aw, on, dpad, wp, wq, sb, s);
  else if (e == hipSuccess && want_dx)
    e = run_product(pl.dx, pl.both.dx, dtype, ax, on, dpad, sb + sc.planes, s);
  else if (e == hipSuccess && dw)
    e = run_product(pl.dw, pl.both.dw, dtype, aw, wp, wq, sb + sc.planes_dw, s);
  return status(e);
}

int gated_backward(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                   const void* pg, const void* pu, const void* dh, void* dx, void* dwg, void* dwu,
                   void* dbg, void* dbu, void* scratch, uint64_t scratch_bytes, void* stream) {
  GatedGeo g;
  BackwardPlan pl;
  const int st = gated_backward_checked(p, dtype, x, wg, wu, pg, pu, dh, dx, dwg, dwu, dbg, dbu,
                                        scratch, scratch_bytes, &g, &pl);
  if (st) return st;
  const BackwardScratch& sc = pl.scratch;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* sb = static_cast<char*>(scratch);
  const ColsumPlan cp = plan_colsum(g.m, g.f);
  DzArgs a{};
  a.dy = at(dh, p->dh_off, g.es);
  a.z[0] = at(pg, p->pg_off, g.es);
  a.z[1] = at(pu, p->pu_off, g.es);
  a.dz = sb + sc.dz;
  a.sums = dbg ? reinterpret_cast<float*>(sb + sc.sums) : nullptr;
  a.ldy = g.ldh; a.ldz = g.ldp; a.lddz = sc.dz_ld;
  a.m = g.m; a.rows = cp.rows;
  a.n = (int)g.f; a.np = (int)round_up(g.f, 8);
  a.act = p->activation; a.alpha = p->act_alpha; a.beta = p->act_beta;
  hipError_t e = dz_pass(dtype, a, true, (int)cp.chunks, s);
  if (e == hipSuccess && dbg) {
    SumsArgs q{};
    q.sums = a.sums;
    q.db[0] = at(dbg, p->dbg_off, g.es);
    q.db[1] = at(dbu, p->dbu_off, g.es);
    q.chunks = (int)cp.chunks; q.n = a.n; q.np = a.np; q.parts = 2;
    e = sums_pass(dtype, q, s);
  }
  const char* dg = sb + sc.dz;
  const char* du = dg + (int64_t)a.np * g.es;
  const bool want_dx = dx && g.m > 0;
  const void* src[3] = {dwg ? at(x, p->x_off, g.es) : nullptr,
                        want_dx ? at(wg, p->wg_off, g.es) : nullptr,
                        want_dx ? at(wu, p->wu_off, g.es) : nullptr};
  int64_t ld[3] = {g.ldx, g.ldw, g.ldw};
  if (e == hipSuccess) e = run_pack(pl.pack, dtype, src, ld, scratch, s);
  const bool on = pl.pack.on;
  ProductArgs ax{}, aw{};
  if (want_dx) {
    ax.P[0] = src[1];
    ax.P[1] = src[2];
    ax.Q[0] = dg;
    ax.Q[1] = du;
    ax.ldp = ld[1]; ax.ldq = sc.dz_ld;
    ax.e.out[0] = at(dx, p->dx_off, g.es);
    ax.e.ldo = g.lddx;
  }
  if (dwg) {
    aw.P[0] = src[0];
    aw.Q[0] = dg;
    aw.Q[1] = du;
    aw.ldp = ld[0]; aw.ldq = sc.dz_ld;
    aw.e.out[0] = at(dwg, p->dwg_off, g.es);
    aw.e.out[1] = at(dwu, p->dwu_off, g.es);
    aw.e.ldo = g.lddw;
  }
  if (e == hipSuccess && want_dx && dwg)
    e = run_both(pl, dtype, ax, aw, on, true, on, true, sb, s);
  else if (e == hipSuccess && want_dx)
    e = run_product(pl.dx, pl.both.dx, dtype, ax, on, true, sb + sc.planes, s);
  else if (e == hipSuccess && dwg)
    e = run_product(pl.dw, pl.both.dw, dtype, aw, on, true, sb + sc.planes_dw, s);
  return status(e);
}

}  // extern "C"
