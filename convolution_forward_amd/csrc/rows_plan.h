// Shape-only planner of the row operators (include/layer_norm.h, include/dropout.h,
// quantize_rows of include/linear_int8.h): validation, kernel choice, scratch layout.
// Plain C++ with no HIP include.
#pragma once

#include <stdint.h>

#include "dropout.h"
#include "layer_norm.h"
#include "linear_int8.h"
#include "operand_checks.h"

namespace convfwd {

struct NormGeo {
  int64_t m, n;
  int64_t ldx, ldr, ldy, lds, ldds, lddx, lddr;
  int es;
};

// How a row is held: by `threads` threads, up to `runs` runs of 8 elements each; or,
// parts > 0, cut into parts of that size, in two launches.
struct RowPlan {
  int threads, runs;
  int64_t parts;
};

struct NormPlan {
  RowPlan row;
  int64_t scratch;
};

// Rows up to which dw and db can be summed by workgroups of their own, all rows each.
constexpr int kOnceRows = 1024;

// Backward: `groups` workgroups, each with a partial row of dw and of db; `teams`
// rows at a time in a workgroup.  once: dw and db by
// workgroups of their own and no partial rows; whole rows (`groups` workgroups of a row
// a team) then go in the same launch and need no scratch.
struct NormBackwardPlan {
  RowPlan row;
  bool once;
  int teams;
  int64_t groups;     // workgroups along the rows
  int64_t sums;       // byte offsets: row sums (split), partial rows of dw and db
  int64_t partials;
  int64_t scratch;
};

struct DropGeo {
  int64_t m, n, ldx, ldr, ldy;
  int es;
  int runs;  // of 8 elements a thread
};

struct QuantGeo {
  int64_t m, n, ldx, ldq;
  int es;
  RowPlan row;  // parts > 0: the row is read twice
};

// Rows of one launch of a row kernel: fewer than 2^32 work-items, `items` a row, in whole
// workgroups of `teams` rows.  A kernel knows the last row of the call, not that of its launch:
// a last workgroup with room left would take rows of the next launch, which would then
// be worked on twice, outputs over inputs as well.
constexpr int64_t rows_of_launch(int64_t items, int64_t teams) {
  return 0xff000000LL / items / teams * teams;
}

// Drop threshold of 16 random bits.
int drop_threshold(float p);

int layer_norm_validate(const layer_norm_problem* p, int dtype, NormGeo* g);
NormPlan plan_layer_norm(const NormGeo& g);
NormBackwardPlan plan_layer_norm_backward(const NormGeo& g);

// The checks of the headers; a call that passes gets its geometry and plan.
int layer_norm_checked(const layer_norm_problem* p, int dtype, const void* x, const void* r,
                       const void* w, const void* b, const void* y, const void* s,
                       const void* mean, const void* rstd, const void* step, const void* scratch,
                       uint64_t scratch_bytes, NormGeo* g, NormPlan* plan);
int layer_norm_backward_checked(const layer_norm_problem* p, int dtype, const void* s,
                                const void* w, const void* mean, const void* rstd, const void* dy,
                                const void* ds, const void* dx, const void* dr, const void* dw,
                                const void* db, const void* step, const void* scratch,
                                uint64_t scratch_bytes, NormGeo* g, NormBackwardPlan* plan);
int dropout_checked(const dropout_problem* p, int dtype, const void* x, const void* r,
                    const void* y, const void* step, DropGeo* g);
int dropout_backward_checked(const dropout_problem* p, int dtype, const void* dy, const void* dx,
                             const void* step, DropGeo* g);
int quantize_checked(const quantize_problem* p, int dtype, const void* x, const void* q,
                     const void* scale, QuantGeo* g);

}  // namespace convfwd
