// Shape-only planner of the 8-bit linear layer (include/linear_int8.h).  Plain C++ with
// no HIP include.
#pragma once

#include "linear_int8.h"
#include "linear_plan.h"
#include "operand_checks.h"

namespace convfwd {

constexpr int64_t kInt8MaxK = 131071;  // 2^14 k of them stay below 2^31

struct Int8Geo {
  int64_t m, n, k;
  int64_t ldx, ldw, ldr, ldy;
  int es;  // of b, r and y
};

int int8_validate(const linear_int8_problem* p, int dtype, Int8Geo* g);
LinearPlan plan_linear_int8(const linear_int8_problem* p, const Int8Geo& g);
// The checks of the header; a call that passes gets its geometry and plan.
int linear_int8_checked(const linear_int8_problem* p, int dtype, const void* x, const void* xs,
                        const void* w, const void* ws, const void* b, const void* r, const void* y,
                        const void* scratch, uint64_t scratch_bytes, Int8Geo* g, LinearPlan* plan);

}  // namespace convfwd
