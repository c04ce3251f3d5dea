// Shape-only half of include/grad_clip.h: validation and the cut of the tensors
// into chunks and launches.  Plain C++ with no HIP include.
#pragma once

#include <stdint.h>

#include "grad_clip.h"
#include "plan.h"

namespace convfwd {

constexpr int kClipTable = 112;      // tensors per launch (their table is a kernel argument)
constexpr int kClipSmall = 16;       // or of a launch with a small table, if they are that few
constexpr int kClipPartials = 1024;  // partial norms per launch

struct ClipPlan {
  int64_t total;     // elements
  int64_t chunk;     // elements per chunk: a power of two, a function of the total
  int64_t launches;  // of up to kClipTable tensors
  int64_t scratch;   // bytes
};

int clip_validate(const grad_clip_problem* p, ClipPlan* pl);

}  // namespace convfwd
