// Host half of include/grad_clip.h that never touches the device.
#include "grad_clip_plan.h"

#include <algorithm>

namespace convfwd {

int clip_validate(const grad_clip_problem* p, ClipPlan* out) {
  if (!p || p->reserved != 0) return CONV_ERR_ARG;
  if (p->kind < GRAD_NORM_1 || p->kind > GRAD_NORM_INF) return CONV_ERR_ARG;
  if (!(p->max_norm >= 0.0f) || !(p->eps >= 0.0f)) return CONV_ERR_ARG;
  if (p->count < 0 || p->count > 65536) return CONV_ERR_SHAPE;
  if (p->count > 0 && !p->tensors) return CONV_ERR_ARG;
  ClipPlan pl{};
  int with_out = 0, with_data = 0;
  for (int64_t i = 0; i < p->count; ++i) {
    const grad_tensor& t = p->tensors[i];
    if ((t.dtype != CONV_F32 && t.dtype != CONV_F16 && t.dtype != CONV_BF16) || t.reserved != 0)
      return CONV_ERR_ARG;
    if (t.elems < 0 || t.elems > (1LL << 38)) return CONV_ERR_SHAPE;
    pl.total += t.elems;  // at most 2^54
    if (t.elems == 0) continue;
    if (!t.g) return CONV_ERR_ARG;
    const uintptr_t es = (uintptr_t)dtype_size(t.dtype);
    if ((uintptr_t)t.g % es != 0 || (uintptr_t)t.out % es != 0) return CONV_ERR_ARG;
    ++with_data;
    with_out += t.out != nullptr;
  }
  if (with_out != 0 && with_out != with_data) return CONV_ERR_ARG;
  if (pl.total > (1LL << 40)) return CONV_ERR_SHAPE;
  // about two chunks for each of the 1024 workgroups of the norm, between 1024
  // elements (one vector a thread of 16 bits) and 32768
  pl.chunk = 1024;
  while (pl.chunk < 32768 && pl.chunk * 2 * kClipPartials < pl.total) pl.chunk *= 2;
  pl.launches = std::max<int64_t>(1, ceil_div(p->count, kClipTable));
  pl.scratch = (pl.launches * kClipPartials + 1) * 8;
  pl.scratch = ceil_div(pl.scratch, 256) * 256;
  *out = pl;
  return CONV_OK;
}

}  // namespace convfwd

using namespace convfwd;

extern "C" {

int grad_clip_scratch_size(const grad_clip_problem* p, uint64_t* bytes) {
  if (!bytes) return CONV_ERR_ARG;
  ClipPlan pl;
  const int st = clip_validate(p, &pl);
  if (st) return st;
  *bytes = (uint64_t)pl.scratch;
  return CONV_OK;
}

int grad_clip_check(const grad_clip_problem* p, const void* norm, const void* scratch,
                    uint64_t scratch_bytes) {
  ClipPlan pl;
  const int st = clip_validate(p, &pl);
  if (st) return st;
  if (!norm || (uintptr_t)norm % 4 != 0) return CONV_ERR_ARG;
  if (scratch_bytes < (uint64_t)pl.scratch) return CONV_ERR_SCRATCH;
  if (!scratch || (uintptr_t)scratch % 256 != 0) return CONV_ERR_ARG;
  const uintptr_t s0 = (uintptr_t)scratch, s1 = s0 + (uintptr_t)pl.scratch;
  const uintptr_t n0 = (uintptr_t)norm, n1 = n0 + 4;
  if (n0 < s1 && s0 < n1) return CONV_ERR_OVERLAP;
  for (int64_t i = 0; i < p->count; ++i) {
    const grad_tensor& t = p->tensors[i];
    if (t.elems == 0) continue;
    const uintptr_t len = (uintptr_t)t.elems * (uintptr_t)dtype_size(t.dtype);
    const uintptr_t g = (uintptr_t)t.g, o = (uintptr_t)t.out;
    if (t.out && o != g && o < g + len && g < o + len) return CONV_ERR_OVERLAP;
    for (uintptr_t b : {g, o}) {
      if (b == 0) continue;
      if ((b < s1 && s0 < b + len) || (b < n1 && n0 < b + len)) return CONV_ERR_OVERLAP;
    }
  }
  return CONV_OK;
}

}  // extern "C"
