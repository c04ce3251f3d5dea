// Plans random linear, gated and clipping problems over the whole range of their
// sizes, for a build with address and undefined-behaviour checks.
#include <math.h>
#include <stdio.h>

#include <random>

#include "grad_clip_plan.h"
#include "linear_plan.h"

int main(int argc, char**) {
  std::mt19937_64 gen(argc);
  auto size = [&](double bits) {
    return (int64_t)pow(2.0, std::uniform_real_distribution<double>(0, bits)(gen));
  };
  long good = 0;
  char text[256];
  for (int i = 0; i < 20000; ++i) {
    linear_problem p{};
    p.m = i % 7 == 0 ? 0 : size(31) - 1;
    p.n = size(20);
    p.k = size(20);
    p.activation = (int32_t)(gen() % 11);
    p.has_bias = (int32_t)(gen() % 2);
    p.has_residual = (int32_t)(gen() % 3);
    p.w_layout = (int32_t)(gen() % 2);
    if (gen() % 2) {
      p.ldx = p.k + (int64_t)(gen() % 9);
      p.ldw = (p.w_layout ? p.n : p.k) + (int64_t)(gen() % 9);
    }
    if (gen() % 4 == 0) p.x_off = (int64_t)(gen() % 9);
    gated_problem q{};
    q.m = p.m;
    q.f = p.n;
    q.k = p.k;
    q.activation = p.activation;
    q.ldx = p.ldx;
    const int dtype = (int)(gen() % 3);
    uint64_t bytes;
    if (linear_scratch_size(&p, dtype, &bytes) == CONV_OK)
      good += linear_describe_variant(&p, dtype, text, sizeof text) == CONV_OK;
    if (linear_backward_scratch_size(&p, dtype, &bytes) == CONV_OK)
      good += linear_backward_describe_variant(&p, dtype, text, sizeof text) == CONV_OK;
    if (gated_scratch_size(&q, dtype, &bytes) == CONV_OK)
      good += gated_describe_variant(&q, dtype, text, sizeof text) == CONV_OK;
    if (gated_backward_scratch_size(&q, dtype, &bytes) == CONV_OK)
      good += gated_backward_describe_variant(&q, dtype, text, sizeof text) == CONV_OK;
    grad_tensor t[3] = {};
    for (grad_tensor& e : t) {
      e.g = (const void*)(uintptr_t)4096;
      e.elems = size(39) - 1;
      e.dtype = (int32_t)(gen() % 3);
    }
    grad_clip_problem c{t, 3, GRAD_NORM_2, 1.0f, 1e-6f, 0};
    good += grad_clip_scratch_size(&c, &bytes) == CONV_OK;
  }
  printf("%ld plans\n", good);
  return good > 40000 ? 0 : 1;
}
