// Plans and checks random layer norm, dropout, quantization and 8-bit linear problems
// over the whole range of their sizes, for a build with address and
// undefined-behaviour checks.
#include <math.h>
#include <stdio.h>

#include <random>

#include "linear_int8_plan.h"
#include "rows_plan.h"

int main(int argc, char**) {
  std::mt19937_64 gen(argc);
  auto size = [&](double bits) {
    return (int64_t)pow(2.0, std::uniform_real_distribution<double>(0, bits)(gen));
  };
  auto place = [&] { return (const void*)(uintptr_t)((gen() % (1 << 20) + 1) << 24); };
  long good = 0;
  char text[256];
  for (int i = 0; i < 20000; ++i) {
    const int dtype = (int)(gen() % 3);
    uint64_t bytes = 0;
    layer_norm_problem p{};
    p.m = i % 7 == 0 ? 0 : size(31) - 1;
    p.n = size(20);
    p.eps = 1e-5f;
    p.drop = (float)(gen() % 11) / 10;
    p.has_weight = p.has_bias = 1;
    p.has_residual = (int32_t)(gen() % 2);
    if (gen() % 2) p.ldx = p.n + (int64_t)(gen() % 9);
    if (gen() % 4 == 0) p.x_off = (int64_t)(gen() % 9);
    const void* q[12];
    for (const void*& e : q) e = place();
    if (layer_norm_scratch_size(&p, dtype, &bytes) == CONV_OK) {
      good += layer_norm_describe_variant(&p, dtype, text, sizeof text) == CONV_OK;
      layer_norm_check(&p, dtype, q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7], q[8], q[9], bytes);
    }
    if (layer_norm_backward_scratch_size(&p, dtype, &bytes) == CONV_OK) {
      good += layer_norm_backward_describe_variant(&p, dtype, text, sizeof text) == CONV_OK;
      layer_norm_backward_check(&p, dtype, q[0], q[1], q[2], q[3], q[4], q[5], q[6], nullptr, q[7],
                                q[8], q[9], q[10], bytes);
    }
    dropout_problem d{};
    d.m = p.m;
    d.n = p.n;
    d.ldx = p.ldx;
    d.drop = p.drop;
    good += dropout_describe_variant(&d, dtype, text, sizeof text) == CONV_OK;
    dropout_check(&d, dtype, q[0], q[1], q[2], q[3]);
    quantize_problem z{};
    z.m = p.m;
    z.n = p.n;
    z.ldx = p.ldx;
    quantize_check(&z, dtype, q[0], q[1], q[2]);
    linear_int8_problem l{};
    l.m = p.m;
    l.n = size(20);
    l.k = size(16.9);
    l.activation = (int32_t)(gen() % 11);
    if (gen() % 2) l.ldx = l.k + (int64_t)(gen() % 17);
    if (linear_int8_scratch_size(&l, dtype, &bytes) == CONV_OK) {
      good += linear_int8_describe_variant(&l, dtype, text, sizeof text) == CONV_OK;
      linear_int8_check(&l, dtype, q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7], bytes);
    }
  }
  printf("%ld plans\n", good);
  return good > 60000 ? 0 : 1;
}
