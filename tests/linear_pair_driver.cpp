// Plans of both gradients in one launch of large tiles: what each product runs as by
// itself (one gradient wanted, or operands that cannot go to LDS directly) is the plan
// that it gets alone.
#include <math.h>
#include <stdio.h>

#include <random>

#include "linear_plan.h"

using namespace convfwd;

int main() {
  std::mt19937_64 gen(1);
  auto size = [&](double lo, double hi) {
    return (int64_t)pow(2.0, std::uniform_real_distribution<double>(lo, hi)(gen));
  };
  long pairs = 0, bad = 0;
  for (int i = 0; i < 200000; ++i) {
    int64_t m = size(4, 14), n = size(5, 14), k = size(5, 14);
    if (i == 0) m = 960, n = 896, k = 4352;
    if (i % 2) m = round_up(m, 64), n = round_up(n, 64), k = round_up(k, 64);
    const int seg = i % 3 == 1 ? 2 : 1;
    const ProductShape dx{k, m, n, seg, 1, true, false, false, true};
    const ProductShape dw{k, n, m, 1, seg, true, true, false, true};
    const PairPlan p = plan_pair(dx, dw, 2);
    if (p.tile < 0 || p.tile == TILE_64) continue;
    ++pairs;
    const ProductPlan x = plan_product(dx, 2), w = plan_product(dw, 2);
    if (x.tile == p.dx.tile && x.splits == p.dx.splits && x.planes_bytes == p.dx.planes_bytes &&
        w.tile == p.dw.tile && w.splits == p.dw.splits && w.planes_bytes == p.dw.planes_bytes)
      continue;
    if (bad++ < 5)
      printf("m %lld n %lld k %lld: dx %d/%d, alone %d/%d; dw %d/%d, alone %d/%d\n", (long long)m, (long long)n,
             (long long)k, p.dx.tile, p.dx.splits, x.tile, x.splits, p.dw.tile, p.dw.splits, w.tile, w.splits);
  }
  printf("%ld pairs, %ld bad\n", pairs, bad);
  return pairs > 1000 && bad == 0 ? 0 : 1;
}
