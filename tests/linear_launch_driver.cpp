// Every launch of the linear and gated calls over random problems of the whole range
// of their sizes: below 2^32 work-items, and row counts that 32 bits hold with a tile's
// padding.  For a build with address and undefined-behaviour checks.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <random>

#include "linear_plan.h"

using namespace convfwd;

namespace {

struct Kind {
  int tile;
  int64_t r, c, threads;
};
const Kind kKinds[] = {{TILE_256, 256, 256, 512}, {TILE_256X128, 256, 128, 512},
                       {TILE_128, 128, 128, 256}, {TILE_64, 64, 64, 256}};
long bad = 0, cut = 0;

void fail(const char* what, const ProductShape& s) {
  if (bad++ < 10)
    printf("%s: R %lld C %lld K %lld gated %d\n", what, (long long)s.R, (long long)s.C, (long long)s.K, s.gated);
}

// work-items of a product's largest launch
int64_t items(const ProductShape& s, const ProductPlan& pl) {
  if (s.C < 1) return 0;
  if (pl.tile == TILE_STREAM) return ceil_div(s.R, pl.stream_rows) * 512;
  const int64_t rows = launch_rows(s, pl.splits);
  if (rows < 256 || rows % 256 != 0 || rows > (1LL << 30)) fail("rows", s);
  if (rows < s.C) {
    ++cut;
    if (pl.splits > 1) fail("a split product is cut", s);
  }
  int64_t most = 0;
  for (const Kind& k : kKinds)  // operands that cannot go to LDS directly take a smaller tile
    if (k.tile == pl.tile || k.tile == TILE_128)
      most = std::max(most, ceil_div(s.gated ? 2 * s.R : s.R, k.r) * ceil_div(std::min(rows, s.C), k.c) *
                                s.nz * pl.splits * k.threads);
  return most;
}

void look(const ProductShape& s, const ProductPlan& pl) {
  if (items(s, pl) >= (1LL << 32)) fail("work-items", s);
}

void look(const BackwardPlan& b) {
  look(b.dx, b.both.dx);
  look(b.dw, b.both.dw);
  if (b.both.tile < 0 || b.dx.C < 1 || launch_rows(b.dx, b.both.dx.splits) < b.dx.C ||
      launch_rows(b.dw, b.both.dw.splits) < b.dw.C)
    return;
  ProductPlan x = b.both.dx, w = b.both.dw;
  x.tile = w.tile = b.both.tile;
  if (items(b.dx, x) + items(b.dw, w) >= (1LL << 32)) fail("work-items of a pair", b.dx);
}

void look(const Packing& k, const ProductShape& s, int es) {
  if (!k.on) return;
  int64_t groups = 0;
  for (int i = 0; i < k.n; ++i)
    if (k.item[i].need) groups += ceil_div(k.item[i].rows * k.item[i].packed_ld * es / 16, 1024);
  if (groups * 256 >= (1LL << 32)) fail("work-items of the copies", s);
}

}  // namespace

int main(int argc, char**) {
  std::mt19937_64 gen(argc);
  auto size = [&](double bits) {
    return (int64_t)pow(2.0, std::uniform_real_distribution<double>(0, bits)(gen));
  };
  const int64_t rows[] = {2147483647, 2147483647 - 63, 2147483647 - 127, 1100000000, (1LL << 30) + 77};
  long good = 0;
  for (int i = 0; i < 60000; ++i) {
    linear_problem p{};
    p.m = i % 3 == 0 ? rows[gen() % 5] : size(31) - 1;
    p.n = size(i % 2 ? 8 : 20);
    p.k = size(i % 2 ? 8 : 20);
    p.activation = (int32_t)(gen() % 11);
    p.w_layout = (int32_t)(gen() % 2);
    gated_problem q{};
    q.m = p.m;
    q.f = p.n;
    q.k = p.k;
    const int dtype = (int)(gen() % 3);
    LinearGeo g;
    if (linear_validate(&p, dtype, &g) == CONV_OK) {
      const LinearPlan f = plan_linear(&p, g);
      look(f.product, f.run);
      look(f.pack, f.product, dtype == CONV_F32 ? 4 : 2);
      const BackwardPlan b = plan_linear_backward(&p, g);
      look(b);
      look(b.pack, b.dx, dtype == CONV_F32 ? 4 : 2);
      ++good;
    }
    GatedGeo h;
    if (gated_validate(&q, dtype, &h) == CONV_OK) {
      const GatedPlan f = plan_gated(&q, h);
      look(f.product, f.run);
      look(f.pack, f.product, dtype == CONV_F32 ? 4 : 2);
      const BackwardPlan b = plan_gated_backward(&q, h);
      look(b);
      look(b.pack, b.dx, dtype == CONV_F32 ? 4 : 2);
      ++good;
    }
  }
  printf("%ld problems, %ld products cut, %ld bad\n", good, cut, bad);
  return bad == 0 && good > 20000 && cut > 100 ? 0 : 1;
}
