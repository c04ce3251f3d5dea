// Shape-only planner of the linear and gated feed-forward calls
// (include/linear.h): validation, the kernel choice for each matrix product and
// the scratch layout.  Plain C++ with no HIP include, like the convolution's.
#pragma once

#include <stdint.h>

#include "linear.h"
#include "plan.h"

namespace convfwd {

// One matrix product out[c][r] = sum_k P(r, k) Q(c, k).  An operand is k-major
// (its rows run along k) or, "transposed", r- or c-major (rows of constant k).
struct ProductShape {
  int64_t R, C, K;  // K of one segment
  int nseg;         // segments of the contraction (dx of the gated backward: 2)
  int nz;           // products of one shape in a launch (gated weight gradients: 2)
  bool pt, qt;      // operand transposed
  bool gated;       // P is two matrices of R rows (gate and up), joined in the epilogue
  bool aligned;     // rows of whole 16-byte vectors (strides, extents, offsets)
};

enum ProductTile { TILE_256 = 0, TILE_128 = 1, TILE_64 = 2, TILE_STREAM = 3, TILE_256X128 = 4 };

struct ProductPlan {
  int tile;
  int splits;       // contraction ranges, joined in order by a second kernel
  int64_t ktiles;   // 128-byte contraction steps of one segment
  int64_t per_split;
  int stream_t;     // stream: 16-row blocks of Q
  int64_t plane_ld; // floats per plane row
  int64_t planes_bytes;
  double time;      // estimated, us
};

struct LinearGeo {
  int64_t m, n, k;
  int64_t ldx, ldw, ldr, ldy, ldz, lddx, lddw, lddr;
  int es;
  bool kn;
};

struct GatedGeo {
  int64_t m, f, k;
  int64_t ldx, ldw, ldh, ldp, lddx, lddw;
  int es;
};

// Column sums of dz: rows in chunks, one float32 partial row per chunk.
struct ColsumPlan {
  int64_t rows;    // rows per chunk
  int64_t chunks;  // <= 256
};

// Scratch layout of a backward call (byte offsets; every part 256-byte aligned).
struct BackwardScratch {
  int64_t dz;      // dz [m, dz_ld] (gated: dg and du side by side)
  int64_t dz_ld;   // elements
  int64_t sums;    // column-sum partials
  int64_t planes;  // split planes (the two products run one after the other)
  int64_t total;
};

constexpr int64_t kLinMaxExtent = 1 << 20;

int linear_validate(const linear_problem* p, int dtype, LinearGeo* g);
int gated_validate(const gated_problem* p, int dtype, GatedGeo* g);

ProductPlan plan_product(const ProductShape& s, int es);
// The tile (TILE_256 or TILE_256X128) of one launch for both products of a backward
// pass, or -1 where they run one after the other.
int plan_pair(const ProductShape& dx, const ProductShape& dw, int es);
ColsumPlan plan_colsum(int64_t m, int64_t n);

// The products of each call, from the geometry and offsets alone.
ProductShape linear_product(const linear_problem* p, const LinearGeo& g);
ProductShape linear_dx_product(const linear_problem* p, const LinearGeo& g);
ProductShape linear_dw_product(const linear_problem* p, const LinearGeo& g);
ProductShape gated_product(const gated_problem* p, const GatedGeo& g);
ProductShape gated_dx_product(const gated_problem* p, const GatedGeo& g);
ProductShape gated_dw_product(const gated_problem* p, const GatedGeo& g);

BackwardScratch linear_backward_scratch(const linear_problem* p, const LinearGeo& g);
BackwardScratch gated_backward_scratch(const gated_problem* p, const GatedGeo& g);

inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace convfwd
