// Shape-only planner of the linear and gated feed-forward calls
// (include/linear.h): validation, the kernel choice for each matrix product and
// the scratch layout.  Plain C++ with no HIP include, like the convolution's.
#pragma once

#include <stdint.h>

#include <stddef.h>

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
  bool aligned;     // rows of whole 16-byte pieces at multiples of 4 bytes (strides, extents, offsets)
};

enum ProductTile { TILE_256 = 0, TILE_128 = 1, TILE_64 = 2, TILE_STREAM = 3, TILE_256X128 = 4 };

struct ProductPlan {
  int tile;
  int splits;       // contraction ranges, joined in order by a second kernel
  int64_t ktiles;   // 128-byte contraction steps of one segment
  int64_t per_split;
  int stream_t;     // stream: 16-row blocks of Q
  int stream_rows;  // stream: weight rows of a workgroup
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

// Operands whose rows do not start on multiples of 4 bytes or are no whole 16-byte
// pieces can be copied to scratch first, rows padded with zeros, which lets the
// products load them to LDS directly.  Planned where the model finds it cheaper than
// products that gather through registers.
struct PackItem {
  int64_t rows, cols, ld;
  bool need;
  int64_t off, packed_ld;  // in the call's scratch (bytes), elements
};
struct Packing {
  bool on;
  int n;
  PackItem item[3];
  int64_t bytes;
};

// Scratch layout of a backward call (byte offsets; every part 256-byte aligned).
struct BackwardScratch {
  int64_t dz;      // dz [m, dz_ld] (gated: dg and du side by side)
  int64_t dz_ld;   // elements
  int64_t sums;    // column-sum partials
  int64_t planes;  // split planes (dw's behind dx's where they run in one launch)
  int64_t planes_dw;
  int64_t pack;    // packed operands
  int64_t total;
};

constexpr int64_t kLinMaxExtent = 1 << 20;

int linear_validate(const linear_problem* p, int dtype, LinearGeo* g);
int gated_validate(const gated_problem* p, int dtype, GatedGeo* g);

ProductPlan plan_product(const ProductShape& s, int es);
// Rows c that one launch may take (a multiple of 256): a launch holds fewer than 2^32
// work-items, and the kernels count rows in 32 bits.  More run one launch after the other.
int64_t launch_rows(const ProductShape& s, int splits);
// Both products of a backward pass: in one launch of a tile (TILE_256, TILE_256X128,
// or TILE_64, each with its splits), or one after the other (tile -1).
struct PairPlan {
  int tile;
  double time;         // estimated, us
  ProductPlan dx, dw;  // of each alone; for TILE_64 in that launch
};
// 8-bit products: tiles of 256 x 256 of the last round that are cut in two (0: none).  At most
// half of the units would have one in it (8192 x 11008 x 4096: 322 us for 340).
inline int64_t cut_tiles(int64_t tiles) {
  const int64_t rest = tiles % 256;
  return tiles > 256 && rest <= 128 ? rest : 0;
}
PairPlan plan_pair(const ProductShape& dx, const ProductShape& dw, int es);
ColsumPlan plan_colsum(int64_t m, int64_t n);

// A call's plan: its products as they will run, and its scratch.
struct LinearPlan {
  ProductShape product;
  ProductPlan run;
  Packing pack;  // x, w
  int64_t planes, total;
};
struct GatedPlan {
  ProductShape product;
  ProductPlan run;
  Packing pack;  // x, wg, wu
  int64_t planes, total;
};
struct BackwardPlan {
  ProductShape dx, dw;
  PairPlan both;
  Packing pack;  // linear: x, w, dy (identity); gated: x, wg, wu
  BackwardScratch scratch;
};
LinearPlan plan_linear(const linear_problem* p, const LinearGeo& g);
// Products of 8-bit operands (include/linear_int8.h): the same kernels and planes of
// int32 sums; a contraction step is 128 bytes of every type, so the times are alike.
LinearPlan plan_int8(int64_t m, int64_t n, int64_t k, int64_t ldx, int64_t ldw, int64_t x_off,
                     int64_t w_off);
GatedPlan plan_gated(const gated_problem* p, const GatedGeo& g);
BackwardPlan plan_linear_backward(const linear_problem* p, const LinearGeo& g);
BackwardPlan plan_gated_backward(const gated_problem* p, const GatedGeo& g);

// A plan's part of a variant's name ("tile64x64.split4").
void product_name(const ProductPlan& pl, char* buf, size_t len);

// The checks of include/linear.h; a call that passes gets its geometry and plan.
int linear_checked(const linear_problem* p, int dtype, const void* x, const void* w, const void* b,
                   const void* r, const void* y, const void* z, const void* scratch,
                   uint64_t scratch_bytes,
                   LinearGeo* g, LinearPlan* plan);
int linear_backward_checked(const linear_problem* p, int dtype, const void* x, const void* w,
                            const void* z, const void* dy, const void* dx, const void* dw,
                            const void* db, const void* dr, const void* scratch,
                            uint64_t scratch_bytes,
                            LinearGeo* g, BackwardPlan* plan);
int gated_checked(const gated_problem* p, int dtype, const void* x, const void* wg, const void* wu,
                  const void* bg, const void* bu, const void* h, const void* pg, const void* pu,
                  const void* scratch, uint64_t scratch_bytes,
                  GatedGeo* g, GatedPlan* plan);
int gated_backward_checked(const gated_problem* p, int dtype, const void* x, const void* wg,
                           const void* wu, const void* pg, const void* pu, const void* dh,
                           const void* dx, const void* dwg, const void* dwu, const void* dbg,
                           const void* dbu, const void* scratch, uint64_t scratch_bytes,
                           GatedGeo* g, BackwardPlan* plan);

inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

}  // namespace convfwd
