// Kernel arguments and launchers of the linear and gated feed-forward products
// (include/linear.h), shared by the launch half and the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "internal.h"

namespace convfwd {

// What becomes of a float32 sum: bias, residual, activation, stores.  Output
// element (c, r) lies at out + c * ldo + r.  For the gated product the two sums
// of an element come together, bias[1] and save[1] being the second one's.
struct LinEpilogue {
  const void* bias[2];
  const void* res;
  void* out[2];   // per batch z
  void* save[2];  // the sums before the activation (optional)
  long long ldo, ldres, ldsave;
  int R;          // valid r
  int res_mode;   // LINEAR_RES_*
  int act;
  float alpha, beta;
  const float *xs, *ws;  // 8-bit operands: scales of the rows c and of r
};

// out[c][r] = sum_k P(r, k) Q(c, k), see linear_plan.h.
struct ProductArgs {
  const void* P[2];  // by segment of the contraction, or gate / up
  const void* Q[2];  // by segment, or by batch z
  long long ldp, ldq;
  int R, C, K;
  int nseg, nz;
  int ntr, ntc;        // tiles along r and c
  int ktiles;          // contraction steps of one segment
  int splits, per_split;
  float* planes;       // splits > 1: [split][z][half][C][plane_ld]
  long long plane_ld;
  LinEpilogue e;
};

// Two products of one launch (split on small tiles only).
struct PairArgs {
  ProductArgs dx, dw;
  int first;     // workgroups of the one that comes first
  int dw_first;  // which one that is
};

// Second pass of a split contraction.
struct JoinArgs {
  const float* planes;
  long long plane_ld, plane_stride;  // floats; stride between splits
  int splits, C, nz;
  LinEpilogue e;
};

// Up to three matrices copied into rows of whole 16-byte pieces, zeros past the end.
struct PackArgs {
  const void* src[3];
  void* dst[3];
  long long ld[3], packed_ld[3], pieces[3];  // strides in elements; 16-byte pieces of all rows
  int cols[3];
  int first[4];  // first workgroup of each; the last entry is the grid
  int n;
};

// dz and its column sums (see k_linear_grad.hip).
struct DzArgs {
  const void* dy;
  const void* z[2];  // linear: z; gated: pg, pu
  void* dz;          // [m, ldz_out], columns up to np written (zeros past n); may be null
  void* dr;          // optional copy (linear)
  float* sums;       // [chunk][gated 2][np] partial column sums; may be null
  long long ldy, ldz, lddz, lddr;
  long long m, rows;  // rows per chunk
  int n, np;
  int dr_is_dy;
  int act;
  float alpha, beta;
};

struct SumsArgs {
  const float* sums;  // [chunk][width]
  void* db[2];
  int chunks, n, np, parts;
};

// layout: 0 both operands k-major, 1 P transposed, 2 both transposed.
// dma: rows of whole aligned 16-byte vectors (global to LDS directly).
template <typename E>
hipError_t launch_product(const ProductArgs& a, int tile, int layout, bool gated, bool dma,
                          hipStream_t s);
template <typename E>
hipError_t launch_pack(const PackArgs& a, hipStream_t s);
// tile: TILE_256, TILE_256X128 (16 bits) or TILE_64; operands that go to LDS directly.
template <typename E>
hipError_t launch_pair(const PairArgs& a, int tile, bool dx_transposed, hipStream_t s);
template <typename E>
hipError_t launch_stream(const ProductArgs& a, int blocks16, int rows, bool gated, bool vec,
                         hipStream_t s);
template <typename E>
hipError_t launch_join(const JoinArgs& a, bool gated, hipStream_t s);
template <typename E>
hipError_t launch_join_pair(const JoinArgs& a, const JoinArgs& b, hipStream_t s);
// 8-bit operands, outputs of type O.
template <typename O>
hipError_t launch_int8_product(const ProductArgs& a, int tile, bool dma, hipStream_t s);
template <typename O>
hipError_t launch_int8_stream(const ProductArgs& a, int blocks16, int rows, bool vec, hipStream_t s);
template <typename O>
hipError_t launch_int8_join(const JoinArgs& a, hipStream_t s);
template <typename E>
hipError_t launch_dz(const DzArgs& a, bool gated, int chunks, hipStream_t s);
template <typename E>
hipError_t launch_sums(const SumsArgs& a, hipStream_t s);

}  // namespace convfwd
