// Instantiation and launch of the tile kernel for one element type; included by
// one source file per type.
#pragma once

#include "linear_pingpong.h"
#include "linear_plan.h"

namespace convfwd {

template <typename E, bool PT, bool QT, int BR, int BC, int WVR, int WVC, bool DMA, bool GATED>
static hipError_t launch_tile(ProductArgs a, hipStream_t s) {
  a.ntr = (a.R + (GATED ? BR / 2 : BR) - 1) / (GATED ? BR / 2 : BR);
  a.ntc = (a.C + BC - 1) / BC;
  const int grid = a.ntr * a.ntc * a.nz * a.splits;
  hipLaunchKernelGGL((linear_tile_kernel<E, PT, QT, BR, BC, WVR, WVC, DMA, GATED>), dim3(grid),
                     dim3(WVR * WVC * 64), 0, s, a);
  return hipGetLastError();
}

template <typename E, bool PT, bool QT, int BC, bool GATED>
static hipError_t launch_pingpong(ProductArgs a, hipStream_t s) {
  constexpr int BR = GATED ? 128 : 256;
  a.ntr = (a.R + BR - 1) / BR;
  a.ntc = (a.C + BC - 1) / BC;
  const int grid = a.ntr * a.ntc * a.nz * a.splits;
  hipLaunchKernelGGL((linear_pingpong_kernel<E, PT, QT, BC, GATED>), dim3(grid), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename E, bool PT, bool QT>
static hipError_t launch_layout(const ProductArgs& a, int tile, bool dma, hipStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (tile == TILE_256 && dma) return launch_pingpong<E, PT, QT, 256, false>(a, s);
    if (tile == TILE_256X128 && dma) return launch_pingpong<E, PT, QT, 128, false>(a, s);
  }
  if (tile == TILE_64)
    return dma ? launch_tile<E, PT, QT, 64, 64, 2, 2, true, false>(a, s)
               : launch_tile<E, PT, QT, 64, 64, 2, 2, false, false>(a, s);
  return dma ? launch_tile<E, PT, QT, 128, 128, 2, 2, true, false>(a, s)
             : launch_tile<E, PT, QT, 128, 128, 2, 2, false, false>(a, s);
}

template <typename E>
hipError_t launch_product(const ProductArgs& a, int tile, int layout, bool gated, bool dma,
                          hipStream_t s) {
  if (gated) {
    if constexpr (sizeof(E) == 2) {
      if (tile == TILE_256 && dma) return launch_pingpong<E, false, false, 256, true>(a, s);
      if (tile == TILE_256X128 && dma) return launch_pingpong<E, false, false, 128, true>(a, s);
    }
    if (tile == TILE_64)
      return dma ? launch_tile<E, false, false, 64, 64, 1, 4, true, true>(a, s)
                 : launch_tile<E, false, false, 64, 64, 1, 4, false, true>(a, s);
    return dma ? launch_tile<E, false, false, 128, 128, 2, 2, true, true>(a, s)
               : launch_tile<E, false, false, 128, 128, 2, 2, false, true>(a, s);
  }
  if (layout == 0) return launch_layout<E, false, false>(a, tile, dma, s);
  if (layout == 1) return launch_layout<E, true, false>(a, tile, dma, s);
  return launch_layout<E, true, true>(a, tile, dma, s);
}

template <typename E>
hipError_t launch_pair(const PairArgs& pair, int tile, bool dx_transposed, hipStream_t s) {
  PairArgs a = pair;
  const int br = tile == TILE_64 ? 64 : 256;
  const int bc = tile == TILE_64 ? 64 : tile == TILE_256 ? 256 : 128;
  int grid[2], i = 0;
  for (ProductArgs* p : {&a.dx, &a.dw}) {
    p->ntr = (p->R + br - 1) / br;
    p->ntc = (p->C + bc - 1) / bc;
    grid[i++] = p->ntr * p->ntc * p->nz * p->splits;
  }
  // the longer contraction first: the shorter tiles then even out the last round
  a.dw_first = a.dw.per_split > a.dx.per_split;
  a.first = grid[a.dw_first];
  const dim3 g(grid[0] + grid[1]);
  if (tile == TILE_64) {
    if (dx_transposed) hipLaunchKernelGGL((linear_tile_pair_kernel<E, true>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((linear_tile_pair_kernel<E, false>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (sizeof(E) == 2) {
    const dim3 b(512);
    if (dx_transposed) {
      if (bc == 256) hipLaunchKernelGGL((linear_pair_kernel<E, true, 256>), g, b, 0, s, a);
      else hipLaunchKernelGGL((linear_pair_kernel<E, true, 128>), g, b, 0, s, a);
    } else {
      if (bc == 256) hipLaunchKernelGGL((linear_pair_kernel<E, false, 256>), g, b, 0, s, a);
      else hipLaunchKernelGGL((linear_pair_kernel<E, false, 128>), g, b, 0, s, a);
    }
    return hipGetLastError();
  }
  return hipErrorInvalidValue;  // the large tiles take 16-bit operands
}

}  // namespace convfwd
