// Tile layout and workgroup order shared by the fused GEMM kernels.
#pragma once

#include "device_common.h"

namespace qlora {

__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// byte offset of 16-byte chunk c of row `row` in a swizzled 256 x 64 bf16 tile
__device__ __forceinline__ int tile_off(int row, int c) { return row * 128 + ((c ^ swz(row)) << 4); }

// Map the linear workgroup id b to (token tile, output tile): workgroups are dispatched
// round-robin over the 8 XCDs, so consecutive tiles of the grouped raster order are
// given to the same XCD (sharing its L2); groups of 4 token tiles sweep the outputs.
__device__ __forceinline__ void tile_coords(int b, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int T = tiles_m * tiles_n;
  if ((T & 7) == 0) b = (b & 7) * (T >> 3) + (b >> 3);
  constexpr int G = 4;
  const int group = b / (G * tiles_n);
  const int first = group * G;
  const int gsize = min(tiles_m - first, G);
  const int in = b - group * G * tiles_n;
  tm = first + in % gsize;
  tn = in / gsize;
}

}  // namespace qlora
