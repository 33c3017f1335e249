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

// Keep decisions of a lane's 32 elements of two neighbouring 32 x 32 accumulator blocks (a row
// of `group0 * 8 ..`, element e of block j in bit 16 j + e, its column 32 j + 8 (e / 4) + 4 (l /
// 32) + e % 4): the eight columns of a generator group are held by lanes l and l + 32, four
// each.  Of each pair of groups the lower half makes the first one's block and the upper half
// the second one's; a half-wave swap of two word pairs then gives every lane the two words of
// its own elements of both groups.
__device__ __forceinline__ uint32_t keep_word(const DropKey &dk, uint32_t group0) {
  const uint32_t top = dk.thr << 16;
  uint32_t bits = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // groups 2 q and 2 q + 1 of the eight
    const u32x4_t w = drop_words(group0 + 2 * q + ((threadIdx.x & 63) >> 5), 0u, dk);
    const auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t v[2] = {g ? lo[1] : lo[0], g ? hi[1] : hi[0]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h = (e & 1) ? v[e / 2] : v[e / 2] << 16;  // the element's bits on top
        bits |= h >= top ? 1u << (8 * q + 4 * g + e) : 0u;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // one block's registers at a time
  }
  return bits;
}

}  // namespace qlora
