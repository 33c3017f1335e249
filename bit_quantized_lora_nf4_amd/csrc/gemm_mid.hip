// The fused NF4 forward on smaller tiles (gfx950): Y = X W'^T + U Bl^T, and the gated
// projections H = act(G) L, for calls whose 256 x 256 tiles would leave most CUs idle.
//
// A 256-thread workgroup computes 32 NI tokens x 128 weight rows (NI = 1, 2, 4); wave w owns
// all the tokens and 32 of the rows, one 32x32x16 MFMA block per 32 tokens.  As in the large
// kernel the weight is the MFMA's A operand, decoded per lane straight into fragments (lane
// l: weight row l % 32), and X tiles go to LDS by
// direct buffer loads in the same swizzled layout.  What differs:
//   - the contraction advances two 64-steps at a time, and lane half h decodes the whole
//     64-weight block of step h (as the MFMA's contraction half h), so that the 16 table
//     entries of a block constant are made once instead of in both halves: 133 vector
//     instructions a step instead of 152, which is what bounds the kernel;
//   - several workgroups share a CU (16 to 64 KB of LDS each, at most 256 registers a
//     lane), so that one wave's decode overlaps another's MFMAs without hand scheduling;
//   - X tiles are fetched two steps ahead through a ring of four, and the codes and
//     constants of four steps (a row's 128-byte line) together, a group ahead;
//   - gated: the 32 rows of a wave are 16 gate rows and the same 16 up rows, which the
//     accumulator layout puts in one lane (elements e and e + 8 of a block);
//   - the LoRA term runs over 64 ranks at a time staged like an X tile; gated, the two
//     projections' ranks are staged side by side and summed apart;
//   - SPLIT: the contraction is divided over several workgroups that write their fp32
//     accumulators, and gemm_mid_join adds them in a fixed order and does the epilogue.
// Bound by the decode's vector instructions (at 16 tokens they issue in 65 % of the cycles, and
// two fifths of them are permutes, which take two slots).
// Measured, whole calls: 16 x 8192 -> 2 x 22016 of rank 64 83 us (2.35 TB/s; the 256 x 256
// tiles and the small-M kernel take 150), 777 x 4096 -> 2 x 11008 184 us (201), 333 x 1280 ->
// 2 x 1001 of rank 12, copies of its operands included, 28 us (82).

#include <type_traits>

#include "gemm_tile.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int NT = 256;
constexpr int TK = 64;
constexpr int TN = 128;    // weight rows of a tile (gated: 64 columns of each projection)
constexpr int RING = 4;    // X tiles in flight or in use, and steps of a code group
constexpr int kBlockFloats = 32 * 32;

struct MidParams {
  WeightView w;
  const uint16_t *X;   // [M, K]
  const uint16_t *U;   // [M, ldu] or unused (r = 0)
  const uint16_t *Bl;  // [N, r]
  uint16_t *Y;         // [M, N]; gated: [M, 2 P] or NULL
  uint16_t *H;         // gated: [M, P]
  float *part;         // SPLIT: fp32 partial sums
  int M, N, K, r, ldu;
  int part_rows;       // gated: P; else rows per part of fused linears, or 0
  int act;
  int tiles_m, tiles_n, splits, ksteps;
  LevelTable lvl;
};

// The weight row of lane row x (0..31) of block column base c (gated: of the projections'
// column c), or -1 past the edge.
template <bool GATED>
__device__ __forceinline__ int weight_row(const MidParams &p, int c, int x) {
  if constexpr (GATED) {
    const int h = c + (x & 15);
    return h < p.part_rows ? (x >> 4) * p.part_rows + h : -1;
  }
  return c + x < p.N ? c + x : -1;
}

// Four bf16 values v at row[col..], of which those below `cols` exist.
__device__ __forceinline__ void put4(uint16_t *row, int col, int cols, const float (&v)[4]) {
  if (cols % 4 == 0) {
    if (col < cols)
      *reinterpret_cast<u32x2_t *>(row + col) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < cols) row[col + e] = to_bf16(v[e]);
}

// A finished block: lane holds token m (when below M) and rows 8 g + 4 (l / 32) + 0..3 of
// the block's 32 weight rows in a[4 g + 0..3].
template <bool GATED>
__device__ __forceinline__ void store_block(const MidParams &p, int m, int c, const f32x16_t &a) {
  if (m >= p.M) return;
  const int half = (threadIdx.x >> 5) & 1;
  if constexpr (!GATED) {
    uint16_t *row = p.Y + static_cast<int64_t>(m) * p.N;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float v[4] = {a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
      put4(row, c + 8 * g + 4 * half, p.N, v);
    }
  } else {
    const int P = p.part_rows;
    uint16_t *hrow = p.H + static_cast<int64_t>(m) * P;
    uint16_t *yrow = p.Y + static_cast<int64_t>(m) * 2 * P;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float G[4] = {a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
      const float L[4] = {a[4 * g + 8], a[4 * g + 9], a[4 * g + 10], a[4 * g + 11]};
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[e] = (p.act == kActSilu ? act_value<kActSilu>(G[e]) : act_value<kActGeluTanh>(G[e])) * L[e];
      const int col = c + 8 * g + 4 * half;
      put4(hrow, col, P, h);
      if (p.Y) {
        put4(yrow, col, P, G);
        put4(yrow + P, col, P, L);
      }
    }
  }
}

// One 16-byte piece a lane from a buffer straight into LDS (lane l at dst + 16 l).  A named
// function: from a lambda of the kernel template the builtin keeps the host compilation from
// emitting the instantiations' launch stubs.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char *dst, uint32_t off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, off, soff, 0, 0);
}

// The codes of a lane's blocks among four consecutive steps (steps h and 2 + h of the group
// for lane half h, 32 bytes each) and the row's four block constants: the fp32 ones, or two
// aligned dwords that cover the four 8-bit codes.  The group scale and offset of the double-quantized types are loaded once: a
// workgroup's steps are at most kMaxSteps blocks of the row, so they lie in two groups.
template <int CT>
struct Codes {
  u32x4_t code[RING];
  typename std::conditional<CT == kConstF32, u32x4_t, u32x2_t>::type q;
};
constexpr int kCodeLoads = RING + 1;  // vector loads of one Codes
constexpr int kMaxSteps = 256;

// One tile of 32 NI tokens from m0 on; SLOT: 32-token blocks of a tile in the partial sums.
template <int CT, bool GATED, int NI, bool SPLIT, int SLOT>
__device__ __forceinline__ void mid_body(const MidParams &p, char *sX, int m0, int tni, int split) {
  constexpr int TILE = NI * 32 * 128;  // bytes of an X tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = tni * (GATED ? TN / 2 : TN) + wave * (GATED ? 16 : 32);  // this wave's first column

  const int K = p.K;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.X, static_cast<uint32_t>(uint64_t(p.M) * K * 2));
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.w.codes, static_cast<uint32_t>(uint64_t(p.N) * K / 2));
  const ConstRsrc rq = make_const_rsrc<CT>(p.w, static_cast<uint32_t>(uint64_t(p.N) * K / 64));
  // this workgroup's contraction steps: nk of them from step s0
  const int s0 = SPLIT ? split * p.ksteps : 0;
  const int nk = SPLIT ? min(K / TK - s0, p.ksteps) : K / TK;

  // X loads: load i of a wave writes tile rows 8 (NI w + i) .. + 7 (1 KB, lane l at byte
  // 16 l); rows past M are clamped to the last one and feed only outputs never stored
  uint32_t xoff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int x = (wave * NI + i) * 8 + (lane >> 3);
    xoff[i] = (static_cast<uint32_t>(min(m0 + x, p.M - 1)) * K + ((lane & 7) ^ swz(x)) * 8) * 2;
  }
  // codes and constants of this lane's weight row (lanes past the edge read row 0's: they
  // feed only outputs never stored)
  const int n = weight_row<GATED>(p, c0, lane & 31);
  const bool row_ok = n >= 0;
  const int half = lane >> 5;
  const uint32_t coff = row_ok ? static_cast<uint32_t>(n) * (K / 2) : 0;
  const uint32_t boff = row_ok ? static_cast<uint32_t>(n) * (K / 64) : 0;
  const uint32_t b0 = boff + s0, grp0 = b0 >> 8, grp1 = (b0 + nk - 1) >> 8;
  float gs[2] = {0.0f, 0.0f}, go[2] = {0.0f, 0.0f};
  if constexpr (CT != kConstF32) {
    gs[0] = __uint_as_float(buf_load4(rq.s, grp0 * 4u));
    gs[1] = __uint_as_float(buf_load4(rq.s, grp1 * 4u));
    go[0] = __uint_as_float(buf_load4(rq.o, grp0 * 4u));
    go[1] = __uint_as_float(buf_load4(rq.o, grp1 * 4u));
  }
  // the 8-bit codes as aligned dwords: from the dword that holds the array's first byte (the
  // array may start anywhere) to the one that holds its last
  const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.w.absmax_q)) & 3u;
  const __amdgpu_buffer_rsrc_t r8 =
      make_rsrc(p.w.absmax_q - mis, static_cast<uint32_t>((uint64_t(p.N) * K / 64 + mis + 3) & ~uint64_t(3)));
  // c' (rounded once) of the block of step it = 4 a + 2 jp + half
  auto constant = [&](const Codes<CT> &cs, int jp, int it) {
    if constexpr (CT == kConstF32) return __uint_as_float(half ? cs.q[2 * jp + 1] : cs.q[2 * jp]);
    const uint32_t first = b0 + (it - 2 * jp - half) + mis;
    const uint32_t four = __builtin_amdgcn_alignbit(cs.q[1], cs.q[0], (first & 3u) * 8u);
    const bool low = ((b0 + it) >> 8) == grp0;
    return __builtin_fmaf(c8_value<CT>((four >> (8 * (2 * jp + half))) & 0xFFu), low ? gs[0] : gs[1],
                          low ? go[0] : go[1]);
  };
  // the codes of steps it .. it + 3 (steps past the end repeat the last one's codes and are
  // not used; their constants read the following bytes)
  auto issue_codes = [&](int it, Codes<CT> &cs) {
#pragma unroll
    for (int jp = 0; jp < 2; ++jp) {
      const uint32_t off = coff + (s0 + min(it + 2 * jp + half, nk - 1)) * (TK / 2);
      cs.code[2 * jp] = buf_load16(rc, off);
      cs.code[2 * jp + 1] = buf_load16(rc, off + 16);
    }
    const uint32_t b = b0 + min(it, nk - 1);
    if constexpr (CT == kConstF32)
      cs.q = buf_load16(rq.s, b * 4u);
    else
      cs.q = buf_load8(r8, (b + mis) & ~3u);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto issue_x = [&](int it) {
    char *dst = sX + (it % RING) * TILE + wave * NI * 1024;
#pragma unroll
    for (int i = 0; i < NI; ++i) dma16(rx, dst + i * 1024, xoff[i], (s0 + min(it, nk - 1)) * TK * 2);
    __builtin_amdgcn_sched_barrier(0);  // each step's loads stay together, in step order
  };
  // fragments of chunk c of a staged tile's rows: token 32 i + l % 32
  auto frag = [&](const char *t, int c, int i) {
    return *reinterpret_cast<const u32x4_t *>(t + tile_off(i * 32 + (lane & 31), c));
  };

  f32x16_t acc[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;

  // The LoRA term first, 64 ranks at a time through the ring's last buffer (U rows past M
  // clamped like X's, ranks past the end read as zero); split 0 adds it.  Gated: both
  // projections' ranks at a time, the up projection's through the buffer before it and into sums
  // of their own, of which its rows (elements 8..15 of a block) are taken: in common sums a
  // projection's infinities would meet the zeros of the other's rows.
  if (p.r > 0 && split == 0) {
    constexpr int PARTS = GATED ? 2 : 1;
    const int qc = !GATED && p.part_rows > 0 ? (c0 / p.part_rows) * p.r : 0;
    const __amdgpu_buffer_rsrc_t ru = make_rsrc(p.U, static_cast<uint32_t>(uint64_t(p.M) * p.ldu * 2));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.Bl, static_cast<uint32_t>(uint64_t(p.N) * p.r * 2));
    f32x16_t up[GATED ? NI : 1];
#pragma unroll
    for (int i = 0; i < (GATED ? NI : 1); ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) up[i][e] = 0.0f;
    for (int t = 0; t < p.r; t += TK) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int x = (wave * NI + i) * 8 + (lane >> 3);
          const int j = t + ((lane & 7) ^ swz(x)) * 8;
          const uint32_t off =
              j < p.r ? (static_cast<uint32_t>(min(m0 + x, p.M - 1)) * p.ldu + (GATED ? q * p.r : qc) + j) * 2 : kOOB;
          dma16(ru, sX + (RING - 1 - q) * TILE + (wave * NI + i) * 1024, off, 0);
        }
      // 8 ranks of this lane's row (every lane's row takes part in one of the two sums)
      u32x4_t wl[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int j = t + (GATED ? 16 * s + 8 * half : 32 * half + 8 * s);
        wl[s] = buf_load16(rb, row_ok && j < p.r ? (static_cast<uint32_t>(n) * p.r + j) * 2 : kOOB);
      }
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (GATED && t + 16 * s >= p.r) break;  // (no ranks left for this sub-step)
        const int c = GATED ? 2 * s + half : 4 * half + s;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          acc[i] = mfma32x32x16(wl[s], frag(sX + (RING - 1) * TILE, c, i), acc[i]);
          if constexpr (GATED) up[i] = mfma32x32x16(wl[s], frag(sX + (RING - 2) * TILE, c, i), up[i]);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // read before it is loaded again
    }
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 8; e < 16; ++e) acc[i][e] = up[i][e];
    }
  }

  // Two steps, 4 a + 2 jp and the next: lane half h takes the whole block of step h from tile
  // t + h; with `single` there is no second step, and half 1 adds zeros (its tile is cleared
  // too: zero weights alone would make NaN of an infinity).  The codes' fragments are decoded
  // and the X fragments read one sub-step ahead of the MFMAs that use them.
  auto compute = [&](const char *tiles2, const Codes<CT> &cs, int jp, int it, bool single) {
    const char *t = tiles2 + half * TILE;
    float c = constant(cs, jp, it + half);
    if (single && half) c = 0.0f;
    const Planes pl = make_planes(c, p.lvl);
    u32x4_t wa = lookup8(cs.code[2 * jp][0], pl), xb[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) xb[i] = frag(t, 0, i);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      u32x4_t wan, xbn[NI];
      if (s < 7) {
#pragma unroll
        for (int i = 0; i < NI; ++i) xbn[i] = frag(t, s + 1, i);
        wan = lookup8(cs.code[2 * jp + (s + 1) / 4][(s + 1) & 3], pl);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] = mfma32x32x16(wa, xb[i], acc[i]);
      if (s < 7) {
        wa = wan;
#pragma unroll
        for (int i = 0; i < NI; ++i) xb[i] = xbn[i];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Four steps of the group `cur`, two at a time: the two tiles that the next two steps read
  // are loaded first, then (once a group) the next group's codes, which may stay in flight at
  // the barrier that publishes those tiles.
  auto group = [&](int it, const Codes<CT> &cur, Codes<CT> &nxt) {
#pragma unroll
    for (int jp = 0; jp < 2; ++jp) {
      // tiles it + 2 jp and the next have landed for every wave, and no wave still reads the
      // buffers that the next loads overwrite
      if (jp == 0)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kCodeLoads) : "memory");
      issue_x(it + 2 * jp + 2);
      issue_x(it + 2 * jp + 3);
      if (jp == 0) issue_codes(it + RING, nxt);
      compute(sX + 2 * jp * TILE, cur, jp, it + 2 * jp, false);
    }
  };
  Codes<CT> ca, cb;
  issue_codes(0, ca);
#pragma unroll
  for (int j = 0; j < 2; ++j) issue_x(j);
  int it = 0;
  for (; it + 2 * RING <= nk; it += 2 * RING) {
    group(it, ca, cb);
    group(it + RING, cb, ca);
  }
  if (it + RING <= nk) {
    group(it, ca, cb);
    it += RING;
    ca = cb;
  }
  // the last nk % 4 steps; a wave clears its part of the tile behind an odd last one
  auto clear_x = [&](int slot) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      *reinterpret_cast<u32x4_t *>(sX + slot * TILE + (wave * NI + i) * 1024 + lane * 16) = u32x4_t{0u, 0u, 0u, 0u};
  };
  const int rem = nk - it;
  if (rem > 0) {
    if (rem == 1) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // slot 1 still takes the repeated last tile
      clear_x(1);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    issue_x(it + 2);
    if (rem == 3) clear_x(3);  // (no load into slot 3 is in flight, and no wave reads it any more)
    compute(sX, ca, 0, it, rem == 1);
    if (rem == 3) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      compute(sX + 2 * TILE, ca, 1, it + 2, true);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may land after the kernel ends

  if constexpr (SPLIT) {
    float *const base = p.part + (static_cast<int64_t>(blockIdx.x) * 4 + wave) * (SLOT * kBlockFloats);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (m0 + 32 * i >= p.M) break;
      f32x4_t *dst = reinterpret_cast<f32x4_t *>(base + i * kBlockFloats) + lane;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        dst[64 * g] = f32x4_t{acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) store_block<GATED>(p, m0 + 32 * i + (lane & 31), c0, acc[i]);
  }
}

// TAIL: the 32-token blocks of the last tile, when that many hold its tokens (0: as many as the
// others'): a step for 32 tokens takes 0.55 of the time of one for 128 (777 x 4096 -> 2 x 11008:
// 189.6 us with 128 for the last 9 tokens, 183.0 with 32).
template <int CT, bool GATED, int NI, bool SPLIT, int TAIL>
__global__ __launch_bounds__(NT, 2) void gemm_mid_kernel(MidParams p) {
  __shared__ __attribute__((aligned(16))) char sX[RING * NI * 32 * 128];
  const int tiles = p.tiles_m * p.tiles_n;
  const int split = SPLIT ? static_cast<int>(blockIdx.x) / tiles : 0;
  const int tile = static_cast<int>(blockIdx.x) - split * tiles;
  int tmi, tni;
  tile_coords(tile, p.tiles_m, p.tiles_n, tmi, tni);
  if constexpr (TAIL > 0) {
    if (tmi == p.tiles_m - 1) {
      mid_body<CT, GATED, TAIL, SPLIT, NI>(p, sX, tmi * 32 * NI, tni, split);
      return;
    }
  }
  mid_body<CT, GATED, NI, SPLIT, NI>(p, sX, tmi * 32 * NI, tni, split);
}

// The join of a split forward: a wave adds one block's partial sums in split order, four
// splits' loads in flight at a time, and finishes the block.
template <bool GATED, int NI>
__global__ __launch_bounds__(NT) void gemm_mid_join_kernel(MidParams p) {
  const int lane = threadIdx.x & 63;
  const int tiles = p.tiles_m * p.tiles_n;
  const int unit = static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 6);
  const int i = unit % NI, wave = (unit / NI) & 3, tile = unit / (4 * NI);
  if (tile >= tiles) return;
  int tmi, tni;
  tile_coords(tile, p.tiles_m, p.tiles_n, tmi, tni);
  const int m0 = tmi * 32 * NI + 32 * i;
  if (m0 >= p.M) return;
  const f32x4_t *src = reinterpret_cast<const f32x4_t *>(p.part) +
                       ((static_cast<int64_t>(tile) * 4 + wave) * NI + i) * (kBlockFloats / 4) + lane;
  const int64_t pitch = static_cast<int64_t>(tiles) * 4 * NI * (kBlockFloats / 4);
  f32x16_t a;
#pragma unroll
  for (int e = 0; e < 16; ++e) a[e] = 0.0f;
  for (int k = 0; k < p.splits; k += 4) {
    f32x4_t v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int g = 0; g < 4; ++g) v[u][g] = src[min(k + u, p.splits - 1) * pitch + 64 * g];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k + u < p.splits) {
#pragma unroll
        for (int e = 0; e < 16; ++e) a[e] += v[u][e >> 2][e & 3];
      }
  }
  const int c0 = tni * (GATED ? TN / 2 : TN) + wave * (GATED ? 16 : 32);
  store_block<GATED>(p, m0 + (lane & 31), c0, a);
}

}  // namespace

namespace {
// The tile height (NI blocks of 32 tokens, no more than hold M) and the number of splits, by
// the time they take: a step of a workgroup costs its CU about 0.32 / 0.44 / 0.58 us (NI = 1 /
// 2 / 4; measured on 4096 -> 2 x 11008 and 8192 -> 2 x 22016), 15% more when it is alone
// there; splits add the join's launch and the partial sums, written and read once.  Lower
// tiles decode the weight more often but spread few tokens over more CUs without a join
// (whole calls, us, the best with NI = 1, 2, 4: 128 x 4096 -> 2 x 2000: 25.9, 26.9, 28.9; 500
// x 1536 -> 2 x 1200: 26.9, 21.4, 25.5; 160 x 8192 -> 2 x 4000: 70.6, 58.3, 57.1).
struct MidPlan {
  int ni, tiles_m, tiles_n, splits, ksteps;
  double cost;
};
MidPlan mid_plan(int64_t M, int64_t K, int64_t cols) {
  MidPlan b;
  b.cost = 1e30;
  const int64_t nk = K / TK, tiles_n = (cols + TN - 1) / TN, s_min = (nk + kMaxSteps - 1) / kMaxSteps;
  for (int ni = M <= 32 ? 1 : M <= 64 ? 2 : 4; ni >= 1; ni /= 2) {
    const int64_t tiles_m = (M + 32 * ni - 1) / (32 * ni), tiles = tiles_m * tiles_n;
    const double step = ni == 4 ? 0.58 : ni == 2 ? 0.44 : 0.32;
    for (int64_t s = s_min; s == s_min || (s * tiles <= 1024 && 2 * s <= nk); ++s) {
      // whole code groups, which are whole lines when the rows are
      const int64_t steps = s == 1 ? nk : (nk + s * RING - 1) / (s * RING) * RING, used = (nk + steps - 1) / steps;
      const int64_t per_cu = (tiles * used + 255) / 256;
      const double cost = (per_cu == 1 ? 1.15 : double(per_cu)) * step * steps + 5.0 +
                          (used > 1 ? 5.0 + double(M) * cols * 8.0 * used / 4.5e6 : 0.0);
      if (cost < b.cost - 1e-9)
        b = {ni, static_cast<int>(tiles_m), static_cast<int>(tiles_n), static_cast<int>(used),
             static_cast<int>(steps), cost};
    }
  }
  return b;
}

// The 256 x 256 tiles' time: a step of a round that fills the card takes about 1.65 us (the
// card's power bounds it), 1.2 us when few CUs work, and each round about 4 us around its steps.
double big_cost(int64_t M, int64_t K, int64_t cols) {
  const int64_t tiles = ((M + 255) / 256) * ((cols + 255) / 256), full = tiles / 256, rest = tiles % 256;
  const double nk = double(K / TK);
  return full * (1.65 * nk + 4.0) + (rest ? (1.2 + 0.45 * rest / 256.0) * nk + 4.0 : 0.0);
}

int64_t tile_cols(int64_t N, bool gated) { return gated ? (N / 2 + 63) / 64 * 128 : N; }
}  // namespace

// Measured (whole calls, us, 256 x 256 tiles against these): 20 x 4096 -> 2 x 11008: 90, 35;
// 128: 90, 51; 256: 93, 77; 512: 109, 121; 777: 205, 191; 1024: 212, 226; 136 x 5696 -> 2 x
// 832: 118, 33; 1000 x 2048 -> 2 x 2048: 54, 33.
bool mid_takes(int64_t M, int64_t K, int64_t N, bool gated) {
  const int64_t cols = tile_cols(N, gated);
  return mid_plan(M, K, cols).cost < big_cost(M, K, cols);
}

// The one-launch small-M kernel reads the weight once for all tokens but every token's X
// again for each 16 weight rows; measured it takes about 4 + (0.23 + 0.008 M) us per million
// weights (gated, 1 x 4096 -> 2 x 11008: 24.5; 16: 38; 1 x 8192 -> 2 x 22016: 88; 16: 134),
// these tiles their plan's time and two launches of about 5 us for U (33, 33, 74, 78).
bool gemv_takes(int64_t M, int64_t K, int64_t N, int r, bool gated) {
  if (!gemv_shape_ok(M, N, K)) return false;
  const double gemv = 4.0 + double(N) * K * 1e-6 * (0.23 + 0.008 * M);
  return gemv < mid_plan(M, K, tile_cols(N, gated)).cost + (r > 0 ? 10.0 : 0.0);
}

size_t gemm_mid_workspace(int64_t M, int64_t K, int64_t N, bool gated) {
  const MidPlan b = mid_plan(M, K, tile_cols(N, gated));
  return b.splits > 1 ? size_t(b.splits) * b.tiles_m * b.tiles_n * 4 * b.ni * kBlockFloats * sizeof(float) : 0;
}

hipError_t launch_gemm_mid(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U, int ldu,
                           const uint16_t *Bl, int r, int64_t part_rows, bool gated, int act, uint16_t *H, uint16_t *Y,
                           float *part, hipStream_t stream) {
  const int64_t N = w.n_rows, K = w.n_cols, P = N / 2;
  if (!gemm_supported(w, M, ldu) || (r > 0 && (r % 8 != 0 || ldu % 8 != 0))) return hipErrorInvalidValue;
  if (gated ? (N % 2 != 0 || (r > 0 && ldu != 2 * r)) : (part_rows > 0 && (part_rows % TN != 0 || N % part_rows != 0)))
    return hipErrorInvalidValue;
  const MidPlan b = mid_plan(M, K, tile_cols(N, gated));
  MidParams p;
  p.w = w;
  p.X = X;
  p.U = U;
  p.Bl = Bl;
  p.Y = Y;
  p.H = H;
  p.part = part;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.r = r;
  p.ldu = ldu;
  p.part_rows = static_cast<int>(gated ? P : part_rows);
  p.act = act;
  p.tiles_m = b.tiles_m;
  p.tiles_n = b.tiles_n;
  p.splits = b.splits;
  p.ksteps = b.ksteps;
  p.lvl = level_table(w.quant_type);
  const int64_t wgs = int64_t(b.tiles_m) * b.tiles_n * b.splits;
  if (wgs > 0x7fffffff || (b.splits > 1 && !part)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(wgs)), block(NT);
  auto go = [&](auto ct, auto g, auto ni, auto tail) -> hipError_t {
    constexpr int CT = decltype(ct)::value, NI = decltype(ni)::value, TAIL = decltype(tail)::value;
    constexpr bool GATED = decltype(g)::value;
    if (b.splits == 1) {
      hipLaunchKernelGGL((gemm_mid_kernel<CT, GATED, NI, false, TAIL>), grid, block, 0, stream, p);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((gemm_mid_kernel<CT, GATED, NI, true, TAIL>), grid, block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 jgrid(static_cast<unsigned>(int64_t(b.tiles_m) * b.tiles_n * NI));
    hipLaunchKernelGGL((gemm_mid_join_kernel<GATED, NI>), jgrid, block, 0, stream, p);
    return hipGetLastError();
  };
  const int64_t last = M - int64_t(b.tiles_m - 1) * 32 * b.ni;  // tokens of the last tile
  auto with_ni = [&](auto ct, auto g) {
    using std::integral_constant;
    if (b.ni == 1) return go(ct, g, integral_constant<int, 1>{}, integral_constant<int, 0>{});
    if (b.ni == 2)
      return last <= 32 ? go(ct, g, integral_constant<int, 2>{}, integral_constant<int, 1>{})
                        : go(ct, g, integral_constant<int, 2>{}, integral_constant<int, 0>{});
    return last <= 32   ? go(ct, g, integral_constant<int, 4>{}, integral_constant<int, 1>{})
           : last <= 64 ? go(ct, g, integral_constant<int, 4>{}, integral_constant<int, 2>{})
                        : go(ct, g, integral_constant<int, 4>{}, integral_constant<int, 0>{});
  };
  auto with_g = [&](auto ct) { return gated ? with_ni(ct, std::true_type{}) : with_ni(ct, std::false_type{}); };
  switch (w.const_type) {
    case kConstDqInt8: return with_g(std::integral_constant<int, kConstDqInt8>{});
    case kConstDqFp8: return with_g(std::integral_constant<int, kConstDqFp8>{});
    case kConstF32: return with_g(std::integral_constant<int, kConstF32>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qlora
