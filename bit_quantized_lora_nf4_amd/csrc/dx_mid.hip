// The extended dX GEMM on smaller tiles (gfx950): dX = dY W' + m (V A) for calls whose 256 x
// 256 tiles would leave most CUs idle (the backward of the forwards in gemm_mid.hip).
//
// A 256-thread workgroup computes 32 NI tokens x 256 weight columns (NI = 1, 2, 4); wave w owns
// all the tokens and 64 of the columns.  A step contracts 64 weight rows: lane l decodes row
// l's whole 64-weight block of the wave's columns into the wave's own 8 KB of LDS, from where
// the transposing reads give the MFMA's weight operand; only the dY tile, fetched two steps
// ahead through a ring of three, is shared, so there is one barrier a step.  Two or three
// workgroups share a CU, so that one's decode overlaps another's MFMAs without hand scheduling.
//   - dY comes in padded column blocks and the LoRA term carries the dropout mask, as in the
//     large kernel (DxExt in gemm.hip);
//   - SPLIT: the contraction is divided over several workgroups that write their fp32
//     accumulators, and dx_mid_join_kernel adds them in a fixed order.
// Bound by the decode's vector instructions (287 a step and wave, 130 of them permutes at half
// rate) and, split, by the partial sums.  Whole backward calls against the 256 x 256 tiles: 64
// x 4096 -> 4096 36 us (44), 400 x 4096 -> 1000 35 (47), 1319 x 3392 -> 1608 72 (82).  Decoding
// a step ahead between the MFMAs changed nothing at NI = 1 and 2 and spilled at NI = 4.

#include <type_traits>

#include "gemm_tile.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

typedef short v4i16_t __attribute__((ext_vector_type(4)));

constexpr int NT = 256;
constexpr int TK = 64;
constexpr int TC = 256;   // weight columns of a tile
constexpr int RING = 3;   // dY tiles in flight or in use
constexpr int kWaveW = 64 * 128;  // bytes of a wave's decoded weights
constexpr int kBlockFloats = 32 * 32;

struct DxMidParams {
  WeightView w;
  const uint16_t *dY;  // [M, Kc]
  const uint16_t *V;   // [M, r] or unused (r = 0)
  const uint16_t *At;  // [K, r]
  uint16_t *dX;        // [M, K]
  float *part;         // SPLIT: fp32 partial sums
  int M, K, N, Kc, r;  // N weight rows; Kc contraction positions (padded column blocks)
  int half, skip;      // position k stands for row k, or k - skip from `half` on
  int tiles_m, tiles_n, splits, ksteps;
  int fin_wgs;         // workgroups after the tiles, which do the finalize job
  Dropout drop;
  LevelTable lvl;
  FinalizeJob fin;
};

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char *dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
}

// One 32 x 32 block: lane holds token m and columns c + 8 g + 4 (l / 32) + 0..3 (g = 0..3).
__device__ __forceinline__ void store_block(const DxMidParams &p, int m, int c, const f32x16_t &a) {
  if (m >= p.M) return;
  uint16_t *row = p.dX + static_cast<int64_t>(m) * p.K + c + 4 * ((threadIdx.x >> 5) & 1);
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<u32x2_t *>(row + 8 * g) =
        u32x2_t{pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
}

struct CodeStage {
  u32x4_t code[2];
  ConstRaw c;
};

template <int CT, int NI, bool SPLIT>
__global__ __launch_bounds__(NT, 2) void dx_mid_kernel(DxMidParams p) {
  constexpr int TILE = NI * 32 * 128;  // bytes of a dY tile
  // the ring's buffers are objects of their own, so that the compiler can tell reads of one
  // from the loads into the others
  __shared__ __attribute__((aligned(16))) char sY0[TILE];
  __shared__ __attribute__((aligned(16))) char sY1[TILE];
  __shared__ __attribute__((aligned(16))) char sY2[TILE];
  __shared__ __attribute__((aligned(16))) char sW[4 * kWaveW];
  const int tiles = p.tiles_m * p.tiles_n;
  const int tile_wgs = SPLIT ? tiles * p.splits : tiles;
  if (static_cast<int>(blockIdx.x) >= tile_wgs) {
    finalize_part(p.fin, blockIdx.x - tile_wgs, p.fin_wgs);
    return;
  }
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = SPLIT ? static_cast<int>(blockIdx.x) / tiles : 0;
  const int tile = static_cast<int>(blockIdx.x) - split * tiles;
  int tmi, tni;
  tile_coords(tile, p.tiles_m, p.tiles_n, tmi, tni);
  const int m0 = tmi * 32 * NI, c0 = tni * TC + 64 * wave;
  const int K = p.K, Kc = p.Kc;
  const bool col_ok = c0 < K;  // K is a multiple of 64
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.dY, static_cast<uint32_t>(uint64_t(p.M) * Kc * 2));
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.w.codes, static_cast<uint32_t>(uint64_t(p.N) * K / 2));
  const ConstRsrc rq = make_const_rsrc<CT>(p.w, static_cast<uint32_t>(uint64_t(p.N) * K / 64));
  // this workgroup's contraction steps: nk of them from step s0
  const int all = (Kc + TK - 1) / TK, s0 = SPLIT ? split * p.ksteps : 0;
  const int nk = SPLIT ? min(all - s0, p.ksteps) : all;
  char *const sw = sW + wave * kWaveW;

  // dY loads: load i of a wave writes tile rows 8 (NI w + i) .. + 7 (1 KB, lane l at byte 16
  // l); rows past M are clamped to the last one and feed only outputs never stored; chunks
  // past the contraction read as zero
  uint32_t yoff[NI];
  int ych[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int x = (wave * NI + i) * 8 + (lane >> 3);
    ych[i] = ((lane & 7) ^ swz(x)) * 8;
    yoff[i] = static_cast<uint32_t>(min(m0 + x, p.M - 1)) * Kc * 2;
  }
  auto issue_y = [&](int it, char *tile_y) {
    const int kt = (s0 + min(it, nk - 1)) * TK;
    char *dst = tile_y + wave * NI * 1024;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      dma16(ry, dst + i * 1024, kt + ych[i] < Kc ? yoff[i] + (kt + ych[i]) * 2 : kOOB);
    __builtin_amdgcn_sched_barrier(0);  // each step's loads stay together, in step order
  };
  // the block of row l of the step; padding positions of the first column block take rows of
  // the second one, times zeros, positions past the last row are zero
  auto issue_codes = [&](int it, CodeStage &cs) {
    int n = (s0 + min(it, nk - 1)) * TK + lane;
    n -= n >= p.half ? p.skip : 0;
    const bool ok = col_ok && n < p.N;
    const uint32_t off = static_cast<uint32_t>(n) * (K / 2) + c0 / 2;
    cs.code[0] = buf_load16(rc, ok ? off : kOOB);
    cs.code[1] = buf_load16(rc, ok ? off + 16 : kOOB);
    cs.c = fetch_constant<CT>(rq, static_cast<uint32_t>(n) * (K / 64) + c0 / 64, ok);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int CODE_LOADS = 2 + (CT == kConstF32 ? 1 : 3);
  // token fragments of chunk c of a staged tile
  auto frag = [&](const char *t, int c, int i) {
    return *reinterpret_cast<const u32x4_t *>(t + tile_off(i * 32 + (lane & 31), c));
  };
  // weight fragments: columns 32 j + l % 32 of rows 16 s + 8 (l / 32) .. + 7 of the wave's tile
  // (within a 16-lane group, lane i reads 8 bytes of row base + i / 4 at column 4 (i % 4) of
  // its 16-column half and receives column i of those four rows)
  uint32_t trb[2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = lane & 15, g = lane >> 4;
      const int row = 8 * (g >> 1) + 4 * e + (i >> 2), col = 32 * j + (g & 1) * 16 + 4 * (i & 3);
      trb[e][j] = tile_off(row, col >> 3) + (col & 7) * 2;  // rows 16 apart swizzle alike
    }
  auto wfrag = [&](int s, int j) {
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const v4i16_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4i16_t *)(sw + trb[e][j] + 2048 * s));
      const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
      r[2 * e] = u[0];
      r[2 * e + 1] = u[1];
    }
    return r;
  };

  f32x16_t acc[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // The LoRA term first, 64 ranks at a time through the ring's last buffer (V rows past M
  // clamped like dY's, ranks past the end read as zero); split 0 adds it.
  if (p.r > 0 && split == 0) {
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(p.V, static_cast<uint32_t>(uint64_t(p.M) * p.r * 2));
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.At, static_cast<uint32_t>(uint64_t(K) * p.r * 2));
    char *const sV = sY2;
    for (int t = 0; t < p.r; t += TK) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int x = (wave * NI + i) * 8 + (lane >> 3);
        const int q = t + ych[i];
        dma16(rv, sV + (wave * NI + i) * 1024,
              q < p.r ? (static_cast<uint32_t>(min(m0 + x, p.M - 1)) * p.r + q) * 2 : kOOB);
      }
      u32x4_t al[4][2];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int q = t + 16 * s + 8 * half, k = c0 + 32 * j + (lane & 31);
          al[s][j] = buf_load16(ra, col_ok && q < p.r ? (static_cast<uint32_t>(k) * p.r + q) * 2 : kOOB);
        }
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const u32x4_t v = frag(sV, 2 * s + half, i);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(al[s][j], v, acc[i][j]);
        }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // read before it is loaded again
    }
    if (p.drop.thr != 0) {
      const DropKey dk = drop_key(p.drop);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t keep = keep_word(
            dk, static_cast<uint32_t>(m0 + 32 * i + (lane & 31)) * static_cast<uint32_t>(K / 8) + c0 / 8);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int m = static_cast<int>(keep << (31 - (16 * j + e))) >> 31;
            const float v = acc[i][j][e];
            acc[i][j][e] = __uint_as_float(__float_as_uint(v) & static_cast<uint32_t>(m));
          }
      }
    }
  }

  // A step: decode its codes, then multiply its tile.
  auto compute = [&](const char *t, const CodeStage &cs) {
    const Planes pl = make_planes(const_value<CT>(cs.c), p.lvl);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<u32x4_t *>(sw + tile_off(lane, q)) = lookup8(cs.code[q >> 2][q & 3], pl);
    // the wave's own writes, in order before its reads
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    u32x4_t wa[2], yb[NI];
#pragma unroll
    for (int j = 0; j < 2; ++j) wa[j] = wfrag(0, j);
#pragma unroll
    for (int i = 0; i < NI; ++i) yb[i] = frag(t, half, i);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t wan[2], ybn[NI];
      if (s < 3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) wan[j] = wfrag(s + 1, j);
#pragma unroll
        for (int i = 0; i < NI; ++i) ybn[i] = frag(t, 2 * (s + 1) + half, i);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(wa[j], yb[i], acc[i][j]);
      if (s < 3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) wa[j] = wan[j];
#pragma unroll
        for (int i = 0; i < NI; ++i) yb[i] = ybn[i];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // In the main loop the barrier leaves the next step's loads in flight.  After it every wave
  // has step it's tile and no wave still reads the buffer that the next loads overwrite.
  auto step = [&](int it, const char *t, char *next, const CodeStage &cur, CodeStage &ld) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(NI + CODE_LOADS) : "memory");
    issue_y(it + 2, next);
    issue_codes(it + 2, ld);
    compute(t, cur);
  };
  CodeStage S0, S1, S2;
  issue_y(0, sY0);
  issue_codes(0, S0);
  issue_y(1, sY1);
  issue_codes(1, S1);
  int it = 0;
  for (; it + RING <= nk; it += RING) {
    step(it, sY0, sY2, S0, S2);
    step(it + 1, sY1, sY0, S1, S0);
    step(it + 2, sY2, sY1, S2, S1);
  }
  // the last nk % 3 steps
  if (it < nk) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    compute(sY0, S0);
    if (it + 1 < nk) compute(sY1, S1);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may land after the kernel ends
  if (!col_ok) return;

  if constexpr (SPLIT) {
    float *const base = p.part + (static_cast<int64_t>(blockIdx.x) * 4 + wave) * (2 * NI * kBlockFloats);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (m0 + 32 * i >= p.M) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x4_t *dst = reinterpret_cast<f32x4_t *>(base + (2 * i + j) * kBlockFloats) + lane;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          dst[64 * g] = f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) store_block(p, m0 + 32 * i + (lane & 31), c0 + 32 * j, acc[i][j]);
  }
}

// The join of a split dX: a wave adds one block's partial sums in split order, four splits'
// loads in flight at a time, and rounds once.
template <int NI>
__global__ __launch_bounds__(NT) void dx_mid_join_kernel(DxMidParams p) {
  const int lane = threadIdx.x & 63;
  const int tiles = p.tiles_m * p.tiles_n;
  const int unit = static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 6);
  const int b = unit % (2 * NI), wave = (unit / (2 * NI)) & 3, tile = unit / (8 * NI);
  if (tile >= tiles) return;
  int tmi, tni;
  tile_coords(tile, p.tiles_m, p.tiles_n, tmi, tni);
  const int m0 = tmi * 32 * NI + 32 * (b >> 1), c0 = tni * TC + 64 * wave;
  if (m0 >= p.M || c0 >= p.K) return;
  const f32x4_t *src = reinterpret_cast<const f32x4_t *>(p.part) +
                       ((static_cast<int64_t>(tile) * 4 + wave) * (2 * NI) + b) * (kBlockFloats / 4) + lane;
  const int64_t pitch = static_cast<int64_t>(tiles) * 8 * NI * (kBlockFloats / 4);
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
  store_block(p, m0 + (lane & 31), c0 + 32 * (b & 1), a);
}

// Tile height and splits by the time they take, as for the forward (mid_plan in gemm_mid.hip): a
// step takes a workgroup alone on its CU 0.92 / 1.06 / 1.4 us (NI = 1 / 2 / 4), a CU with
// several 0.75 / 0.85 / 0.9 for each (the decode: a CU's vector units are shared), a fifth more
// when the launch is long enough for the card's power to set the clock; 8 us around the steps,
// 2 more for every workgroup past a CU's second; a split adds the join's launch, the partial
// sums, and a little for each part.
struct DxMidPlan {
  int ni, tiles_m, tiles_n, splits, ksteps;
  double cost;
};
DxMidPlan dx_mid_plan(int64_t M, int64_t K, int64_t Kc) {
  DxMidPlan b;
  b.cost = 1e30;
  const int64_t nk = (Kc + TK - 1) / TK, tiles_n = (K + TC - 1) / TC;
  for (int ni = M <= 32 ? 1 : M <= 64 ? 2 : 4; ni >= 1; ni /= 2) {
    const int64_t tiles_m = (M + 32 * ni - 1) / (32 * ni), tiles = tiles_m * tiles_n;
    const double lone = ni == 4 ? 1.4 : ni == 2 ? 1.06 : 0.92, shared = ni == 4 ? 0.9 : ni == 2 ? 0.85 : 0.75;
    for (int64_t s = 1; s == 1 || (s * tiles <= 1024 && 2 * s <= nk); ++s) {
      const int64_t steps = (nk + s - 1) / s, used = (nk + steps - 1) / steps;
      const int64_t per_cu = (tiles * used + 255) / 256;
      const double run = (per_cu == 1 ? lone : per_cu * shared) * steps * (per_cu * steps > 60 ? 1.2 : 1.0) +
                         (per_cu > 2 ? 2.0 * (per_cu - 2) : 0.0);
      const double cost = run + 8.0 + (used > 1 ? 7.0 + 0.3 * used + double(M) * K * 8.0 * used / 4.5e6 : 0.0);
      if (cost < b.cost - 1e-9)
        b = {ni, static_cast<int>(tiles_m), static_cast<int>(tiles_n), static_cast<int>(used),
             static_cast<int>(steps), cost};
    }
  }
  return b;
}

}  // namespace

double dx_mid_cost(int64_t M, int64_t K, int64_t Kc) { return dx_mid_plan(M, K, Kc).cost; }

size_t dx_mid_workspace(int64_t M, int64_t K, int64_t Kc) {
  const DxMidPlan b = dx_mid_plan(M, K, Kc);
  return b.splits > 1 ? size_t(b.splits) * b.tiles_m * b.tiles_n * 8 * b.ni * kBlockFloats * sizeof(float) : 0;
}

hipError_t launch_dx_mid(const WeightView &w, const uint16_t *dY, int64_t M, int64_t Kc, int64_t half, int64_t skip,
                         const uint16_t *V, const uint16_t *At, int r, uint16_t *dX, const Dropout &d, float *part,
                         hipStream_t stream, const FinalizeJob *fin) {
  const int64_t N = w.n_rows, K = w.n_cols;
  if (K % 64 != 0 || Kc % 8 != 0 || r % 8 != 0) return hipErrorInvalidValue;
  const DxMidPlan b = dx_mid_plan(M, K, Kc);
  DxMidParams p;
  p.w = w;
  p.dY = dY;
  p.V = V;
  p.At = At;
  p.dX = dX;
  p.part = part;
  p.M = static_cast<int>(M);
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.Kc = static_cast<int>(Kc);
  p.r = r;
  p.half = static_cast<int>(half);
  p.skip = static_cast<int>(skip);
  p.tiles_m = b.tiles_m;
  p.tiles_n = b.tiles_n;
  p.splits = b.splits;
  p.ksteps = b.ksteps;
  p.drop = d;
  p.lvl = level_table(w.quant_type);
  p.fin_wgs = 0;
  p.fin = FinalizeJob{nullptr, 0, 0, 0, 0, 0.0f, nullptr};
  if (fin && fin->splits > 0) {
    p.fin = *fin;
    p.fin_wgs = static_cast<int>(finalize_workgroups(*fin));
  }
  const int64_t wgs = int64_t(b.tiles_m) * b.tiles_n * b.splits + p.fin_wgs;
  if (wgs > 0x7fffffff || (b.splits > 1 && !part)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(wgs)), block(NT);
  auto go = [&](auto ct, auto ni) -> hipError_t {
    constexpr int CT = decltype(ct)::value, NI = decltype(ni)::value;
    if (b.splits == 1) {
      hipLaunchKernelGGL((dx_mid_kernel<CT, NI, false>), grid, block, 0, stream, p);
      return hipGetLastError();
    }
    hipLaunchKernelGGL((dx_mid_kernel<CT, NI, true>), grid, block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 jgrid(static_cast<unsigned>(int64_t(b.tiles_m) * b.tiles_n * 2 * NI));
    hipLaunchKernelGGL((dx_mid_join_kernel<NI>), jgrid, block, 0, stream, p);
    return hipGetLastError();
  };
  auto with_ni = [&](auto ct) {
    return b.ni == 1 ? go(ct, std::integral_constant<int, 1>{})
           : b.ni == 2 ? go(ct, std::integral_constant<int, 2>{}) : go(ct, std::integral_constant<int, 4>{});
  };
  switch (w.const_type) {
    case kConstDqInt8: return with_ni(std::integral_constant<int, kConstDqInt8>{});
    case kConstDqFp8: return with_ni(std::integral_constant<int, kConstDqFp8>{});
    case kConstF32: return with_ni(std::integral_constant<int, kConstF32>{});
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qlora
