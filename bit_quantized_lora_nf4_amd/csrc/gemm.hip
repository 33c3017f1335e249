// Fused NF4-decode GEMMs on bf16 MFMA (gfx950): the forward Y = X W'^T + U Bl^T
// and the input gradient dX = dY W' + V At^T.
//
// W' is never written to HBM: the kernels stream packed 4-bit codes plus int8 block
// constants and decode them to bf16 on the fly ([Digest] "方法步骤与流程" step 3 and
// [QLoRA note] "5. QLoRA 训练方式本身": the 4-bit weight is decoded to BF16 inside
// the operator): w' = bf16_rne(q[code] * c'), c' = fma(c8, s, o).  The LoRA product
// is added to the same fp32 accumulators as r extra contraction steps (before the
// weight's) ahead of the single bf16 rounding of each output.
//
// Tile: a 256-thread workgroup (four waves, one per SIMD) computes a 256 x 256 output
// tile, 256 fp32 accumulators per lane.  In the forward, wave w owns all 256
// activation rows and output columns [64 w, 64 w + 64), i.e. 8 x 2 tiles of the
// 32x32x16 MFMA; in dX the waves split the tile 2 x 2 (4 x 4 MFMA tiles each).  The
// MFMA "A" operand is the weight side (rows = output columns) and "B" the activation
// side (columns = tokens), so each lane ends with 4 consecutive output columns of one
// token: 8-byte stores.  The contraction advances 64 at a time.
//
// Activation tiles (X or dY, 256 rows x 64) are staged in LDS (a three-deep ring in
// the forward, two stages in dX) with an XOR swizzle of the eight 16-byte chunks of
// each 128-byte row, chunk c of row r at slot c ^ f(r), f(r) = (r & 7) ^ ((r >> 3) & 1):
// the 16-byte fragment reads of 16 consecutive rows hit distinct banks for either 32
// or 64 LDS banks.
//
// Decode: per block constant c a lane builds the 16 possible outputs
// bf16_rne(q[j] * c) as byte planes in registers and looks codes up with byte
// permutes (no LDS table; about four VALU instructions per weight).
//
// Forward: the weight operand is decoded privately per lane straight into MFMA
// fragments (lane l of wave w: weight rows 64 w + 32 j + l % 32, contraction half
// l / 32 of each 64-step, i.e. one 16-byte code load and one block constant per row
// and step); no weight bytes touch LDS.  The contraction order inside a step is
// permuted identically on both operands (lane half h takes k in [32 h, 32 h + 32)).
// Backward: the contraction runs over weight rows, so the 64 x 256 weight tile is
// decoded cooperatively into LDS in its natural row-major layout (16-byte chunk c of
// row n at slot c ^ g(n), with g(n) = (n1, n0, n1 ^ n3, n2) in the bits of n) and read
// with the gfx950 transposing LDS read ds_read_b64_tr_b16, which hands each lane four
// consecutive weight rows of one column; the dY tiles come through LDS like the
// forward's activations, and the four waves split the output tile 2 x 2.

#include "device_common.h"
#include "gemm_tile.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int NT = 256;
constexpr int TM = 256, TN = 256, TK = 64;
#ifndef LORA_RQ
#define LORA_RQ 4
#endif
constexpr int TILE_BYTES = TM * TK * 2;  // 32 KB per staged operand tile

struct GemmParams {
  const uint16_t *A;  // fwd: X [M, K]; bwd: dY [M, N]; row length Kc
  WeightView w;
  const uint16_t *A2;  // U or V [M, r]
  const uint16_t *B2;  // fwd: Bl [N, r]; bwd: At [K, r]
  uint16_t *C;         // [M, No]
  int M, No, Kc, r;
  LevelTable lvl;  // NF4 codebook
  int lda2;       // row pitch of A2 (r, or the stacked rank of fused linears)
  int part_rows;  // fused linears: output columns [q P, q P + P) use A2 columns
                  // [q r, q r + r); 0 = one linear (tiles never straddle parts)
  int tiles;         // dX: workgroups [0, tiles) compute output tiles; the fin_wgs after
  int fin_wgs;       // them do the finalize job `fin` (the dA pass of the same backward)
  FinalizeJob fin;
};

// The dX GEMM's extension (launch_gemm_dx_ext): the dropout mask of the LoRA term, and dY
// in column blocks of `half` columns of which the last `skip` are padding (zeros in dY):
// contraction position k stands for weight row k, or k - skip from `half` on.  The padding
// positions thus read rows of the next block (past the last one: zeros) times zero.  Only
// two blocks or none (half = the whole contraction) are needed.
// With splits > 1 workgroup s tiles + t computes the contraction steps [s ksteps, (s + 1)
// ksteps) of tile t and writes its fp32 accumulators to `part` (dx_join_kernel adds them);
// the LoRA term belongs to split 0.
struct DxExt {
  Dropout drop;
  int half, skip;
  int splits, ksteps;
  float *part;
};

// ---- activation tile staging: 256 rows x 64 columns, 8 chunks of 16 B per thread ----
struct ActStage {
  u32x4_t v[8];
};

// thread t handles rows (t >> 3) + 32 i, chunk t & 7
__device__ __forceinline__ void act_load(__amdgpu_buffer_rsrc_t rs, int m0, int M, int Kc, int kt,
                                         bool vec, const uint16_t *base, ActStage &st) {
  const int tid = threadIdx.x;
  const int c = tid & 7;
  const int col = kt + c * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m0 + (tid >> 3) + 32 * i;
    if (vec) {
      const bool ok = row < M && col < Kc;
      st.v[i] = buf_load16(rs, ok ? (static_cast<uint32_t>(row) * Kc + col) * 2 : kOOB);
    } else {
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (row < M) {
        const uint16_t *src = base + static_cast<int64_t>(row) * Kc;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const uint32_t lo = (col + e < Kc) ? src[col + e] : 0u;
          const uint32_t hi = (col + e + 1 < Kc) ? src[col + e + 1] : 0u;
          v[e / 2] = lo | (hi << 16);
        }
      }
      st.v[i] = v;
    }
  }
}

__device__ __forceinline__ void act_store(char *s, const ActStage &st) {
  const int tid = threadIdx.x;
  const int c = tid & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (tid >> 3) + 32 * i;
    *reinterpret_cast<u32x4_t *>(s + tile_off(row, c)) = st.v[i];
  }
}

__device__ __forceinline__ void zero_acc(f32x16_t (&acc)[8][2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
}

// One MFMA operand fragment of a LoRA matrix: 8 consecutive ranks j0 .. j0 + 7 of row
// `row` (row pitch ld elements); rows past `rows` and ranks past r read as zero.  With
// 16-byte aligned rows it is one 16-byte load, else eight 2-byte loads; both are
// straight-line buffer loads.
__device__ __forceinline__ u32x4_t lora_frag(__amdgpu_buffer_rsrc_t rs, bool vec, int row, int rows, int ld,
                                             int j0, int r) {
  const bool ok = row < rows;
  if (vec) return buf_load16(rs, (ok && j0 < r) ? (static_cast<uint32_t>(row) * ld + j0) * 2 : kOOB);
  u32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = j0 + 2 * e;
    const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(
        rs, (ok && j < r) ? (static_cast<uint32_t>(row) * ld + j) * 2 : kOOB, 0, 0);
    const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(
        rs, (ok && j + 1 < r) ? (static_cast<uint32_t>(row) * ld + j + 1) * 2 : kOOB, 0, 0);
    v[e] = lo | (hi << 16);
  }
  return v;
}

// LoRA steps: acc[i][j] += A2 rows (tokens) x B2 rows (output columns), r in steps of 16.
// LORA_RQ rank steps at a time: every fragment load of a chunk is issued before its
// first MFMA, so the chunk pays one memory latency instead of one per 16 ranks.
__device__ __forceinline__ void lora_steps(const GemmParams &p, int m0, int c0,
                                           f32x16_t (&acc)[8][2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = p.r, lda2 = p.lda2;
  const bool vec = (r % 8) == 0 && (lda2 % 8) == 0;
  // fused linears: this tile's part picks its rank columns of A2
  const uint16_t *const A2 = p.A2 + (p.part_rows > 0 ? (c0 / p.part_rows) * r : 0);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(A2, static_cast<uint32_t>(uint64_t(p.M) * lda2 * 2));
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B2, static_cast<uint32_t>(uint64_t(p.No) * r * 2));
  constexpr int RQ = LORA_RQ;
  for (int r0 = 0; r0 < r; r0 += 16 * RQ) {
    u32x4_t wa[RQ][2], xb[RQ][8];
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
      const int j0 = r0 + 16 * q + (lane >> 5) * 8;
#pragma unroll
      for (int j = 0; j < 2; ++j) wa[q][j] = lora_frag(rb, vec, c0 + wave * 64 + j * 32 + (lane & 31), p.No, r, j0, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) xb[q][i] = lora_frag(ra, vec, m0 + i * 32 + (lane & 31), p.M, lda2, j0, r);
    }
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
      if (r0 + 16 * q < r) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(wa[q][j], xb[q][i], acc[i][j]);
      }
    }
  }
}

// Epilogue: lane holds token m = m0 + 32 i + l % 32 and output columns
// c0 + 64 w + 32 j + 8 g + 4 (l / 32) + 0..3 for g = 0..3.
__device__ __forceinline__ void store_out(const GemmParams &p, int m0, int c0,
                                          const f32x16_t (&acc)[8][2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool vec = (p.No % 4) == 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + i * 32 + (lane & 31);
    if (m >= p.M) continue;
    uint16_t *row = p.C + static_cast<int64_t>(m) * p.No;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = c0 + wave * 64 + j * 32 + g * 8 + (lane >> 5) * 4;
        const f32x16_t &a = acc[i][j];
        if (vec) {
          if (col < p.No) {
            u32x2_t o = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
            *reinterpret_cast<u32x2_t *>(row + col) = o;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.No) row[col + e] = to_bf16(a[4 * g + e]);
        }
      }
  }
}

// The same epilogue through LDS, for outputs with 16-byte aligned rows (No % 8 == 0):
// each wave stages its 256 x 64 output block in two halves of 128 tokens (rows of 136
// bytes, so that the 32 token rows of a lane half's 8-byte writes fall in distinct
// banks) and writes it back 8 rows x 128 bytes per store instruction, where the
// register layout would give 32 pieces of 16 bytes.  `lds` holds 4 x 128 x 136 bytes
// that no wave reads any more.
constexpr int kOutPitch = 136;
__device__ __forceinline__ void store_out_lds(const GemmParams &p, int m0, int c0, const f32x16_t (&acc)[8][2],
                                              char *lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  char *const reg = lds + wave * (128 * kOutPitch);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int ii = 0; ii < 4; ++ii)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16_t &a = acc[4 * h + ii][j];
          const int tok = ii * 32 + (lane & 31), col = j * 32 + g * 8 + (lane >> 5) * 4;
          const u32x2_t o = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
          *reinterpret_cast<u32x2_t *>(reg + tok * kOutPitch + col * 2) = o;
        }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's writes have landed
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int tok = 8 * q + (lane >> 3), ch = lane & 7;
      const u32x2_t lo = *reinterpret_cast<const u32x2_t *>(reg + tok * kOutPitch + ch * 16);
      const u32x2_t hi = *reinterpret_cast<const u32x2_t *>(reg + tok * kOutPitch + ch * 16 + 8);
      const int m = m0 + 128 * h + tok, col = c0 + wave * 64 + ch * 8;
      if (m < p.M && col < p.No)
        *reinterpret_cast<u32x4_t *>(p.C + static_cast<int64_t>(m) * p.No + col) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read back before the next half overwrites it
  }
}

// ---- gated projections ------------------------------------------------------------------
// Outputs of the gated forward: H [M, P], and Y [M, 2 P] = [G | L] or NULL.
struct GatedOut {
  uint16_t *H, *Y;
  int act;
};

// The rank steps of the gated forward from memory (lora_steps with one part per 32-column
// block j: acc[i][0] takes the gate's ranks, acc[i][1] the up projection's).
__device__ __forceinline__ void lora_steps_gated(const GemmParams &p, int m0, int h, f32x16_t (&acc)[8][2]) {
  const int lane = threadIdx.x & 63;
  const int r = p.r, lda2 = p.lda2, P = p.part_rows;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A2, static_cast<uint32_t>(uint64_t(p.M) * lda2 * 2));
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B2, static_cast<uint32_t>(uint64_t(p.No) * r * 2));
#pragma unroll
  for (int j = 0; j < 2; ++j)
    for (int r0 = 0; r0 < r; r0 += 16) {
      const int j0 = r0 + (lane >> 5) * 8;
      const u32x4_t wa = lora_frag(rb, true, h < P ? j * P + h : p.No, p.No, r, j0, r);
      u32x4_t xb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // columns [j r, j r + r) of U; ranks past r are zero on both sides
        const int row = m0 + i * 32 + (lane & 31);
        xb[i] = buf_load16(ra, row < p.M && j0 < r ? (static_cast<uint32_t>(row) * lda2 + j * r + j0) * 2 : kOOB);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][j] = mfma32x32x16(wa, xb[i], acc[i][j]);
    }
}

// Epilogue of the gated forward: lane holds token m0 + 32 i + l % 32 and columns
// h0 + 32 w + 8 g + 4 (l / 32) + 0..3 of G in acc[i][0] and of L in acc[i][1].  The
// workgroup's 128 columns of H (and G, L when they are kept) go through LDS, 128 tokens at
// a time (rows of 264 bytes: the 32 token rows of a lane half fall in distinct banks), and
// are written back 4 rows x 256 bytes per store instruction, or element by element when P
// is not a multiple of 8.  `lds` holds 3 x 128 x 264 bytes that no wave reads any more.
constexpr int kGatedPitch = 264;
constexpr int kGatedStage = 128 * kGatedPitch;
template <int ACT>
__device__ __forceinline__ void store_gated(const GemmParams &p, const GatedOut &o, int m0, int h0,
                                            const f32x16_t (&acc)[8][2], char *lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int P = p.part_rows;
  const bool keep = o.Y != nullptr, vec = P % 8 == 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int ii = 0; ii < 4; ++ii)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x16_t &a = acc[4 * h + ii][0], &b = acc[4 * h + ii][1];
        const int off = (ii * 32 + (lane & 31)) * kGatedPitch + (wave * 32 + g * 8 + (lane >> 5) * 4) * 2;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = act_value<ACT>(a[4 * g + e]) * b[4 * g + e];
        *reinterpret_cast<u32x2_t *>(lds + off) = u32x2_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        if (keep) {
          *reinterpret_cast<u32x2_t *>(lds + kGatedStage + off) =
              u32x2_t{pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
          *reinterpret_cast<u32x2_t *>(lds + 2 * kGatedStage + off) =
              u32x2_t{pack_bf16x2(b[4 * g], b[4 * g + 1]), pack_bf16x2(b[4 * g + 2], b[4 * g + 3])};
        }
        __builtin_amdgcn_sched_barrier(0);  // a few elements' registers at a time
      }
    __syncthreads();
    for (int t = 0; t < (keep ? 3 : 1); ++t) {
      const char *const src = lds + t * kGatedStage;
      uint16_t *const out = t == 0 ? o.H : o.Y + (t == 2 ? P : 0);
      const int64_t ld = t == 0 ? P : 2 * int64_t(P);
      if (vec) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int tok = 16 * q + (tid >> 4), ch = tid & 15;
          const u32x2_t lo = *reinterpret_cast<const u32x2_t *>(src + tok * kGatedPitch + ch * 16);
          const u32x2_t hi = *reinterpret_cast<const u32x2_t *>(src + tok * kGatedPitch + ch * 16 + 8);
          const int m = m0 + 128 * h + tok, col = h0 + ch * 8;
          if (m < p.M && col < P)
            *reinterpret_cast<u32x4_t *>(out + m * ld + col) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
        }
      } else {
        for (int q = tid; q < 128 * 128; q += NT) {
          const int tok = q >> 7, c = q & 127;
          const int m = m0 + 128 * h + tok;
          if (m < p.M && h0 + c < P)
            out[m * ld + h0 + c] = *reinterpret_cast<const uint16_t *>(src + tok * kGatedPitch + c * 2);
        }
      }
    }
    __syncthreads();  // read back before the next half overwrites it
  }
}

// ===================================== forward =====================================
// Per-lane code prefetch for one contraction step: two weight rows (j = 0, 1).
struct CodeStage {
  u32x4_t code[2];
  ConstRaw c[2];
};

template <int V>
struct Ic {
  static constexpr int v = V;
};

// X fragments (B operand) of contraction sub-step s from a staged tile: rows
// 32 i + l % 32, contraction half l / 32 -> chunk 4 (l / 32) + s.
__device__ __forceinline__ void read_xfrags_fwd(const char *sx, int s, u32x4_t (&xb)[8]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    xb[i] = *reinterpret_cast<const u32x4_t *>(sx + tile_off(i * 32 + (lane & 31), (lane >> 5) * 4 + s));
}

// Instruction-scheduling template for one forward sub-step (16 MFMAs), applied to a
// region fenced by sched_barrier: the 8 LDS fragment reads for the next sub-step go
// first, then each MFMA is followed by `NV` VALU instructions of decode work; the
// sub-step's `NG` global loads are spread evenly between the MFMAs, so that the four
// waves of a workgroup (which run in step) never queue all their loads at once.
template <int NV, int NG>
__device__ __forceinline__ void substep_schedule() {
  __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);  // DS reads
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    if constexpr (NG > 0)
      if (q % (16 / NG) == 0) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // VMEM
    __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);  // VALU
  }
}

// Global loads per wave and contraction step: per weight row (2) the codes and the
// constant's pieces (three, or one fp32 constant) of the step two ahead, then eight
// activation DMA loads, the last four after the step's barrier.  The barrier's wait
// leaves in flight the loads issued since the previous barrier and retires everything
// older, which includes the tile read right after it.  The last one or two steps of a
// launch issue no code loads (nothing would read them; left in the source, the
// compiler would delete them as dead and the count would no longer hold), so their
// barriers leave only their own DMA loads in flight.
constexpr int kDmaPerHalf = 4;  // DMA loads per wave and half tile (issue_dma)
template <int CT>
constexpr int code_loads_per_row() {
  return 1 + (CT == kConstF32 ? 1 : 3);  // issue_codes
}
template <int CT, bool CODES>
constexpr int loads_before_barrier() {
  return (CODES ? 2 * code_loads_per_row<CT>() : 0) + kDmaPerHalf;
}

// The forward is software-pipelined by contraction sub-step (16 of each 64-step):
// while the 16 MFMAs of sub-step s run, the weight fragments of sub-step s + 1 are
// decoded in registers and its activation fragments read from LDS.  Activation tiles
// rotate through three LDS buffers filled by direct buffer -> LDS loads: step i
// computes from buffer i % 3, issues the loads of tile i + 2 (into (i + 2) % 3, last
// read in step i - 1) during its second half, and reads the first fragments of tile
// i + 1 in its last sub-step, after a barrier that waits only for the loads of
// earlier steps.  Code stages and
// buffer indices are compile-time roles of a three-way unrolled loop, so no
// register copy ever waits for a load in flight.
constexpr int NBUF = 3;

// GATED: a tile is 256 tokens x 128 gate columns and the same 128 up columns; wave w owns
// 32 of each (its two 32-column blocks j = 0, 1 are weight rows of the two projections at
// the same column), so that act(G) L of an element is formed in one lane's registers and
// neither projection is read back; H, and G and L where they are kept, leave through LDS in
// whole rows.  Bound like the plain forward by the matrix units at the clock that the card's
// power leaves them: 4096 x 4096 -> 2 x 11008 with rank 64, dropout and [G | L] kept, whole
// call: 695 us, 1086 TFLOP/s (a bf16 library product of that size: 1186); 2048 x 8192 -> 2 x
// 22016: 1314 us, 1137 (1356).
template <int CT, bool GATED>
__device__ __forceinline__ void gemm_fwd_body(GemmParams p, GatedOut o) {
  __shared__ __attribute__((aligned(16))) char sX[(NBUF + (GATED ? 1 : 0)) * TILE_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tmi, tni;
  if constexpr (GATED)
    tile_coords(blockIdx.x, (p.M + TM - 1) / TM, (p.part_rows + TN / 2 - 1) / (TN / 2), tmi, tni);
  else
    tile_coords(blockIdx.x, (p.M + TM - 1) / TM, (p.No + TN - 1) / TN, tmi, tni);
  const int m0 = tmi * TM, n0 = tni * (GATED ? TN / 2 : TN);

  const int K = p.Kc;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.A, static_cast<uint32_t>(uint64_t(p.M) * K * 2));
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.w.codes, static_cast<uint32_t>(uint64_t(p.No) * K / 2));
  const ConstRsrc rq = make_const_rsrc<CT>(p.w, static_cast<uint32_t>(uint64_t(p.No) * K / 64));
  const int nk = K / TK;
  const int last = nk - 1;

  // Per-lane load offsets; the contraction position enters as the scalar offset.
  // Rows past M and weight rows past N are clamped to the last valid one: they feed
  // only outputs that are never stored, and every load stays inside its buffer.
  // DMA: each wave-wide load writes 1 KB of LDS contiguously (lane l at byte 16 l),
  // so lane l fetches the chunk that belongs at that swizzled slot: tile row
  // r = 8 q + l / 8, slot l % 8 holds chunk (l % 8) ^ f(r); wave w issues q = 8 w + i.
  uint32_t xoff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (wave * 8 + i) * 8 + (lane >> 3);
    const int row = min(m0 + r, p.M - 1);
    xoff[i] = (static_cast<uint32_t>(row) * K + ((lane & 7) ^ swz(r)) * 8) * 2;
  }
  uint32_t coff[2], boff[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = GATED ? j * p.part_rows + min(n0 + wave * 32 + (lane & 31), p.part_rows - 1)
                        : min(n0 + wave * 64 + j * 32 + (lane & 31), p.No - 1);
    coff[j] = static_cast<uint32_t>(n) * (K / 2) + (lane >> 5) * 16;
    boff[j] = static_cast<uint32_t>(n) * (K / 64);
  }
  auto issue_codes = [&](int kt, int j, CodeStage &cs) {
    cs.code[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rc, coff[j], kt / 2, 0));
    if constexpr (CT == kConstF32) {
      cs.c[j] = {0u, __builtin_amdgcn_raw_buffer_load_b32(rq.s, boff[j] * 4u, kt / 16, 0), 0u};
    } else {
      cs.c[j].c8 = __builtin_amdgcn_raw_buffer_load_b8(rq.q8, boff[j], kt / 64, 0);
      const uint32_t g4 = ((boff[j] + kt / 64) >> 8) * 4u;
      cs.c[j].s = __builtin_amdgcn_raw_buffer_load_b32(rq.s, g4, 0, 0);
      cs.c[j].o = __builtin_amdgcn_raw_buffer_load_b32(rq.o, g4, 0, 0);
    }
  };
  auto issue_dma = [&](int kt, int h, char *buf) {
    char *dst = buf + wave * 8 * 1024;
#pragma unroll
    for (int i = kDmaPerHalf * h; i < kDmaPerHalf * (h + 1); ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (__attribute__((address_space(3))) void *)(dst + i * 1024),
                                               16, xoff[i], kt * 2, 0, 0);
  };

  f32x16_t acc[8][2];
  zero_acc(acc);

  CodeStage S0, S1, S2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    issue_codes(0, h, S0);
    issue_codes(min(1, last) * TK, h, S1);
    issue_dma(0, h, sX);
    issue_dma(min(1, last) * TK, h, sX + TILE_BYTES);
  }
  // The LoRA term first, while the first tiles' loads are in flight.  Up to 64 ranks
  // with 16-byte aligned rows: the U_s tile of the 256 tokens (the rank columns of this
  // tile's part, zeros past r) is staged in the third activation buffer like one
  // contraction step of X and read with the same fragment reads, so every wave reads it
  // from LDS and loads only its own weight rows' B fragments (sub-step s: ranks
  // 8 s .. 8 s + 7 and 32 + 8 s .. in the two lane halves, as X's contraction order).
  // Otherwise the rank steps load both operands' fragments from memory.
  const bool lds_lora = p.r > 0 && p.r <= TK && (p.r % 8) == 0 && (p.lda2 % 8) == 0;
  u32x4_t wl[4][2];
  char *const sU = sX + 2 * TILE_BYTES;  // not written by the prologue's tile loads
  if (lds_lora) {
    const int qc = !GATED && p.part_rows > 0 ? (n0 / p.part_rows) * p.r : 0;
    const __amdgpu_buffer_rsrc_t ru = make_rsrc(p.A2, static_cast<uint32_t>(uint64_t(p.M) * p.lda2 * 2));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B2, static_cast<uint32_t>(uint64_t(p.No) * p.r * 2));
    char *dst = sU + wave * 8 * 1024;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = (wave * 8 + i) * 8 + (lane >> 3);
      const int row = min(m0 + rr, p.M - 1);
      const int c = (lane & 7) ^ swz(rr);
      const uint32_t off = c * 8 < p.r ? (static_cast<uint32_t>(row) * p.lda2 + qc + c * 8) * 2 : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (__attribute__((address_space(3))) void *)(dst + i * 1024), 16,
                                               off, 0, 0, 0);
      // GATED: the up projection's rank columns in a fourth buffer
      if constexpr (GATED)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ru, (__attribute__((address_space(3))) void *)(dst + TILE_BYTES + i * 1024), 16,
            c * 8 < p.r ? off + p.r * 2 : kOOB, 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = n0 + wave * 32 + (lane & 31);
        const int row = GATED ? (h < p.part_rows ? j * p.part_rows + h : p.No) : n0 + wave * 64 + j * 32 + (lane & 31);
        wl[s][j] = lora_frag(rb, true, row, p.No, p.r, 32 * (lane >> 5) + 8 * s, p.r);
      }
  } else if (p.r > 0) {
    if constexpr (GATED)
      lora_steps_gated(p, m0, n0 + wave * 32 + (lane & 31), acc);
    else
      lora_steps(p, m0, n0, acc);
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (lds_lora) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (8 * s < p.r) {
        u32x4_t xu[8];
        read_xfrags_fwd(sU, s, xu);
        if constexpr (GATED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i][0] = mfma32x32x16(wl[s][0], xu[i], acc[i][0]);
          read_xfrags_fwd(sU + TILE_BYTES, s, xu);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i][1] = mfma32x32x16(wl[s][1], xu[i], acc[i][1]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(wl[s][j], xu[i], acc[i][j]);
        }
      }
    }
    __syncthreads();  // no wave reads the U_s tile any more when step 0 loads tile 2 there
  }

  Planes pl[2], pln[2];
  u32x4_t wa[2], xb[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    pl[j] = make_planes(const_value<CT>(S0.c[j]), p.lvl);
    wa[j] = lookup8(S0.code[j][0], pl[j]);
  }
  read_xfrags_fwd(sX, 0, xb);

  auto mfmas = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(wa[j], xb[i], acc[i][j]);
  };

  // One contraction step; B is the LDS buffer of the step's tile (it % 3); CODES says
  // whether the codes of step it + 2 are loaded (every step but the last one or two).
  auto step = [&](auto B, auto CODES, int it, CodeStage &cur, CodeStage &nxt, CodeStage &nn) {
    constexpr int b = decltype(B)::v;
    constexpr bool codes = decltype(CODES)::v != 0;
    const char *sx = sX + b * TILE_BYTES;
    const char *sxn = sX + ((b + 1) % NBUF) * TILE_BYTES;
    char *sxw = sX + ((b + 2) % NBUF) * TILE_BYTES;
    const int ktn = min(it + 2, last) * TK;
    float cn0, cn1;  // block constants of the next step's two rows
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t wan[2], xbn[8];
      if (codes && s < 2) issue_codes(ktn, s, nn);  // codes first: they are needed soonest
      // the next step's planes, half a row per sub-step (row 1's last half is needed
      // by this step's last sub-step)
      if (s == 0) {
        cn0 = const_value<CT>(nxt.c[0]);
        make_planes_half(cn0, p.lvl, 0, pln[0]);
      }
      if (s == 1) make_planes_half(cn0, p.lvl, 1, pln[0]);
      if (s == 2) {
        cn1 = const_value<CT>(nxt.c[1]);
        make_planes_half(cn1, p.lvl, 0, pln[1]);
      }
      if (s == 3) make_planes_half(cn1, p.lvl, 1, pln[1]);
      if (s == 2) issue_dma(ktn, 0, sxw);
      if (s == 3) {
        // tile it + 1 (issued a step ago) must have landed for every wave, and no wave
        // may still read the buffer that the next step's loads will overwrite
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(loads_before_barrier<CT, codes>())
                     : "memory");
        issue_dma(ktn, 1, sxw);
        read_xfrags_fwd(sxn, 0, xbn);
#pragma unroll
        for (int j = 0; j < 2; ++j) wan[j] = lookup8(nxt.code[j][0], pln[j]);
      } else {
        read_xfrags_fwd(sx, s + 1, xbn);
#pragma unroll
        for (int j = 0; j < 2; ++j) wan[j] = lookup8(cur.code[j][s + 1], pl[j]);
      }
      mfmas();
#pragma unroll
      for (int j = 0; j < 2; ++j) wa[j] = wan[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) xb[i] = xbn[i];
      substep_schedule<5, 4>();
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) pl[j] = pln[j];
  };

  int it = 0;
  for (; it + 3 <= nk; it += 3) {
    step(Ic<0>{}, Ic<1>{}, it, S0, S1, S2);
    step(Ic<1>{}, Ic<1>{}, it + 1, S1, S2, S0);
    step(Ic<2>{}, Ic<1>{}, it + 2, S2, S0, S1);
  }
  // the last one or two steps: the codes of steps past the end are not loaded
  if (it < nk) step(Ic<0>{}, Ic<0>{}, it, S0, S1, S2);
  if (it + 1 < nk) step(Ic<1>{}, Ic<0>{}, it + 1, S1, S2, S0);
  // drain the clamped prefetches of the last steps before the epilogue
  __builtin_amdgcn_s_waitcnt(0);
  if constexpr (GATED) {
    static_assert(3 * kGatedStage <= (NBUF + 1) * TILE_BYTES, "output staging");
    __syncthreads();  // every wave is done reading the activation buffers
    if (o.act == kActSilu)
      store_gated<kActSilu>(p, o, m0, n0, acc, sX);
    else
      store_gated<kActGeluTanh>(p, o, m0, n0, acc, sX);
  } else if (p.No % 8 == 0) {
    static_assert(4 * 128 * kOutPitch <= NBUF * TILE_BYTES, "output staging");
    __syncthreads();  // every wave is done reading the activation buffers
    store_out_lds(p, m0, n0, acc, sX);
  } else {
    store_out(p, m0, n0, acc);
  }
}

template <int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_fwd_kernel(
    GemmParams p) {
  gemm_fwd_body<CT, false>(p, GatedOut{});
}
template <int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_gated_kernel(
    GemmParams p, GatedOut o) {
  gemm_fwd_body<CT, true>(p, o);
}

// ===================================== backward ====================================
// Weight tile for contraction rows [kt, kt + 64) and output columns [k0, k0 + 256),
// natural layout: 64 rows of 512 bytes, 16-byte chunk c of row n at slot c ^ g(n).
// Thread t decodes row kt + (t % 64), columns k0 + 64 (t / 64) .. + 64: one block
// constant, 32 bytes of codes, eight 16-byte LDS stores.  With n = (n3 n2 n1 n0) in
// binary, g(n) = (n1, n0, n1 ^ n3, n2): the 8 (16) consecutive rows of one store
// hit 8 (16) distinct 16-byte bank groups of a 128-byte (256-byte) bank cycle, and
// the 4 rows x 2 (4) chunks of a transposing read's 16 (32) lanes do too.
__device__ __forceinline__ int gswz(int n) {
  return ((n & 3) << 2) | ((((n >> 1) ^ (n >> 3)) & 1) << 1) | ((n >> 2) & 1);
}
__device__ __forceinline__ int wtile_off(int n, int col) {
  return n * 512 + ((((col >> 3) ^ gswz(n)) & 31) << 4) + (col & 7) * 2;
}

struct CodeStageB {
  u32x4_t code[2];
  ConstRaw c;
};

template <int CT>
__device__ __forceinline__ void code_load_bwd(const GemmParams &p, __amdgpu_buffer_rsrc_t rc,
                                              const ConstRsrc &rq, int k0, int kt, CodeStageB &cs) {
  const int tid = threadIdx.x;
  const int K = p.No, N = p.Kc;  // output columns are weight columns; contraction over rows
  const int n = kt + (tid & 63);
  const int k = k0 + (tid >> 6) * 64;
  const bool ok = n < N && k < K;
  const uint32_t off = static_cast<uint32_t>(n) * (K / 2) + k / 2;
  cs.code[0] = buf_load16(rc, ok ? off : kOOB);
  cs.code[1] = buf_load16(rc, ok ? off + 16 : kOOB);
  cs.c = fetch_constant<CT>(rq, static_cast<uint32_t>(n) * (K / 64) + k / 64, ok);
}

template <int CT>
__device__ __forceinline__ void code_store_bwd(const GemmParams &p, const CodeStageB &cs, char *sw) {
  const int tid = threadIdx.x;
  const int n = tid & 63, c0 = (tid >> 6) * 64;
  const Planes pl = make_planes(const_value<CT>(cs.c), p.lvl);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4_t *>(sw + wtile_off(n, c0 + h * 32 + i * 8)) = lookup8(cs.code[h][i], pl);
}


// Weight-side MFMA fragment for contraction step s (16 rows) and output-column tile
// j of this wave: two transposing reads of 4 rows each.  Within a 16-lane group, lane
// i reads row nbase + i / 4 at column cbase + 4 (i % 4) and receives column cbase + i
// of rows nbase .. nbase + 3.
__device__ __forceinline__ u32x4_t wfrag_tr(const char *sw, int s, int j) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int cbase = wave * 64 + j * 32 + (g & 1) * 16;
  const int col = cbase + 4 * (i & 3);
  u32x4_t r;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int n = 16 * s + 8 * (g >> 1) + 4 * e + (i >> 2);
    const v4i16_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16_t *)(sw + wtile_off(n, col)));
    const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
    r[2 * e] = u[0];
    r[2 * e + 1] = u[1];
  }
  return r;
}

template <bool VEC, int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_dx_kernel(
    GemmParams p) {
  __shared__ __attribute__((aligned(16))) char sX[2][TILE_BYTES];
  __shared__ __attribute__((aligned(16))) char sW[2][TILE_BYTES];
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    finalize_part(p.fin, blockIdx.x - p.tiles, p.fin_wgs);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  int tmi, tni;
  tile_coords(blockIdx.x, (p.M + TM - 1) / TM, (p.No + TN - 1) / TN, tmi, tni);
  const int m0 = tmi * TM, k0 = tni * TN;

  const int N = p.Kc, K = p.No;
  const __amdgpu_buffer_rsrc_t rdy = make_rsrc(p.A, static_cast<uint32_t>(uint64_t(p.M) * N * 2));
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.w.codes, static_cast<uint32_t>(uint64_t(N) * K / 2));
  const ConstRsrc rq = make_const_rsrc<CT>(p.w, static_cast<uint32_t>(uint64_t(N) * K / 64));
  const int nk = (N + TK - 1) / TK;
  const int last = nk - 1;

  f32x16_t acc[8][2];
  zero_acc(acc);

  ActStage st;
  CodeStageB cs;
  act_load(rdy, m0, p.M, N, 0, VEC, p.A, st);
  code_load_bwd<CT>(p, rc, rq, k0, 0, cs);
  act_store(sX[0], st);
  code_store_bwd<CT>(p, cs, sW[0]);
  __syncthreads();

  auto step = [&](int it, const char *sx, const char *sw, char *sx_next, char *sw_next) {
    const int nt = min(it + 1, last) * TK;
    act_load(rdy, m0, p.M, N, nt, VEC, p.A, st);
    code_load_bwd<CT>(p, rc, rq, k0, nt, cs);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t wa[2], xb[8];
      const int chunk = 2 * s + (lane >> 5);
#pragma unroll
      for (int j = 0; j < 2; ++j) wa[j] = wfrag_tr(sw, s, j);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        xb[i] = *reinterpret_cast<const u32x4_t *>(sx + tile_off(i * 32 + (lane & 31), chunk));
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32x32x16(wa[j], xb[i], acc[i][j]);
    }
    act_store(sx_next, st);
    code_store_bwd<CT>(p, cs, sw_next);
    __syncthreads();
  };
  int it = 0;
  for (; it + 1 < nk; it += 2) {
    step(it, sX[0], sW[0], sX[1], sW[1]);
    step(it + 1, sX[1], sW[1], sX[0], sW[0]);
  }
  if (it < nk) step(it, sX[0], sW[0], sX[1], sW[1]);
  if (p.r > 0) lora_steps(p, m0, k0, acc);
  store_out(p, m0, k0, acc);
}

// Pipelined dX for dY rows of whole 16-byte chunks (N % 8 == 0).
//
// Layout: 2 x 2 waves; wave w owns tokens m0 + 128 (w / 2) .. + 128 (four 32-token
// MFMA tiles) and output columns k0 + 128 (w % 2) .. + 128 (four 32-column tiles),
// acc[i][j], so per sub-step it reads 4 weight and 4 dY fragments for 16 MFMAs.  Each
// step's 256 x 64 dY slice is fetched one step ahead by direct buffer -> LDS loads
// into one of two stages, wave w loading rows 64 w .. + 64 (whole 128-byte row
// segments per load, in the swizzled row layout of tile_off); the MFMA fragments are
// read back with ds_read_b128 (lane l: token 32 i + l % 32, 8 contraction rows at
// 16 s + 8 (l / 32)).  The step's barrier, after each wave's own load wait,
// publishes the next stage.  The decoded weight tile (64 rows x 256 columns) is
// shared through LDS (each wave reads its 128 columns) with the transposing
// ds_read_b64_tr_b16.  During step i
// every thread decodes its 64 weights of step i + 1 (one block constant, eight
// lookups) into the other of two weight tiles, spread over the first three
// sub-steps; the single barrier per step, before the last sub-step, publishes that
// tile, whose first fragments the last sub-step then reads.  dY columns past N read
// as zero and weight rows past N decode to zero, so the contraction tail adds nothing.

// Weight-side fragment for contraction sub-step s and output-column tile j (32
// columns) of the block: two transposing reads of 4 rows each.  Within a 16-lane
// group, lane i reads row nbase + i / 4 at column cbase + 4 (i % 4) and receives
// column cbase + i of rows nbase .. nbase + 3.  The swizzle g(n) depends on the row
// only through n % 16, and j / 4 moves the chunk index by 16, past the bits that
// g(n) touches, so a lane's read addresses are eight per-lane bases trb[e][j % 4]
// (sub-step 0, j < 4) plus the constants 8192 s + 256 (j / 4).
__device__ __forceinline__ void wfrag_bases(uint32_t (&trb)[2][4]) {
  const int lane = threadIdx.x & 63;
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
      trb[e][jj] = wtile_off(8 * (g >> 1) + 4 * e + (i >> 2), jj * 32 + (g & 1) * 16 + 4 * (i & 3));
}
__device__ __forceinline__ u32x4_t wfrag_tr_all(const char *sw, const uint32_t (&trb)[2][4], int s, int j) {
  u32x4_t r;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const v4i16_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16_t *)(sw + trb[e][j & 3] + (8192 * s + 256 * (j >> 2))));
    const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
    r[2 * e] = u[0];
    r[2 * e + 1] = u[1];
  }
  return r;
}

// Epilogue of the dX layout: lane holds tokens tb + 32 i + l % 32 and output columns
// cb + 32 j + 8 g + 4 (l / 32) + 0..3 (g = 0..3) of acc[i][j].
template <int NI, int NJ>
__device__ __forceinline__ void store_out_dx(const GemmParams &p, int tb, int cb,
                                             const f32x16_t (&acc)[NI][NJ]) {
  const int lane = threadIdx.x & 63;
  const bool vec = (p.No % 4) == 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int m = tb + i * 32 + (lane & 31);
    if (m >= p.M) continue;
    uint16_t *row = p.C + static_cast<int64_t>(m) * p.No;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = cb + j * 32 + g * 8 + (lane >> 5) * 4;
        const f32x16_t &a = acc[i][j];
        if (vec) {
          if (col < p.No) {
            u32x2_t o = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
            *reinterpret_cast<u32x2_t *>(row + col) = o;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.No) row[col + e] = to_bf16(a[4 * g + e]);
        }
      }
  }
}

// The dX epilogue through LDS, for 16-byte aligned output rows (No % 8 == 0): each
// wave stages its 128 x 128 output block in its own 32 KB buffer `reg`, in two halves
// of 64 tokens (rows of 264 bytes, so that a lane half's 32 token rows fall in
// distinct banks), and writes it back 4 rows x 256 bytes per store instruction.
constexpr int kOutPitchDx = 264;
__device__ __forceinline__ void store_out_dx_lds(const GemmParams &p, int tb, int cb, const f32x16_t (&acc)[4][4],
                                                 char *reg) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int ii = 0; ii < 2; ++ii)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16_t &a = acc[2 * h + ii][j];
          const int tok = ii * 32 + (lane & 31), col = j * 32 + g * 8 + (lane >> 5) * 4;
          const u32x2_t o = {pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3])};
          *reinterpret_cast<u32x2_t *>(reg + tok * kOutPitchDx + col * 2) = o;
        }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's writes have landed
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int tok = 4 * q + (lane >> 4), ch = lane & 15;
      const u32x2_t lo = *reinterpret_cast<const u32x2_t *>(reg + tok * kOutPitchDx + ch * 16);
      const u32x2_t hi = *reinterpret_cast<const u32x2_t *>(reg + tok * kOutPitchDx + ch * 16 + 8);
      const int m = tb + 64 * h + tok, col = cb + ch * 8;
      if (m < p.M && col < p.No)
        *reinterpret_cast<u32x4_t *>(p.C + static_cast<int64_t>(m) * p.No + col) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read back before the next half overwrites it
  }
}

// LoRA steps of the dX layout: acc[i][j] += A2 rows (tokens tb + 32 i + ..) x B2 rows
// (output columns cb + 32 j + ..), rank in steps of 16.
template <int NI, int NJ>
__device__ __forceinline__ void lora_steps_dx(const GemmParams &p, int tb, int cb, f32x16_t (&acc)[NI][NJ]) {
  const int lane = threadIdx.x & 63;
  const int r = p.r;
  const bool vec = (r % 8) == 0;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A2, static_cast<uint32_t>(uint64_t(p.M) * r * 2));
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B2, static_cast<uint32_t>(uint64_t(p.No) * r * 2));
  constexpr int RQ = LORA_RQ;  // rank steps per chunk, all loads before the MFMAs
  for (int r0 = 0; r0 < r; r0 += 16 * RQ) {
    u32x4_t wa[RQ][NJ], vb[RQ][NI];
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
      const int j0 = r0 + 16 * q + (lane >> 5) * 8;
#pragma unroll
      for (int j = 0; j < NJ; ++j) wa[q][j] = lora_frag(rb, vec, cb + j * 32 + (lane & 31), p.No, r, j0, r);
#pragma unroll
      for (int i = 0; i < NI; ++i) vb[q][i] = lora_frag(ra, vec, tb + i * 32 + (lane & 31), p.M, r, j0, r);
    }
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
      if (r0 + 16 * q < r) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) acc[i][j] = mfma32x32x16(wa[q][j], vb[q][i], acc[i][j]);
      }
    }
  }
}

template <int NR, int NV, int NG, int NW>
__device__ __forceinline__ void dx_schedule() {
  __builtin_amdgcn_sched_group_barrier(0x100, NR, 0);  // DS reads
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    if constexpr (NG > 0)
      if (q % (16 / NG) == 0) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // VMEM
    if constexpr (NW > 0)
      if (q % (16 / NW) == (16 / NW) - 1) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // DS write
    __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);  // VALU
  }
}

// dY rows that one wave loads per step: 64 tokens x 64 contraction rows (8 KB); a stage
// holds the four waves' slices.
constexpr int YWAVE_BYTES = 64 * TK * 2;

// The dropout mask of X on the LoRA term of dX (acc[i][j]: tokens tb + 32 i + l % 32,
// output columns cb + 32 j + 8 g + 4 (l / 32) + 0..3).  keep_bits packs a lane's keep
// decisions, element e of acc[i][j] in bit 16 (j % 2) + e of word [i][j / 2] (keep_word in
// gemm_tile.h), so that the generator runs while the first tiles' loads are in flight;
// mask_lora applies them.
__device__ __forceinline__ void keep_bits(const DropKey &dk, int tb, int cb, int K, uint32_t (&keep)[4][2]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t row = static_cast<uint32_t>(tb + 32 * i + (lane & 31)) * static_cast<uint32_t>(K / 8);
#pragma unroll
    for (int jp = 0; jp < 2; ++jp) keep[i][jp] = keep_word(dk, row + (cb + 64 * jp) / 8);
  }
}
__device__ __forceinline__ void mask_lora(const uint32_t (&keep)[4][2], f32x16_t (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x16_t t = acc[i][j];
      asm volatile("" : "+a"(t));
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int m = static_cast<int>(keep[i][j >> 1] << (31 - (16 * (j & 1) + e))) >> 31;
        t[e] = __uint_as_float(__float_as_uint(t[e]) & static_cast<uint32_t>(m));
      }
      // back in the accumulation registers tile by tile (left to itself the compiler
      // carries all the tiles in the other half of the register file and spills)
      asm volatile("" : "+a"(t));
      acc[i][j] = t;
      __builtin_amdgcn_sched_barrier(0);
    }
}

// Partial sums of a split dX: accumulators acc[i][j] of wave w of tile t, split s, go to
// part[((s tiles + t) 4 + w) 16 + 4 i + j] as four 16-byte pieces a lane ([g][lane]), so that
// every store and the join's loads cover 1 KB contiguously.  32 x 32 blocks past M or K hold
// nothing and are skipped on both sides.
constexpr int kPartBlock = 32 * 32;  // floats of one accumulator block
__device__ __forceinline__ int64_t part_index(int tiles, int split, int tile, int wave, int i, int j) {
  return ((static_cast<int64_t>(split) * tiles + tile) * 4 + wave) * 16 + 4 * i + j;
}
__device__ __forceinline__ void store_dx_part(const GemmParams &p, float *part, int split, int tile, int tb, int cb,
                                              const f32x16_t (&acc)[4][4]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *const base = part + part_index(p.tiles, split, tile, wave, 0, 0) * kPartBlock;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (tb + 32 * i >= p.M || cb + 32 * j >= p.No) continue;
      f32x4_t *dst = reinterpret_cast<f32x4_t *>(base + (4 * i + j) * kPartBlock) + lane;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        dst[64 * g] = f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      __builtin_amdgcn_sched_barrier(0);
    }
}

// EXT: dX = dY W' + m (V A) with dY in padded column blocks (DxExt).  The LoRA term comes
// first, so the mask is applied to the accumulators once, before the base product is added
// to them; the kept elements, one bit each in the accumulators' layout, are generated while
// the first tiles' loads are in flight.  4096 x 4096 -> 4096, rank 64: 7 us over the same
// product without a mask (144.5, 137.1; 1083 TFLOP/s on 4096 x 22016 -> 4096), bound by the
// matrix units as the kernel without EXT is.
// SPLIT: one part of the contraction, see dx_split.
template <int CT, bool EXT, bool SPLIT = false>
__device__ __forceinline__ void dx_pipe_body(GemmParams p, DxExt x) {
  // two weight tiles and two dY stages, 128 KB; separate objects, so that the
  // compiler can tell reads of one stage or tile from the loads into the other stage
  __shared__ __attribute__((aligned(16))) char sW0[TILE_BYTES];
  __shared__ __attribute__((aligned(16))) char sW1[TILE_BYTES];
  __shared__ __attribute__((aligned(16))) char sY0[TILE_BYTES];
  __shared__ __attribute__((aligned(16))) char sY1[TILE_BYTES];
  // the workgroups after the tiles (dispatched last, so in CUs the tiles have left) do
  // the finalize job that rides in this launch
  const int tile_wgs = SPLIT ? p.tiles * x.splits : p.tiles;
  if (static_cast<int>(blockIdx.x) >= tile_wgs) {
    finalize_part(p.fin, blockIdx.x - tile_wgs, p.fin_wgs);
    return;
  }
  const int split = SPLIT ? static_cast<int>(blockIdx.x) / p.tiles : 0;
  const int tile = static_cast<int>(blockIdx.x) - split * p.tiles;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // 2 x 2 waves: wave w computes tokens 128 (w / 2) .. + 128 and output columns
  // 128 (w % 2) .. + 128; it loads the dY rows 64 w .. + 64 of the block
  const int wr = wave >> 1, wc = wave & 1;
  char *const sYw[2] = {sY0 + wave * YWAVE_BYTES, sY1 + wave * YWAVE_BYTES};
  int tmi, tni;
  tile_coords(tile, (p.M + TM - 1) / TM, (p.No + TN - 1) / TN, tmi, tni);
  const int m0 = tmi * TM, k0 = tni * TN;

  // contraction over weight rows (EXT: over the padded column blocks of dY that stand for
  // them), outputs are weight columns
  const int N = p.Kc, K = p.No, NW = EXT ? static_cast<int>(p.w.n_rows) : N;
  const __amdgpu_buffer_rsrc_t rdy = make_rsrc(p.A, static_cast<uint32_t>(uint64_t(p.M) * N * 2));
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(p.w.codes, static_cast<uint32_t>(uint64_t(NW) * K / 2));
  const ConstRsrc rq = make_const_rsrc<CT>(p.w, static_cast<uint32_t>(uint64_t(NW) * K / 64));
  // this workgroup's contraction steps: from kb on, nk of them
  const int kb = SPLIT ? split * x.ksteps * TK : 0;
  const int nk = SPLIT ? min((N + TK - 1) / TK - split * x.ksteps, x.ksteps) : (N + TK - 1) / TK;
  const int last = nk - 1;
  const int r = SPLIT && split > 0 ? 0 : p.r;

  // dY loads: load q of a step writes rows 8 q .. 8 q + 7 of the wave's slice (1 KB,
  // lane l at byte 16 l), so lane l fetches the chunk that belongs at slot l % 8 of
  // row r = 8 q + l / 8: chunk (l % 8) ^ swz(r), which depends on q only through its
  // parity.  Rows past M are clamped to the last one; they feed only outputs that are
  // never stored.
  const int ych[2] = {(lane & 7) ^ (lane >> 3), (lane & 7) ^ (lane >> 3) ^ 1};
  uint32_t yoff[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int row = min(m0 + wave * 64 + 8 * q + (lane >> 3), p.M - 1);
    yoff[q] = (static_cast<uint32_t>(row) * N + ych[q & 1] * 8) * 2;
  }
  // CHK: the step may reach past N (the last one); chunks at or past N read as zero
  auto issue_y = [&](auto CHK, int kt, char *dst) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      auto *d = (__attribute__((address_space(3))) void *)(dst + q * 1024);
      if constexpr (decltype(CHK)::v) {
        const uint32_t off = kt + ych[q & 1] * 8 < N ? yoff[q] + kt * 2 : kOOB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rdy, d, 16, off, 0, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rdy, d, 16, yoff[q], kt * 2, 0, 0);
      }
    }
  };
  // dY fragments of sub-step s from a stage: token 128 wr + 32 i + l % 32 is row
  // 32 (i % 2) + l % 32 of the slice loaded by wave 2 wr + i / 2; swz() sees only the
  // row's low five bits, so token tile i adds the constant 4096 i to one base per
  // sub-step
  uint32_t yrb[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) yrb[s] = wr * 2 * YWAVE_BYTES + tile_off(lane & 31, 2 * s + (lane >> 5));
  auto read_y = [&](const char *sy, int s, u32x4_t (&yb)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) yb[i] = *reinterpret_cast<const u32x4_t *>(sy + yrb[s] + 4096 * i);
  };
  // weight fragments of this wave's column tiles j = 0..3 (block tiles 4 wc + j)
  uint32_t trb[2][4];
  wfrag_bases(trb);
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int j = 0; j < 4; ++j) trb[e][j] += 256 * wc;
  // Weight decode: thread t owns tile row t % 64 and columns 64 (t / 64) .. + 64.
  const int dn = tid & 63, dc = (tid >> 6) * 64;
  const bool col_ok = k0 + dc < K;
  auto issue_codes = [&](int kt, CodeStageB &cs) {
    // EXT: padding positions of the first block take rows of the second one, times zeros
    int n = kt + dn;
    if constexpr (EXT) n -= n >= x.half ? x.skip : 0;
    const bool ok = col_ok && n < NW;
    const uint32_t off = static_cast<uint32_t>(n) * (K / 2) + (k0 + dc) / 2;
    cs.code[0] = buf_load16(rc, ok ? off : kOOB);
    cs.code[1] = buf_load16(rc, ok ? off + 16 : kOOB);
    cs.c = fetch_constant<CT>(rq, static_cast<uint32_t>(n) * (K / 64) + (k0 + dc) / 64, ok);
  };
  // global loads of one issue_codes: two code chunks and the constant's pieces
  constexpr int CODE_LOADS = 2 + (CT == kConstF32 ? 1 : 3);
  // lookups q0 .. q1 - 1 of the eight (q = 4 h + i: 16-byte code half h, word i)
  auto decode_part = [&](const CodeStageB &cs, const Planes &pd, char *sw, int q0, int q1) {
#pragma unroll
    for (int q = q0; q < q1; ++q)
      *reinterpret_cast<u32x4_t *>(sw + wtile_off(dn, dc + q * 8)) = lookup8(cs.code[q >> 2][q & 3], pd);
  };

  f32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  CodeStageB S0, S1;
  issue_codes(kb, S0);
  issue_codes(kb + min(1, last) * TK, S1);
  issue_y(Ic<1>{}, kb, sYw[0]);
  // The LoRA term first, while the first tiles' loads are in flight.  Up to 64 ranks
  // with 16-byte aligned rows: the V tile of the 256 tokens (zeros past r) is loaded
  // into the second dY stage laid out like a dY stage and read with the same fragment
  // reads (sub-step s: ranks 16 s .. 16 s + 15); each wave loads only its own output
  // columns' At fragments.  Otherwise the rank steps load both operands from memory.
  const bool lds_lora = r > 0 && r <= TK && (r % 8) == 0;
  u32x4_t wl[4][4];
  if (lds_lora) {
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(p.A2, static_cast<uint32_t>(uint64_t(p.M) * p.r * 2));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B2, static_cast<uint32_t>(uint64_t(p.No) * p.r * 2));
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = min(m0 + wave * 64 + 8 * q + (lane >> 3), p.M - 1);
      const int c = ych[q & 1];
      const uint32_t off = c * 8 < p.r ? (static_cast<uint32_t>(row) * p.r + c * 8) * 2 : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (__attribute__((address_space(3))) void *)(sYw[1] + q * 1024), 16,
                                               off, 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wl[s][j] = lora_frag(rb, true, k0 + 128 * wc + j * 32 + (lane & 31), p.No, p.r, 16 * s + (lane >> 5) * 8, p.r);
  } else if (r > 0) {
    lora_steps_dx(p, m0 + 128 * wr, k0 + 128 * wc, acc);
  }
  uint32_t keep[4][2];
  if constexpr (EXT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) keep[i][0] = keep[i][1] = ~0u;
    if (x.drop.thr != 0 && split == 0) keep_bits(drop_key(x.drop), m0 + 128 * wr, k0 + 128 * wc, K, keep);
  }
  {
    const Planes pd = make_planes(const_value<CT>(S0.c), p.lvl);
    decode_part(S0, pd, sW0, 0, 8);
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (lds_lora) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (16 * s < p.r) {
        u32x4_t vb[4];
        read_y(sY1, s, vb);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma32x32x16(wl[s][j], vb[i], acc[i][j]);
      }
    }
    __syncthreads();  // no wave reads the V tile any more when step 0 loads dY step 1 there
  }
  if constexpr (EXT) {
    mask_lora(keep, acc);
  }

  u32x4_t wa[4], yb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) wa[j] = wfrag_tr_all(sW0, trb, 0, j);
  read_y(sY0, 0, yb);

  // Step it: weight tile and dY stage b2 = it % 2 are this step's; the other stage
  // receives the dY slice of step it + 1, `dec` holds the codes of step it + 1
  // (decoded now into the other weight tile), `ld` receives those of step it + 2.
  // In the main loop (CHK = 0) the barrier leaves the code loads of step it + 2 in
  // flight.  In the last one to three steps (CHK = 1) some of those loads feed nothing,
  // and the compiler may delete them on some paths, so the count of loads in flight
  // would not hold there: those steps wait for all of their loads at the barrier.
  auto step = [&](auto B2, auto CHK, int it, CodeStageB &dec, CodeStageB &ld) {
    constexpr int b2 = decltype(B2)::v;
    constexpr bool tail = decltype(CHK)::v != 0;
    const char *sw = b2 ? sW1 : sW0;
    char *swn = b2 ? sW0 : sW1;
    const char *sy = b2 ? sY1 : sY0;
    const char *syn = b2 ? sY0 : sY1;
    const int kt1 = kb + min(it + 1, last) * TK, kt2 = kb + min(it + 2, last) * TK;
    Planes pd;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t wan[4], ybn[4];
      if (s == 0) {
        pd = make_planes(const_value<CT>(dec.c), p.lvl);
        // the other stage was last read two sub-steps ago, and every LDS read has
        // completed at the previous step's barrier
        issue_y(CHK, kt1, sYw[1 - b2]);
        decode_part(dec, pd, swn, 0, 2);
      }
      if (s == 1) {
        issue_codes(kt2, ld);
        decode_part(dec, pd, swn, 2, 5);
      }
      if (s == 2) decode_part(dec, pd, swn, 5, 8);
      if (s == 3) {
        // this wave's dY slice of step it + 1 has landed (only the code loads of
        // sub-step 1 were issued after it), and after the barrier every wave's has;
        // every thread's part of the next weight tile is written; no wave still
        // reads the tile or stage that the next step overwrites
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(tail ? 0 : CODE_LOADS) : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) wan[j] = wfrag_tr_all(swn, trb, 0, j);
        read_y(syn, 0, ybn);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) wan[j] = wfrag_tr_all(sw, trb, s + 1, j);
        read_y(sy, s + 1, ybn);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma32x32x16(wa[j], yb[i], acc[i][j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) wa[j] = wan[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) yb[i] = ybn[i];
      if (s == 0)
        dx_schedule<12, 5, 8, 2>();
      else if (s == 1)
        dx_schedule<12, 4, CODE_LOADS, 3>();
      else if (s == 2)
        dx_schedule<12, 4, 0, 3>();
      else
        dx_schedule<12, 1, 0, 0>();
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Two steps per trip (stages, code stages and weight tiles alternate) while the
  // dY prefetch stays inside N; the last steps check the contraction tail.
  int it = 0;
  for (; it + 4 <= nk; it += 2) {
    step(Ic<0>{}, Ic<0>{}, it, S1, S0);
    step(Ic<1>{}, Ic<0>{}, it + 1, S0, S1);
  }
  if (it < nk) step(Ic<0>{}, Ic<1>{}, it, S1, S0);
  if (it + 1 < nk) step(Ic<1>{}, Ic<1>{}, it + 1, S0, S1);
  if (it + 2 < nk) step(Ic<0>{}, Ic<1>{}, it + 2, S1, S0);
  __builtin_amdgcn_s_waitcnt(0);
  if constexpr (SPLIT) {
    store_dx_part(p, x.part, split, tile, m0 + 128 * wr, k0 + 128 * wc, acc);
  } else if (EXT || p.No % 8 == 0) {  // (K is a multiple of 64)
    static_assert(64 * kOutPitchDx <= TILE_BYTES, "output staging");
    __syncthreads();  // every wave is done reading the weight tiles and dY stages
    char *const reg = wave == 0 ? sW0 : wave == 1 ? sW1 : wave == 2 ? sY0 : sY1;
    store_out_dx_lds(p, m0 + 128 * wr, k0 + 128 * wc, acc, reg);
  } else {
    store_out_dx(p, m0 + 128 * wr, k0 + 128 * wc, acc);
  }
}

// The join of a split dX (bound by memory: 4 bytes read an element and split, 2 written; 1000
// x 8192 in two splits 15 us, 5.5 TB/s): a wave adds one 32 x 32 block's partial sums in split order (the
// loads of four splits in flight at a time: with few tiles and many splits the chain of
// loads is what the join waits for), rounds once and writes four columns a lane.
__global__ __launch_bounds__(NT) void dx_join_kernel(const float *__restrict__ part, int splits, int tiles, int M,
                                                     int K, uint16_t *__restrict__ dX) {
  const int lane = threadIdx.x & 63;
  const int unit = static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 6);
  const int j = unit & 3, i = (unit >> 2) & 3, w = (unit >> 4) & 3, tile = unit >> 6;
  int tmi, tni;
  tile_coords(tile, (M + TM - 1) / TM, (K + TN - 1) / TN, tmi, tni);
  const int tb = tmi * TM + 128 * (w >> 1) + 32 * i, cb = tni * TN + 128 * (w & 1) + 32 * j;
  if (tb >= M || cb >= K) return;
  const f32x4_t *src = reinterpret_cast<const f32x4_t *>(part + part_index(tiles, 0, tile, w, i, j) * kPartBlock) + lane;
  const int64_t pitch = static_cast<int64_t>(tiles) * 64 * (kPartBlock / 4);
  f32x4_t s[4];
  for (int k = 0; k < splits; k += 4) {
    f32x4_t v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int g = 0; g < 4; ++g) v[u][g] = src[min(k + u, splits - 1) * pitch + 64 * g];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k + u < splits) {
#pragma unroll
        for (int g = 0; g < 4; ++g) s[g] = k + u == 0 ? v[u][g] : s[g] + v[u][g];
      }
  }
  const int m = tb + (lane & 31);
  if (m >= M) return;
  uint16_t *row = dX + static_cast<int64_t>(m) * K + cb + (lane >> 5) * 4;  // K is a multiple of 64
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<u32x2_t *>(row + 8 * g) = u32x2_t{pack_bf16x2(s[g][0], s[g][1]), pack_bf16x2(s[g][2], s[g][3])};
}

template <int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_dx_pipe_kernel(
    GemmParams p) {
  dx_pipe_body<CT, false>(p, DxExt{});
}
template <int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_dx_ext_kernel(
    GemmParams p, DxExt x) {
  dx_pipe_body<CT, true>(p, x);
}
template <int CT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_dx_split_kernel(
    GemmParams p, DxExt x) {
  dx_pipe_body<CT, true, true>(p, x);
}

bool fits_32bit(int64_t M, int64_t N, int64_t K, int r) {
  const uint64_t lim = 0xFFFFFFF0ull;
  return uint64_t(M) * K * 2 <= lim && uint64_t(M) * N * 2 <= lim && uint64_t(N) * K / 2 <= lim &&
         uint64_t(M) * r * 2 <= lim && uint64_t(N) * r * 2 <= lim && uint64_t(K) * r * 2 <= lim;
}

GemmParams make_params(const uint16_t *A, const WeightView &w, const uint16_t *A2,
                       const uint16_t *B2, uint16_t *C, int64_t M, int64_t No, int64_t Kc, int r) {
  GemmParams p{A, w, A2, B2, C, static_cast<int>(M), static_cast<int>(No), static_cast<int>(Kc), r, {}, r, 0};
  p.lvl = level_table(w.quant_type);
  p.tiles = static_cast<int>(((M + TM - 1) / TM) * ((No + TN - 1) / TN));
  p.fin_wgs = 0;
  p.fin = FinalizeJob{nullptr, 0, 0, 0, 0, 0.0f, nullptr};
  return p;
}

unsigned grid_size(int64_t M, int64_t No) {
  return static_cast<unsigned>(((M + TM - 1) / TM) * ((No + TN - 1) / TN));
}

}  // namespace

bool gemm_supported(const WeightView &w, int64_t M, int r) {
  return M <= 0x7fffffff && fits_32bit(M, w.n_rows, w.n_cols, r);
}

hipError_t launch_gemm_fwd(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U,
                           int ldu, const uint16_t *Bl, int r, int64_t part_rows, uint16_t *Y,
                           hipStream_t stream) {
  if (!fits_32bit(M, w.n_rows, w.n_cols, ldu) || M > 0x7fffffff) return hipErrorInvalidValue;
  if (part_rows > 0 && (part_rows % TN != 0 || w.n_rows % part_rows != 0)) return hipErrorInvalidValue;
  GemmParams p = make_params(X, w, U, Bl, Y, M, w.n_rows, w.n_cols, r);
  p.lda2 = ldu;
  p.part_rows = static_cast<int>(part_rows);
  const dim3 grid(grid_size(M, w.n_rows));
  switch (w.const_type) {
    case kConstDqInt8: hipLaunchKernelGGL(gemm_fwd_kernel<kConstDqInt8>, grid, dim3(NT), 0, stream, p); break;
    case kConstDqFp8: hipLaunchKernelGGL(gemm_fwd_kernel<kConstDqFp8>, grid, dim3(NT), 0, stream, p); break;
    case kConstF32: hipLaunchKernelGGL(gemm_fwd_kernel<kConstF32>, grid, dim3(NT), 0, stream, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_gemm_dx(const WeightView &w, const uint16_t *dY, int64_t M, const uint16_t *V,
                          const uint16_t *At, int r, uint16_t *dX, hipStream_t stream, const FinalizeJob *fin) {
  if (!fits_32bit(M, w.n_rows, w.n_cols, r) || M > 0x7fffffff) return hipErrorInvalidValue;
  GemmParams p = make_params(dY, w, V, At, dX, M, w.n_cols, w.n_rows, r);
  if (fin && fin->splits > 0) {
    p.fin = *fin;
    p.fin_wgs = static_cast<int>(finalize_workgroups(*fin));
  }
  if (int64_t(p.tiles) + p.fin_wgs > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(p.tiles + p.fin_wgs));
  const bool pipe = w.n_rows % 8 == 0;
  auto go = [&](auto pipe_kern, auto plain_kern) {
    if (pipe)
      hipLaunchKernelGGL(pipe_kern, grid, dim3(NT), 0, stream, p);
    else
      hipLaunchKernelGGL(plain_kern, grid, dim3(NT), 0, stream, p);
    return hipGetLastError();
  };
  switch (w.const_type) {
    case kConstDqInt8: return go(gemm_dx_pipe_kernel<kConstDqInt8>, gemm_dx_kernel<false, kConstDqInt8>);
    case kConstDqFp8: return go(gemm_dx_pipe_kernel<kConstDqFp8>, gemm_dx_kernel<false, kConstDqFp8>);
    case kConstF32: return go(gemm_dx_pipe_kernel<kConstF32>, gemm_dx_kernel<false, kConstF32>);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm_gated(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U, int ldu,
                             const uint16_t *Bl, int r, int act, uint16_t *H, uint16_t *Y, hipStream_t stream) {
  const int64_t P = w.n_rows / 2;
  if (w.n_rows % 2 != 0 || P < 1 || (r > 0 && (r % 8 != 0 || ldu != 2 * r))) return hipErrorInvalidValue;
  if (!fits_32bit(M, w.n_rows, w.n_cols, ldu) || M > 0x7fffffff) return hipErrorInvalidValue;
  GemmParams p = make_params(X, w, U, Bl, nullptr, M, w.n_rows, w.n_cols, r);
  p.lda2 = ldu;
  p.part_rows = static_cast<int>(P);
  const int64_t tiles = ((M + TM - 1) / TM) * ((P + TN / 2 - 1) / (TN / 2));
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  const GatedOut o{H, Y, act};
  switch (w.const_type) {
    case kConstDqInt8: hipLaunchKernelGGL(gemm_gated_kernel<kConstDqInt8>, grid, dim3(NT), 0, stream, p, o); break;
    case kConstDqFp8: hipLaunchKernelGGL(gemm_gated_kernel<kConstDqFp8>, grid, dim3(NT), 0, stream, p, o); break;
    case kConstF32: hipLaunchKernelGGL(gemm_gated_kernel<kConstF32>, grid, dim3(NT), 0, stream, p, o); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

namespace {
// Splits of the extended dX GEMM's contraction: the tiles of 256 x 256 alone leave CUs idle
// when there are few tokens.  A step of the tile costs about 1.6 us and a workgroup about
// 8 us around its steps; the partial sums are written and read once (256 KB a workgroup at
// about 4.5 TB/s over the card) and joined by one more launch of about 5 us.  The number of
// splits minimises that sum (1000 x 24576 -> 8192: 128 tiles, 2 splits, 642 -> 374 us).
struct DxSplit {
  int splits, ksteps;
  double cost;
};
DxSplit dx_split(int64_t M, int64_t K, int64_t Kc) {
  const int64_t tiles = ((M + TM - 1) / TM) * ((K + TN - 1) / TN), nk = (Kc + TK - 1) / TK;
  DxSplit best{1, static_cast<int>(nk), double((tiles + 255) / 256) * (1.6 * nk + 8.0)};
  if (tiles >= 256) return best;
  const double kb = double(M) * K * 8.0 / 4.5e6;  // us per split of partial sums, written and read
  for (int64_t s = 2; s * tiles <= 512 && s * 2 <= nk; ++s) {
    const int64_t steps = (nk + s - 1) / s, used = (nk + steps - 1) / steps;
    const double rounds = double((tiles * used + 255) / 256);
    const double cost = rounds * (1.6 * steps + 8.0) + 5.0 + kb * used;
    if (cost < best.cost - 1e-9) best = {static_cast<int>(used), static_cast<int>(steps), cost};
  }
  return best;
}
// The smaller tiles of dx_mid.hip (whole backward calls, us, these tiles against those: 64 x
// 4096 -> 4096 44, 36; 512 x 2048 -> 2048 47, 38; 270 x 4416 -> 9730 89, 81; 1319 x 3392 ->
// 1608 82, 72; 400 x 4096 -> 1000 47, 35; 512 x 4096 -> 22016 140, 146; 1000 x 8192 -> 24576
// 429, 489; the sums above leave out about 6 us that these tiles take longer to start and end).
bool dx_mid_takes(int64_t M, int64_t K, int64_t Kc) { return dx_mid_cost(M, K, Kc) < dx_split(M, K, Kc).cost + 6.0; }
}  // namespace

size_t gemm_dx_ext_workspace(int64_t M, int64_t K, int64_t Kc) {
  if (dx_mid_takes(M, K, Kc)) return dx_mid_workspace(M, K, Kc);
  const DxSplit sp = dx_split(M, K, Kc);
  const int64_t tiles = ((M + TM - 1) / TM) * ((K + TN - 1) / TN);
  return sp.splits > 1 ? static_cast<size_t>(sp.splits) * tiles * TM * TN * sizeof(float) : 0;
}

hipError_t launch_gemm_dx_ext(const WeightView &w, const uint16_t *dY, int64_t M, int parts, const uint16_t *V,
                              const uint16_t *At, int r, uint16_t *dX, const Dropout &d, float *part,
                              hipStream_t stream, const FinalizeJob *fin) {
  const int64_t Np = w.n_rows / parts, half = (Np + 7) / 8 * 8, Kc = parts > 1 ? parts * half : half;
  if (w.n_rows % parts != 0 || (parts > 2 && half != Np)) return hipErrorInvalidValue;
  // the padding is dY's alone: the weight's arrays have n_rows rows (as gemm_supported counts them)
  if (!gemm_supported(w, M, r) || uint64_t(M) * Kc * 2 > 0xFFFFFFF0ull) return hipErrorInvalidValue;
  if (dx_mid_takes(M, w.n_cols, Kc))
    return launch_dx_mid(w, dY, M, Kc, half == Np ? Kc : half, half - Np, V, At, r, dX, d, part, stream, fin);
  GemmParams p = make_params(dY, w, V, At, dX, M, w.n_cols, Kc, r);
  if (fin && fin->splits > 0) {
    p.fin = *fin;
    p.fin_wgs = static_cast<int>(finalize_workgroups(*fin));
  }
  const DxSplit sp = dx_split(M, w.n_cols, Kc);
  if (int64_t(p.tiles) * sp.splits + p.fin_wgs > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(p.tiles * sp.splits + p.fin_wgs));
  // without padding the column blocks are the contraction as it is
  const DxExt x{d, static_cast<int>(half == Np ? Kc : half), static_cast<int>(half - Np), sp.splits, sp.ksteps, part};
  auto go = [&](auto whole, auto split) {
    if (sp.splits > 1)
      hipLaunchKernelGGL(split, grid, dim3(NT), 0, stream, p, x);
    else
      hipLaunchKernelGGL(whole, grid, dim3(NT), 0, stream, p, x);
  };
  switch (w.const_type) {
    case kConstDqInt8: go(gemm_dx_ext_kernel<kConstDqInt8>, gemm_dx_split_kernel<kConstDqInt8>); break;
    case kConstDqFp8: go(gemm_dx_ext_kernel<kConstDqFp8>, gemm_dx_split_kernel<kConstDqFp8>); break;
    case kConstF32: go(gemm_dx_ext_kernel<kConstF32>, gemm_dx_split_kernel<kConstF32>); break;
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.splits == 1) return e;
  hipLaunchKernelGGL(dx_join_kernel, dim3(static_cast<unsigned>(16 * p.tiles)), dim3(NT), 0, stream, part, sp.splits,
                     p.tiles, static_cast<int>(M), static_cast<int>(w.n_cols), dX);
  return hipGetLastError();
}

}  // namespace qlora
