// Products of few tokens with a group-scaled 4-bit weight (gfx950):
//
//   Y[m, n] = bf16( sum over the groups G of row n of  s_G  sum_{k in G} (q[n, k] - z_G) x[m, k] )
//
// Nothing of the weight is rounded: the inner sum runs on matrix instructions over exact
// small integers in bf16, the group's scale multiplies its fp32 sum.  A code becomes bf16 by
// a shift and an and-or, 16 + q (the bf16 of exponent 4 counts in eighths, so q is the
// mantissa's upper four bits); the sum of (16 + q) x exceeds that of (q - z) x by
// (16 + z) sum x, and sum x comes from one more matrix instruction against ones, shared by
// all rows of the tile.  The terms of those sums are (16 + q) |x| and (16 + z) |x| where the
// result's are |q - z| |x|: with zeros up to 15 at most 31 times as large each (codes spread over 0 to 15
// about a zero of 8: six times on average), so the difference costs up to five bits of the fp32
// sums of terms next to the zero; zeros above 15, up to 255, cost more.  It does not hold when x is infinite
// or so large that a sum overflows; a wave whose result is not finite computes its part again
// from the integers 2^-16 (q - z) themselves, whose sums with finite x stay in range whatever x, and
// s takes the 2^16 back (never taken on ordinary data).
//
// A workgroup owns 16 NT rows.  Its waves split K: each takes every W-th round of 512 columns
// (four blocks of 128), and their fp32 sums are added in wave order through LDS.  A lane
// (row l % 16, l / 16) loads 16 bytes of a block, 32 consecutive codes; four swaps between
// the lane groups turn four such dwords into the fragments of four matrix instructions of 32
// consecutive columns each, so that one instruction never spans two groups.  A row's scales
// (and zeros) of a round are one load, lane group g holding those of block g.  X is loaded in
// whole contiguous pieces and passed through LDS of the wave's own (no barrier), in the order of
// the codes, the 16-byte chunk c of a token's block at slot c ^ token, so that the sixteen
// token lanes of a fragment read fall in distinct banks.
//
// Times here are of a product in a graph; an empty node takes 1.8 us of each.  One token x 4096 ->
// 11008 takes 7.8 us (23.2 MB, 3.9 TB/s past the node's 1.8): most of it is the start, the first
// loads' way and the sums' way out.  16 x 8192 -> 22016 takes 28.6 us (93 MB, 3.5 TB/s; one token of the
// same weight 23.6): memory, with the codes in flight that the registers have room for.  64 x 4096 ->
// 11008 takes 22.1 us in groups of 32 and 17.7 in groups of 128: the scales are applied by vector
// instructions, two for each sum of a group.

#include <type_traits>

#include "device_common.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

// dword j of lane group g  <->  dword g of lane group j
__device__ __forceinline__ u32x4_t transpose_lane_groups(u32x4_t d) {
  const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// Eight codes -> four bf16 pairs in the order (0, 4), (1, 5), (2, 6), (3, 7): 16 + q, or q - z.
// The two constants stand in registers that the compiler cannot see through (as literals they would
// take an instruction each: an and-or has no room for them).
struct CodeBits {
  uint32_t mask, base;
  __device__ __forceinline__ void init() {
    asm("s_mov_b32 %0, 0x780078" : "=s"(mask));
    asm("v_mov_b32 %0, 0x41804180" : "=v"(base));
  }
};
__device__ __forceinline__ u32x4_t offset_codes(uint32_t c, const CodeBits &k) {
  return u32x4_t{((c << 3) & k.mask) | k.base, ((c >> 1) & k.mask) | k.base, ((c >> 5) & k.mask) | k.base,
                 ((c >> 9) & k.mask) | k.base};
}
// Times 2^-16, which is exact (|q - z| < 2^8): a group's sum of up to 128 products with the largest x stays
// in range.
constexpr float kPlain = 0x1p-16f;
__device__ __forceinline__ u32x4_t plain_codes(uint32_t c, float z) {
  u32x4_t r;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    r[p] = pack_bf16x2((static_cast<float>((c >> (4 * p)) & 15u) - z) * kPlain,
                       (static_cast<float>((c >> (4 * p + 16)) & 15u) - z) * kPlain);
  return r;
}
// Eight consecutive values of X in the codes' order.
__device__ __forceinline__ u32x4_t code_order(u32x4_t x) {
  return u32x4_t{pack_lo(x[0], x[2]), pack_hi(x[0], x[2]), pack_lo(x[1], x[3]), pack_hi(x[1], x[3])};
}

// The value of lane group q (of four) made known to all lanes: by lane moves, or through the LDS
// crossbar, which leaves the vector pipe alone.  Measured (us a product in a graph, moves / crossbar):
// 1 x 11008 -> 4096 in groups of 64 8.7 / 8.2, 64 x 4096 -> 11008 in groups of 32 22.9 / 22.0, but
// 16 x 8192 -> 22016 28.6 / 30.2: there LDS serves X at the rate at which the weight arrives.
template <bool CROSSBAR>
__device__ __forceinline__ uint32_t from_lane_group(uint32_t v, int q, uint32_t lane) {
  if constexpr (CROSSBAR) {
    return __builtin_amdgcn_ds_bpermute(4 * (lane % 16) + 64 * q, v);
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // lane groups (0 1 0 1), (2 3 2 3)
    const uint32_t u = h[q >> 1];
    const auto o = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return o[q & 1];
  }
}

// Waits until at most N of the wave's loads are on their way (they complete in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// What a wave holds.  XR: tokens kept in LDS (a power of two; MT tiles of 16 of them).  FS:
// columns between two uses of a scale: 128 where that divides the group, 64 for groups of 64
// in whole blocks, else 32.  VS: a block's scales of a row are one aligned load.
template <int XR, int NT, int FS, bool S16, bool VS>
struct Product {
  static constexpr int MT = (XR + 15) / 16;
  static constexpr int kScales = 128 / FS;  // scales of a row in a block
  static constexpr int kFlush = XR >= 16 && FS == 128 ? 64 : FS;
  static constexpr int kSRegs = S16 && VS ? kScales / 2 : kScales;
  static constexpr int kZRegs = VS ? 1 : kScales;
  static constexpr int kXLoads = XR < 16 ? XR : XR / 8;  // of a round (few tokens) or half a block
  // Scales and zeros of a round, those of block g held by lane group g.
  struct Scales {
    uint32_t s[NT][kSRegs], z[NT][kZRegs];
  };
  struct Codes {
    u32x4_t c[NT];
  };
  struct Xs {
    u32x4_t x[kXLoads];
  };

  __amdgpu_buffer_rsrc_t codes, scales, zeros, X;
  CodeBits bits;
  bool zp;  // zeros are given (else 8 everywhere)
  uint32_t lane, row_bytes, row_groups, x_bytes, per, magic, n_steps;
  char *xs;  // the wave's LDS, [4][XR][256] bytes (few tokens)
  f32x4_t y[MT][NT];

  __device__ __forceinline__ void init(const GroupView &w, int64_t n0, const uint16_t *x, uint32_t tokens,
                                       uint32_t magic_) {
    lane = threadIdx.x & 63;
    row_bytes = static_cast<uint32_t>(w.n_cols / 2);
    x_bytes = static_cast<uint32_t>(2 * w.n_cols);
    per = static_cast<uint32_t>(w.group / 32);
    magic = magic_;
    n_steps = static_cast<uint32_t>(w.n_cols / 32);
    row_groups = group_of(n_steps);
    // Reads past the tile's own rows, and past the last one of the tensor, give zeros.
    const uint32_t rows = static_cast<uint32_t>(min(w.n_rows - n0, int64_t(16 * NT)));
    const uint32_t n_groups = rows * row_groups;
    constexpr uint32_t kBytes = S16 ? 2 : 4;
    const int64_t g0 = n0 * row_groups;
    bits.init();
    codes = make_rsrc(w.codes + n0 * row_bytes, rows * row_bytes);
    scales = make_rsrc(static_cast<const char *>(w.scales) + g0 * kBytes, n_groups * kBytes);
    zp = w.zeros != nullptr;
    zeros = make_rsrc(zp ? w.zeros + g0 : nullptr, zp ? n_groups : 0u);
    X = make_rsrc(x, tokens * x_bytes);
  }
  __device__ __forceinline__ uint32_t group_of(uint32_t step) const { return per == 1 ? step : __umulhi(step, magic); }

  __device__ __forceinline__ void load_scales(Scales &b, uint32_t round) const {
    const uint32_t r = lane % 16, block = 4 * round + lane / 16;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t row = (16 * t + r) * row_groups;
      if constexpr (VS) {
        const bool in = 4 * block < n_steps;
        const uint32_t i = row + block * kScales;
        if constexpr (S16 && kScales == 2) {
          b.s[t][0] = buf_load4(scales, in ? 2 * i : kOOB);
        } else if constexpr (S16 || kScales == 2) {
          const u32x2_t v = buf_load8(scales, in ? (S16 ? 2 : 4) * i : kOOB);
          b.s[t][0] = v[0], b.s[t][1] = v[1];
        } else {
          const u32x4_t v = buf_load16(scales, in ? 4 * i : kOOB);
          b.s[t][0] = v[0], b.s[t][1] = v[1], b.s[t][2] = v[2], b.s[t][3] = v[3];
        }
        b.z[t][0] = 0x08080808u;
        if (zp)
          b.z[t][0] = kScales == 2 ? __builtin_amdgcn_raw_buffer_load_b16(zeros, in ? i : kOOB, 0, 0)
                                   : buf_load4(zeros, in ? i : kOOB);
      } else {
#pragma unroll
        for (int k = 0; k < kScales; ++k) {
          const uint32_t step = 4 * block + k * (FS / 32), i = row + group_of(step);
          const bool in = step < n_steps;
          b.s[t][k] = S16 ? __builtin_amdgcn_raw_buffer_load_b16(scales, in ? 2 * i : kOOB, 0, 0)
                          : buf_load4(scales, in ? 4 * i : kOOB);
          b.z[t][k] = 8u;
          if (zp) b.z[t][k] = __builtin_amdgcn_raw_buffer_load_b8(zeros, in ? i : kOOB, 0, 0);
        }
      }
    }
  }
  // Blocks past the last read as zeros, without a memory access.
  __device__ __forceinline__ void load_codes(Codes &b, uint32_t block) const {
    const uint32_t o = (lane % 16) * row_bytes + block * 64 + 16 * (lane / 16);
#pragma unroll
    for (int t = 0; t < NT; ++t) b.c[t] = buf_load16(codes, 4 * block < n_steps ? o + 16 * t * row_bytes : kOOB);
  }
  // Few tokens: a round of X, a token a load.  More: half a block, eight tokens a load.
  __device__ __forceinline__ void load_round(Xs &b, uint32_t round) const {
    const uint32_t o = round * 1024 + 16 * lane;
#pragma unroll
    for (int m = 0; m < kXLoads; ++m) b.x[m] = buf_load16(X, o < x_bytes ? m * x_bytes + o : kOOB);
  }
  __device__ __forceinline__ void load_half(char *to, uint32_t half) const {
    const uint32_t o = half * 128 + 16 * ((lane % 8) ^ (lane / 8));
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(X, (__attribute__((address_space(3))) void *)(to + 1024 * i), 16,
                                               o < x_bytes ? (8 * i + lane / 8) * x_bytes + o : kOOB, 0, 0, 0);
  }
  __device__ __forceinline__ void stage_round(const Xs &b) const {
#pragma unroll
    for (int m = 0; m < kXLoads; ++m)
      *reinterpret_cast<u32x4_t *>(xs + ((lane / 16) * XR + m) * 256 + 16 * ((lane % 16) ^ m)) = code_order(b.x[m]);
  }
  // Fragments of a round's block q (few tokens) and of the half block in LDS.
  __device__ __forceinline__ u32x4_t frag_round(int q, int j) const {
    const uint32_t m = (lane % 16) % XR;
    return *reinterpret_cast<const u32x4_t *>(xs + (q * XR + m) * 256 + 16 * ((4 * j + lane / 16) ^ m));
  }
  __device__ __forceinline__ u32x4_t frag_half(const char *from, int m, int j) const {
    const uint32_t r = lane % 16;
    return *reinterpret_cast<const u32x4_t *>(from + (16 * m + r) * 128 + 16 * ((4 * (j & 1) + lane / 16) ^ (r % 8)));
  }

  // Scales and zeros of a block as every lane knows them.
  struct Known {
    uint32_t s[NT][kSRegs], z[NT][kZRegs];
    __device__ __forceinline__ float scale(int t, int k) const {
      if constexpr (S16 && VS) return (k & 1) ? bf16_hi(s[t][k / 2]) : bf16_lo(s[t][k / 2]);
      return __uint_as_float(S16 ? s[t][k] << 16 : s[t][k]);
    }
    __device__ __forceinline__ float zero(int t, int k) const {
      return static_cast<float>(VS ? (z[t][0] >> (8 * k)) & 255u : z[t][VS ? 0 : k]);
    }
  };
  __device__ __forceinline__ Known known(const Scales &b, int q) const {
    Known v;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < kSRegs; ++k) v.s[t][k] = from_lane_group<XR != 16>(b.s[t][k], q, lane);
#pragma unroll
      for (int k = 0; k < kZRegs; ++k) v.z[t][k] = zp ? from_lane_group<XR != 16>(b.z[t][k], q, lane) : b.z[t][k];
    }
    return v;
  }

  struct Sums {
    f32x4_t acc[MT][NT], sum[MT];
  };
  // Steps j0 .. j1 - 1 (of 32 columns) of a block: X's fragment of step j and token tile m is
  // frag(m, j).  A group that ends inside goes to y; what is left stays in `a`.
  template <bool EXACT, int J0, int J1, typename FRAG>
  __device__ __forceinline__ void multiply(Sums &a, const Codes &c, const Known &v, uint32_t block, FRAG frag) {
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    u32x4_t x[J1 - J0][MT];
#pragma unroll
    for (int j = J0; j < J1; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) x[j - J0][m] = frag(m, j);
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      if (4 * block + j >= n_steps) break;
      const int k = j / (FS / 32);
      if (j % (kFlush / 32) == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          a.sum[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int t = 0; t < NT; ++t) a.acc[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
      u32x4_t w[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t cj = c.c[t][j];
        w[t] = EXACT ? plain_codes(cj, v.zero(t, k)) : offset_codes(cj, bits);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4_t f = XR < 16 ? x[j - J0][m] : code_order(x[j - J0][m]);  // (few: stored in this order)
        if constexpr (!EXACT) a.sum[m] = mfma16x16x32(f, ones, a.sum[m]);
#pragma unroll
        for (int t = 0; t < NT; ++t) a.acc[m][t] = mfma16x16x32(f, w[t], a.acc[m][t]);
      }
      if ((j + 1) % (kFlush / 32) == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float off = -16.0f - v.zero(t, k);
          float s = v.scale(t, k), back = 1.0f;
          // plain_codes' 2^16 goes to the scale, or to the sum of a scale that it would take out of range
          if constexpr (EXACT) (fabsf(s) < 0x1p100f ? s : back) *= 1.0f / kPlain;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = EXACT ? a.acc[m][t][i] * back : __builtin_fmaf(off, a.sum[m][i], a.acc[m][t][i]);
              y[m][t][i] = __builtin_fmaf(s, u, y[m][t][i]);
            }
        }
      }
    }
  }
  __device__ __forceinline__ static void transpose(Codes &c) {
#pragma unroll
    for (int t = 0; t < NT; ++t) c.c[t] = transpose_lane_groups(c.c[t]);
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) y[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ bool finite() const {
    float v = 0.0f;  // becomes NaN with the first value that is not finite
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) v = __builtin_fmaf(0.0f, y[m][t][i], v);
    return v == 0.0f;
  }

  // The waves' sums added in wave order through LDS, [wave][m tile][t][token][row] (the waves
  // from `half` on in `part1`), and stored.
  __device__ __forceinline__ void finish(float *part0, float *part1, uint32_t half, uint32_t wave, uint32_t waves,
                                         uint32_t tokens, uint32_t rows, uint16_t *Y, int64_t ldy) const {
    constexpr uint32_t kTok = XR < 16 ? XR : 16, kPart = MT * NT * kTok * 16;
    auto part = [&](uint32_t k) { return k < half ? part0 + k * kPart : part1 + (k - half) * kPart; };
    float *mine = part(wave);
    __syncthreads();  // the waves' X pieces are read
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t tok = 4 * (lane / 16) + i;
          if (tok < kTok) mine[((m * NT + t) * kTok + tok) * 16 + lane % 16] = y[m][t][i];
        }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < kPart; e += blockDim.x) {
      const uint32_t mt = e / (16 * kTok), m = 16 * (mt / NT) + (e / 16) % kTok, n = 16 * (mt % NT) + e % 16;
      if (m >= tokens || n >= rows) continue;
      float v = part0[e];
      for (uint32_t k = 1; k < waves; ++k) v += part(k)[e];
      Y[m * ldy + n] = to_bf16(v);
    }
  }
};

// Up to 8 tokens: a round of everything in flight at once.  W: the most waves of a workgroup.
template <int XR, int NT, int W, int FS, bool S16, bool VS>
__global__ __launch_bounds__(64 * W) void group_few_kernel(GroupView w, const uint16_t *__restrict__ X, uint32_t M,
                                                           uint32_t magic, uint16_t *__restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  using P = Product<XR, NT, FS, S16, VS>;
  P T;
  T.init(w, n0, X, M, magic);
  T.xs = lds + wave * (XR * 1024);
  T.clear();
  auto rounds = [&](auto exact) {
#pragma nounroll
    for (uint32_t k = wave; 16 * k < T.n_steps; k += waves) {
      typename P::Xs x;
      typename P::Scales s;
      typename P::Codes c[4];
      typename P::Sums a;
      T.load_round(x, k);
      T.load_scales(s, k);
#pragma unroll
      for (int q = 0; q < 4; ++q) T.load_codes(c[q], 4 * k + q);
      __builtin_amdgcn_sched_barrier(0);
      T.stage_round(x);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * (4 * k + q) >= T.n_steps) break;
        T.transpose(c[q]);
        T.template multiply<decltype(exact)::value, 0, 4>(a, c[q], T.known(s, q), 4 * k + q,
                                                          [&](int, int j) { return T.frag_round(q, j); });
      }
    }
  };
  rounds(std::false_type());
  if (__any(!T.finite())) {
    T.clear();
    rounds(std::true_type());
  }
  float *part = reinterpret_cast<float *>(lds);
  T.finish(part, part, 64, wave, waves, M, static_cast<uint32_t>(min(w.n_rows - n0, int64_t(16 * NT))), Y + n0,
           w.n_rows);
}

// More tokens, XR of them a workgroup.  X goes straight from memory to LDS, half a block to each of
// two stages of the wave's own, and a stage is asked for again as soon as it is multiplied; the
// next block of codes is in flight while one is multiplied.  The stages are separate objects, so that
// the waits the compiler puts before one's reads leave the other's loads in flight.  (Four
// stages: 32 us instead of 28.5 at 16 x 8192 -> 22016, fewer workgroups fit.)
template <int XR, int NT, int W, int FS, bool S16, bool VS>
__global__ __launch_bounds__(64 * W) void group_many_kernel(GroupView w, const uint16_t *__restrict__ X, int64_t M,
                                                            uint32_t magic, uint16_t *__restrict__ Y) {
  using P = Product<XR, NT, FS, S16, VS>;
  static_assert(P::MT * NT * 1024 * ((W + 1) / 2) <= W * XR * 128, "partial sums of half the waves fit a stage");
  __shared__ __attribute__((aligned(16))) char x0[W * XR * 128];
  __shared__ __attribute__((aligned(16))) char x1[W * XR * 128];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT), m0 = static_cast<int64_t>(blockIdx.y) * XR;
  const uint32_t tokens = static_cast<uint32_t>(min(M - m0, int64_t(XR)));
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  P T;
  T.init(w, n0, X + m0 * w.n_cols, tokens, magic);
  T.clear();
  auto rounds = [&](auto exact) {
    typename P::Scales s, s2;
    typename P::Codes c, c2;
    typename P::Sums a;
    char *const stage[2] = {x0 + wave * (XR * 128), x1 + wave * (XR * 128)};
    T.load_scales(s, wave);
    T.load_codes(c, 4 * wave);
    T.load_half(stage[0], 8 * wave);
    T.load_half(stage[1], 8 * wave + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma nounroll
    for (uint32_t k = wave; 16 * k < T.n_steps; k += waves) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t block = 4 * k + q, next = q < 3 ? block + 1 : 4 * (k + waves);
        T.load_codes(c2, next);
        if (q == 3) T.load_scales(s2, k + waves);
        __builtin_amdgcn_sched_barrier(0);
        const typename P::Known v = T.known(s, q);
        T.transpose(c);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          auto frag = [&](int m, int j) { return T.frag_half(stage[h], m, j); };
          // The stage's loads have landed when only what was asked for after them is on its way: the
          // other stage's and the next block's codes.  (The waits that the compiler derives are not
          // enough: it takes a direct load for a store of one lane's 16 bytes.)
          wait_loads<P::kXLoads + NT>();
          if (h == 0)
            T.template multiply<decltype(exact)::value, 0, 2>(a, c, v, block, frag);
          else
            T.template multiply<decltype(exact)::value, 2, 4>(a, c, v, block, frag);
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage is read
          T.load_half(stage[h], 2 * next + h);
          __builtin_amdgcn_sched_barrier(0);
        }
        c = c2;
      }
      s = s2;
    }
  };
  rounds(std::false_type());
  if (__any(!T.finite())) {
    T.clear();
    rounds(std::true_type());
  }
  // the loads asked for past the last round write zeros to the stages, which become the sums' place
  wait_loads<0>();
  T.finish(reinterpret_cast<float *>(x0), reinterpret_cast<float *>(x1), W / 2, wave, waves, tokens,
           static_cast<uint32_t>(min(w.n_rows - n0, int64_t(16 * NT))), Y + m0 * w.n_rows + n0, w.n_rows);
}

// FEW: group_few_kernel, else group_many_kernel.
template <bool FEW, int XR, int NT, int W>
hipError_t go(const GroupView &w, const uint16_t *X, int64_t M, uint16_t *Y, hipStream_t stream) {
  const int64_t gx = (w.n_rows + 16 * NT - 1) / (16 * NT), gy = (M + XR - 1) / XR;
  // as many waves as share the rounds evenly
  const int64_t rounds = (w.n_cols + 511) / 512, each = (rounds + W - 1) / W;
  const int waves = static_cast<int>((rounds + each - 1) / each);
  if (gx * 64 * waves > kMaxThreads || gy > 0xffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(64 * waves);
  static_assert(!FEW || W * XR <= 64, "64 KB of dynamic LDS");
  const size_t lds = FEW ? static_cast<size_t>(waves) * XR * 1024 : 0;  // (holds the partial sums too)
  const uint32_t magic = group_magic(static_cast<uint32_t>(w.group / 32));
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, w, X, M, magic, Y);
    return hipGetLastError();
  };
  // Groups of whole blocks take one scale a block; groups of 64 and 32 theirs by one aligned load;
  // any other group (and unaligned arrays) a load for each 32 columns.
  const int64_t per_block = 128 / w.group;
  const bool aligned = (w.group == 64 || w.group == 32) && w.n_cols % 128 == 0 &&
                       reinterpret_cast<uintptr_t>(w.scales) % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(w.zeros) % per_block == 0;
  const int kind = w.group % 128 == 0 ? 0 : !aligned ? 3 : w.group == 64 ? 1 : 2;
  switch (2 * kind + (w.scale_bf16 ? 1 : 0)) {
#define QLORA_ONE(n, fs, s16, vs)                                           \
  case n:                                                                   \
    if constexpr (FEW)                                                      \
      return launch(group_few_kernel<XR, NT, W, fs, s16, vs>);              \
    else                                                                    \
      return launch(group_many_kernel<XR, NT, W, fs, s16, vs>);
    QLORA_ONE(0, 128, false, false)
    QLORA_ONE(1, 128, true, false)
    QLORA_ONE(2, 64, false, true)
    QLORA_ONE(3, 64, true, true)
    QLORA_ONE(4, 32, false, true)
    QLORA_ONE(5, 32, true, true)
    QLORA_ONE(6, 32, false, false)
    QLORA_ONE(7, 32, true, false)
#undef QLORA_ONE
    default: return hipErrorInvalidValue;
  }
}

// Tiles of XR tokens and 16 NT rows for more than 8 tokens.  Below 256 workgroups, one to a CU, a
// launch takes what its tile takes (in us at K = 8192, beside 3.5 of the launch itself: small
// tiles are sooner done, each reads X for itself), above it as many times that as it has rounds
// of 256.  58 tokens x 8064 -> 560: 8.4 us with the smallest tile, 26.1 with the largest; 64 x
// 8192 -> 8192: 55.8 and 28.1, 23.6 with 64 x 32; 64 x 4096 -> 11008: 34.0 and 17.7, 26.4 with 64 x 32.
struct TileCost {
  int tokens, rows16;
  double us;
};
constexpr TileCost kTiles[] = {{16, 1, 4.9}, {16, 2, 7.5}, {16, 3, 10.8}, {32, 2, 10.6},
                               {32, 3, 14.9}, {64, 2, 17.2}, {64, 3, 22.9}};
int best_tile(int64_t M, int64_t rows) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 7; ++i) {
    const TileCost &t = kTiles[i];
    const int64_t wgs = (rows + 16 * t.rows16 - 1) / (16 * t.rows16) * ((M + t.tokens - 1) / t.tokens);
    const double us = t.us * static_cast<double>((wgs + 255) / 256);
    if (i == 0 || us < least) best = i, least = us;
  }
  return best;
}

template <int XR>
hipError_t few(const GroupView &w, const uint16_t *X, int64_t M, uint16_t *Y, hipStream_t stream) {
  if (w.n_rows >= 16 * 1024) return go<true, XR, 2, 8>(w, X, M, Y, stream);
  return go<true, XR, 1, XR < 8 ? 16 : 8>(w, X, M, Y, stream);
}

}  // namespace

// Up to 8 tokens a wave has the whole of its round in flight, with 16 rows a workgroup, or 32 where
// they are so many that the card's CUs have several workgroups each all the same: 1, 4 and 8 tokens
// x 8192 -> 22016 23.6, 25.0, 28.1 us with 32 rows, 26.4, 35.9, 32.5 with 16; 1 x 4096 -> 11008 8.8 and 7.8,
// 8 x 11008 -> 4096 13.2 and 10.2.
hipError_t launch_group_linear(const GroupView &w, const uint16_t *X, int64_t M, uint16_t *Y, hipStream_t stream) {
  if (M == 1) return few<1>(w, X, M, Y, stream);
  if (M <= 4) return few<4>(w, X, M, Y, stream);
  if (M <= 8) return few<8>(w, X, M, Y, stream);
  switch (best_tile(M, w.n_rows)) {
    case 0: return go<false, 16, 1, 16>(w, X, M, Y, stream);
    case 1: return go<false, 16, 2, 8>(w, X, M, Y, stream);
    case 2: return go<false, 16, 3, 8>(w, X, M, Y, stream);
    case 3: return go<false, 32, 2, 8>(w, X, M, Y, stream);
    case 4: return go<false, 32, 3, 8>(w, X, M, Y, stream);
    case 5: return go<false, 64, 2, 8>(w, X, M, Y, stream);
    default: return go<false, 64, 3, 8>(w, X, M, Y, stream);
  }
}

}  // namespace qlora
