// Products of few tokens with a group-scaled 4-bit weight (gfx950):
//
//   Y[m, n] = bf16( sum over the groups G of row n of  s_G  sum_{k in G} (q[n, k] - z_G) x[m, k] )
//
// Nothing of the weight is rounded: the inner sum runs on matrix instructions over exact
// small integers in bf16, the group's scale multiplies its fp32 sum.  A code becomes bf16 by
// a shift and an and-or, 16 + q (the bf16 of exponent 4 counts in eighths, so q is the
// mantissa's upper four bits); the sum of (16 + q) x exceeds that of (q - z) x by
// (16 + z) sum x, and sum x comes from one more matrix instruction against ones, shared by
// all rows of the tile.  That difference is of sums at most a few times larger than the
// result's terms, so it costs two bits of the fp32 sums.  It does not hold when x is infinite
// or so large that a sum overflows; a wave whose result is not finite computes its part again
// from the integers q - z themselves (never taken on ordinary data).
//
// A wave owns 16 NT rows and, of K, every W-th block of 128 columns (W waves in the
// workgroup); the waves' fp32 sums are added in wave order through LDS.  A lane (row l % 16,
// l / 16) loads 16 bytes, 32 consecutive codes; four swaps between the lane groups turn four
// such dwords into the fragments of four matrix instructions of 32 consecutive columns each.
// One instruction then never spans two groups, and X is read in whole 64-byte pieces.

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
__device__ __forceinline__ u32x4_t offset_codes(uint32_t c) {
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
  return u32x4_t{((c << 3) & kMask) | kBase, ((c >> 1) & kMask) | kBase, ((c >> 5) & kMask) | kBase,
                 ((c >> 9) & kMask) | kBase};
}
__device__ __forceinline__ u32x4_t plain_codes(uint32_t c, float z) {
  u32x4_t r;
#pragma unroll
  for (int p = 0; p < 4; ++p)
    r[p] = pack_bf16x2(static_cast<float>((c >> (4 * p)) & 15u) - z, static_cast<float>((c >> (4 * p + 16)) & 15u) - z);
  return r;
}
// Eight consecutive values of X in the codes' order.
__device__ __forceinline__ u32x4_t code_order(u32x4_t x) {
  return u32x4_t{pack_lo(x[0], x[2]), pack_hi(x[0], x[2]), pack_lo(x[1], x[3]), pack_hi(x[1], x[3])};
}

// FS: columns between two uses of a scale, the largest of 32, 64 and 128 that divides the group.
template <int MT, int NT, int FS>
struct Tile {
  static constexpr int kScales = 128 / FS;  // scales of a row in a block of 128 columns
  struct Block {
    u32x4_t codes[NT], x[MT][4];
    float s[NT][kScales], z[NT][kScales];
  };

  __amdgpu_buffer_rsrc_t codes, scales, zeros, X;
  bool s16, zp;
  uint32_t lane, row_bytes, row_groups, x_bytes, per, magic, n_steps;
  f32x4_t y[MT][NT];

  __device__ __forceinline__ uint32_t group_of(uint32_t step32) const {
    return per == 1 ? step32 : __umulhi(step32, magic);
  }

  __device__ __forceinline__ void load(Block &b, uint32_t block) const {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      b.codes[t] = buf_load16(codes, (16 * t + lane % 16) * row_bytes + block * 64 + 16 * (lane / 16));
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b.x[m][j] = buf_load16(X, (16 * m + lane % 16) * x_bytes + block * 256 + 64 * j + 16 * (lane / 16));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int g = 0; g < kScales; ++g) {
        const uint32_t i = (16 * t + lane % 16) * row_groups + group_of(4 * block + g * (FS / 32));
        b.s[t][g] = s16 ? __uint_as_float(uint32_t(__builtin_amdgcn_raw_buffer_load_b16(scales, 2 * i, 0, 0)) << 16)
                        : __uint_as_float(buf_load4(scales, 4 * i));
        b.z[t][g] = zp ? static_cast<float>(__builtin_amdgcn_raw_buffer_load_b8(zeros, i, 0, 0)) : 8.0f;
      }
  }

  template <bool EXACT>
  __device__ __forceinline__ void multiply(const Block &b, uint32_t block) {
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    u32x4_t c[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) c[t] = transpose_lane_groups(b.codes[t]);
#pragma unroll
    for (int g = 0; g < kScales; ++g) {
      f32x4_t acc[MT][NT], sum[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int jj = 0; jj < FS / 32; ++jj) {
        const int j = g * (FS / 32) + jj;
        if (4 * block + j < n_steps) {
          u32x4_t w[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t cj = c[t][j];
            w[t] = EXACT ? plain_codes(cj, b.z[t][g]) : offset_codes(cj);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4_t x = code_order(b.x[m][j]);
            if constexpr (!EXACT) sum[m] = mfma16x16x32(x, ones, sum[m]);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = mfma16x16x32(x, w[t], acc[m][t]);
          }
        }
      }
      if (4 * block + g * (FS / 32) >= n_steps) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float off = -16.0f - b.z[t][g];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = EXACT ? acc[m][t][i] : __builtin_fmaf(off, sum[m][i], acc[m][t][i]);
            y[m][t][i] = __builtin_fmaf(b.s[t][g], a, y[m][t][i]);
          }
      }
    }
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
};

template <int MT, int NT, int FS>
__global__ __launch_bounds__(512) void group_linear_kernel(GroupView w, const uint16_t *__restrict__ X, int64_t M,
                                                           uint32_t magic, uint16_t *__restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) float part[];
  constexpr int kRows = 16 * NT, kTokens = 16 * MT;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kRows, m0 = static_cast<int64_t>(blockIdx.y) * kTokens;
  const uint32_t rows = static_cast<uint32_t>(min(w.n_rows - n0, int64_t(kRows)));
  const uint32_t tokens = static_cast<uint32_t>(min(M - m0, int64_t(kTokens)));
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;

  Tile<MT, NT, FS> T;
  T.lane = threadIdx.x & 63;
  T.row_bytes = static_cast<uint32_t>(w.n_cols / 2);
  T.x_bytes = static_cast<uint32_t>(2 * w.n_cols);
  T.per = static_cast<uint32_t>(w.group / 32);
  T.magic = magic;
  T.n_steps = static_cast<uint32_t>(w.n_cols / 32);
  T.row_groups = T.n_steps / T.per;
  T.s16 = w.scale_bf16;
  T.zp = w.zeros != nullptr;
  // Reads past the tile's own rows, and past the last one of the tensor, give zeros.
  const int64_t g0 = n0 * T.row_groups;
  const uint32_t n_groups = rows * T.row_groups, s_size = T.s16 ? 2 : 4;
  T.codes = make_rsrc(w.codes + n0 * T.row_bytes, rows * T.row_bytes);
  T.scales = make_rsrc(static_cast<const char *>(w.scales) + g0 * s_size, n_groups * s_size);
  T.zeros = make_rsrc(T.zp ? w.zeros + g0 : nullptr, T.zp ? n_groups : 0u);
  T.X = make_rsrc(X + m0 * w.n_cols, tokens * T.x_bytes);

  const uint32_t blocks = (T.n_steps + 3) / 4;
  T.clear();
  typename Tile<MT, NT, FS>::Block b;
  for (uint32_t k = wave; k < blocks; k += waves) {
    T.load(b, k);
    T.template multiply<false>(b, k);
  }
  if (__any(!T.finite())) {
    T.clear();
#pragma nounroll
    for (uint32_t k = wave; k < blocks; k += waves) {
      T.load(b, k);
      T.template multiply<true>(b, k);
    }
  }

  // part[wave][m][t][i][lane]
  constexpr uint32_t kPart = MT * NT * 4 * 64;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave * kPart + ((m * NT + t) * 4 + i) * 64 + T.lane] = T.y[m][t][i];
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < kPart; e += blockDim.x) {
    const uint32_t l = e & 63, i = (e >> 6) & 3, mt = e >> 8;
    const uint32_t m = 16 * (mt / NT) + 4 * (l / 16) + i, n = 16 * (mt % NT) + l % 16;
    if (m >= tokens || n >= rows) continue;
    float v = part[e];
    for (uint32_t k = 1; k < waves; ++k) v += part[k * kPart + e];
    Y[(m0 + m) * w.n_rows + n0 + n] = to_bf16(v);
  }
}

template <int MT, int NT>
hipError_t go(const GroupView &w, const uint16_t *X, int64_t M, int waves, uint16_t *Y, hipStream_t stream) {
  const int64_t gx = (w.n_rows + 16 * NT - 1) / (16 * NT), gy = (M + 16 * MT - 1) / (16 * MT);
  if (gx > 0x7fffffff || gy > 0xffff) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(64 * waves);
  const size_t lds = static_cast<size_t>(waves) * MT * NT * 1024;
  const uint32_t magic = group_magic(static_cast<uint32_t>(w.group / 32));
  if (w.group % 128 == 0)
    hipLaunchKernelGGL((group_linear_kernel<MT, NT, 128>), grid, block, lds, stream, w, X, M, magic, Y);
  else if (w.group % 64 == 0)
    hipLaunchKernelGGL((group_linear_kernel<MT, NT, 64>), grid, block, lds, stream, w, X, M, magic, Y);
  else
    hipLaunchKernelGGL((group_linear_kernel<MT, NT, 32>), grid, block, lds, stream, w, X, M, magic, Y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_group_linear(const GroupView &w, const uint16_t *X, int64_t M, uint16_t *Y, hipStream_t stream) {
  const int64_t blocks = (w.n_cols + 127) / 128;
  const int waves = static_cast<int>(blocks < 8 ? blocks : 8);
  if (M <= 16) return go<1, 2>(w, X, M, waves, Y, stream);
  if (M <= 32) return go<2, 2>(w, X, M, waves, Y, stream);
  return go<4, 2>(w, X, M, waves, Y, stream);
}

}  // namespace qlora
