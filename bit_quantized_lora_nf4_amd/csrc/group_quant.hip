// 4-bit weights with one scale (and zero) for each group of consecutive elements of a row
// (gfx950): quantization and its inverse.
//
//   without zeros  s = ST(RN(max |w| RN(1 / 7))),  z = 8
//   with zeros     lo = min(w, 0), hi = max(w, 0), s = ST(RN(RN(hi - lo) RN(1 / 15))),
//                  z = clamp(rint(RN(-lo RN(1 / s))), 0, 15)
//   code = clamp(rint(RN(w RN(1 / s))) + z, 0, 15),   w' = RN((code - z) s)
//
// RN rounds to fp32, ST to the scales' type (bf16 or fp32); s below 2^-126 counts as 0 and
// 1 / s as 0 then, so that a group of zeros (or of subnormal numbers) stands for zeros; s that is not
// finite (an infinity or a NaN in the group) becomes NaN, and 1 / s counts as 0.  The
// reciprocal is taken once a group, the weights are multiplied by it.  Both kernels are bound
// by memory: 2 or 4 bytes a weight on one side, 0.5 and the scales on the other.

#include "device_common.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

constexpr int kEach = 2, kUnroll = 4;  // chunks of a thread of the quantizer, and of the inverse
constexpr int64_t kMemorySideCache = int64_t(256) << 20;

// 1.5 x 2^23: added to a number below 2^22 it leaves the number rounded to an integer, ties to even,
// in the sum's last bits.
constexpr float kRound = 12582912.0f;

struct GroupStep {
  float s, inv, z;
  float least, most;  // kRound - z, kRound + 15 - z: where a rounded weight may be
};
// Scale, its reciprocal and the zero of a group from its extremes (lo <= 0 <= hi with zeros,
// else hi = max |w|).
template <bool S16, bool ZP>
__device__ __forceinline__ GroupStep group_step(float lo, float hi) {
  constexpr float kPer7 = 1.0f / 7.0f, kPer15 = 1.0f / 15.0f;
  float s = ZP ? (hi - lo) * kPer15 : hi * kPer7;
  if constexpr (S16) s = bf16_to_f32(to_bf16(s));
  const bool any = s >= 0x1p-126f && s < __builtin_inff();
  const float inv = any ? 1.0f / s : 0.0f;
  s = any ? s : s < 0x1p-126f ? 0.0f : __builtin_nanf("");
  float z = 8.0f;
  if constexpr (ZP) z = any ? __builtin_amdgcn_fmed3f(__builtin_rintf(-lo * inv), 0.0f, 15.0f) : 0.0f;
  return {s, inv, z, kRound - z, kRound + (15.0f - z)};
}
template <bool S16, bool ZP>
__device__ __forceinline__ void store_step(const GroupStep &g, int64_t i, void *scales, uint8_t *zeros) {
  if constexpr (S16)
    static_cast<uint16_t *>(scales)[i] = to_bf16(g.s);
  else
    static_cast<float *>(scales)[i] = g.s;
  if constexpr (ZP) zeros[i] = static_cast<uint8_t>(g.z);
}

// V consecutive weights as fp32: eight of bf16 or four of fp32, 16 bytes.
template <bool W16>
struct Chunk {
  static constexpr int V = W16 ? 8 : 4;
  float v[V];
};
template <bool W16, bool STREAM>
__device__ __forceinline__ Chunk<W16> load_chunk(const void *W, int64_t c) {
  Chunk<W16> x;
  const u32x4_t *p = reinterpret_cast<const u32x4_t *>(W) + c;
  const u32x4_t u = STREAM ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = u[i];
    if constexpr (W16) {
      x.v[2 * i] = bf16_lo(b);
      x.v[2 * i + 1] = bf16_hi(b);
    } else {
      x.v[i] = __uint_as_float(b);
    }
  }
  return x;
}
// NaN if either is.
__device__ __forceinline__ float lesser(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float greater(float a, float b) { return __builtin_elementwise_maximum(a, b); }
// The extreme over `lanes` neighbouring lanes (a power of two), known to all of them; by moves
// within rows of 16 lanes, then between rows.
template <int MOVE>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), MOVE, 0xF, 0xF, true));
}
template <typename F>
__device__ __forceinline__ float lanes_extreme(float v, int lanes, F of) {
  if (lanes > 1) v = of(v, moved<0xB1>(v));   // lanes 1 0 3 2
  if (lanes > 2) v = of(v, moved<0x4E>(v));   // lanes 2 3 0 1
  if (lanes > 4) v = of(v, moved<0x141>(v));  // mirrored within 8
  if (lanes > 8) v = of(v, moved<0x140>(v));  // mirrored within 16
  if (lanes > 16) v = of(v, __shfl_xor(v, 16, 64));
  if (lanes > 32) v = of(v, __shfl_xor(v, 32, 64));
  return v;
}
template <bool ZP>
__device__ __forceinline__ void lanes_extremes(float &lo, float &hi, int lanes) {
  hi = lanes_extreme(hi, lanes, greater);
  if constexpr (ZP) lo = lanes_extreme(lo, lanes, lesser);
}
template <bool W16, bool ZP>
__device__ __forceinline__ void extremes(const Chunk<W16> &x, float &lo, float &hi) {
#pragma unroll
  for (int i = 0; i < Chunk<W16>::V; ++i) {
    if constexpr (ZP) lo = lesser(lo, x.v[i]);
    hi = greater(hi, ZP ? x.v[i] : fabsf(x.v[i]));
  }
}
template <bool W16>
__device__ __forceinline__ void store_codes(const Chunk<W16> &x, const GroupStep &g, int64_t c, void *codes) {
  // Each code is the rounded weight's last bits less those of kRound - z, which come off all of them at
  // once (modulo 2^32).
  uint32_t p = 0;
#pragma unroll
  for (int i = Chunk<W16>::V - 1; i >= 0; --i)
    p = (p << 4) + __float_as_uint(__builtin_amdgcn_fmed3f(x.v[i] * g.inv + kRound, g.least, g.most));
  p -= __float_as_uint(g.least) * (W16 ? 0x11111111u : 0x1111u);
  if constexpr (W16)
    static_cast<uint32_t *>(codes)[c] = p;
  else
    static_cast<uint16_t *>(codes)[c] = static_cast<uint16_t>(p);
}

// Groups of a power of two of chunks, at most a wave's 64: `lanes` neighbouring lanes hold a
// group, a thread takes two chunks, both loaded before the first is used (11008 x 4096 bf16 with zeros:
// 21.7 us, 23.9 with four; 22016 x 8192 fp32, streamed: 128.5 and 128.3).  Whole groups fall out together
// at the end, so no lane misses a partner.  Vector instructions are what bounds it beside memory: about
// six a weight with the minima, maxima and codes, 23.8 us for the first of these weights with ten.
// STREAM: W is larger than the memory-side cache and is read past it (22016 x 8192 fp32, 721 MB: 128
// us, 146 through the caches; 90 MB of bf16 are read faster through them, 21.7 us and 26.4).
template <bool W16, bool S16, bool ZP, bool STREAM>
__global__ __launch_bounds__(kThreads) void group_quantize_kernel(const void *__restrict__ W, int64_t chunks,
                                                                  int lanes, int shift, void *__restrict__ codes,
                                                                  void *__restrict__ scales,
                                                                  uint8_t *__restrict__ zeros) {
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kEach) * kThreads + threadIdx.x;
  Chunk<W16> x[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int64_t c = first + u * kThreads;
    if (c < chunks) x[u] = load_chunk<W16, STREAM>(W, c);
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int64_t c = first + u * kThreads;
    if (c >= chunks) return;
    float lo = 0.0f, hi = 0.0f;
    extremes<W16, ZP>(x[u], lo, hi);
    lanes_extremes<ZP>(lo, hi, lanes);
    const GroupStep g = group_step<S16, ZP>(lo, hi);
    store_codes<W16>(x[u], g, c, codes);
    if ((threadIdx.x & (lanes - 1)) == 0) store_step<S16, ZP>(g, c >> shift, scales, zeros);
  }
}

// Any other group size: a wave to a group, which it reads twice (the second time from the
// caches).
template <bool W16, bool S16, bool ZP>
__global__ __launch_bounds__(kThreads) void group_quantize_any_kernel(const void *__restrict__ W, int64_t groups,
                                                                      int64_t per_group, void *__restrict__ codes,
                                                                      void *__restrict__ scales,
                                                                      uint8_t *__restrict__ zeros) {
  const int lane = threadIdx.x & 63;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 64);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); i < groups; i += step) {
    const int64_t base = i * per_group;
    float lo = 0.0f, hi = 0.0f;
    for (int64_t c = lane; c < per_group; c += 64) extremes<W16, ZP>(load_chunk<W16, false>(W, base + c), lo, hi);
    lanes_extremes<ZP>(lo, hi, 64);
    const GroupStep g = group_step<S16, ZP>(lo, hi);
    for (int64_t c = lane; c < per_group; c += 64) store_codes<W16>(load_chunk<W16, false>(W, base + c), g, base + c, codes);
    if (lane == 0) store_step<S16, ZP>(g, i, scales, zeros);
  }
}

// A wave takes spans of kUnroll x 64 chunks of one row (V codes and 16 bytes of output a
// lane), so the group of a chunk is a 32-bit division by the group's chunks (four at least), done
// by a multiplication (exact for the row lengths that the caller allows).  The output is stored past the
// caches, which hold the codes (11008 x 4096 bf16: 16.1 us, 19.9 through them; 22016 x 8192 fp32: 120
// us, 6.7 TB/s, and 179).
template <bool O16>
__global__ __launch_bounds__(kThreads) void group_dequantize_kernel(GroupView w, uint32_t row_chunks, uint32_t spans,
                                                                    uint32_t row_groups, uint32_t magic,
                                                                    void *__restrict__ out) {
  constexpr int V = O16 ? 8 : 4;
  const uint32_t lane = threadIdx.x & 63;
  const int64_t total = w.n_rows * spans, step = static_cast<int64_t>(gridDim.x) * (kThreads / 64);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); i < total; i += step) {
    const int64_t row = i / spans;
    const uint32_t c0 = static_cast<uint32_t>(i - row * spans) * (kUnroll * 64) + lane;
    const int64_t chunk0 = row * row_chunks, group0 = row * row_groups;
    uint32_t code[kUnroll];
    float s[kUnroll], z[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t c = c0 + 64 * u;
      if (c >= row_chunks) continue;
      if constexpr (O16)
        code[u] = reinterpret_cast<const uint32_t *>(w.codes)[chunk0 + c];
      else
        code[u] = reinterpret_cast<const uint16_t *>(w.codes)[chunk0 + c];
      const int64_t g = group0 + __umulhi(c, magic);
      s[u] = w.scale_bf16 ? bf16_to_f32(static_cast<const uint16_t *>(w.scales)[g])
                          : static_cast<const float *>(w.scales)[g];
      z[u] = w.zeros ? static_cast<float>(w.zeros[g]) : 8.0f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t c = c0 + 64 * u;
      if (c >= row_chunks) continue;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = (static_cast<float>((code[u] >> (4 * e)) & 15u) - z[u]) * s[u];
      u32x4_t o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (O16)
          o[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        else
          o[e] = __float_as_uint(v[e]);
      }
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t *>(out) + chunk0 + c);
    }
  }
}

template <bool W16, bool S16, bool ZP>
hipError_t quantize_go(const void *W, int64_t n, int64_t group, void *codes, void *scales, uint8_t *zeros,
                       hipStream_t stream) {
  constexpr int V = Chunk<W16>::V;
  const int64_t chunks = n / V, per_group = group / V;
  if (per_group <= 64 && (per_group & (per_group - 1)) == 0) {
    const int64_t blocks = (chunks + kThreads * kEach - 1) / (kThreads * kEach);
    if (blocks * kThreads > kMaxThreads) return hipErrorInvalidValue;
    int shift = 0;
    while ((int64_t(1) << shift) < per_group) ++shift;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
    const int lanes = static_cast<int>(per_group);
    if (16 * chunks > kMemorySideCache)
      hipLaunchKernelGGL((group_quantize_kernel<W16, S16, ZP, true>), grid, block, 0, stream, W, chunks, lanes, shift,
                         codes, scales, zeros);
    else
      hipLaunchKernelGGL((group_quantize_kernel<W16, S16, ZP, false>), grid, block, 0, stream, W, chunks, lanes, shift,
                         codes, scales, zeros);
  } else {
    const int64_t groups = n / group;
    int64_t blocks = (groups + kThreads / 64 - 1) / (kThreads / 64);
    if (blocks > 256 * 16) blocks = 256 * 16;
    hipLaunchKernelGGL((group_quantize_any_kernel<W16, S16, ZP>), dim3(static_cast<unsigned>(blocks)), dim3(kThreads),
                       0, stream, W, groups, per_group, codes, scales, zeros);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_group_quantize(const void *W, bool w_bf16, int64_t n_rows, int64_t n_cols, int64_t group,
                                 bool scale_bf16, uint8_t *codes, void *scales, uint8_t *zeros, hipStream_t stream) {
  const int64_t n = n_rows * n_cols;
  switch ((w_bf16 ? 4 : 0) + (scale_bf16 ? 2 : 0) + (zeros ? 1 : 0)) {
    case 0: return quantize_go<false, false, false>(W, n, group, codes, scales, zeros, stream);
    case 1: return quantize_go<false, false, true>(W, n, group, codes, scales, zeros, stream);
    case 2: return quantize_go<false, true, false>(W, n, group, codes, scales, zeros, stream);
    case 3: return quantize_go<false, true, true>(W, n, group, codes, scales, zeros, stream);
    case 4: return quantize_go<true, false, false>(W, n, group, codes, scales, zeros, stream);
    case 5: return quantize_go<true, false, true>(W, n, group, codes, scales, zeros, stream);
    case 6: return quantize_go<true, true, false>(W, n, group, codes, scales, zeros, stream);
    default: return quantize_go<true, true, true>(W, n, group, codes, scales, zeros, stream);
  }
}

hipError_t launch_group_dequantize(const GroupView &w, void *out, bool out_bf16, hipStream_t stream) {
  const int V = out_bf16 ? 8 : 4;
  const uint32_t row_chunks = static_cast<uint32_t>(w.n_cols / V), per_group = static_cast<uint32_t>(w.group / V);
  const uint32_t spans = (row_chunks + kUnroll * 64 - 1) / (kUnroll * 64);
  int64_t blocks = (w.n_rows * spans + kThreads / 64 - 1) / (kThreads / 64);
  if (blocks > 256 * 16) blocks = 256 * 16;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  const uint32_t magic = group_magic(per_group);
  if (out_bf16)
    hipLaunchKernelGGL(group_dequantize_kernel<true>, grid, block, 0, stream, w, row_chunks, spans,
                       row_chunks / per_group, magic, out);
  else
    hipLaunchKernelGGL(group_dequantize_kernel<false>, grid, block, 0, stream, w, row_chunks, spans,
                       row_chunks / per_group, magic, out);
  return hipGetLastError();
}

}  // namespace qlora
