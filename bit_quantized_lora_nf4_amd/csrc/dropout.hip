// Dropout from a counter-based generator (gfx950) and the row copies that bring operands
// of unaligned row length into 16-byte rows.
//
//   out[e] = m[e] c x[e],  c = 1 / (1 - p),  m a function of (seed, offset, e)
//
// (lora_dropout of the adapter configuration, [Repro] "官方代码阅读路线".)  No mask is
// stored: the backward of the operator is the operator itself with the same seed and
// offset.  A thread takes whole groups of eight elements, one generator block each
// (drop_words in device_common.h): 16-byte accesses for bf16, two of them for fp32.  The
// kernel is bound by memory: a block costs about 14 32x32-bit products for 32 bytes moved
// (bf16).

#include "device_common.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int NT = 256;

template <bool BF16>
__global__ __launch_bounds__(NT) void dropout_kernel(const void *X, int64_t n, Dropout d, float c, void *out) {
  const DropKey dk = drop_key(d);
  const int64_t groups = n / 8, stride = static_cast<int64_t>(gridDim.x) * NT;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
  for (int64_t g = t0; g < groups; g += stride) {
    const u32x4_t w = drop_words(static_cast<uint32_t>(g), static_cast<uint32_t>(g >> 32), dk);
    if constexpr (BF16) {
      const u32x4_t x = reinterpret_cast<const u32x4_t *>(X)[g];
      const u32x4_t m = drop_mask(w, dk.thr);
      u32x4_t y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = pack_bf16x2(bf16_lo(x[i]) * c, bf16_hi(x[i]) * c) & m[i];
      reinterpret_cast<u32x4_t *>(out)[g] = y;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t x = reinterpret_cast<const f32x4_t *>(X)[2 * g + h];
        f32x4_t y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = w[2 * h + i / 2];
          y[i] = ((i & 1) ? v >> 16 : v & 0xFFFFu) >= dk.thr ? x[i] * c : 0.0f;
        }
        reinterpret_cast<f32x4_t *>(out)[2 * g + h] = y;
      }
    }
  }
  // the last n % 8 elements
  const int64_t e = 8 * groups + t0;
  if (t0 < 8 && e < n) {
    const u32x4_t w = drop_words(static_cast<uint32_t>(groups), static_cast<uint32_t>(groups >> 32), dk);
    const uint32_t v = t0 < 2 ? w[0] : t0 < 4 ? w[1] : t0 < 6 ? w[2] : w[3];
    const bool keep = ((t0 & 1) ? v >> 16 : v & 0xFFFFu) >= dk.thr;
    if constexpr (BF16) {
      const float x = bf16_to_f32(static_cast<const uint16_t *>(X)[e]);
      static_cast<uint16_t *>(out)[e] = keep ? to_bf16(x * c) : static_cast<uint16_t>(0);
    } else {
      const float x = static_cast<const float *>(X)[e];
      static_cast<float *>(out)[e] = keep ? x * c : 0.0f;
    }
  }
}

// Row copies with zero padding (CopyJob): a row of the grid per job, a thread per 8 columns
// (16 bytes) of the destination.  A side whose rows are 16-byte aligned is accessed whole,
// the other one element by element, all in flight together.  The jobs are adapter operands
// of unaligned rank (a few MB: the launch is what they take, 3.4 us for A [24, 1280] and B
// [2002, 12]) or a gradient of odd width.
struct CopyJobs {
  CopyJob j[kMaxCopyJobs];
};
__global__ __launch_bounds__(NT) void copy_rows_kernel(CopyJobs jobs) {
  const CopyJob jb = jobs.j[blockIdx.y];
  const uint32_t chunks = static_cast<uint32_t>((jb.dcols + 7) / 8);
  const uint32_t n = static_cast<uint32_t>(jb.rows) * chunks;  // of 16 bytes of a tensor below 4 GiB
  const bool vs = jb.lds % 8 == 0, vd = jb.ldd % 8 == 0;
  for (uint32_t i = blockIdx.x * NT + threadIdx.x; i < n; i += gridDim.x * NT) {
    const uint32_t row = i / chunks, c = (i - row * chunks) * 8;
    const uint16_t *src = jb.src + row * jb.lds + c;
    uint16_t *dst = jb.dst + row * jb.ldd + c;
    const int64_t have = jb.cols - c, want = jb.dcols - c;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (vs && have >= 8) {
      v = *reinterpret_cast<const u32x4_t *>(src);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = 2 * e < have ? src[2 * e] : 0u, hi = 2 * e + 1 < have ? src[2 * e + 1] : 0u;
        v[e] = lo | (hi << 16);
      }
    }
    if (vd && want >= 8) {
      *reinterpret_cast<u32x4_t *>(dst) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = v[e];
        if (2 * e < want) dst[2 * e] = static_cast<uint16_t>(w);
        if (2 * e + 1 < want) dst[2 * e + 1] = static_cast<uint16_t>(w >> 16);
      }
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void *X, bool bf16, int64_t n, const Dropout &d, float c, void *out,
                          hipStream_t stream) {
  if (d.thr == 0) {
    if (X == out) return hipSuccess;
    return hipMemcpyAsync(out, X, static_cast<size_t>(n) * (bf16 ? 2 : 4), hipMemcpyDeviceToDevice, stream);
  }
  int64_t blocks = (n / 8 + NT - 1) / NT;
  if (blocks > 256 * 16) blocks = 256 * 16;
  if (blocks < 1) blocks = 1;
  const dim3 grid(static_cast<unsigned>(blocks)), block(NT);
  if (bf16)
    hipLaunchKernelGGL(dropout_kernel<true>, grid, block, 0, stream, X, n, d, c, out);
  else
    hipLaunchKernelGGL(dropout_kernel<false>, grid, block, 0, stream, X, n, d, c, out);
  return hipGetLastError();
}

hipError_t launch_copy_rows(const CopyJob *jobs, int n, hipStream_t stream) {
  CopyJobs a;
  int used = 0;
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    if (jobs[i].rows <= 0) continue;
    const int64_t units = jobs[i].rows * ((jobs[i].dcols + 7) / 8);
    if (used == kMaxCopyJobs || units > 0x7fffffff) return hipErrorInvalidValue;
    a.j[used++] = jobs[i];
    most = units > most ? units : most;
  }
  if (used == 0) return hipSuccess;
  for (int i = used; i < kMaxCopyJobs; ++i) a.j[i] = CopyJob{nullptr, nullptr, 0, 0, 0, 0, 0};
  int64_t blocks = (most + NT - 1) / NT;
  if (blocks > 2048) blocks = 2048;
  hipLaunchKernelGGL(copy_rows_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(used)), dim3(NT), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace qlora
