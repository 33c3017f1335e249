// Backward of the gated projections' activation and product (gfx950):
//
//   [dG | dL] = [dH L act'(G) | dH act(G)]   from the saved bf16 [G | L]
//
// in one pass over the three inputs, 8 columns (16 bytes of each) a thread.  The kernel is
// bound by memory: 10 bytes an element of H move.  The result is what the linear's backward
// reads as dY: rows of two column blocks of round_up(P, 8) columns, zeros in the padding,
// so that odd P keeps 16-byte rows.

#include "device_common.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int NT = 256;

// Eight bf16 values of a row at `src`, of which n >= 1 exist; 16-byte load when `vec`.
__device__ __forceinline__ u32x4_t load_chunk(const uint16_t *src, bool vec, int n) {
  if (vec) return *reinterpret_cast<const u32x4_t *>(src);
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < n ? src[2 * i] : 0u, hi = 2 * i + 1 < n ? src[2 * i + 1] : 0u;
    v[i] = lo | (hi << 16);
  }
  return v;
}

template <int ACT>
__global__ __launch_bounds__(NT) void gated_grad_kernel(const uint16_t *__restrict__ dH,
                                                        const uint16_t *__restrict__ Y, uint32_t M, uint32_t P,
                                                        uint16_t *__restrict__ dY) {
  const uint32_t chunks = (P + 7) / 8, P8 = chunks * 8;
  const bool vec = P % 8 == 0;
  const uint32_t n = M * chunks;
  for (uint32_t i = blockIdx.x * NT + threadIdx.x; i < n; i += gridDim.x * NT) {
    const uint32_t m = i / chunks, c = (i - m * chunks) * 8;
    const int cols = min(P - c, 8u);
    const int64_t row = m;
    const u32x4_t h = load_chunk(dH + row * P + c, vec, cols);
    const u32x4_t g = load_chunk(Y + row * 2 * P + c, vec, cols);
    const u32x4_t l = load_chunk(Y + row * 2 * P + P + c, vec, cols);
    u32x4_t dg, dl;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f0, d0, f1, d1;
      act_grad<ACT>(bf16_lo(g[k]), f0, d0);
      act_grad<ACT>(bf16_hi(g[k]), f1, d1);
      const float h0 = bf16_lo(h[k]), h1 = bf16_hi(h[k]);
      dg[k] = pack_bf16x2(h0 * bf16_lo(l[k]) * d0, h1 * bf16_hi(l[k]) * d1);
      dl[k] = pack_bf16x2(h0 * f0, h1 * f1);  // zero past P: h is zero there
    }
    uint16_t *const out = dY + row * 2 * P8 + c;
    *reinterpret_cast<u32x4_t *>(out) = dg;
    *reinterpret_cast<u32x4_t *>(out + P8) = dl;
  }
}

}  // namespace

hipError_t launch_gated_grad(const uint16_t *dH, const uint16_t *Y, int64_t M, int64_t P, int act, uint16_t *dY,
                             hipStream_t stream) {
  const int64_t P8 = (P + 7) / 8 * 8;
  if (uint64_t(M) * 2 * P8 * 2 > 0xFFFFFFF0ull) return hipErrorInvalidValue;
  int64_t blocks = (M * (P8 / 8) + NT - 1) / NT;
  if (blocks > 256 * 32) blocks = 256 * 32;
  const dim3 grid(static_cast<unsigned>(blocks)), block(NT);
  const uint32_t m = static_cast<uint32_t>(M), p = static_cast<uint32_t>(P);
  if (act == kActSilu)
    hipLaunchKernelGGL(gated_grad_kernel<kActSilu>, grid, block, 0, stream, dH, Y, m, p, dY);
  else
    hipLaunchKernelGGL(gated_grad_kernel<kActGeluTanh>, grid, block, 0, stream, dH, Y, m, p, dY);
  return hipGetLastError();
}

}  // namespace qlora
