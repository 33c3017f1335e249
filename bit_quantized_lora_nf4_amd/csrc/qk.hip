// Norms of query and key heads with the position rotation in the same pass (gfx950), forward
// and backward.
//
// The rows are the fused projections' [q heads | k heads | v heads], d elements a head.  For a
// q or k head x of a token at position p:
//
//   n = x r w,  r = 1 / sqrt(mean x^2 + eps)          (without a norm: n = x)
//   pair i of the first `rot` elements, (a, b), turns by t_i = p f_i:
//     (a cos t_i - b sin t_i,  b cos t_i + a sin t_i)
//   pair i is (i, i + rot / 2), or interleaved (2 i, 2 i + 1); the other elements pass
//
// and backward, with dn the rotation by -t of the output's gradient:
//   dw = sum dn x r,   dx = r (g - x r (r mean(g x))),  g = dn w
//
// The angle in turns, p f / (2 pi), is formed and reduced to [-1/2, 1/2] in 64 bits (at
// position 131071 a product in fp32 would be off by up to 2^-8 radians); one sine and cosine
// a pair and token, shared by the token's heads through LDS.  Both directions are bound by
// memory; every row is read once and every result written once.
//
// A head's elements lie on L lanes (a power of two), 2 V a lane: for a rotated unit u the two
// chunks of V elements that turn into each other, so no value ever crosses lanes except the
// sums of the norm.  A wave takes 64 / L heads of a token at a time.

#include "device_common.h"
#include "qlora_internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxPairs = kQkMaxDim / 2;

// V values as fp32 from / to memory of T16 ? bf16 : fp32; the access is V * size bytes wide.
template <bool T16, int V>
__device__ __forceinline__ void load_values(const void *p, int64_t i, float *v) {
  if constexpr (T16) {
    const uint16_t *q = static_cast<const uint16_t *>(p) + i;
    uint32_t u[V / 2];
    if constexpr (V == 8) {
      const u32x4_t t = *reinterpret_cast<const u32x4_t *>(q);
      u[0] = t[0], u[1] = t[1], u[2] = t[2], u[3] = t[3];
    } else if constexpr (V == 4) {
      const u32x2_t t = *reinterpret_cast<const u32x2_t *>(q);
      u[0] = t[0], u[1] = t[1];
    } else {
      u[0] = *reinterpret_cast<const uint32_t *>(q);
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) v[2 * e] = bf16_lo(u[e]), v[2 * e + 1] = bf16_hi(u[e]);
  } else {
    const float *q = static_cast<const float *>(p) + i;
    if constexpr (V == 4) {
      const f32x4_t t = *reinterpret_cast<const f32x4_t *>(q);
      v[0] = t[0], v[1] = t[1], v[2] = t[2], v[3] = t[3];
    } else {
      const u32x2_t t = *reinterpret_cast<const u32x2_t *>(q);
      v[0] = __uint_as_float(t[0]), v[1] = __uint_as_float(t[1]);
    }
  }
}
template <bool T16, int V>
__device__ __forceinline__ void store_values(void *p, int64_t i, const float *v) {
  if constexpr (T16) {
    uint16_t *q = static_cast<uint16_t *>(p) + i;
    uint32_t u[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) u[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    if constexpr (V == 8)
      *reinterpret_cast<u32x4_t *>(q) = u32x4_t{u[0], u[1], u[2], u[3]};
    else if constexpr (V == 4)
      *reinterpret_cast<u32x2_t *>(q) = u32x2_t{u[0], u[1]};
    else
      *reinterpret_cast<uint32_t *>(q) = u[0];
  } else {
    float *q = static_cast<float *>(p) + i;
    if constexpr (V == 4)
      *reinterpret_cast<f32x4_t *>(q) = f32x4_t{v[0], v[1], v[2], v[3]};
    else
      *reinterpret_cast<u32x2_t *>(q) = u32x2_t{__float_as_uint(v[0]), __float_as_uint(v[1])};
  }
}

// What a lane holds of every head: chunks at elements o0 and o1 (has0, has1: within the
// head), turned into each other (rotated units) or passed on.
struct Unit {
  int o0, o1;
  bool has0, has1, turns;
};
template <int V, bool INTER>
__device__ __forceinline__ Unit unit_of(int u, const QkShape &s) {
  const int turning = s.rot / (2 * V);
  Unit x;
  x.turns = u < turning;
  if (!x.turns || INTER) {
    x.o0 = 2 * u * V;
    x.o1 = x.o0 + V;
  } else {
    x.o0 = u * V;
    x.o1 = x.o0 + s.rot / 2;
  }
  x.has0 = x.o0 < s.d;
  x.has1 = x.o1 < s.d;
  return x;
}

// Sines and cosines of a token's pairs into the wave's own LDS, then the V pairs of this
// lane's unit.  LDS accesses of one wave stay in order, so no barrier is needed.
template <int V>
__device__ __forceinline__ void angles(int64_t position, const float *inv_freq, const QkShape &s, int lane, int u,
                                       bool turns, float *lds, float *co, float *si) {
  const double p = static_cast<double>(position);
  __builtin_amdgcn_wave_barrier();
  for (int i = lane; i < s.rot / 2; i += 64) {
    const double turn = p * (static_cast<double>(inv_freq[i]) * 0.15915494309189535);
    const float half_turns = static_cast<float>(2.0 * (turn - __builtin_rint(turn)));
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    lds[i] = cs;
    lds[kMaxPairs + i] = sn;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int e = 0; e < V; ++e) {
    co[e] = turns ? lds[u * V + e] : 1.0f;
    si[e] = turns ? lds[kMaxPairs + u * V + e] : 0.0f;
  }
}

// (x0, x1) of one lane turned by its V angles.
template <int V, bool INTER>
__device__ __forceinline__ void turn(float *x, const float *co, const float *si, float sign) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int a = INTER ? 2 * e : e, b = INTER ? 2 * e + 1 : V + e;
    const float sn = sign * si[e], va = x[a], vb = x[b];
    x[a] = va * co[e] - vb * sn;
    x[b] = vb * co[e] + va * sn;
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

template <bool T16, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_fwd_kernel(const void *__restrict__ Y, QkShape s,
                                                          const int64_t *__restrict__ positions,
                                                          const float *__restrict__ inv_freq,
                                                          const void *__restrict__ qw, const void *__restrict__ kw,
                                                          void *__restrict__ Q, void *__restrict__ K) {
  __shared__ float lds[kWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = lane & (s.lanes - 1), heads_per = 64 / s.lanes, sub = lane / s.lanes, heads = s.nq + s.nk;
  const Unit un = unit_of<V, INTER>(u, s);
  const bool norm = qw != nullptr;
  float wq[2 * V], wk[2 * V];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) wq[e] = wk[e] = 1.0f;
  if (norm) {
    if (un.has0) load_values<T16, V>(qw, un.o0, wq), load_values<T16, V>(kw, un.o0, wk);
    if (un.has1) load_values<T16, V>(qw, un.o1, wq + V), load_values<T16, V>(kw, un.o1, wk + V);
  }
  const int64_t tasks = s.M * s.split, step = static_cast<int64_t>(gridDim.x) * kWaves;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + wave; task < tasks; task += step) {
    const int64_t m = task / s.split;
    const int part = static_cast<int>(task - m * s.split);
    float co[V], si[V];
    angles<V>(positions[m], inv_freq, s, lane, u, un.turns, lds[wave], co, si);
    const int h1 = min(heads, (part + 1) * s.per * heads_per);
    for (int h = part * s.per * heads_per + sub; h < h1; h += heads_per) {
      float x[2 * V];
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[e] = 0.0f;
      const int64_t at = m * s.row + static_cast<int64_t>(h) * s.d;
      if (un.has0) load_values<T16, V>(Y, at + un.o0, x);
      if (un.has1) load_values<T16, V>(Y, at + un.o1, x + V);
      if (norm) {
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) sq = __builtin_fmaf(x[e], x[e], sq);
        sq = lanes_sum(sq, s.lanes);
        const float r = 1.0f / sqrtf(sq * s.inv_d + s.eps);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) x[e] = x[e] * r * (h < s.nq ? wq[e] : wk[e]);
      }
      turn<V, INTER>(x, co, si, 1.0f);
      void *out = h < s.nq ? Q : K;
      const int64_t to = h < s.nq ? (m * s.nq + h) * s.d : (m * s.nk + h - s.nq) * s.d;
      if (un.has0) store_values<T16, V>(out, to + un.o0, x);
      if (un.has1) store_values<T16, V>(out, to + un.o1, x + V);
    }
  }
}

template <bool T16, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_bwd_kernel(const void *__restrict__ dQ, const void *__restrict__ dK,
                                                          const void *__restrict__ dV, const void *__restrict__ Y,
                                                          QkShape s, const int64_t *__restrict__ positions,
                                                          const float *__restrict__ inv_freq,
                                                          const void *__restrict__ qw, const void *__restrict__ kw,
                                                          void *__restrict__ dY, float *__restrict__ part_dw) {
  __shared__ float lds[kWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = lane & (s.lanes - 1), heads_per = 64 / s.lanes, sub = lane / s.lanes, heads = s.nq + 2 * s.nk;
  const Unit un = unit_of<V, INTER>(u, s);
  const bool norm = qw != nullptr;
  float wq[2 * V], wk[2 * V], dwq[2 * V], dwk[2 * V];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) wq[e] = wk[e] = 1.0f, dwq[e] = dwk[e] = 0.0f;
  if (norm) {
    if (un.has0) load_values<T16, V>(qw, un.o0, wq), load_values<T16, V>(kw, un.o0, wk);
    if (un.has1) load_values<T16, V>(qw, un.o1, wq + V), load_values<T16, V>(kw, un.o1, wk + V);
  }
  const int64_t tasks = s.M * s.split, step = static_cast<int64_t>(gridDim.x) * kWaves;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + wave; task < tasks; task += step) {
    const int64_t m = task / s.split;
    const int part = static_cast<int>(task - m * s.split);
    float co[V], si[V];
    angles<V>(positions[m], inv_freq, s, lane, u, un.turns, lds[wave], co, si);
    const int h1 = min(heads, (part + 1) * s.per * heads_per);
    for (int h = part * s.per * heads_per + sub; h < h1; h += heads_per) {
      const bool is_q = h < s.nq, is_v = h >= s.nq + s.nk;
      const void *src = is_q ? dQ : is_v ? dV : dK;
      const int64_t from = is_q ? (m * s.nq + h) * s.d : (m * s.nk + (h - s.nq - (is_v ? s.nk : 0))) * s.d;
      const int64_t at = m * s.row + static_cast<int64_t>(h) * s.d;
      float g[2 * V];
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) g[e] = 0.0f;
      if (un.has0) load_values<T16, V>(src, from + un.o0, g);
      if (un.has1) load_values<T16, V>(src, from + un.o1, g + V);
      if (!is_v) {
        turn<V, INTER>(g, co, si, -1.0f);
        if (norm) {
          float x[2 * V];
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) x[e] = 0.0f;
          if (un.has0) load_values<T16, V>(Y, at + un.o0, x);
          if (un.has1) load_values<T16, V>(Y, at + un.o1, x + V);
          float sq = 0.0f, gx = 0.0f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            sq = __builtin_fmaf(x[e], x[e], sq);
            gx = __builtin_fmaf(g[e] * (is_q ? wq[e] : wk[e]), x[e], gx);
          }
          sq = lanes_sum(sq, s.lanes);
          gx = lanes_sum(gx, s.lanes);
          const float r = 1.0f / sqrtf(sq * s.inv_d + s.eps);
          const float back = r * (gx * s.inv_d);
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            const float xh = x[e] * r, d = g[e] * xh;
            dwq[e] += is_q ? d : 0.0f;
            dwk[e] += is_q ? 0.0f : d;
            g[e] = r * (g[e] * (is_q ? wq[e] : wk[e]) - xh * back);
          }
        }
      }
      if (un.has0) store_values<T16, V>(dY, at + un.o0, g);
      if (un.has1) store_values<T16, V>(dY, at + un.o1, g + V);
    }
  }
  if (!norm) return;

  // the wave's sums over its heads, then the workgroup's over its waves, in a fixed order
  __shared__ float dw[kWaves][2][kQkMaxDim];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) {
    for (int m = s.lanes; m < 64; m <<= 1) {
      dwq[e] += __shfl_xor(dwq[e], m, 64);
      dwk[e] += __shfl_xor(dwk[e], m, 64);
    }
    const int o = e < V ? un.o0 + e : un.o1 + e - V;
    if (lane < s.lanes && (e < V ? un.has0 : un.has1)) dw[wave][0][o] = dwq[e], dw[wave][1][o] = dwk[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * s.d; i += kThreads) {
    const int which = i >= s.d, o = which ? i - s.d : i;
    float v = dw[0][which][o];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += dw[k][which][o];
    part_dw[static_cast<int64_t>(blockIdx.x) * 2 * s.d + i] = v;
  }
}

// The workgroups' partial sums [parts][2 d] added in a fixed order: 32 columns and 32 slices
// of the parts to a workgroup, the slices' sums added in slice order.
template <bool T16>
__global__ __launch_bounds__(1024) void qk_dw_kernel(const float *__restrict__ P, int parts, int d,
                                                     void *__restrict__ dqw, void *__restrict__ dkw) {
  __shared__ float sums[32][33];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5, i = blockIdx.x * 32 + col;
  float v = 0.0f;
  if (i < 2 * d)
    for (int k = slice; k < parts; k += 32) v += P[static_cast<int64_t>(k) * 2 * d + i];
  sums[slice][col] = v;
  __syncthreads();
  if (slice != 0 || i >= 2 * d) return;
  for (int k = 1; k < 32; ++k) v += sums[k][col];
  void *out = i < d ? dqw : dkw;
  const int o = i < d ? i : i - d;
  if constexpr (T16)
    static_cast<uint16_t *>(out)[o] = to_bf16(v);
  else
    static_cast<float *>(out)[o] = v;
}

// Elements of a lane's chunk: the widest access (16 bytes) that divides the head and half the
// rotated part.
int chunk_of(const QkShape &s, bool t16) {
  int v = t16 ? 8 : 4;
  while (v > 2 && (s.d % v != 0 || s.rot % (2 * v) != 0)) v /= 2;
  return v;
}

// Lanes of a head, and how a token's heads are split over waves: all of them to one wave (one
// computation of the angles) unless the tokens are too few for the card.
constexpr int64_t kWantedWaves = 256 * 16;
void plan(QkShape *s, int v, int heads) {
  const int units = (s->d + 2 * v - 1) / (2 * v);
  s->lanes = 1;
  while (s->lanes < units) s->lanes *= 2;
  const int heads_per = 64 / s->lanes, rounds = (heads + heads_per - 1) / heads_per;
  int64_t split = (kWantedWaves + s->M - 1) / s->M;
  if (split > rounds) split = rounds;
  s->per = static_cast<int>((rounds + split - 1) / split);
  s->split = (rounds + s->per - 1) / s->per;
  s->row = static_cast<int64_t>(s->nq + 2 * s->nk) * s->d;
  s->inv_d = 1.0f / static_cast<float>(s->d);
}
int64_t workgroups(const QkShape &s, int64_t most) {
  const int64_t wgs = (s.M * s.split + kWaves - 1) / kWaves;
  return wgs < most ? wgs : most;
}
constexpr int64_t kFwdWorkgroups = 256 * 8, kBwdWorkgroups = 256 * 4;

}  // namespace

size_t qk_bwd_workspace(QkShape s, bool t16, bool norm) {
  if (!norm) return 0;
  plan(&s, chunk_of(s, t16), s.nq + 2 * s.nk);
  return static_cast<size_t>(workgroups(s, kBwdWorkgroups)) * 2 * s.d * sizeof(float);
}

hipError_t launch_qk_fwd(const void *Y, QkShape s, bool t16, bool interleaved, const int64_t *positions,
                         const float *inv_freq, const void *qw, const void *kw, void *Q, void *K,
                         hipStream_t stream) {
  const int v = chunk_of(s, t16);
  plan(&s, v, s.nq + s.nk);
  const dim3 grid(static_cast<unsigned>(workgroups(s, kFwdWorkgroups))), block(kThreads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, Y, s, positions, inv_freq, qw, kw, Q, K);
    return hipGetLastError();
  };
  switch ((t16 ? 100 : 0) + 10 * v + (interleaved ? 1 : 0)) {
    case 180: return go(qk_fwd_kernel<true, 8, false>);
    case 181: return go(qk_fwd_kernel<true, 8, true>);
    case 140: return go(qk_fwd_kernel<true, 4, false>);
    case 141: return go(qk_fwd_kernel<true, 4, true>);
    case 120: return go(qk_fwd_kernel<true, 2, false>);
    case 121: return go(qk_fwd_kernel<true, 2, true>);
    case 40: return go(qk_fwd_kernel<false, 4, false>);
    case 41: return go(qk_fwd_kernel<false, 4, true>);
    case 20: return go(qk_fwd_kernel<false, 2, false>);
    default: return go(qk_fwd_kernel<false, 2, true>);
  }
}

hipError_t launch_qk_bwd(const void *dQ, const void *dK, const void *dV, const void *Y, QkShape s, bool t16,
                         bool interleaved, const int64_t *positions, const float *inv_freq, const void *qw,
                         const void *kw, void *dY, void *dqw, void *dkw, float *part, hipStream_t stream) {
  const int v = chunk_of(s, t16);
  plan(&s, v, s.nq + 2 * s.nk);
  const int64_t wgs = workgroups(s, kBwdWorkgroups);
  const dim3 grid(static_cast<unsigned>(wgs)), block(kThreads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, dQ, dK, dV, Y, s, positions, inv_freq, qw, kw, dY, part);
    return hipGetLastError();
  };
  hipError_t e;
  switch ((t16 ? 100 : 0) + 10 * v + (interleaved ? 1 : 0)) {
    case 180: e = go(qk_bwd_kernel<true, 8, false>); break;
    case 181: e = go(qk_bwd_kernel<true, 8, true>); break;
    case 140: e = go(qk_bwd_kernel<true, 4, false>); break;
    case 141: e = go(qk_bwd_kernel<true, 4, true>); break;
    case 120: e = go(qk_bwd_kernel<true, 2, false>); break;
    case 121: e = go(qk_bwd_kernel<true, 2, true>); break;
    case 40: e = go(qk_bwd_kernel<false, 4, false>); break;
    case 41: e = go(qk_bwd_kernel<false, 4, true>); break;
    case 20: e = go(qk_bwd_kernel<false, 2, false>); break;
    default: e = go(qk_bwd_kernel<false, 2, true>); break;
  }
  if (e != hipSuccess || !qw) return e;
  const dim3 dgrid(static_cast<unsigned>((2 * s.d + 31) / 32));
  if (t16)
    hipLaunchKernelGGL(qk_dw_kernel<true>, dgrid, dim3(1024), 0, stream, part, static_cast<int>(wgs), s.d, dqw, dkw);
  else
    hipLaunchKernelGGL(qk_dw_kernel<false>, dgrid, dim3(1024), 0, stream, part, static_cast<int>(wgs), s.d, dqw, dkw);
  return hipGetLastError();
}

}  // namespace qlora
