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
// The angle in turns, p f / (2 pi), its reduction, sine and cosine are formed in 64 bits (at
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

constexpr int kThreads = 256, kWaves = kThreads / 64;           // forward
constexpr int kBwdThreads = 1024, kBwdWaves = kBwdThreads / 64;  // backward: few partial sums
constexpr int kMaxPairs = kQkMaxDim / 2;

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef double f64x2_t __attribute__((ext_vector_type(2)));

// V values of a tensor (T16: bf16, else fp32) as loaded: one access of 16, 8 or 4 bytes.
template <bool T16, int V>
struct Raw {
  static constexpr int kWords = T16 ? V / 2 : V;
  uint32_t w[kWords];
};
template <bool T16, int V>
__device__ __forceinline__ void load_raw(Raw<T16, V> &r, const void *p, int64_t i) {
  const char *q = static_cast<const char *>(p) + i * (T16 ? 2 : 4);
  if constexpr (Raw<T16, V>::kWords == 4) {
    const u32x4_t t = *reinterpret_cast<const u32x4_t *>(q);
    r.w[0] = t[0], r.w[1] = t[1], r.w[2] = t[2], r.w[3] = t[3];
  } else if constexpr (Raw<T16, V>::kWords == 2) {
    const u32x2_t t = *reinterpret_cast<const u32x2_t *>(q);
    r.w[0] = t[0], r.w[1] = t[1];
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t *>(q);
  }
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store_as(T v, char *q) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<T *>(q));
  else
    *reinterpret_cast<T *>(q) = v;
}
template <bool STREAM, bool T16, int V>
__device__ __forceinline__ void store_raw(const Raw<T16, V> &r, void *p, int64_t i) {
  char *q = static_cast<char *>(p) + i * (T16 ? 2 : 4);
  if constexpr (Raw<T16, V>::kWords == 4)
    store_as<STREAM>(u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]}, q);
  else if constexpr (Raw<T16, V>::kWords == 2)
    store_as<STREAM>(u32x2_t{r.w[0], r.w[1]}, q);
  else
    store_as<STREAM>(r.w[0], q);
}
template <bool T16, int V>
__device__ __forceinline__ void to_values(const Raw<T16, V> &r, float *v) {
#pragma unroll
  for (int e = 0; e < Raw<T16, V>::kWords; ++e) {
    if constexpr (T16)
      v[2 * e] = bf16_lo(r.w[e]), v[2 * e + 1] = bf16_hi(r.w[e]);
    else
      v[e] = __uint_as_float(r.w[e]);
  }
}
template <bool T16, int V>
__device__ __forceinline__ Raw<T16, V> from_values(const float *v) {
  Raw<T16, V> r;
#pragma unroll
  for (int e = 0; e < Raw<T16, V>::kWords; ++e) r.w[e] = T16 ? pack_bf16x2(v[2 * e], v[2 * e + 1]) : __float_as_uint(v[e]);
  return r;
}

// What a lane holds of every head: chunks at elements o0 and o1 (has0, has1: within the
// head), turned into each other (rotated units) or passed on.
struct Unit {
  int o0, o1;
  bool has0, has1, turns;
};
template <int V, bool INTER>
__device__ __forceinline__ Unit unit_of(int u, const QkShape &s) {
  Unit x;
  x.turns = u < s.rot / (2 * V);
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
// A lane's two chunks of a head at element i of a tensor (zeros where there is none).
template <bool T16, int V>
struct Both {
  Raw<T16, V> c[2];
  __device__ __forceinline__ void load(const void *p, int64_t i, const Unit &u, bool on) {
#pragma unroll
    for (int e = 0; e < Raw<T16, V>::kWords; ++e) c[0].w[e] = c[1].w[e] = 0u;
    if (on && u.has0) load_raw(c[0], p, i + u.o0);
    if (on && u.has1) load_raw(c[1], p, i + u.o1);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(void *p, int64_t i, const Unit &u) const {
    if (u.has0) store_raw<STREAM>(c[0], p, i + u.o0);
    if (u.has1) store_raw<STREAM>(c[1], p, i + u.o1);
  }
  __device__ __forceinline__ void values(float *v) const {
    to_values(c[0], v);
    to_values(c[1], v + V);
  }
  __device__ __forceinline__ void set(const float *v) {
    c[0] = from_values<T16, V>(v);
    c[1] = from_values<T16, V>(v + V);
  }
  // The other's where `changed`; else the bits as loaded, which a conversion would not keep of a NaN.
  __device__ __forceinline__ void take(const Both &o, bool changed) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < Raw<T16, V>::kWords; ++e) c[k].w[e] = changed ? o.c[k].w[e] : c[k].w[e];
  }
};

// 1 / OVER in a scalar register that is set where it is used: the compiler would keep every constant of
// a series in vector registers over the whole kernel, 16 more of them, and fewer waves would fit.
template <int64_t OVER>
__device__ __forceinline__ double one_over() {
  constexpr uint64_t bits = __builtin_bit_cast(uint64_t, 1.0 / OVER);
  uint32_t lo, hi;
  asm volatile("s_mov_b32 %0, %1" : "=s"(lo) : "n"(static_cast<uint32_t>(bits)));
  asm volatile("s_mov_b32 %0, %1" : "=s"(hi) : "n"(static_cast<uint32_t>(bits >> 32)));
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Sine and cosine of an angle given in turns, all in 64 bits and each rounded once: within half a step of
// fp32, also at far positions.  The angle is reduced to an eighth of a turn on either side of a quarter's
// multiple (1.5 x 2^52 added leaves the multiple in the sum's last bits), where the power series to
// x^11 and x^12 are off by less than 2^-36.  (An angle rounded to fp32 before its sine is taken leaves a
// cosine off by up to 1.1e-7, the cosine's own rounding by 3.0e-8.)
__device__ __forceinline__ void sine_cosine(double turn, float &sn, float &cs) {
  const double t = turn - __builtin_rint(turn);
  const double k = __builtin_fma(4.0, t, 0x1.8p52);
  const uint32_t quarter = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, k));
  const double x = __builtin_fma(-0.25, k - 0x1.8p52, t) * 6.283185307179586;
  const double x2 = x * x;
  double s = one_over<-39916800>(), c = one_over<479001600>();
  s = __builtin_fma(s, x2, one_over<362880>());
  s = __builtin_fma(s, x2, one_over<-5040>());
  s = __builtin_fma(s, x2, one_over<120>());
  s = __builtin_fma(s, x2, one_over<-6>());
  c = __builtin_fma(c, x2, one_over<-3628800>());
  c = __builtin_fma(c, x2, one_over<40320>());
  c = __builtin_fma(c, x2, one_over<-720>());
  c = __builtin_fma(c, x2, one_over<24>());
  c = __builtin_fma(c, x2, -0.5);
  const float fs = static_cast<float>(__builtin_fma(x * x2, s, x)), fc = static_cast<float>(__builtin_fma(c, x2, 1.0));
  const bool odd = quarter & 1;
  sn = __uint_as_float(__float_as_uint(odd ? fc : fs) ^ ((quarter & 2) << 30));
  cs = __uint_as_float(__float_as_uint(odd ? fs : fc) ^ (((quarter + 1) & 2) << 30));
}

// Sines and cosines of a token's pairs into the wave's own LDS, then the V pairs of this
// lane's unit.  LDS accesses of one wave stay in order, so no barrier is needed.
template <int V>
__device__ __forceinline__ void angles(int64_t position, const float *inv_freq, const QkShape &s, int lane, int u,
                                       bool turns, float *lds, float *co, float *si) {
  const double p = static_cast<double>(position);
  __builtin_amdgcn_wave_barrier();
  for (int i = lane; i < s.rot / 2; i += 64) {
    float sn, cs;
    sine_cosine(p * (static_cast<double>(inv_freq[i]) * 0.15915494309189535), sn, cs);
    lds[i] = cs;
    lds[kMaxPairs + i] = sn;
  }
  __builtin_amdgcn_wave_barrier();
  const int at = turns ? u * V : 0;  // (the result of a lane that does not turn is not used)
#pragma unroll
  for (int e = 0; e < V; ++e) {
    co[e] = lds[at + e];
    si[e] = lds[kMaxPairs + at + e];
  }
}

// (x0, x1) of one lane turned by its V angles.  Of a lane whose elements only pass the result is not
// used: times 1 and 0 an infinity or a NaN of one would reach the other, and a negative zero lose its sign.
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

constexpr int kJoin = 16;  // rows of partial sums that one workgroup adds
constexpr int kJoinLoads = kJoin * kQkMaxDim / kBwdThreads;  // of a thread, for the longest rows
constexpr int kSC1 = 16;       // buffer cache policy: agent-coherent access

// Sum over the `lanes` lanes of a head (a power of two, the same for the whole launch), known
// to all of them: neighbours within 16 lanes by data-parallel moves, then rows of 16.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xF, 0xF, true));
}
// The sum of each lane with its partner 16 (32) lanes away.
template <int STEP>
__device__ __forceinline__ float rows_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  uint32_t a, b;
  if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    a = r[0], b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    a = r[0], b = r[1];
  }
  return __uint_as_float(a) + __uint_as_float(b);
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  if (lanes > 1) v += moved<0xB1>(v);   // lanes 1 0 3 2
  if (lanes > 2) v += moved<0x4E>(v);   // lanes 2 3 0 1
  if (lanes > 4) v += moved<0x141>(v);  // mirrored within 8
  if (lanes > 8) v += moved<0x140>(v);  // mirrored within 16
  if (lanes > 16) v = rows_sum<16>(v);
  if (lanes > 32) v = rows_sum<32>(v);
  return v;
}
// The same in 64 bits, for the weights' gradients: two values at a time.  Lanes 0 to 31 (STEP 16: the even
// rows of 16) get a's sum over the partner lanes, the others b's.
template <int STEP>
__device__ __forceinline__ double two_sums(double a, double b) {
  const uint64_t ua = __builtin_bit_cast(uint64_t, a), ub = __builtin_bit_cast(uint64_t, b);
  uint64_t x = 0, y = 0;
#pragma unroll
  for (int k = 0; k < 64; k += 32) {
    const uint32_t wa = static_cast<uint32_t>(ua >> k), wb = static_cast<uint32_t>(ub >> k);
    if constexpr (STEP == 16) {
      const auto r = __builtin_amdgcn_permlane16_swap(wa, wb, false, false);
      x |= static_cast<uint64_t>(r[0]) << k, y |= static_cast<uint64_t>(r[1]) << k;
    } else {
      const auto r = __builtin_amdgcn_permlane32_swap(wa, wb, false, false);
      x |= static_cast<uint64_t>(r[0]) << k, y |= static_cast<uint64_t>(r[1]) << k;
    }
  }
  return __builtin_bit_cast(double, x) + __builtin_bit_cast(double, y);
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u), CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Sum over the lanes of a row of 16 that are a multiple of `lanes` apart.
__device__ __forceinline__ double row_sum(double v, int lanes) {
  if (lanes <= 1) v += moved<0x121>(v);  // the row turned by 1, 2, 4, 8
  if (lanes <= 2) v += moved<0x122>(v);
  if (lanes <= 4) v += moved<0x124>(v);
  if (lanes <= 8) v += moved<0x128>(v);
  return v;
}
// 1 / sqrt(mean + eps): the hardware's reciprocal root is within a unit in the last place; its
// argument may not be subnormal, which only a zero eps allows (scaled by 2^48 then).
__device__ __forceinline__ float inverse_rms(float sum, const QkShape &s) {
  const float m = sum * s.inv_d + s.eps;
  return m < 0x1p-100f ? __builtin_amdgcn_rsqf(m * 0x1p48f) * 0x1p24f : __builtin_amdgcn_rsqf(m);
}

// A choice of values: the operator's own is one of places where both sides are variables, which
// keeps what a lambda captures in memory.
template <typename T>
__device__ __forceinline__ T pick(bool first, T a, T b) {
  return first ? a : b;
}

// A wave's work: rounds of 64 / lanes heads of one token.  The q heads' rounds come first, then
// the k heads' (then, backward, the v heads'); a round never holds heads of two kinds, so what a
// head is is the same for the whole wave.
struct Rounds {
  int heads_per, q, k, total;
  __device__ __forceinline__ Rounds(const QkShape &s, bool with_v) {
    heads_per = 64 / s.lanes;
    q = (s.nq + heads_per - 1) / heads_per;
    k = (s.nk + heads_per - 1) / heads_per;
    total = q + (with_v ? 2 * k : k);
  }
};

// STREAM: queries and keys larger than the L2s together are stored past them (2048 tokens of 64 + 64
// heads of 128, 67 MB: 20.6 us, 6.5 TB/s; 24.3 through them).  The backward gains nothing by it.
template <bool T16, int V, bool INTER, bool STREAM>
__global__ __launch_bounds__(kThreads) void qk_fwd_kernel(const void *__restrict__ Y, QkShape s,
                                                          const int64_t *__restrict__ positions,
                                                          const float *__restrict__ inv_freq,
                                                          const void *__restrict__ qw, const void *__restrict__ kw,
                                                          void *__restrict__ Q, void *__restrict__ K) {
  __shared__ float lds[kWaves][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = lane & (s.lanes - 1), sub = lane / s.lanes;
  const Unit un = unit_of<V, INTER>(u, s);
  const Rounds R(s, false);
  const bool norm = qw != nullptr;
  using B = Both<T16, V>;
  B wq, wk;
  wq.load(qw, 0, un, norm);
  wk.load(kw, 0, un, norm);
  const int64_t tasks = s.M * s.split, step = static_cast<int64_t>(gridDim.x) * kWaves;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(wave); task < tasks;
       task += step) {
    const int64_t m = task / s.split;
    const int first = static_cast<int>(task - m * s.split) * s.per, last = min(first + s.per, R.total);
    // head of this lane in a round: of q or k, and among the row's
    auto load = [&](B &x, int r) {
      const bool is_q = r < R.q;
      const int h = (is_q ? r : r - R.q) * R.heads_per + sub;
      x.load(Y, m * s.row + static_cast<int64_t>(is_q ? h : s.nq + h) * s.d, un, h < pick(is_q, s.nq, s.nk));
    };
    B next;
    load(next, first);
    float co[V], si[V];
    angles<V>(positions[m], inv_freq, s, lane, u, un.turns, lds[wave], co, si);
    for (int r = first; r < last; ++r) {
      B x = next;
      if (r + 1 < last) load(next, r + 1);
      const bool is_q = r < R.q;
      const int h = (is_q ? r : r - R.q) * R.heads_per + sub, heads = pick(is_q, s.nq, s.nk);
      float v[2 * V];
      x.values(v);
      if (norm) {
        float sq = 0.0f, w[2 * V];
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) sq = __builtin_fmaf(v[e], v[e], sq);
        const float rms = inverse_rms(lanes_sum(sq, s.lanes), s);
        if (is_q)
          wq.values(w);
        else
          wk.values(w);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) v[e] = v[e] * rms * w[e];
      }
      if (un.turns) turn<V, INTER>(v, co, si, 1.0f);
      if (norm || un.turns) x.set(v);  // (else the bits as loaded: a conversion would quiet a NaN)
      if (h < heads) x.template store<STREAM>(pick(is_q, Q, K), (m * heads + h) * s.d, un);
    }
  }
}

// With a norm the waves of large workgroups sum the weights' gradients (few partial sums), in 64 bits: a
// sum over all tokens and heads in fp32 loses what its terms still hold.  The partial sums of 16
// workgroups are added by the last of them to finish, the groups' by the last group: a single workgroup
// would read all of them (512 KB for heads of 128) at one CU's rate (2048 tokens of 64 + 64 heads 57.3 us,
// 60.7 with one level; 1024 tokens of 32 + 8 heads of 256 22.4 and 30.0).  Two values a lane move
// (two_sums) instead of one took 333 tokens of 15 + 5 heads of 80 in fp32 from 13.6 to 12.2 us.  Without
// one nothing is summed, and the kernel is the forward's with the other sign and the v heads, on eight
// waves a SIMD (62 registers; with 65, and seven, 2048 tokens of 64 + 64 + 64 heads of 128 take 35.3 us
// instead of 34.3).
template <bool T16, int V, bool INTER, bool NORM>
__global__ __launch_bounds__(NORM ? kBwdThreads : kThreads, NORM ? 4 : 8) void qk_bwd_kernel(const void *__restrict__ dQ, const void *__restrict__ dK,
                                                          const void *__restrict__ dV, const void *__restrict__ Y,
                                                          QkShape s, const int64_t *__restrict__ positions,
                                                          const float *__restrict__ inv_freq,
                                                          const void *__restrict__ qw, const void *__restrict__ kw,
                                                          void *__restrict__ dY, void *__restrict__ dqw, void *__restrict__ dkw,
                                                          double *__restrict__ part, uint32_t *__restrict__ ticket) {
  constexpr int kW = NORM ? kBwdWaves : kWaves;
  __shared__ float lds[kW][2 * kMaxPairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = lane & (s.lanes - 1), sub = lane / s.lanes;
  const Unit un = unit_of<V, INTER>(u, s);
  const Rounds R(s, true);
  using B = Both<T16, V>;
  B wq, wk;
  wq.load(qw, 0, un, NORM);
  wk.load(kw, 0, un, NORM);
  double dwq[2 * V], dwk[2 * V];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) dwq[e] = dwk[e] = 0.0;
  const int64_t tasks = s.M * s.split, step = static_cast<int64_t>(gridDim.x) * kW;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kW + __builtin_amdgcn_readfirstlane(wave); task < tasks;
       task += step) {
    const int64_t m = task / s.split;
    const int first = static_cast<int>(task - m * s.split) * s.per, last = min(first + s.per, R.total);
    auto head = [&](int r) __attribute__((always_inline)) { return (r < R.q ? r : r < R.q + R.k ? r - R.q : r - R.q - R.k) * R.heads_per + sub; };
    auto row_at = [&](int r, int h) __attribute__((always_inline)) {
      return m * s.row + static_cast<int64_t>(r < R.q ? h : r < R.q + R.k ? s.nq + h : s.nq + s.nk + h) * s.d;
    };
    auto load = [&](B &g, B &x, int r) __attribute__((always_inline)) {
      const int h = head(r), heads = pick(r < R.q, s.nq, s.nk);
      g.load(pick(r < R.q, dQ, pick(r < R.q + R.k, dK, dV)), (m * heads + h) * s.d, un, h < heads);
      x.load(Y, row_at(r, h), un, NORM && r < R.q + R.k && h < heads);
    };
    B next_g, next_x;
    load(next_g, next_x, first);
    float co[V], si[V];
    angles<V>(positions[m], inv_freq, s, lane, u, un.turns, lds[wave], co, si);
    // one round of q or k heads; the gradients of w are summed in dw.  on: this lane has a head (with a
    // zero eps the root of another's zeros is infinite, and its product with them NaN)
    auto round = [&](B &g, const B &x, const B &weight, double *dw, bool on) __attribute__((always_inline)) {
      float v[2 * V];
      g.values(v);
      if (!NORM || un.turns) turn<V, INTER>(v, co, si, -1.0f);
      if constexpr (NORM) {
        float xv[2 * V], w[2 * V], sq = 0.0f, gx = 0.0f;
        x.values(xv);
        weight.values(w);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
          sq = __builtin_fmaf(xv[e], xv[e], sq);
          gx = __builtin_fmaf(v[e] * w[e], xv[e], gx);
        }
        sq = lanes_sum(sq, s.lanes);
        gx = lanes_sum(gx, s.lanes);
        const float r = on ? inverse_rms(sq, s) : 0.0f, back = r * r * (gx * s.inv_d);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
          dw[e] += static_cast<double>(v[e] * r * xv[e]);
          v[e] = r * (v[e] * w[e] - xv[e] * back);
        }
      }
      if constexpr (NORM) {
        g.set(v);
      } else {  // (by a choice of words: with a branch around it 40.1 us instead of 39.0, interleaved)
        B turned;
        turned.set(v);
        g.take(turned, un.turns);
      }
    };
    for (int r = first; r < last; ++r) {
      B g = next_g, x = next_x;
      if (r + 1 < last) load(next_g, next_x, r + 1);
      const int h = head(r);
      const bool on = h < pick(r < R.q, s.nq, s.nk);
      if (r < R.q)
        round(g, x, wq, dwq, on);
      else if (r < R.q + R.k)
        round(g, x, wk, dwk, on);
      if (on) g.template store<false>(dY, row_at(r, h), un);
    }
  }
  if constexpr (NORM) {

    // the wave's sums over its heads, then the workgroup's over its waves, in a fixed order
    __shared__ __attribute__((aligned(16))) double dw[kBwdWaves][2][kQkMaxDim];
    auto put = [&](const double *v, int weight, bool second) {
      if (second ? un.has1 : un.has0)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[wave][weight][(second ? un.o1 : un.o0) + e] = v[e];
    };
    if (s.lanes == 64) {
      put(dwq, 0, false), put(dwq + V, 0, true), put(dwk, 1, false), put(dwk + V, 1, true);
    } else {
      double v[2 * V];  // (lanes 32 on: dkw)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) v[e] = two_sums<32>(dwq[e], dwk[e]);
      if (s.lanes == 32) {
        put(v, lane / 32, false), put(v + V, lane / 32, true);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)  // (odd rows of 16 lanes: the second chunk)
          v[e] = row_sum(two_sums<16>(v[e], v[V + e]), s.lanes);
        if (lane % 16 < s.lanes) put(v, lane / 32, lane / 16 % 2);
      }
    }
    __syncthreads();
    // Partial sums leave as rows of `cols`, two columns a thread: those of the workgroups, then those of
    // groups of kJoin of them; agent-coherent (SC1: the L2 of one XCD is not coherent with the others).
    const int cols = 2 * s.d, pairs = s.d, first_pair = 2 * static_cast<int>(threadIdx.x);
    const uint32_t groups = (gridDim.x + kJoin - 1) / kJoin, group = blockIdx.x / kJoin;
    const __amdgpu_buffer_rsrc_t P = make_rsrc(part, (gridDim.x + groups) * cols * 8u);
    auto leave = [&](f64x2_t v, uint32_t row) {
      const uint32_t at = (row * cols + first_pair) * 8u;
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), P, at, 0, kSC1);
    };
    // Whether this workgroup is the last of n to leave its sums, which have completed before the ticket
    // is taken: so whoever takes the last ticket sees them all.
    __shared__ uint32_t taken;
    auto last_of = [&](uint32_t *t, uint32_t n) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (threadIdx.x == 0) taken = __hip_atomic_fetch_add(t, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      const bool last = taken == n - 1;
      if (last && threadIdx.x == 0) __hip_atomic_store(t, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return last;
    };
    // The sums of n <= kJoin rows, known to the first `pairs` threads: slices of the workgroup add every
    // slices-th row each, the slices are added in their order.
    auto join = [&](uint32_t first, uint32_t n) {
      double *sums = &dw[0][0][0];
      const uint32_t slices = kBwdThreads / pairs, slice = threadIdx.x / pairs, col = 2 * (threadIdx.x - slice * pairs);
      u32x4_t t[kJoinLoads];
#pragma unroll
      for (int e = 0; e < kJoinLoads; ++e) {
        const uint32_t row = slice + e * slices;  // past the last: zeros
        t[e] = __builtin_amdgcn_raw_buffer_load_b128(
            P, slice < slices && row < n ? ((first + row) * cols + col) * 8u : kOOB, 0, kSC1);
      }
      f64x2_t v = {0.0, 0.0};
#pragma unroll
      for (int e = 0; e < kJoinLoads; ++e) v += __builtin_bit_cast(f64x2_t, t[e]);
      if (slice < slices) *reinterpret_cast<f64x2_t *>(sums + slice * cols + col) = v;
      __syncthreads();
      if (threadIdx.x < pairs) {
        v = *reinterpret_cast<const f64x2_t *>(sums + first_pair);
        for (uint32_t k = 1; k < min(slices, n); ++k)
          v += *reinterpret_cast<const f64x2_t *>(sums + k * cols + first_pair);
      }
      return v;
    };
    const int which = first_pair >= s.d, o = which ? first_pair - s.d : first_pair;
    if (threadIdx.x < pairs) {
      f64x2_t v = *reinterpret_cast<const f64x2_t *>(&dw[0][which][o]);
      for (int k = 1; k < kBwdWaves; ++k) v += *reinterpret_cast<const f64x2_t *>(&dw[k][which][o]);
      leave(v, blockIdx.x);
    }
    const uint32_t members = min(gridDim.x - group * kJoin, static_cast<uint32_t>(kJoin));
    if (!last_of(ticket + 1 + group, members)) return;
    f64x2_t v = join(group * kJoin, members);
    if (groups > 1) {
      if (threadIdx.x < pairs) leave(v, gridDim.x + group);
      if (!last_of(ticket, groups)) return;
      v = join(gridDim.x, groups);
    }
    if (threadIdx.x < pairs) {
      const float a = static_cast<float>(v[0]), b = static_cast<float>(v[1]);
      void *out = pick(which != 0, dkw, dqw);
      if constexpr (T16)
        static_cast<uint32_t *>(out)[o / 2] = pack_bf16x2(a, b);
      else
        static_cast<f32x2_t *>(out)[o / 2] = f32x2_t{a, b};
    }
  }
}

// Elements of a lane's chunk: the widest access that divides the head and half the rotated part, of
// up to 16 bytes.  The backward with a norm (sums) stops at 8 bytes (4 of bf16): with 16 a lane holds
// twice the values and half as many waves fit (2048 tokens of 64 + 64 + 64 heads of 128: 50.5 us with
// 8 bytes, 59.4 with 16, the sums in fp32 as they were then; forward 28.0 and 24.5).
int chunk_of(const QkShape &s, bool t16, bool sums) {
  int v = t16 && !sums ? 8 : 4;
  while (v > 2 && (s.d % v != 0 || s.rot % (2 * v) != 0)) v /= 2;
  return v;
}

// Lanes of a head, and how a token's rounds are split over waves: enough of them to fill the card
// (eight a SIMD, four of the backward with a norm, where a wave holds more), and no more, since each
// computes the token's angles.
constexpr int64_t kFwdWaves = 1024 * 8, kBwdAllWaves = 1024 * 4;
void plan(QkShape *s, int v, bool with_v, bool sums) {
  const int units = (s->d + 2 * v - 1) / (2 * v);
  s->lanes = 1;
  while (s->lanes < units) s->lanes *= 2;
  const int heads_per = 64 / s->lanes;
  const int rounds = (s->nq + heads_per - 1) / heads_per + (with_v ? 2 : 1) * ((s->nk + heads_per - 1) / heads_per);
  int64_t split = ((sums ? kBwdAllWaves : kFwdWaves) + s->M - 1) / s->M;
  if (split > rounds) split = rounds;
  s->per = static_cast<int>((rounds + split - 1) / split);
  s->split = (rounds + s->per - 1) / s->per;
  s->row = static_cast<int64_t>(s->nq + 2 * s->nk) * s->d;
  s->inv_d = 1.0f / static_cast<float>(s->d);
}
int64_t workgroups(const QkShape &s, int waves, int64_t most) {
  const int64_t wgs = (s.M * s.split + waves - 1) / waves;
  return wgs < most ? wgs : most;
}
// The backward's workgroups each leave partial sums, so no more than are on the card at once.
constexpr int64_t kFwdWorkgroups = 256 * 16, kBwdWorkgroups = 256;
static_assert(kBwdWorkgroups <= kJoin * kJoin, "two levels join them all");

}  // namespace

size_t qk_bwd_workspace(QkShape s, bool t16, bool norm) {
  if (!norm) return 0;
  plan(&s, chunk_of(s, t16, true), true, true);
  const int64_t wgs = workgroups(s, kBwdWaves, kBwdWorkgroups);
  return static_cast<size_t>(wgs + (wgs + kJoin - 1) / kJoin) * 2 * s.d * sizeof(double);
}

hipError_t launch_qk_fwd(const void *Y, QkShape s, bool t16, bool interleaved, const int64_t *positions,
                         const float *inv_freq, const void *qw, const void *kw, void *Q, void *K,
                         hipStream_t stream) {
  const int v = chunk_of(s, t16, false);
  plan(&s, v, false, false);
  const dim3 grid(static_cast<unsigned>(workgroups(s, kWaves, kFwdWorkgroups))), block(kThreads);
  const bool stream_out = s.M * (s.nq + s.nk) * s.d * (t16 ? 2 : 4) > (int64_t(32) << 20);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, Y, s, positions, inv_freq, qw, kw, Q, K);
    return hipGetLastError();
  };
#define QLORA_FWD(t16, v, inter) \
  return stream_out ? launch(qk_fwd_kernel<t16, v, inter, true>) : launch(qk_fwd_kernel<t16, v, inter, false>);
  switch ((t16 ? 100 : 0) + 10 * v + (interleaved ? 1 : 0)) {
    case 180: QLORA_FWD(true, 8, false)
    case 181: QLORA_FWD(true, 8, true)
    case 140: QLORA_FWD(true, 4, false)
    case 141: QLORA_FWD(true, 4, true)
    case 120: QLORA_FWD(true, 2, false)
    case 121: QLORA_FWD(true, 2, true)
    case 40: QLORA_FWD(false, 4, false)
    case 41: QLORA_FWD(false, 4, true)
    case 20: QLORA_FWD(false, 2, false)
    default: QLORA_FWD(false, 2, true)
  }
#undef QLORA_FWD
}

hipError_t launch_qk_bwd(const void *dQ, const void *dK, const void *dV, const void *Y, QkShape s, bool t16,
                         bool interleaved, const int64_t *positions, const float *inv_freq, const void *qw,
                         const void *kw, void *dY, void *dqw, void *dkw, double *part, uint32_t *ticket,
                         hipStream_t stream) {
  const bool norm = qw != nullptr;
  const int v = chunk_of(s, t16, norm);
  plan(&s, v, true, norm);
  const int64_t wgs = norm ? workgroups(s, kBwdWaves, kBwdWorkgroups) : workgroups(s, kWaves, kFwdWorkgroups);
  const dim3 grid(static_cast<unsigned>(wgs)), block(norm ? kBwdThreads : kThreads);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, dQ, dK, dV, Y, s, positions, inv_freq, qw, kw, dY, dqw, dkw,
                       part, ticket);
    return hipGetLastError();
  };
#define QLORA_BWD(t16, v, inter) \
  return norm ? launch(qk_bwd_kernel<t16, v, inter, true>) : launch(qk_bwd_kernel<t16, v, inter, false>);
  switch ((t16 ? 100 : 0) + 10 * v + (interleaved ? 1 : 0)) {
    case 180: return launch(qk_bwd_kernel<true, 8, false, false>);
    case 181: return launch(qk_bwd_kernel<true, 8, true, false>);
    case 140: QLORA_BWD(true, 4, false)
    case 141: QLORA_BWD(true, 4, true)
    case 120: QLORA_BWD(true, 2, false)
    case 121: QLORA_BWD(true, 2, true)
    case 40: QLORA_BWD(false, 4, false)
    case 41: QLORA_BWD(false, 4, true)
    case 20: QLORA_BWD(false, 2, false)
    default: QLORA_BWD(false, 2, true)
  }
#undef QLORA_BWD
}

}  // namespace qlora
