// Internal declarations shared by the host API and the kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlora {

constexpr int kBlock = 64;     // weights per first-level block
constexpr int kGroup = 256;    // block constants per double-quantization group
constexpr int kBuckets = 129;  // quantizer bucket table entries (x in [-1, 1])
constexpr int kMaxRank = 256;  // largest LoRA rank
// Bytes at the start of every workspace layout reserved for the small-M forward's
// cross-workgroup counters; no other kernel writes them.
constexpr size_t kGemvSyncBytes = 256 + 4096 * 16;  // QLORA_WORKSPACE_HEADER_BYTES

// Level tables of the 4-bit codes and encodings of the block constants (the values
// of the weight descriptor's quant_type and const_type).
enum : int { kQuantNF4 = 0, kQuantFP4 = 1 };
enum : int { kConstDqInt8 = 0, kConstDqFp8 = 1, kConstF32 = 2 };

struct Codebook {
  float q[16];                  // levels, ascending
  float thr[15];                // decision thresholds
  float bucket_thr[kBuckets];   // the threshold inside each bucket window (2.0 if none)
  int bucket_base[kBuckets];    // thresholds below each bucket window
  bool bucket_ok;               // every window holds at most one threshold
};

// kQuantNF4 or kQuantFP4 (any other value: NF4).
const Codebook &codebook(int quant_type = kQuantNF4);

// Kernel arguments passed by value (kernarg segment).
struct QuantTable {
  float thr[kBuckets];
  int base[kBuckets];
};
struct LevelTable {
  float q[16];
};
LevelTable level_table(int quant_type);

// Device view of a quantized weight.  Double-quantized constants (kConstDqInt8,
// kConstDqFp8) use absmax_q / dq_scale / dq_offset; kConstF32 uses absmax.
struct WeightView {
  const uint8_t *codes;
  const int8_t *absmax_q;
  const float *dq_scale;
  const float *dq_offset;
  int64_t n_rows;  // N = d_out
  int64_t n_cols;  // K = d_in
  const float *absmax;
  int quant_type;
  int const_type;
};

// Dropout from a counter-based generator (drop_words in device_common.h): an element is
// kept when its 16 bits are >= thr; thr == 0: no dropout.  `counter` (nullable) is a
// device word added to the offset when the kernel runs.
struct Dropout {
  uint32_t thr, k0, k1;
  uint64_t offset;
  const uint64_t *counter;
};

// Activations of the gated projections (the header's qlora_act values).
enum : int { kActSilu = 0, kActGeluTanh = 1 };

// ---- launchers (each returns the HIP error of its launches) -----------------
// out = x c m of n elements (n >= 1): bf16 or fp32.
hipError_t launch_dropout(const void *X, bool bf16, int64_t n, const Dropout &d, float c, void *out,
                          hipStream_t stream);
// One row of a copy job: `rows` rows of `cols` bf16 values from src (row pitch lds) to dst
// (row pitch ldd); dst columns cols .. dcols - 1 are cleared.  launch_copy_rows runs all
// jobs of the list (at most kMaxCopyJobs, rows == 0 skipped) in one launch.
struct CopyJob {
  const uint16_t *src;
  uint16_t *dst;
  int64_t rows, cols, dcols, lds, ldd;
};
constexpr int kMaxCopyJobs = 4;
hipError_t launch_copy_rows(const CopyJob *jobs, int n, hipStream_t stream);
// absmax_f32 receives the fp32 block constants (required for kConstF32, optional
// otherwise); absmax_q / dq_scale / dq_offset are written for the double-quantized types.
hipError_t launch_quantize(const void *W, bool w_bf16, int64_t n_rows, int64_t n_cols, int quant_type,
                           int const_type, uint8_t *codes, int8_t *absmax_q, float *dq_scale,
                           float *dq_offset, float *absmax_f32, hipStream_t stream);
hipError_t launch_dequantize(const WeightView &w, void *out, bool out_bf16, hipStream_t stream);

// OUT[M, r] (row pitch ldout, bf16) = bf16(scale * IN[M, Kc] . WT[r, Kc]^T);  IN rows
// have pitch ldin, WT rows pitch ldwt (column slices of wider matrices are allowed).
// `ws` holds lora_down_workspace(M, Kc, r) bytes of fp32 partial sums.
size_t lora_down_workspace(int64_t M, int64_t Kc, int r);
// A rank padded with zeros: parts of `width` columns, of which the first `live` are the rank's
// own and the others of OUT are set to zero (live = width: none padded).
struct RankPad {
  int width = 0, live = 0;
};
hipError_t launch_lora_down(const uint16_t *IN, int64_t M, int64_t Kc, int64_t ldin, const uint16_t *WT,
                            int64_t ldwt, int r, float scale, uint16_t *OUT, int64_t ldout, float *ws,
                            hipStream_t stream, RankPad pad = {});
// The same with the dropout mask on IN, a dense [M, Kc] tensor: OUT = bf16(scale (m IN) WT^T).
// Needs r % 8 == 0 and the fast-path shapes (drop_shape_ok).
hipError_t launch_lora_down_drop(const uint16_t *IN, int64_t M, int64_t Kc, const uint16_t *WT, int r, float scale,
                                 uint16_t *OUT, float *ws, const Dropout &d, hipStream_t stream, RankPad pad = {});
bool drop_shape_ok(int64_t M, int64_t Kc, int r);
// OUT_q[C_q, R_q] = IN_q[R_q, C_q]^T for two bf16 matrices (dense row-major) in one
// launch; IN1 may be NULL (one transpose).
hipError_t launch_transpose2_bf16(const uint16_t *IN0, int64_t R0, int64_t C0, uint16_t *OUT0, const uint16_t *IN1,
                                  int64_t R1, int64_t C1, uint16_t *OUT1, hipStream_t stream);
// The last pass of a split reduction: OUT = bf16(scale * (P_0 + P_1 + ...)) for the
// `count` partial sums of each of `splits` splits (count % 4 == 0), laid out as rows of
// `cols` values written with row pitch ldout.  splits == 0: nothing to do.
struct FinalizeJob {
  const float *P;
  int splits;
  int64_t count, cols, ldout;
  float scale;
  uint16_t *OUT;
};
// Workgroups of 256 threads a finalize job is spread over when it rides in another
// launch (the dX GEMM's); finalize_part (device_common.h) does one workgroup's share.
inline int64_t finalize_workgroups(const FinalizeJob &j) {
  if (j.splits <= 0) return 0;
  const int64_t w = (j.count / 4 + 4 * 256 - 1) / (4 * 256);  // four groups of four values per thread
  return w < 1 ? 1 : w;
}

// P[s][No][r] fp32 partials of sum over m in split s of IN[m][no] * S[m][j]; then
// OUT = bf16(sum_s P) written as [No, r] (trans_out = false) or [r, No] (true).
// IN rows have pitch ldin, S rows pitch lds.  If `defer` is not NULL and the fast path
// runs, the finalize pass is not launched but described in *defer (else defer->splits
// is 0), for a later launch to do.
size_t reduce_m_workspace(int64_t M, int64_t No, int r);
hipError_t launch_reduce_m(const uint16_t *IN, int64_t M, int64_t No, int64_t ldin, const uint16_t *S,
                           int64_t lds, int r, float *partials, uint16_t *OUT, bool trans_out,
                           hipStream_t stream, FinalizeJob *defer = nullptr);
// dA [r, Kc] = bf16((V + V_lo)^T (m IN)) with the dropout mask on IN, a dense [M, Kc] tensor
// (drop.thr = 0: none); V dense [M, r], V_lo `lo` elements (a multiple of 8) behind it.
// V's rounding to bf16 would be as large an error of dA as its own last one, so what it
// takes off is multiplied too: X is read once for both, and the second product costs 3 us
// (4096 x 4096, rank 64: 18.8 us, 16.0 with V alone; rank 128: 27.2, 24.4).  pair_shape_ok:
// the shapes it takes.
size_t reduce_pair_workspace(int64_t M, int64_t Kc, int r);
bool pair_shape_ok(int64_t M, int64_t Kc, int r, int64_t lo);
hipError_t launch_reduce_pair(const uint16_t *IN, int64_t M, int64_t Kc, const uint16_t *V, int64_t lo, int r,
                              float *partials, uint16_t *OUT, const Dropout &d, hipStream_t stream,
                              FinalizeJob *defer);

// The backward's two products over dY in one launch plus one finalize launch:
// V[M, r] (row pitch ldu) = bf16(scale dY B) and dB[Np, r] = bf16(dY^T U), where dY has
// row pitch ldy (a column slice of width Np), B is [Np, r] (dense rows) and U [M, r]
// with row pitch ldu.  If A and At are given, the same launch also writes At[KA, RA] =
// A[RA, KA]^T.  Needs the fast-path shapes (vdb_fast) and the two fp32 partial regions
// sized by vdb_workspace_v / vdb_workspace_db.  vdb_fast's `padded`: dY's rows hold zeros in
// columns Np .. round_up(Np, 8) - 1 of the slice, and Np need not be a multiple of 8
// (launch_vdb_parts).
bool vdb_fast(int64_t M, int64_t Np, int64_t ldy, int64_t ldu, int r, bool padded = false);
size_t vdb_workspace_v(int64_t M, int64_t Np, int r);
size_t vdb_workspace_db(int64_t M, int64_t Np, int r);
hipError_t launch_vdb(const uint16_t *dY, int64_t M, int64_t Np, int64_t ldy, const uint16_t *B, const uint16_t *U,
                      int64_t ldu, int r, float scale, uint16_t *V, uint16_t *dB, float *ws_v, float *ws_db,
                      const uint16_t *A, int64_t RA, int64_t KA, uint16_t *At, hipStream_t stream);

// launch_vdb for `parts` stacked parts at once (one launch and one finalize): part q's dY
// columns are [q ldp, q ldp + Np) of rows of pitch ldy (zeros up to the next multiple of 8),
// B [parts Np, r], U and V [M, parts r], dB [parts Np, r]; the partial regions are `parts`
// times vdb_workspace_v / vdb_workspace_db; At[KA, parts r] = A^T if both are given.  What
// V's rounding took off goes, rounded in its turn, to the matrix `lo` elements behind V.  V's
// columns from `live` on pad the rank and are set to zero (live = r: none).
hipError_t launch_vdb_parts(int parts, const uint16_t *dY, int64_t M, int64_t Np, int64_t ldp, int64_t ldy,
                            const uint16_t *B, const uint16_t *U, int r, float scale, uint16_t *V, int64_t lo,
                            uint16_t *dB, float *ws_v, float *ws_db, const uint16_t *A, int64_t KA, uint16_t *At,
                            int live, hipStream_t stream);

// AdamW step (fp32 parameter and moments, bf16 gradient, optional bf16 parameter copy).
struct AdamConsts {
  float decay, b1, ob1, b2, ob2, step_size, bc2s, eps;
};
hipError_t launch_adamw(float *p, uint16_t *pb, const uint16_t *g, float *m, float *v, int64_t n,
                        const AdamConsts &c, hipStream_t stream);

// LoRA merge / unmerge of one adapter into a bf16 weight [N, K]:
// out = bf16(W' + scale . B A) from the NF4 weight, or bf16(Wm - scale . B A).
hipError_t launch_lora_merge(const WeightView &w, const uint16_t *A, const uint16_t *B, int r,
                             float scale, uint16_t *out, hipStream_t stream);
hipError_t launch_lora_unmerge(const uint16_t *Wm, int64_t n_rows, int64_t n_cols, const uint16_t *A,
                               const uint16_t *B, int r, float scale, uint16_t *out,
                               hipStream_t stream);

// Whether the fused GEMMs take this shape: X or dY, Y or dX, the codes and the LoRA
// operands (rank or row pitch r) below 0xFFFFFFF0 bytes each (32-bit buffer offsets).
bool gemm_supported(const WeightView &w, int64_t M, int r);
// Y[M, N] = bf16(X . W'^T + U . Bl^T)  (U [M, r] pitch ldu, Bl [N, r]); r may be 0.
// part_rows > 0 (a multiple of 256 dividing N): output rows of part q = n / part_rows
// use U columns [q r, q r + r) (horizontally fused linears with stacked adapters).
hipError_t launch_gemm_fwd(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U,
                           int ldu, const uint16_t *Bl, int r, int64_t part_rows, uint16_t *Y,
                           hipStream_t stream);
// Small-M forward (M <= 16) in one launch: Y = bf16(X W'^T + U_s Bl^T) and
// U_s = bf16(scale X A^T) (written to U_saved if not NULL) over the R stacked ranks of
// A; output row n uses U_s columns [q r, q r + r), q = n / part_rows (part_rows = 0:
// one linear, R = r).  `ws` holds gemv_workspace bytes: a kGemvSyncBytes header of
// counters and flags that must be zero when the call starts (every call leaves it
// zero), then copies of U_s and the partial sums of the down-projection.
// The small-M forward runs for M <= 16, up to 4096 tiles of 16 output rows (one flag word per
// workgroup in the header) and rows of up to 15 x 256 blocks (256 for each of a workgroup's weight
// waves); other shapes take the fused GEMM.
inline bool gemv_shape_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 1 && M <= 16 && (N + 15) / 16 <= 4096 && K <= 15 * 256 * 64;
}
size_t gemv_workspace(int64_t M, int64_t K, int64_t N, int r);
bool gemv_supported(const WeightView &w, int64_t M, int r);
hipError_t launch_gemv(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *A, int R,
                       const uint16_t *Bl, int r, int64_t part_rows, float scale, uint16_t *Y,
                       uint16_t *U_saved, void *ws, hipStream_t stream);
// Its extensions: the dropout mask on X ahead of the adapter (drop.thr > 0), and the gated
// projections (H not NULL: H[M, P] = bf16(act(G) L), Y NULL or receiving [G | L]; r is each
// projection's rank, A [2 r, K], part_rows unused).  gemv_ext_workspace holds for both.
struct GemvExt {
  Dropout drop;
  uint16_t *H;
  int act;
};
size_t gemv_ext_workspace(int64_t M, int64_t K, int64_t N, int r, int parts);
hipError_t launch_gemv_ext(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *A, int R,
                           const uint16_t *Bl, int r, int64_t part_rows, float scale, uint16_t *Y, uint16_t *U_saved,
                           void *ws, const GemvExt &x, hipStream_t stream);
// dX[M, K] = bf16(dY . W' + V . At^T)  (V [M, r], At [K, r]); r may be 0.  A finalize
// job (NULL or splits == 0: none) runs in extra workgroups after the GEMM's tiles.
hipError_t launch_gemm_dx(const WeightView &w, const uint16_t *dY, int64_t M, const uint16_t *V,
                          const uint16_t *At, int r, uint16_t *dX, hipStream_t stream,
                          const FinalizeJob *fin = nullptr);
// Gated projections: weight rows [0, P) are the gate's, [P, 2 P) the up projection's
// (P = n_rows / 2), U [M, 2 r] (pitch ldu) and Bl [2 P, r] their stacked adapter operands.
// H[M, P] = bf16(act(G) L) for [G | L] = X W'^T + U Bl^T before any rounding; Y, if not
// NULL, receives bf16 [G | L] [M, 2 P].
hipError_t launch_gemm_gated(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U, int ldu,
                             const uint16_t *Bl, int r, int act, uint16_t *H, uint16_t *Y, hipStream_t stream);
// The same two forwards on tiles of 128 weight rows, with the contraction split when the
// tiles are few (`part`: gemm_mid_workspace bytes): Y [M, N] as launch_gemm_fwd, or (gated)
// H and Y as launch_gemm_gated.  r % 8 == 0.
// mid_takes: whether this shape runs on them (else on the 256 x 256 tiles).
bool mid_takes(int64_t M, int64_t K, int64_t N, bool gated);
// gemv_takes: whether a small-M call with dropout or gate runs on launch_gemv_ext (else on
// the above).
bool gemv_takes(int64_t M, int64_t K, int64_t N, int r, bool gated);
size_t gemm_mid_workspace(int64_t M, int64_t K, int64_t N, bool gated);
hipError_t launch_gemm_mid(const WeightView &w, const uint16_t *X, int64_t M, const uint16_t *U, int ldu,
                           const uint16_t *Bl, int r, int64_t part_rows, bool gated, int act, uint16_t *H, uint16_t *Y,
                           float *part, hipStream_t stream);
// [dG | dL] = [dH L act'(G) | dH act(G)] from the saved bf16 [G | L] (Y [M, 2 P]), as bf16
// rows of two column blocks of round_up(P, 8) columns, zeros in the padding.
hipError_t launch_gated_grad(const uint16_t *dH, const uint16_t *Y, int64_t M, int64_t P, int act, uint16_t *dY,
                             hipStream_t stream);
// The same with the dropout mask of X on the LoRA term, dX = bf16(dY . W' + m (V . At^T)),
// and with dY given in `parts` column blocks of round_up(Np, 8) columns each (Np = N /
// parts; the padding columns hold zeros), so that odd part heights keep 16-byte rows.  `part`
// holds gemm_dx_ext_workspace(M, K, parts round_up(Np, 8)) bytes: with few output tiles the
// contraction is split and a second launch joins the fp32 partial sums in a fixed order.
size_t gemm_dx_ext_workspace(int64_t M, int64_t K, int64_t Kc);
hipError_t launch_gemm_dx_ext(const WeightView &w, const uint16_t *dY, int64_t M, int parts, const uint16_t *V,
                              const uint16_t *At, int r, uint16_t *dX, const Dropout &d, float *part,
                              hipStream_t stream, const FinalizeJob *fin);

// The same product on smaller tiles (dx_mid.hip), which launch_gemm_dx_ext takes where its own
// are estimated to take longer: dY [M, Kc] with the padding described by half and skip (DxExt
// in gemm.hip); estimated time in us; bytes of partial sums.
double dx_mid_cost(int64_t M, int64_t K, int64_t Kc);
size_t dx_mid_workspace(int64_t M, int64_t K, int64_t Kc);
hipError_t launch_dx_mid(const WeightView &w, const uint16_t *dY, int64_t M, int64_t Kc, int64_t half, int64_t skip,
                         const uint16_t *V, const uint16_t *At, int r, uint16_t *dX, const Dropout &d, float *part,
                         hipStream_t stream, const FinalizeJob *fin);

// ---- weights with one scale for each group of a row's elements -----------------------
// Element k of row n has the value (code - zero) scale of group k / group of that row; zeros
// NULL: 8 everywhere.  n_cols is a multiple of group, group of 32, and n_cols <= kGroupMaxCols.
struct GroupView {
  const uint8_t *codes;
  const void *scales;
  const uint8_t *zeros;
  int64_t n_rows, n_cols, group;
  bool scale_bf16;
};
// group_magic(d): u / d = the high 32 bits of u group_magic(d), for 2 <= d <= u's largest value
// below 2^16 (the rounded-up 2^32 / d is less than d / 2^32 too large, times u less than one);
// rows of at most kGroupMaxCols columns hold that many units of 4 columns or more.
constexpr int64_t kGroupMaxCols = int64_t(1) << 18;
inline uint32_t group_magic(uint32_t d) {
  return d < 2 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / d);
}
// Threads of a launch along one axis: counted in 32 bits.
constexpr int64_t kMaxThreads = 0xffffffff;
hipError_t launch_group_quantize(const void *W, bool w_bf16, int64_t n_rows, int64_t n_cols, int64_t group,
                                 bool scale_bf16, uint8_t *codes, void *scales, uint8_t *zeros, hipStream_t stream);
hipError_t launch_group_dequantize(const GroupView &w, void *out, bool out_bf16, hipStream_t stream);
// Y[M, N] = bf16(X . W^T), fp32 sums; M <= kGroupMaxTokens.
constexpr int64_t kGroupMaxTokens = int64_t(1) << 20;
hipError_t launch_group_linear(const GroupView &w, const uint16_t *X, int64_t M, uint16_t *Y, hipStream_t stream);

// ---- norms of query and key heads with the position rotation --------------------------
constexpr int kQkMaxDim = 256;
// M rows of nq + 2 nk heads of d elements, rot of them rotated; the other members are the
// launchers' own (the distribution of the heads over lanes and waves).
struct QkShape {
  int64_t M;
  int nq, nk, d, rot;
  float eps;
  int lanes, per, split;
  int64_t row;
  float inv_d;
};
// t16: bf16 tensors, else fp32; qw, kw NULL: no norm (Y is not read then by the backward).
hipError_t launch_qk_fwd(const void *Y, QkShape s, bool t16, bool interleaved, const int64_t *positions,
                         const float *inv_freq, const void *qw, const void *kw, void *Q, void *K, hipStream_t stream);
// Norm only: `part`, qk_bwd_workspace bytes of partial sums of dqw and dkw, and `ticket`, 17 words that
// are zero when the call starts and when it has run.
size_t qk_bwd_workspace(QkShape s, bool t16, bool norm);
hipError_t launch_qk_bwd(const void *dQ, const void *dK, const void *dV, const void *Y, QkShape s, bool t16,
                         bool interleaved, const int64_t *positions, const float *inv_freq, const void *qw,
                         const void *kw, void *dY, void *dqw, void *dkw, double *part, uint32_t *ticket,
                         hipStream_t stream);

}  // namespace qlora
