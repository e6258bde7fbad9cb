// loss_common.cuh -- shared by the loss kernels (cross entropy and
// distillation on the RQ-coded head, and their gradients).  Not part of the
// public ABI.
#pragma once

#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rq_common.cuh"

namespace rq {

// Rows of the vocabulary that one block of the gradient index covers: their
// local numbers fit 16 bits, and 3 floats of each, with the sums of 1024 codes,
// fit half an SM's shared memory.
constexpr int kGradRows = 8192;

constexpr float kLog2e = 1.44269504088896340736f;

// Place of no id, after all others in a sorted list.
constexpr int32_t kNoId = 0x7fffffff;

// Code p of row v in any layout, safe for codes >= K (see CodeFix).
struct CodeSrc {
  const void *codes;
  int fmt;
  int64_t V;
  int P, K;
  CodeFix fix;
  // as stored (not yet safe as an index)
  __device__ __forceinline__ uint32_t raw(int64_t v, int p) const {
    if (fmt == RQ_CODES_U16) return __ldg(static_cast<const uint16_t *>(codes) + v * P + p);
    if (fmt == RQ_CODES_U8) return __ldg(static_cast<const uint8_t *>(codes) + v * P + p);
    if (fmt == RQ_CODES_SCHED)
      return sched_code(static_cast<const uint16_t *>(codes), V, v, p, sched_shift(K));
    if (fmt == RQ_CODES_PACKED10_ROT)
      return rot10_code(static_cast<const uint8_t *>(codes), V, P, v, p);
    return packed10_code(static_cast<const uint8_t *>(codes) + v * ((10LL * P + 7) / 8), p);
  }
  __device__ __forceinline__ uint32_t operator()(int64_t v, int p) const { return fix(raw(v, p)); }
};

// ------------------------------------------------------------- fp16 splits
//
// An fp32 operand x of the tensor-core products is scaled by a power of two s
// (exact) with |x| s <= 2^14 and split into hi = fp16_rn(x s) and lo =
// fp16_rn(x s - hi): x s = hi + lo within 2^-22 |x s| as long as lo stays a
// normal number, and within 2^-25 absolutely below that, 2^-39 of the
// largest element.  a b = a_hi b_hi + a_lo b_hi + a_hi b_lo + (dropped
// a_lo b_lo, 2^-22 |a b|).

// Scales.  Every row of h has its own, and so has every row of the logits'
// gradients, bounded by |w| T: a row's scale divides out where its sums leave,
// so that neither a row of large values nor what padding holds costs the other
// rows their bits.  dz^T h sums over the rows; there h_n goes in as
// h_n sdw / scale_z(f_n) with one sdw for all rows (zero where the row has no
// gradient), and the sums leave divided by sdw.  E has one scale.
//
// loss_begin_kernel leaves kAmaxBlocks partial maxima of |C|; sdw follows them.
constexpr int kAmaxBlocks = 128;

// Largest power of two s (clamped to 2^-114 .. 2^112) with bound s < 2^14; 1 for
// a bound that is zero, infinite or NaN.  2^-114 serves the largest floats;
// below 2^-98 the planes lose bits.  A product of two scales or their reciprocals
// may leave float's range where what it scales does not.
__device__ __forceinline__ float pow2_scale(float bound) {
  if (!(bound > 0.f) || !(bound <= FLT_MAX)) return 1.f;
  int e;
  frexpf(bound, &e);
  int k = 14 - e;
  k = k < -114 ? -114 : (k > 112 ? 112 : k);
  return ldexpf(1.f, k);
}

// The scale of decoded rows (sums of L codewords); a whole warp calls it.
__device__ __forceinline__ float scale_e(const float *amax, int L) {
  const int lane = threadIdx.x & 31;
  float m = 0.f;
  for (int i = lane; i < kAmaxBlocks; i += 32) m = fmaxf(m, amax[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return pow2_scale(m * (float)L);
}
// Of a row of the logits' gradients, f = w T times a difference of two
// probabilities each.
__device__ __forceinline__ float scale_z(float f) { return pow2_scale(fabsf(f)); }

__device__ __forceinline__ void split_f16(float x, __half &hi, __half &lo) {
  hi = __float2half_rn(x);
  lo = __float2half_rn(__fsub_rn(x, __half2float(hi)));
}

__device__ __forceinline__ float load_h(const void *h, int bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(h)[i])
              : static_cast<const float *>(h)[i];
}

// ------------------------------------------------------------- launchers

// Tensor-core products of the loss kernels (loss_gemm.cu).
enum LossGemm {
  kGemmStats = 0,   // y = softcap(h E^T): per row and part max and sum of exp(y / T)
  kGemmGrad = 1,    // y again, gradients of the logits as fp16 hi / lo planes
  kGemmDh = 2,      // dz E, fp32, split over the vocabulary
  kGemmDw = 3,      // dz^T h, fp32, pairs of dims: [pair][rows][2]
  kGemmGrad32 = 4   // kGemmGrad with fp32 gradients, unscaled, pairs of tokens
};

// fp16 planes; lo may be null.  Row-major, rows `pitch` elements apart, but for
// the decoded rows, whose columns of 8 dims are `pitch` rows apart (loss_rows.cu).
struct GemmPlanes {
  const void *hi, *lo;
  int64_t rows, cols, pitch; // pitch % 8 == 0
};

struct GemmArgs {
  int m_tiles, n_tiles, splits, kblocks;
  int a_planes, b_planes, chain, stages;
  int rows, cols;            // output extents
  // scales: partial maxima of |C| and sdw, and of h's rows (the logits)
  const float *amax, *sh;
  int L;
  // epilogues
  float inv_cap, cap, beta;
  float2 *stat;              // [parts][stat_ld] (max of y / T, sum of exp(y / T - max))
  int stat_ld;
  int stat_part0;            // first part of this launch
  const float *lse, *f;      // per row: log-sum-exp, w T (0: no gradient)
  __half *dz_hi, *dz_lo;
  float *dz;                 // [token / 2][dz_pitch][2]
  int64_t dz_pitch;
  // listed ids, ascending per row; columns are rows v0 .. of the vocabulary
  const int32_t *sid, *sj;   // [rows][k], places in y's rows (a loss)
  const float *sq;           // [rows][k] (gradients)
  float *y;                  // [rows][k], their logits (a loss)
  int k, v0;
  float *out;                // fp32 output
  int64_t out_pitch, out_split;   // row pitch (kGemmDw: of pairs); stride between splits
  int accumulate;
  unsigned *err;
};

// parts of a row that kGemmStats writes for `rows` rows of the vocabulary
int loss_stats_parts(int64_t tokens, int64_t rows);
cudaError_t launch_loss_gemm(int mode, const GemmPlanes &A, const GemmPlanes &B, const GemmArgs &a,
                             const DevInfo &di, cudaStream_t s);

// Rows of a piece decoded into fp16 hi / lo planes and the other row-wise
// kernels (loss_rows.cu).
//
// h as dz^T h takes it, subspaces of odd dims filled up by a zero, and its scale
// *sdw: written by the CTAs of a decoding.
struct DwPlanes {
  const void *h;
  int bf16, N, M, ds;   // N = 0: none
  int64_t pitch;
  const float *hw, *f;
  float *sdw;
  __half *hi, *lo;      // lo null: bf16 h
};
cudaError_t launch_loss_widen_h(const void *h, int64_t n, float *out, cudaStream_t s);
bool decode_rows_ok(int K, int L, int ds);   // the faster of its kernels has the size
cudaError_t launch_loss_decode(const CodeSrc &cs, const float *C, int M, int L, int ds, int64_t v0,
                               int64_t rows, int64_t pitch, const float *amax, __half *hi,
                               __half *lo, const DwPlanes &dw, const DevInfo &di, cudaStream_t s);
// The sparse probabilities of a loss: target ids (k = 1, val null) or a
// teacher's lists.
struct LossTargets {
  const int32_t *id;     // [N][k]
  const float *val;      // [N][k] or null
  int k;
  float T, beta;
};
// The first launch: maxima of |C| (amax null: none); h's rows as planes hi, lo
// (lo null: bf16 h, which one plane holds; hi null: neither) and their scales
// sh; the sorted lists, for a gradient (sq set) merged, with q and f = weight T
// (0 for rows without a target) and, for dz^T h (hw set), the rows' largest
// |h| / scale_z(f), for a loss with their places sj
struct BeginArgs {
  const float *C;
  int64_t nc;
  float *amax;
  const void *h;
  int bf16, D;
  int64_t pitch;
  __half *hi, *lo;
  float *sh, *hw;
  LossTargets t;
  int64_t rows, V;
  const float *weight;
  int32_t *sid, *sj;
  float *sq, *f;
  unsigned *err;
};
cudaError_t launch_loss_begin(const BeginArgs &a, cudaStream_t s);
// lse and loss from logits [N][V] of a few tokens, or from the parts of
// kGemmStats and the listed ids' logits y [N][k]
cudaError_t launch_loss_logits(const float *logits, int64_t N, int64_t V, const LossTargets &t,
                               float *loss, float *lse, unsigned *err, cudaStream_t s);
cudaError_t launch_loss_finish(const float2 *stat, int parts, int stat_ld, int64_t N, int64_t V,
                               const LossTargets &t, const float *y, float *loss, float *lse,
                               unsigned *err, cudaStream_t s);
// logits [N][V] -> their gradients in pairs of tokens, [(N + 1) / 2][pitch][2],
// dense part
cudaError_t launch_loss_dz(const float *logits, int64_t N, int64_t V, const float *lse,
                           const float *f, float beta, float cap, float *dz, int64_t pitch,
                           cudaStream_t s);
// the same at the listed ids
cudaError_t launch_loss_fix(const int32_t *sid, const float *sq, const float *logits, int k,
                            int64_t N, int64_t V, const float *lse, const float *f, float beta,
                            float cap, float *dz, int64_t pitch, cudaStream_t s);
cudaError_t launch_loss_dh_sum(const float *part, int splits, int64_t stride, int64_t pitch,
                               int64_t N, int D, int bf16, void *dh, cudaStream_t s);

// Rows by code (loss_codebook.cu).
size_t grad_index_bytes(int64_t V, int P, int K);
cudaError_t launch_prepare_grad(const CodeSrc &cs, void *index, const DevInfo &di, cudaStream_t s);
// out[split] (+)= the columns of dw (pairs of dims of a subspace, an odd last
// one half empty: [M][(ds + 1) / 2][pitch][2]; rows v0 .. v0 + rows of the
// vocabulary, v0 % kGradRows == 0) summed by code, each share of the piece's
// blocks in an array like dC; with one share out is dC itself, else
// launch_codebook_join adds them up
int codebook_rows_splits(int64_t V, int64_t rows, int M, int L, int K, int ds);
cudaError_t launch_codebook_rows(const float *dw, int64_t pitch, int64_t v0, int64_t rows,
                                 const void *index, int64_t V, int M, int L, int K, int ds,
                                 int splits, bool accumulate, float *out, const DevInfo &di,
                                 cudaStream_t s);
cudaError_t launch_codebook_join(const float *part, int splits, int64_t n, float *dC,
                                 cudaStream_t s);
// S[pair][split][p][k][2] = sums of dz [(N + 1) / 2][pitch][2] by code, tokens in
// pairs
int codebook_sum_splits(int64_t V, int M, int L, int K, int N);
cudaError_t launch_codebook_sums(const float *dz, int64_t pitch, int N, const void *index, int64_t V,
                                 int M, int L, int K, float *S, const DevInfo &di, cudaStream_t s);
// from S: dC = S h, dhp[p][t][ds] = S C; dh from dhp
cudaError_t launch_codebook_finish(const float *S, int splits, const void *h, int bf16, int N,
                                   const float *f, const float *C, int D, int M, int L, int K,
                                   float *dC, float *dhp, cudaStream_t s);
cudaError_t launch_codebook_dh(const float *dhp, int N, int D, int M, int L, int bf16, void *dh,
                               cudaStream_t s);

}  // namespace rq
