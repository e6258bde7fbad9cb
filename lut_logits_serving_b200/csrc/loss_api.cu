// loss_api.cu -- the losses of the C ABI (see include/rqlut.h): argument
// checks, workspace layout, choice of path and launches.
//
// Two paths.  Few tokens: the logits of the serving kernels (one pass over the
// codes) go to the workspace, and the gradients come from sums of the logits'
// gradients by code (loss_codebook.cu), so the V x D matrix is formed in
// neither direction.  More tokens: pieces of the vocabulary are decoded once
// and multiplied with all tokens on the tensor cores; logits exist one tile at
// a time, gradients of the logits one piece at a time.
#include "loss_common.cuh"

using namespace rq;

namespace {

constexpr int64_t kPieceRows = 4 * kGradRows;   // rows of the vocabulary per piece
constexpr int kTokenChunk = 4096;         // tokens per sweep over the vocabulary
constexpr int kFewTokens = 64;            // up to here a loss takes the serving kernels' logits
constexpr int kFewTokensGrad = 16;        // and a gradient the sums by code
constexpr int kSms = 148;                 // sizes do not depend on the current device
constexpr int kMaxSplits = 32;            // of the vocabulary in dz E
constexpr int kChain = 4;                 // blocks of 64 per accumulation chain
constexpr int kMaxList = 1024;            // a teacher's entries per token
constexpr int kMaxGradK = 4096;           // codewords per codebook, gradients

bool dims_valid(const rq_dims &d) { return rq_lut_bytes(d, 1) != 0; }

bool fmt_known(int fmt) { return fmt >= RQ_CODES_U16 && fmt <= RQ_CODES_PACKED10_ROT; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Problem {
  const void *h;
  int bf16;
  const float *C;
  const void *codes;
  int fmt;
  rq_dims d;
  int N;
  float cap;
  LossTargets t;
  int ds() const { return d.D / d.M; }
  CodeSrc src() const {
    CodeSrc c;
    c.codes = codes;
    c.fmt = fmt;
    c.V = d.V;
    c.P = d.M * d.L;
    c.K = d.K;
    c.fix = make_codefix(d.K);
    return c;
  }
};

// Byte offsets handed out one after the other, 256-byte aligned.
struct Arena {
  size_t at = 0;
  size_t take(int64_t bytes) {
    const size_t o = at;
    at += (size_t)align_up(bytes, 256);
    return o;
  }
};

// A token group's table must fit the table build's shared memory (the rule of
// rq_logits_from_hidden).
bool few_ok(const rq_dims &d, int N, int limit) {
  if (N > limit) return false;
  const int g = N < kTokenGroup ? N : kTokenGroup;
  return (size_t)rq_lut_token_stride(g) * (d.D / d.M) * 4 <= 48 * 1024;
}
bool few_loss(const rq_dims &d, int N) { return few_ok(d, N, kFewTokens); }
bool few_grad(const rq_dims &d, int N) { return few_ok(d, N, kFewTokensGrad) && d.D / d.M <= 128; }

int64_t piece_rows(const rq_dims &d) { return d.V < kPieceRows ? d.V : kPieceRows; }
int64_t pitch16(int64_t n) { return align_up(n, 16); }   // fp16 rows of whole sectors

int total_parts(const rq_dims &d) {
  int n = 0;
  for (int64_t v0 = 0; v0 < d.V; v0 += kPieceRows) {
    const int64_t r = d.V - v0 < kPieceRows ? d.V - v0 : kPieceRows;
    n += 2 * (int)((r + 255) / 256);
  }
  return n;
}

// Splits of dz E over the vocabulary: enough that its 128 x 256 tiles fill the
// SMs.
int dh_splits(const rq_dims &d, int64_t n) {
  const int64_t tiles = (n + 127) / 128 * ((d.D + 255) / 256);
  int64_t s = kSms / tiles;
  const int64_t kb = (piece_rows(d) + 63) / 64;
  if (s > kb) s = kb;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 1 ? 1 : (int)s;
}

struct FewLayout {
  size_t logits, stat, wide, sid, sq, f, dz, S, dhp, fused, fused_bytes, total;
  int splits;
};

FewLayout few_layout(const rq_dims &d, int N, int fmt, int k, bool grad) {
  FewLayout x{};
  Arena a;
  x.logits = a.take((int64_t)N * d.V * 4);
  x.stat = a.take((int64_t)loss_stat_parts(d.V) * N * 8);
  x.wide = a.take((int64_t)N * d.D * 4);
  if (grad) {
    const int P = d.M * d.L;
    x.splits = codebook_sum_splits(d.V, d.M, d.L, d.K, N);
    x.sid = a.take((int64_t)N * k * 4);
    x.sq = a.take((int64_t)N * k * 4);
    x.f = a.take((int64_t)N * 4);
    x.dz = a.take((int64_t)N * pitch16(d.V) * 4);
    x.S = a.take((int64_t)(N + 1) / 2 * x.splits * P * d.K * 8);
    x.dhp = a.take((int64_t)P * N * (d.D / d.M) * 4);
  }
  x.fused_bytes = rq_fused_workspace_bytes(d, N, fmt, 0);
  x.fused = a.take((int64_t)x.fused_bytes);
  x.total = a.at;
  return x;
}

struct ManyLayout {
  size_t amax, hh, hl, wh, wl, stat, y, sid, sq, f, zh, zl, dw, cpart, part, total;
  int64_t hp, zp;      // row pitches: D and the piece's rows, in elements
  int64_t chunk;       // tokens per sweep
  int csplits;         // shares of the codebooks' sums
};

ManyLayout many_layout(const rq_dims &d, int N, int k, bool grad) {
  ManyLayout x{};
  Arena a;
  const int64_t n = N < kTokenChunk ? N : kTokenChunk, rows = piece_rows(d);
  x.chunk = n;
  x.hp = pitch16(d.D);
  x.zp = pitch16(rows);
  x.amax = a.take(3 * kAmaxBlocks * 4);
  x.hh = a.take(n * x.hp * 2);
  x.hl = a.take(n * x.hp * 2);
  x.wh = a.take(rows * x.hp * 2);
  x.wl = a.take(rows * x.hp * 2);
  x.y = a.take(n * k * 4);
  if (!grad) {
    x.stat = a.take((int64_t)total_parts(d) * n * 8);
  } else {
    x.sid = a.take(n * k * 4);
    x.sq = a.take(n * k * 4);
    x.f = a.take(n * 4);
    x.zh = a.take(n * x.zp * 2);
    x.zl = a.take(n * x.zp * 2);
    x.dw = a.take((int64_t)d.D * x.zp * 4);
    x.csplits = codebook_rows_splits(d.V, rows, d.M, d.L, d.K, d.D / d.M);
    x.cpart = a.take(x.csplits > 1 ? (int64_t)x.csplits * d.M * d.L * d.K * (d.D / d.M) * 4 : 0);
    // the last sweep may have fewer tokens and with them more splits
    int64_t part = dh_splits(d, n) * n;
    const int64_t last = N % n == 0 ? n : N % n;
    const int64_t p2 = dh_splits(d, last) * last;
    if (p2 > part) part = p2;
    x.part = a.take(part * x.hp * 4);
  }
  x.total = a.at;
  return x;
}

size_t loss_bytes(const rq_dims &d, int N, int fmt, int k, bool grad) {
  if (grad ? few_grad(d, N) : few_loss(d, N)) return few_layout(d, N, fmt, k, grad).total;
  return many_layout(d, N, k, grad).total;
}

#define RQ_TRY(call)                           \
  do {                                         \
    const cudaError_t e_ = (call);             \
    if (e_ != cudaSuccess) return e_;          \
  } while (0)

template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<unsigned char *>(ws) + off);
}

// Logits [N][V] of a few tokens in the workspace.
int few_logits(const Problem &q, const FewLayout &x, void *ws, cudaStream_t s, cudaError_t *err) {
  const float *h = static_cast<const float *>(q.h);
  if (q.bf16) {
    *err = launch_loss_widen_h(q.h, (int64_t)q.N * q.d.D, at<float>(ws, x.wide), s);
    if (*err != cudaSuccess) return RQ_ERR_CUDA;
    h = at<float>(ws, x.wide);
  }
  return rq_logits_from_hidden(h, q.C, q.codes, q.fmt, q.d, q.N, q.cap, at<float>(ws, x.logits),
                               nullptr, at<void>(ws, x.fused), x.fused_bytes, s);
}

GemmPlanes planes(const void *hi, const void *lo, int64_t rows, int64_t cols, int64_t pitch) {
  GemmPlanes p;
  p.hi = hi;
  p.lo = lo;
  p.rows = rows;
  p.cols = cols;
  p.pitch = pitch;
  return p;
}

GemmArgs gemm_args(const Problem &q, const float *amax, const DevInfo &di) {
  GemmArgs g{};
  g.splits = 1;
  g.chain = kChain;
  g.amax = amax;
  g.L = q.d.L;
  g.cap = q.cap;
  g.inv_cap = q.cap > 0.f ? 1.f / q.cap : 0.f;
  g.beta = q.t.beta;
  g.T = q.t.T;
  g.err = di.err;
  return g;
}

cudaError_t many_loss(const Problem &q, const ManyLayout &x, float *loss, float *lse, void *ws,
                      const DevInfo &di, cudaStream_t s) {
  const rq_dims &d = q.d;
  const int esz = q.bf16 ? 2 : 4;
  float *amax = at<float>(ws, x.amax);
  __half *hh = at<__half>(ws, x.hh), *hl = q.bf16 ? nullptr : at<__half>(ws, x.hl);
  RQ_TRY(launch_loss_amax(q.h, q.bf16, (int64_t)q.N * d.D, q.C, (int64_t)d.M * d.L * d.K * q.ds(),
                          nullptr, 0, amax, s));
  for (int64_t n0 = 0; n0 < q.N; n0 += x.chunk) {
    const int64_t n = q.N - n0 < x.chunk ? q.N - n0 : x.chunk;
    const void *h = static_cast<const char *>(q.h) + n0 * d.D * esz;
    LossTargets t = q.t;
    t.id += n0 * t.k;
    if (t.val) t.val += n0 * t.k;
    RQ_TRY(launch_loss_split_h(h, q.bf16, n, d.D, x.hp, amax, hh, hl, s));
    RQ_TRY(launch_loss_pick(h, q.bf16, q.src(), q.C, d.D, d.M, d.L, t.id, n, t.k, q.cap,
                            at<float>(ws, x.y), s));
    int part0 = 0;
    for (int64_t v0 = 0; v0 < d.V; v0 += kPieceRows) {
      const int64_t rows = d.V - v0 < kPieceRows ? d.V - v0 : kPieceRows;
      RQ_TRY(launch_loss_decode(q.src(), q.C, d.M, d.L, q.ds(), v0, rows, x.hp, amax,
                                at<__half>(ws, x.wh), at<__half>(ws, x.wl), di, s));
      GemmArgs g = gemm_args(q, amax, di);
      g.rows = (int)n;
      g.cols = (int)rows;
      g.stat = at<float2>(ws, x.stat);
      g.stat_ld = (int)x.chunk;
      g.stat_part0 = part0;
      RQ_TRY(launch_loss_gemm(kGemmStats, planes(hh, hl, n, d.D, x.hp),
                              planes(at<void>(ws, x.wh), at<void>(ws, x.wl), rows, d.D, x.hp), g,
                              di, s));
      part0 += 2 * (int)((rows + 255) / 256);
    }
    RQ_TRY(launch_loss_finish(at<float2>(ws, x.stat), part0, (int)x.chunk, n, d.V, t,
                              at<float>(ws, x.y), false, loss + n0, lse + n0, di.err, s));
  }
  return cudaSuccess;
}

cudaError_t many_grad(const Problem &q, const ManyLayout &x, const float *lse, const float *w,
                      const void *index, void *dh, float *dC, void *ws, const DevInfo &di,
                      cudaStream_t s) {
  const rq_dims &d = q.d;
  const int esz = q.bf16 ? 2 : 4;
  float *amax = at<float>(ws, x.amax), *f = at<float>(ws, x.f), *y = at<float>(ws, x.y);
  __half *hh = at<__half>(ws, x.hh), *hl = q.bf16 ? nullptr : at<__half>(ws, x.hl);
  __half *zh = at<__half>(ws, x.zh), *zl = at<__half>(ws, x.zl);
  __half *wh = at<__half>(ws, x.wh), *wl = at<__half>(ws, x.wl);
  int32_t *sid = at<int32_t>(ws, x.sid);
  float *sq = at<float>(ws, x.sq);
  RQ_TRY(launch_loss_amax(q.h, q.bf16, (int64_t)q.N * d.D, q.C, (int64_t)d.M * d.L * d.K * q.ds(), w,
                          q.N, amax, s));
  for (int64_t n0 = 0; n0 < q.N; n0 += x.chunk) {
    const int64_t n = q.N - n0 < x.chunk ? q.N - n0 : x.chunk;
    const void *h = static_cast<const char *>(q.h) + n0 * d.D * esz;
    LossTargets t = q.t;
    t.id += n0 * t.k;
    if (t.val) t.val += n0 * t.k;
    const int splits = dh_splits(d, n);
    RQ_TRY(launch_loss_split_h(h, q.bf16, n, d.D, x.hp, amax, hh, hl, s));
    RQ_TRY(launch_loss_sparse(t, n, d.V, w ? w + n0 : nullptr, sid, sq, f, di.err, s));
    RQ_TRY(launch_loss_pick(h, q.bf16, q.src(), q.C, d.D, d.M, d.L, sid, n, t.k, q.cap, y, s));
    for (int64_t v0 = 0; v0 < d.V; v0 += kPieceRows) {
      const int64_t rows = d.V - v0 < kPieceRows ? d.V - v0 : kPieceRows;
      RQ_TRY(launch_loss_decode(q.src(), q.C, d.M, d.L, q.ds(), v0, rows, x.hp, amax, wh, wl, di,
                                s));
      GemmArgs g = gemm_args(q, amax, di);
      g.rows = (int)n;
      g.cols = (int)rows;
      g.lse = lse + n0;
      g.f = f;
      g.dz_hi = zh;
      g.dz_lo = zl;
      g.dz_pitch = x.zp;
      RQ_TRY(launch_loss_gemm(kGemmGrad, planes(hh, hl, n, d.D, x.hp),
                              planes(wh, wl, rows, d.D, x.hp), g, di, s));
      RQ_TRY(launch_loss_fix_planes(sid, sq, y, t.k, n, v0, rows, lse + n0, f, amax, t.T, t.beta,
                                    q.cap, zh, zl, x.zp, s));
      if (dh) {
        // a bf16 dh keeps 8 bits: the high planes' 11 on either side are
        // within a sixth of its rounding
        GemmArgs p = gemm_args(q, amax, di);
        p.splits = splits;
        p.rows = (int)n;
        p.cols = d.D;
        p.out = at<float>(ws, x.part);
        p.out_pitch = x.hp;
        p.out_split = n * x.hp;
        p.accumulate = v0 > 0;
        RQ_TRY(launch_loss_gemm(kGemmDh, planes(zh, q.bf16 ? nullptr : zl, n, rows, x.zp),
                                planes(wh, q.bf16 ? nullptr : wl, rows, d.D, x.hp), p, di, s));
      }
      if (dC) {
        GemmArgs p = gemm_args(q, amax, di);
        p.rows = d.D;
        p.cols = (int)rows;
        p.out = at<float>(ws, x.dw);
        p.out_pitch = x.zp;
        RQ_TRY(launch_loss_gemm(kGemmDw, planes(hh, hl, n, d.D, x.hp), planes(zh, zl, n, rows, x.zp),
                                p, di, s));
        RQ_TRY(launch_codebook_rows(at<float>(ws, x.dw), x.zp, v0, rows, index, d.V, d.M, d.L, d.K,
                                    q.ds(), x.csplits, n0 > 0 || v0 > 0,
                                    x.csplits > 1 ? at<float>(ws, x.cpart) : dC, di, s));
      }
    }
    if (dh)
      RQ_TRY(launch_loss_dh_sum(at<float>(ws, x.part), splits, n * x.hp, x.hp, n, d.D, q.bf16,
                                static_cast<char *>(dh) + n0 * d.D * esz, s));
  }
  if (dC && x.csplits > 1)
    RQ_TRY(launch_codebook_join(at<float>(ws, x.cpart), x.csplits,
                                (int64_t)d.M * d.L * d.K * q.ds(), dC, s));
  return cudaSuccess;
}

cudaError_t few_gradients(const Problem &q, const FewLayout &x, const float *lse, const float *w,
                          const void *index, void *dh, float *dC, void *ws, const DevInfo &di,
                          cudaStream_t s) {
  const rq_dims &d = q.d;
  const int64_t pitch = pitch16(d.V);
  int32_t *sid = at<int32_t>(ws, x.sid);
  float *sq = at<float>(ws, x.sq), *f = at<float>(ws, x.f), *dz = at<float>(ws, x.dz);
  float *S = at<float>(ws, x.S), *dhp = dh ? at<float>(ws, x.dhp) : nullptr;
  RQ_TRY(launch_loss_sparse(q.t, q.N, d.V, w, sid, sq, f, di.err, s));
  RQ_TRY(launch_loss_dz_small(at<float>(ws, x.logits), q.N, d.V, sid, sq, q.t.k, lse, f, q.t.beta,
                              q.cap, dz, pitch, s));
  RQ_TRY(launch_codebook_sums(dz, pitch, q.N, index, d.V, d.M, d.L, d.K, S, di, s));
  RQ_TRY(launch_codebook_finish(S, x.splits, q.h, q.bf16, q.N, q.C, d.D, d.M, d.L, d.K, dC, dhp, s));
  if (dh) RQ_TRY(launch_codebook_dh(dhp, q.N, d.D, d.M, d.L, q.bf16, dh, s));
  return cudaSuccess;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? RQ_OK : rq::note_cuda_error(e); }

// Checks shared by the losses and their gradients.
int check(const Problem &q, const void *ws) {
  if (!q.h || !q.C || !q.codes || !q.t.id || q.N < 1 || !dims_valid(q.d)) return RQ_ERR_INVALID_ARGUMENT;
  if (q.bf16 != 0 && q.bf16 != 1) return RQ_ERR_INVALID_ARGUMENT;
  if (!fmt_known(q.fmt)) return RQ_ERR_INVALID_ARGUMENT;
  if (q.t.k < 1 || q.t.k > q.d.V) return RQ_ERR_INVALID_ARGUMENT;
  if (!(q.t.T > 0.f) || !(q.t.T <= FLT_MAX) || !(q.t.beta > 0.f) || !(q.t.beta <= FLT_MAX))
    return RQ_ERR_INVALID_ARGUMENT;
  if (rq_codes_bytes(q.d, q.fmt) == 0 || q.t.k > kMaxList) return RQ_ERR_UNSUPPORTED;
  if (!aligned(q.h, q.bf16 ? 2 : 4) || !aligned(q.C, 4) || !aligned(q.codes, 16) ||
      !aligned(q.t.id, 4) || (q.t.val && !aligned(q.t.val, 4)) || (ws && !aligned(ws, 256)))
    return RQ_ERR_MISALIGNED;
  return RQ_OK;
}

int run_loss(const Problem &q, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
  if (!loss || !lse) return RQ_ERR_INVALID_ARGUMENT;
  const int bad = check(q, ws);
  if (bad) return bad;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return RQ_ERR_MISALIGNED;
  if (!ws || ws_bytes < loss_bytes(q.d, q.N, q.fmt, q.t.k, false)) return RQ_ERR_WORKSPACE_TOO_SMALL;
  DevInfo di;
  cudaError_t e = dev_info(&di);
  if (e != cudaSuccess) return status_of(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!few_loss(q.d, q.N)) {
    const ManyLayout x = many_layout(q.d, q.N, q.t.k, false);
    return status_of(many_loss(q, x, loss, lse, ws, di, s));
  }
  const FewLayout x = few_layout(q.d, q.N, q.fmt, q.t.k, false);
  const int st = few_logits(q, x, ws, s, &e);
  if (st != RQ_OK) return e != cudaSuccess ? status_of(e) : st;
  e = launch_loss_logit_stats(at<float>(ws, x.logits), q.N, q.d.V, q.t.beta, at<float2>(ws, x.stat),
                              q.N, s);
  if (e == cudaSuccess)
    e = launch_loss_finish(at<float2>(ws, x.stat), loss_stat_parts(q.d.V), q.N, q.N, q.d.V, q.t,
                           at<float>(ws, x.logits), true, loss, lse, di.err, s);
  return status_of(e);
}

int run_grad(const Problem &q, const float *lse, const float *w, const void *index, void *dh,
             float *dC, void *ws, size_t ws_bytes, void *stream) {
  if (!lse || !index || (!dh && !dC)) return RQ_ERR_INVALID_ARGUMENT;
  const int bad = check(q, ws);
  if (bad) return bad;
  if (q.d.K > kMaxGradK) return RQ_ERR_UNSUPPORTED;
  if (!aligned(lse, 4) || (w && !aligned(w, 4)) || !aligned(index, 16) ||
      (dh && !aligned(dh, q.bf16 ? 2 : 4)) || (dC && !aligned(dC, 4)))
    return RQ_ERR_MISALIGNED;
  if (!ws || ws_bytes < loss_bytes(q.d, q.N, q.fmt, q.t.k, true)) return RQ_ERR_WORKSPACE_TOO_SMALL;
  DevInfo di;
  cudaError_t e = dev_info(&di);
  if (e != cudaSuccess) return status_of(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!few_grad(q.d, q.N)) {
    const ManyLayout x = many_layout(q.d, q.N, q.t.k, true);
    return status_of(many_grad(q, x, lse, w, index, dh, dC, ws, di, s));
  }
  const FewLayout x = few_layout(q.d, q.N, q.fmt, q.t.k, true);
  const int st = few_logits(q, x, ws, s, &e);
  if (st != RQ_OK) return e != cudaSuccess ? status_of(e) : st;
  return status_of(few_gradients(q, x, lse, w, index, dh, dC, ws, di, s));
}

Problem problem(const void *h, int h_bf16, const float *C, const void *codes, int fmt, rq_dims d,
                int N, float cap, const int32_t *id, const float *val, int k, float T) {
  Problem q;
  q.h = h;
  q.bf16 = h_bf16;
  q.C = C;
  q.codes = codes;
  q.fmt = fmt;
  q.d = d;
  q.N = N;
  q.cap = cap;
  q.t.id = id;
  q.t.val = val;
  q.t.k = k;
  q.t.T = T;
  q.t.beta = (float)(1.0 / (double)T);
  return q;
}

}  // namespace

extern "C" {

size_t rq_grad_index_bytes(rq_dims d) {
  if (!dims_valid(d) || d.K > kMaxGradK) return 0;
  return grad_index_bytes(d.V, d.M * d.L, d.K);
}

int rq_prepare_grad(const void *codes, int fmt, rq_dims d, void *index, void *stream) {
  if (!codes || !index || !dims_valid(d) || !fmt_known(fmt)) return RQ_ERR_INVALID_ARGUMENT;
  if (rq_codes_bytes(d, fmt) == 0 || d.K > kMaxGradK) return RQ_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(index, 16)) return RQ_ERR_MISALIGNED;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(codes), b0 = reinterpret_cast<uintptr_t>(index);
  if (a0 < b0 + rq_grad_index_bytes(d) && b0 < a0 + rq_codes_bytes(d, fmt))
    return RQ_ERR_INVALID_ARGUMENT;   // overlap
  DevInfo di;
  cudaError_t e = dev_info(&di);
  if (e != cudaSuccess) return status_of(e);
  const Problem q = problem(nullptr, 0, nullptr, codes, fmt, d, 1, 0.f, nullptr, nullptr, 1, 1.f);
  return status_of(launch_prepare_grad(q.src(), index, di, static_cast<cudaStream_t>(stream)));
}

size_t rq_loss_workspace_bytes(rq_dims d, int N, int fmt, int k, int grad) {
  if (!dims_valid(d) || !fmt_known(fmt) || rq_codes_bytes(d, fmt) == 0 || N < 1 || k < 0 ||
      k > kMaxList || k > d.V)
    return 0;
  if (k < 1) k = 1;
  const size_t a = loss_bytes(d, N, fmt, k, false);
  const size_t b = grad ? loss_bytes(d, N, fmt, k, true) : 0;
  return a > b ? a : b;
}

int rq_xent(const void *h, int h_bf16, const float *C, const void *codes, int fmt, rq_dims d, int N,
            float softcap, const int32_t *target, float *loss, float *lse, void *ws,
            size_t ws_bytes, void *stream) {
  return run_loss(problem(h, h_bf16, C, codes, fmt, d, N, softcap, target, nullptr, 1, 1.f), loss,
                  lse, ws, ws_bytes, stream);
}

int rq_xent_grad(const void *h, int h_bf16, const float *C, const void *codes, int fmt, rq_dims d,
                 int N, float softcap, const int32_t *target, const float *lse, const float *weight,
                 const void *index, void *dh, float *dC, void *ws, size_t ws_bytes, void *stream) {
  return run_grad(problem(h, h_bf16, C, codes, fmt, d, N, softcap, target, nullptr, 1, 1.f), lse,
                  weight, index, dh, dC, ws, ws_bytes, stream);
}

int rq_distill(const void *h, int h_bf16, const float *C, const void *codes, int fmt, rq_dims d,
               int N, float softcap, const float *teacher_val, const int32_t *teacher_idx, int k,
               float temperature, float *loss, float *lse, void *ws, size_t ws_bytes,
               void *stream) {
  if (!teacher_val) return RQ_ERR_INVALID_ARGUMENT;
  return run_loss(
      problem(h, h_bf16, C, codes, fmt, d, N, softcap, teacher_idx, teacher_val, k, temperature),
      loss, lse, ws, ws_bytes, stream);
}

int rq_distill_grad(const void *h, int h_bf16, const float *C, const void *codes, int fmt,
                    rq_dims d, int N, float softcap, const float *teacher_val,
                    const int32_t *teacher_idx, int k, float temperature, const float *lse,
                    const float *weight, const void *index, void *dh, float *dC, void *ws,
                    size_t ws_bytes, void *stream) {
  if (!teacher_val) return RQ_ERR_INVALID_ARGUMENT;
  return run_grad(
      problem(h, h_bf16, C, codes, fmt, d, N, softcap, teacher_idx, teacher_val, k, temperature),
      lse, weight, index, dh, dC, ws, ws_bytes, stream);
}

}  // extern "C"
