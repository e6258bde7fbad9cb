// loss_api.cu -- the losses of the C ABI (see include/rqlut.h): argument
// checks, workspace layout, choice of path and launches.
//
// Logits come from the serving kernels (a few tokens: one pass over the codes,
// tables in shared memory) into the workspace, or from the tensor cores:
// pieces of the vocabulary are decoded once and multiplied with all tokens,
// and logits exist one tile at a time.  Gradients come from sums of the
// logits' gradients by code (a few tokens: the V x D matrix is formed in
// neither direction), or from tensor-core products with the decoded piece and
// the hidden states, one piece at a time.  choose() picks by estimated time.
#include "loss_common.cuh"

using namespace rq;

namespace {

constexpr int kTokenChunk = 4096;         // tokens per sweep over the vocabulary
constexpr int kServeTokens = 64;          // most tokens of a call on the serving kernels' logits
constexpr int kSumTokens = 32;            // and of one on sums by code
constexpr int kSms = 148;                 // sizes do not depend on the current device
constexpr int kMaxSplits = 32;            // of the vocabulary in dz E
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

// Rows of the vocabulary per piece, whole index blocks: 131072, or more where
// rows are short, up to what 1.2 GB of planes and gradients hold.  Fewer pieces
// are fewer launches and ends of waves, more hold more memory (rows of 2304: 1.2
// GB for a loss, 2.4 GB and 0.5 MB per token for gradients).  Rows of 2304, 500
// tokens: 3 blocks a piece 9.1 ms a step, 5 8.7, 8 8.4, 16 8.2; 64 tokens' loss
// 1.60, 1.62, 1.32 and 1.25 ms.
int64_t piece_rows(const rq_dims &d, int64_t tokens) {
  const int64_t fit = 1200000000 / (8 * (int64_t)d.D + 4 * tokens) / kGradRows;
  const int64_t rows = (fit < 16 ? 16 : fit) * kGradRows;
  return d.V < rows ? d.V : rows;
}
int64_t pitch16(int64_t n) { return align_up(n, 16); }   // fp16 rows of whole sectors

int total_parts(const rq_dims &d, int64_t tokens, int64_t piece) {
  int n = 0;
  for (int64_t v0 = 0; v0 < d.V; v0 += piece)
    n += loss_stats_parts(tokens, d.V - v0 < piece ? d.V - v0 : piece);
  return n;
}

// Shares of the vocabulary in dz E: its tiles are few (tokens by dims), so the
// contraction is split until whole waves of them fill the SMs.  A share costs
// its block products (0.85 us for 64 rows) and a pass over its sums.
int dh_splits(const rq_dims &d, int64_t n, int64_t piece) {
  const int64_t mt = (n + 127) / 128, nt = (d.D + 255) / 256, kb = (piece + 63) / 64;
  const bool pairs = mt % 2 == 0 || mt >= 7;
  const int64_t tiles = pairs ? (mt + 1) / 2 * nt : mt * nt, units = pairs ? kSms / 2 : kSms;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= kMaxSplits && s <= kb; ++s) {
    const double us = (double)((tiles * s + units - 1) / units) * (double)((kb + s - 1) / s) * 0.85 +
                      (double)s * (double)n * d.D * 8 / 5e6;
    if (us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

// Where the logits come from and how the gradients are formed.
struct Choice {
  bool serve, sums;
};

// Estimated microseconds of the ways, from measurements at 256000 rows of 768
// codes (V P = 197 million) and at heads a few hundred times smaller:
//   decoding           710 (uint16 codes) to 930 (10 bits) for 295 million pairs
//                      of dims, two levels; 1070 where a thread has a pair of
//                      dims, not a row
//   a tensor product   per million elements of E 0.33 to read them and 0.47
//                      per tile of 128 tokens
//   serving, B <= 4    116 per token (tables in shared memory)
//   serving, groups    tables through L2: 14 TB/s, and at least 0.09 (10 bits
//                      0.13, bytes 0.24) per column and row a thread has;
//                      a rest of tokens behind a group of 32 at least 5 per
//                      million codes (it reads that group's wide tables);
//                      decoded groups: 450 (32 tokens or a rest of 17 and more,
//                      1024 rows per SM), 340 (64, 512).  33 to 63 tokens are two
//                      groups: 63 tokens of 227000 rows 1784 us served, 1093 as
//                      a product; 33 of 256000 1958 and 1246
//   sums by code       1.95 per million codes and pair (of tokens or dims)
// The serving kernels' fallback for odd layouts walks a row's codes one by one
// (385 where the tensor cores take 45) and is never chosen.
double decode_us(const rq_dims &d) {
  return 8 + (double)d.V * d.D / 2e6 * (1.5 + 0.6 * d.L) *
                 (decode_rows_ok(d.K, d.L, d.D / d.M) ? 1.0 : 1.35);
}
double product_us(const rq_dims &d, int N) {
  return 12 + (0.33 + 0.47 * ((N + 127) / 128)) * (double)d.V * d.D / 1e6;
}
double sums_us(const rq_dims &d, int pairs) {
  return 8 + 1.95 * pairs * (double)d.V * d.M * d.L / 1e6;
}

double serve_us(const rq_dims &d, int N, int fmt) {
  const double never = 1e30;
  const int P = d.M * d.L;
  const int g = N < kTokenGroup ? N : kTokenGroup;
  if (N > kServeTokens || (size_t)rq_lut_token_stride(g) * (d.D / d.M) * 4 > 48 * 1024) return never;
  DevInfo di{};
  di.sms = kSms;
  di.max_smem_optin = 232448;
  const double codes = (double)d.V * P / 1e6;
  if (plan_chunk(d.V, P, d.K, N, fmt, di).ok) return 12 + 0.59 * N * codes;
  const bool fast = fmt == RQ_CODES_U16     ? P % 8 == 0
                    : fmt == RQ_CODES_SCHED ? P % 32 == 0
                    : fmt == RQ_CODES_U8    ? P % 16 == 0
                                            : P % 64 == 0;
  if (!fast) return never;
  const bool shape = decode_mma_shape_ok(fmt, d.V, d.D, d.M, d.L, d.K);
  const auto fits = [&](int n) { return decode_mma_smem(d.K, n, fmt) <= (size_t)di.max_smem_optin; };
  const bool tc = shape && fits(32), tc64 = shape && fits(64);
  const int64_t per_sm = (d.V + kSms - 1) / kSms;
  double us = 8;
  for (int left = N; left > 0;) {
    const int nd = decode_group(left, tc, tc64, false, kTcPartialMin);
    if (nd == 64) {
      us += 340.0 * ((per_sm + 511) / 512) * P / 768 + 40;
      left -= 64;
    } else if (nd > 0) {
      us += 450.0 * ((per_sm + 1023) / 1024) * P / 768 + 40;
      left -= nd;
    } else {
      int tok = 4;
      while (tok < left && tok < 32) tok *= 2;
      const int64_t grid = d.V / 256 < 4 * kSms ? (d.V + 255) / 256 : 4 * kSms;
      const int64_t steps = (d.V + grid * (1024 / tok) - 1) / (grid * (1024 / tok));
      const double wait = (fmt == RQ_CODES_U8 ? 0.24 : fmt == RQ_CODES_U16 ? 0.09 : 0.13) * steps * P;
      const double move = codes * tok * 4 / 14;
      const double rest = left < N ? 5 * codes : 0;
      us += 10 + (wait > move ? (wait > rest ? wait : rest) : (move > rest ? move : rest));
      left -= tok;
    }
  }
  return us;
}

Choice choose(const rq_dims &d, int N, int fmt, bool grad) {
  Choice c;
  const int ds = d.D / d.M;
  const double serve = serve_us(d, N, fmt), tensor = decode_us(d) + product_us(d, N);
  c.serve = serve < tensor;
  c.sums = false;
  if (grad) {
    // the products write and read V D floats besides
    const double sums = (c.serve ? serve : tensor) + sums_us(d, (N + 1) / 2);
    const double products = tensor + 2 * product_us(d, N) + (double)d.V * d.D * 4 / 3e6 +
                            sums_us(d, (ds + 1) / 2);
    c.sums = N <= kSumTokens && ds <= 128 && sums < products;
    if (!c.sums) c.serve = false;
  }
  return c;
}

struct Layout {
  Choice how;
  size_t amax, sh, hh, hl, wh, wl, stat, y;        // tensor-core logits and products
  size_t logits, wide, fused, fused_bytes;         // serving logits
  size_t sid, sj, sq, f;                           // sorted lists; gradients
  size_t dz, S, dhp;                               // sums by code
  size_t hw, gh, gl, zh, zl, dw, cpart, part;      // products
  size_t total;
  int64_t hp, gp, zp, vp;  // row pitches: D, D in whole pairs, the piece's rows, V
  int64_t chunk;       // tokens per sweep
  int64_t piece;       // rows of the vocabulary per piece
  int splits;          // shares of the sums by code
};

Layout layout(const rq_dims &d, int N, int fmt, int k, bool grad) {
  Layout x{};
  Arena a;
  x.how = choose(d, N, fmt, grad);
  const int64_t n = N < kTokenChunk ? N : kTokenChunk, rows = piece_rows(d, n);
  const int P = d.M * d.L, ds = d.D / d.M;
  const int64_t last = N % n == 0 ? n : N % n;     // tokens of the last sweep
  x.chunk = n;
  x.piece = rows;
  x.hp = pitch16(d.D);
  x.zp = pitch16(rows);
  x.vp = pitch16(d.V);
  if (!x.how.serve) {
    x.amax = a.take((kAmaxBlocks + 1) * 4);
    x.sh = a.take(n * 4);
    x.hh = a.take(n * x.hp * 2);
    x.hl = a.take(n * x.hp * 2);
    x.wh = a.take((d.D + 7) / 8 * x.zp * 16);        // columns of 8 dims
    x.wl = a.take((d.D + 7) / 8 * x.zp * 16);
    x.y = a.take(n * k * 4);
  } else {
    x.logits = a.take((int64_t)N * d.V * 4);
    x.wide = a.take((int64_t)N * d.D * 4);
    x.fused_bytes = rq_fused_workspace_bytes(d, N, fmt, 0);
    x.fused = a.take((int64_t)x.fused_bytes);
  }
  if (!grad) {
    if (!x.how.serve) {
      int parts = total_parts(d, n, rows);
      if (total_parts(d, last, rows) > parts) parts = total_parts(d, last, rows);
      x.stat = a.take((int64_t)parts * n * 8);
      x.sid = a.take(n * k * 4);
      x.sj = a.take(n * k * 4);
    }
  } else {
    x.sid = a.take(n * k * 4);
    x.sq = a.take(n * k * 4);
    x.f = a.take(n * 4);
    if (x.how.sums) {
      x.splits = codebook_sum_splits(d.V, d.M, d.L, d.K, N);
      x.dz = a.take((int64_t)(N + 1) / 2 * x.vp * 8);
      x.S = a.take((int64_t)(N + 1) / 2 * x.splits * P * d.K * 8);
      x.dhp = a.take((int64_t)P * N * ds * 4);
    } else {
      x.hw = a.take(n * 4);
      x.gp = pitch16((int64_t)d.M * ((ds + 1) & ~1));
      x.gh = a.take(n * x.gp * 2);
      x.gl = a.take(n * x.gp * 2);
      x.zh = a.take(n * x.zp * 2);
      x.zl = a.take(n * x.zp * 2);
      x.dw = a.take((int64_t)d.M * ((ds + 1) / 2) * x.zp * 8);
      x.splits = codebook_rows_splits(d.V, rows, d.M, d.L, d.K, ds);
      x.cpart = a.take(x.splits > 1 ? (int64_t)x.splits * P * d.K * ds * 4 : 0);
      // with fewer tokens there are more shares
      int64_t part = dh_splits(d, n, rows) * n;
      const int64_t p2 = dh_splits(d, last, rows) * last;
      if (p2 > part) part = p2;
      x.part = a.take(part * x.hp * 4);
    }
  }
  x.total = a.at;
  return x;
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

// Logits [N][V] of the serving kernels in the workspace.
int serve_logits(const Problem &q, const Layout &x, void *ws, cudaStream_t s) {
  const float *h = static_cast<const float *>(q.h);
  if (q.bf16) {
    const cudaError_t e =
        launch_loss_widen_h(q.h, (int64_t)q.N * q.d.D, at<float>(ws, x.wide), s);
    if (e != cudaSuccess) return rq::note_cuda_error(e);
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

// The products' common arguments; those of the logits add their own.
GemmArgs gemm_args(const Problem &q, const Layout &x, void *ws, const DevInfo &di) {
  GemmArgs g{};
  g.splits = 1;
  g.amax = at<float>(ws, x.amax);
  g.sh = at<float>(ws, x.sh);
  g.L = q.d.L;
  g.cap = q.cap;
  g.inv_cap = q.cap > 0.f ? 1.f / q.cap : 0.f;
  g.beta = q.t.beta;
  g.err = di.err;
  return g;
}

// The tokens [n0, n0 + n) of a call.
Problem slice(const Problem &q, int64_t n0, int64_t n) {
  Problem p = q;
  p.h = static_cast<const char *>(q.h) + n0 * q.d.D * (q.bf16 ? 2 : 4);
  p.N = (int)n;
  p.t.id += n0 * q.t.k;
  if (p.t.val) p.t.val += n0 * q.t.k;
  return p;
}

// The sorted lists of a sweep's tokens, of a gradient with their probabilities
// and weights, and (`scales`) the hidden states as planes and the tensor cores'
// scales; those of the codebooks with the first sweep.
cudaError_t begin(const Problem &q, const Layout &x, bool scales, bool first, bool grad,
                  const float *w, void *ws, const DevInfo &di, cudaStream_t s) {
  BeginArgs a{};
  a.C = q.C;
  a.nc = (int64_t)q.d.M * q.d.L * q.d.K * q.ds();
  a.amax = scales && first ? at<float>(ws, x.amax) : nullptr;
  a.h = q.h;
  a.bf16 = q.bf16;
  a.D = q.d.D;
  a.pitch = x.hp;
  if (scales) {
    a.hi = at<__half>(ws, x.hh);
    a.lo = q.bf16 ? nullptr : at<__half>(ws, x.hl);
    a.sh = at<float>(ws, x.sh);
  }
  a.hw = grad && !x.how.sums ? at<float>(ws, x.hw) : nullptr;
  a.t = q.t;
  a.rows = q.N;
  a.V = q.d.V;
  a.weight = w;
  a.sid = at<int32_t>(ws, x.sid);
  a.sj = grad ? nullptr : at<int32_t>(ws, x.sj);
  a.sq = grad ? at<float>(ws, x.sq) : nullptr;
  a.f = grad ? at<float>(ws, x.f) : nullptr;
  a.err = di.err;
  return launch_loss_begin(a, s);
}

// Piece [v0, v0 + rows) decoded; with `dw` also the hidden states as dz^T h
// takes them.
cudaError_t decode(const Problem &q, const Layout &x, int64_t v0, int64_t rows, bool dw, void *ws,
                   const DevInfo &di, cudaStream_t s) {
  DwPlanes p{};
  if (dw) {
    p.h = q.h;
    p.bf16 = q.bf16;
    p.N = q.N;
    p.M = q.d.M;
    p.ds = q.ds();
    p.pitch = x.gp;
    p.hw = at<float>(ws, x.hw);
    p.f = at<float>(ws, x.f);
    p.sdw = at<float>(ws, x.amax) + kAmaxBlocks;
    p.hi = at<__half>(ws, x.gh);
    p.lo = q.bf16 ? nullptr : at<__half>(ws, x.gl);
  }
  return launch_loss_decode(q.src(), q.C, q.d.M, q.d.L, q.ds(), v0, rows, x.zp,
                            at<float>(ws, x.amax), at<__half>(ws, x.wh), at<__half>(ws, x.wl), p,
                            di, s);
}

// h and the decoded piece, the factors of the logits.
GemmPlanes h_planes(const Problem &q, const Layout &x, void *ws) {
  return planes(at<void>(ws, x.hh), q.bf16 ? nullptr : at<void>(ws, x.hl), q.N, q.d.D, x.hp);
}
GemmPlanes w_planes(const Problem &q, const Layout &x, int64_t rows, void *ws) {
  return planes(at<void>(ws, x.wh), at<void>(ws, x.wl), rows, q.d.D, x.zp);
}

template <typename Each>
cudaError_t for_pieces(const rq_dims &d, const Layout &x, Each &&each) {
  for (int64_t v0 = 0; v0 < d.V; v0 += x.piece) {
    const cudaError_t e = each(v0, d.V - v0 < x.piece ? d.V - v0 : x.piece);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t tensor_loss(const Problem &all, const Layout &x, float *loss, float *lse, void *ws,
                        const DevInfo &di, cudaStream_t s) {
  float *y = at<float>(ws, x.y);
  for (int64_t n0 = 0; n0 < all.N; n0 += x.chunk) {
    const Problem q = slice(all, n0, all.N - n0 < x.chunk ? all.N - n0 : x.chunk);
    const rq_dims &d = q.d;
    RQ_TRY(begin(q, x, true, n0 == 0, false, nullptr, ws, di, s));
    int part0 = 0;
    RQ_TRY(for_pieces(d, x, [&](int64_t v0, int64_t rows) {
      RQ_TRY(decode(q, x, v0, rows, false, ws, di, s));
      GemmArgs g = gemm_args(q, x, ws, di);
      g.rows = q.N;
      g.cols = (int)rows;
      g.sid = at<int32_t>(ws, x.sid);
      g.k = q.t.k;
      g.v0 = (int)v0;
      g.sj = at<int32_t>(ws, x.sj);
      g.y = y;
      g.stat = at<float2>(ws, x.stat);
      g.stat_ld = (int)x.chunk;
      g.stat_part0 = part0;
      part0 += loss_stats_parts(q.N, rows);
      return launch_loss_gemm(kGemmStats, h_planes(q, x, ws), w_planes(q, x, rows, ws), g, di, s);
    }));
    RQ_TRY(launch_loss_finish(at<float2>(ws, x.stat), part0, (int)x.chunk, q.N, d.V, q.t, y,
                              loss + n0, lse + n0, di.err, s));
  }
  return cudaSuccess;
}

cudaError_t products_grad(const Problem &all, const Layout &x, const float *lse, const float *w,
                          const void *index, void *dh, float *dC, void *ws, const DevInfo &di,
                          cudaStream_t s) {
  float *f = at<float>(ws, x.f);
  __half *zh = at<__half>(ws, x.zh), *zl = at<__half>(ws, x.zl);
  int32_t *sid = at<int32_t>(ws, x.sid);
  float *sq = at<float>(ws, x.sq);
  const int64_t books = (int64_t)all.d.M * all.d.L * all.d.K * all.ds();
  for (int64_t n0 = 0; n0 < all.N; n0 += x.chunk) {
    const Problem q = slice(all, n0, all.N - n0 < x.chunk ? all.N - n0 : x.chunk);
    const rq_dims &d = q.d;
    const float *ql = lse + n0;
    const int splits = dh_splits(d, q.N, x.piece);
    RQ_TRY(begin(q, x, true, n0 == 0, true, w ? w + n0 : nullptr, ws, di, s));
    RQ_TRY(for_pieces(d, x, [&](int64_t v0, int64_t rows) {
      RQ_TRY(decode(q, x, v0, rows, dC && v0 == 0, ws, di, s));
      GemmArgs g = gemm_args(q, x, ws, di);
      g.rows = q.N;
      g.cols = (int)rows;
      g.sid = at<int32_t>(ws, x.sid);
      g.k = q.t.k;
      g.v0 = (int)v0;
      g.sq = sq;
      g.lse = ql;
      g.f = f;
      g.dz_hi = zh;
      g.dz_lo = zl;
      g.dz_pitch = x.zp;
      RQ_TRY(launch_loss_gemm(kGemmGrad, h_planes(q, x, ws), w_planes(q, x, rows, ws), g, di, s));
      if (dh) {
        // Both planes of both factors, for a bf16 dh too: dz sums to about zero
        // over the vocabulary, so a component that the rows of E share cancels, as
        // do like rows of opposite dz, but not what high planes alone (11 bits)
        // lose of them.  With a common part of 200 times the rows' spread those
        // left 5 times the error that a bf16 rounding and fp32 operands may have;
        // a step of 2048 bf16 tokens takes 19.5 ms, 16.7 without the low planes.
        GemmArgs p = gemm_args(q, x, ws, di);
        p.splits = splits;
        p.rows = q.N;
        p.cols = d.D;
        p.f = f;
        p.out = at<float>(ws, x.part);
        p.out_pitch = x.hp;
        p.out_split = q.N * x.hp;
        p.accumulate = v0 > 0;
        RQ_TRY(launch_loss_gemm(kGemmDh, planes(zh, zl, q.N, rows, x.zp),
                                w_planes(q, x, rows, ws), p, di, s));
      }
      if (dC) {
        GemmArgs p = gemm_args(q, x, ws, di);
        p.rows = (int)rows;
        p.cols = d.M * ((q.ds() + 1) & ~1);
        p.out = at<float>(ws, x.dw);
        p.out_pitch = x.zp;
        RQ_TRY(launch_loss_gemm(
            kGemmDw, planes(zh, zl, q.N, rows, x.zp),
            planes(at<void>(ws, x.gh), q.bf16 ? nullptr : at<void>(ws, x.gl), q.N, p.cols, x.gp),
            p, di, s));
        RQ_TRY(launch_codebook_rows(at<float>(ws, x.dw), x.zp, v0, rows, index, d.V, d.M, d.L, d.K,
                                    q.ds(), x.splits, n0 > 0 || v0 > 0,
                                    x.splits > 1 ? at<float>(ws, x.cpart) : dC, di, s));
      }
      return cudaSuccess;
    }));
    if (dh)
      RQ_TRY(launch_loss_dh_sum(at<float>(ws, x.part), splits, q.N * x.hp, x.hp, q.N, d.D, q.bf16,
                                static_cast<char *>(dh) + n0 * d.D * (q.bf16 ? 2 : 4), s));
  }
  if (dC && x.splits > 1)
    RQ_TRY(launch_codebook_join(at<float>(ws, x.cpart), x.splits, books, dC, s));
  return cudaSuccess;
}

// Gradients from sums by code; the serving logits, where chosen, are there.
cudaError_t sums_grad(const Problem &q, const Layout &x, const float *lse, const float *w,
                      const void *index, void *dh, float *dC, void *ws, const DevInfo &di,
                      cudaStream_t s) {
  const rq_dims &d = q.d;
  int32_t *sid = at<int32_t>(ws, x.sid);
  float *sq = at<float>(ws, x.sq), *f = at<float>(ws, x.f), *dz = at<float>(ws, x.dz);
  float *S = at<float>(ws, x.S), *dhp = dh ? at<float>(ws, x.dhp) : nullptr;
  RQ_TRY(begin(q, x, !x.how.serve, true, true, w, ws, di, s));
  if (x.how.serve) {
    const float *y = at<float>(ws, x.logits);
    RQ_TRY(launch_loss_dz(y, q.N, d.V, lse, f, q.t.beta, q.cap, dz, x.vp, s));
    RQ_TRY(launch_loss_fix(sid, sq, y, q.t.k, q.N, d.V, lse, f, q.t.beta, q.cap, dz, x.vp, s));
  } else {
    RQ_TRY(for_pieces(d, x, [&](int64_t v0, int64_t rows) {
      RQ_TRY(decode(q, x, v0, rows, false, ws, di, s));
      GemmArgs g = gemm_args(q, x, ws, di);
      g.rows = q.N;
      g.cols = (int)rows;
      g.sid = at<int32_t>(ws, x.sid);
      g.k = q.t.k;
      g.v0 = (int)v0;
      g.sq = sq;
      g.lse = lse;
      g.f = f;
      g.dz = dz + 2 * v0;
      g.dz_pitch = x.vp;
      return launch_loss_gemm(kGemmGrad32, h_planes(q, x, ws), w_planes(q, x, rows, ws), g, di, s);
    }));
  }
  RQ_TRY(launch_codebook_sums(dz, x.vp, q.N, index, d.V, d.M, d.L, d.K, S, di, s));
  RQ_TRY(launch_codebook_finish(S, x.splits, q.h, q.bf16, q.N, f, q.C, d.D, d.M, d.L, d.K, dC, dhp, s));
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
  // cap tanh(z / cap) needs either factor finite
  if (q.cap > 0.f && !(q.cap <= FLT_MAX && 1.f / q.cap <= FLT_MAX)) return RQ_ERR_INVALID_ARGUMENT;
  if (rq_codes_bytes(q.d, q.fmt) == 0 || q.t.k > kMaxList) return RQ_ERR_UNSUPPORTED;
  if (!aligned(q.h, q.bf16 ? 2 : 4) || !aligned(q.C, 4) || !aligned(q.codes, 16) ||
      !aligned(q.t.id, 4) || (q.t.val && !aligned(q.t.val, 4)) || (ws && !aligned(ws, 256)))
    return RQ_ERR_MISALIGNED;
  return RQ_OK;
}

// What a call reads and writes; a written range may meet no other.
struct Ranges {
  struct One {
    uintptr_t at;
    size_t bytes;
    bool out;
  } r[16];
  int n = 0;
  void add(const void *p, size_t bytes, bool out) {
    if (p) r[n++] = {reinterpret_cast<uintptr_t>(p), bytes, out};
  }
  void add_inputs(const Problem &q) {
    const size_t N = (size_t)q.N;
    add(q.h, N * q.d.D * (q.bf16 ? 2 : 4), false);
    add(q.C, (size_t)q.d.M * q.d.L * q.d.K * q.ds() * 4, false);
    add(q.codes, rq_codes_bytes(q.d, q.fmt), false);
    add(q.t.id, N * q.t.k * 4, false);
    add(q.t.val, N * q.t.k * 4, false);
  }
  bool meet() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((r[i].out || r[j].out) && r[i].at < r[j].at + r[j].bytes &&
            r[j].at < r[i].at + r[i].bytes)
          return true;
    return false;
  }
};

int run_loss(const Problem &q, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
  if (!loss || !lse) return RQ_ERR_INVALID_ARGUMENT;
  const int bad = check(q, ws);
  if (bad) return bad;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return RQ_ERR_MISALIGNED;
  const Layout x = layout(q.d, q.N, q.fmt, q.t.k, false);
  if (!ws || ws_bytes < x.total) return RQ_ERR_WORKSPACE_TOO_SMALL;
  Ranges all;
  all.add_inputs(q);
  all.add(loss, (size_t)q.N * 4, true);
  all.add(lse, (size_t)q.N * 4, true);
  all.add(ws, x.total, true);
  if (all.meet()) return RQ_ERR_INVALID_ARGUMENT;
  DevInfo di;
  cudaError_t e = dev_info(&di);
  if (e != cudaSuccess) return status_of(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!x.how.serve) return status_of(tensor_loss(q, x, loss, lse, ws, di, s));
  const int st = serve_logits(q, x, ws, s);
  if (st != RQ_OK) return st;
  return status_of(
      launch_loss_logits(at<float>(ws, x.logits), q.N, q.d.V, q.t, loss, lse, di.err, s));
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
  const Layout x = layout(q.d, q.N, q.fmt, q.t.k, true);
  if (!ws || ws_bytes < x.total) return RQ_ERR_WORKSPACE_TOO_SMALL;
  Ranges all;
  all.add_inputs(q);
  all.add(lse, (size_t)q.N * 4, false);
  all.add(w, (size_t)q.N * 4, false);
  all.add(index, rq_grad_index_bytes(q.d), false);
  all.add(dh, (size_t)q.N * q.d.D * (q.bf16 ? 2 : 4), true);
  all.add(dC, (size_t)q.d.M * q.d.L * q.d.K * q.ds() * 4, true);
  all.add(ws, x.total, true);
  if (all.meet()) return RQ_ERR_INVALID_ARGUMENT;
  DevInfo di;
  cudaError_t e = dev_info(&di);
  if (e != cudaSuccess) return status_of(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!x.how.sums) return status_of(products_grad(q, x, lse, w, index, dh, dC, ws, di, s));
  if (x.how.serve) {
    const int st = serve_logits(q, x, ws, s);
    if (st != RQ_OK) return st;
  }
  return status_of(sums_grad(q, x, lse, w, index, dh, dC, ws, di, s));
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
  const size_t a = layout(d, N, fmt, k, false).total;
  const size_t b = grad ? layout(d, N, fmt, k, true).total : 0;
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
