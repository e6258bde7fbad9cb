// loss_codebook.cu -- the codebooks' gradient of the losses on the RQ-coded
// head:
//
//   dC[m][l][k] = sum over the rows v with code[v][m][l] = k of dE[v], subspace m
//
// a sum by code, 1 / K of the rows each, for every one of the M L columns of
// the code matrix.  Adding with atomics would make the result depend on the
// order of arrival, so rq_prepare_grad lays out the rows by code once per
// artifact and every sum has one owner that adds its rows in ascending order.
//
// Index.  The vocabulary is cut into blocks of kGradRows rows.  In a (block,
// column) unit the rows of a code are dealt in turn to the code's g lanes (g a
// power of two, so that K g fills some hundred lanes), the lanes are ordered by
// falling length and cut into slices of 32, one per warp, and a slice is
// stored step by step: entry i of its 32 lanes side by side, a lane without an
// i-th row naming row kGradRows, which holds zeros.  So a warp reads its
// entries as whole 64-byte rows, ahead of their use, no lane waits for a
// longer one (with K = 1024 a list has 9 rows on average; in code order the
// longest of 32 would have 17), and there is no branch.  A lane holds at most
// kCap entries; what a code has beyond its g kCap (skewed codes) follows as a
// plain list that one warp adds at the end.
//   uint16 off[slices + 1]   in rows of 32 entries
//   uint16 code[K]           slot s = lanes [s g, (s + 1) g)
//   uint16 over[1 + n + 1]   over[0] = n codes (the first n slots) may have
//                            more; theirs are [over[1 + s], over[2 + s]) of the
//                            entries that follow the slices
//   uint16 entry[]           rows, local numbers, ascending per lane
//
// Two uses.  launch_codebook_rows sums the rows of a piece's dE^T [D][rows]
// (the tensor cores' h^T dz); launch_codebook_sums, for a few tokens, sums the
// logits' gradients themselves, S[p][k][t] = sum of dz[v][t], from which both
// gradients follow without the V x D matrix of either kind:
//   dC[m][l][k] = sum_t S[p][k][t] h_t (subspace m)
//   dh_t (subspace m) = sum_l sum_k S[p][k][t] C[m][l][k]
// Both keep the block's values in shared memory and gather them from there;
// the gathers' bank conflicts (random rows: about 3.4 passes per word) bound
// them.
#include "loss_common.cuh"

namespace rq {

namespace {

constexpr int kCap = 32;

struct IndexShape {
  int64_t V;
  int P, K, blocks, lanes, slices, most;   // most: codes with kCap full rounds
  size_t code_at, over_at, entry_at, unit; // bytes
};

__host__ __device__ inline IndexShape index_shape(int64_t V, int P, int K) {
  IndexShape x;
  x.V = V;
  x.P = P;
  x.K = K;
  x.blocks = (int)((V + kGradRows - 1) / kGradRows);
  x.lanes = 1;
  while (x.lanes < 32 && K * x.lanes < 512) x.lanes *= 2;
  x.slices = (K * x.lanes + 31) / 32;
  const int rows = (int)(V < kGradRows ? V : kGradRows);
  x.most = rows / (x.lanes * (kCap - 1) + 1);
  x.code_at = (size_t)align_up((x.slices + 1) * 2, 16);
  x.over_at = x.code_at + (size_t)align_up(K * 2, 16);
  x.entry_at = (size_t)align_up((int64_t)x.over_at + (x.most + 2) * 2, 64);
  // a slice is as long as its first lane, no longer than the lanes of the slice
  // before, give or take one where codes share lanes: rows + the first slice's
  // padding + one row per slice
  x.unit = x.entry_at +
           (size_t)align_up((rows + 32 * kCap + (x.lanes > 1 ? 32 * x.slices : 0)) * 2, 64);
  return x;
}

struct Unit {
  const uint16_t *off, *code, *over, *entry;
};

__device__ __forceinline__ Unit unit_at(const void *index, const IndexShape &x, int block, int p) {
  const unsigned char *b =
      static_cast<const unsigned char *>(index) + ((size_t)block * x.P + p) * x.unit;
  Unit u;
  u.off = reinterpret_cast<const uint16_t *>(b);
  u.code = reinterpret_cast<const uint16_t *>(b + x.code_at);
  u.over = reinterpret_cast<const uint16_t *>(b + x.over_at);
  u.entry = reinterpret_cast<const uint16_t *>(b + x.entry_at);
  return u;
}

// One block takes `cols` adjacent columns of a block of rows, staged column by
// column in shared memory; a warp per column.  Rows go in ascending order, 32
// at a time; the lanes with one code take consecutive places (match_any), so
// no order of arrival enters.
constexpr int kStagePitch = kGradRows + 8;   // columns 4 banks apart

__global__ void __launch_bounds__(256) prepare_grad_kernel(const CodeSrc cs, const IndexShape x,
                                                           int cols, unsigned char *index) {
  extern __shared__ uint16_t sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (x.P + cols - 1) / cols;
  const int block = blockIdx.x / groups, p0 = blockIdx.x % groups * cols;
  const int nc = x.P - p0 < cols ? x.P - p0 : cols;
  const int64_t v0 = (int64_t)block * kGradRows;
  const int rows = (int)(x.V - v0 < kGradRows ? x.V - v0 : kGradRows);
  for (int i = threadIdx.x; i < rows * cols; i += blockDim.x) {
    const int r = i / cols, c = i - r * cols;
    if (c < nc) sm[c * kStagePitch + r] = (uint16_t)cs(v0 + r, p0 + c);
  }
  __syncthreads();
  if (warp >= nc) return;
  const int p = p0 + warp, g = x.lanes;
  const uint16_t *col = sm + warp * kStagePitch;
  uint16_t *cnt = sm + cols * kStagePitch + (size_t)warp * (2 * x.K + kCap + 32);
  uint16_t *slot = cnt + x.K, *bucket = slot + x.K;
  const unsigned below = (1u << lane) - 1u;
  unsigned char *unit = index + ((size_t)block * x.P + p) * x.unit;
  uint16_t *off = reinterpret_cast<uint16_t *>(unit);
  uint16_t *code = reinterpret_cast<uint16_t *>(unit + x.code_at);
  uint16_t *over = reinterpret_cast<uint16_t *>(unit + x.over_at);
  uint16_t *entry = reinterpret_cast<uint16_t *>(unit + x.entry_at);
  for (int i = lane; i < x.K; i += 32) cnt[i] = 0;
  for (int i = lane; i <= kCap; i += 32) bucket[i] = 0;
  __syncwarp();
  auto sweep = [&](auto &&each) {
    for (int r0 = 0; r0 < rows; r0 += 32) {
      const int r = r0 + lane;
      const uint32_t c = r < rows ? col[r] : 0xFFFFFFFFu;
      const unsigned same = __match_any_sync(0xffffffffu, c);
      if (r < rows) each((int)c, r, same);
      __syncwarp();
    }
  };
  sweep([&](int c, int, unsigned same) {
    if ((same & below) == 0) cnt[c] = (uint16_t)(cnt[c] + __popc(same));
  });
  // codes by falling number of rounds: bucket starts, then places in code order
  auto key = [&](int c) {
    const int n = (cnt[c] + g - 1) / g;
    return kCap - (n < kCap ? n : kCap);
  };
  for (int c0 = 0; c0 < x.K; c0 += 32) {
    const int b = c0 + lane < x.K ? key(c0 + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && (same & below) == 0) bucket[b] = (uint16_t)(bucket[b] + __popc(same));
    __syncwarp();
  }
  // exclusive prefix sums in steps of 32; returns the total
  auto scan = [&](int n, auto &&get, auto &&put) {
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int own = i0 + lane < n ? (int)get(i0 + lane) : 0;
      int y = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      if (i0 + lane < n) put(i0 + lane, run + y - own);
      run += __shfl_sync(0xffffffffu, y, 31);
      __syncwarp();
    }
    return run;
  };
  const int full = bucket[0];                  // codes with kCap rounds
  __syncwarp();
  scan(kCap + 1, [&](int i) { return bucket[i]; },
       [&](int i, int s) { bucket[i] = (uint16_t)s; });
  __syncwarp();
  for (int c0 = 0; c0 < x.K; c0 += 32) {
    const int c = c0 + lane, b = c < x.K ? key(c) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    const int at = b >= 0 ? bucket[b] + __popc(same & below) : 0;
    __syncwarp();
    if (b >= 0) {
      code[at] = (uint16_t)c;
      slot[c] = (uint16_t)at;
      if ((same & below) == 0) bucket[b] = (uint16_t)(bucket[b] + __popc(same));
    }
    __syncwarp();
  }
  __threadfence_block();
  __syncwarp();
  const int total = scan(x.slices, [&](int s) { return kCap - key(code[s * 32 / g]); },
                         [&](int s, int at) { off[s] = (uint16_t)at; });
  if (lane == 0) off[x.slices] = (uint16_t)total;
  const int more = scan(full,
                        [&](int s) {
                          const int n = cnt[code[s]] - g * kCap;
                          return n > 0 ? n : 0;
                        },
                        [&](int s, int at) { over[1 + s] = (uint16_t)at; });
  if (lane == 0) {
    over[0] = (uint16_t)full;
    over[1 + full] = (uint16_t)more;
  }
  for (int i = lane; i < total * 32; i += 32) entry[i] = (uint16_t)kGradRows;
  for (int i = lane; i < x.K; i += 32) cnt[i] = 0;
  __threadfence_block();
  __syncwarp();
  sweep([&](int c, int r, unsigned same) {
    const int e = cnt[c] + __popc(same & below), s = slot[c];
    __syncwarp(same);
    int at;
    if (e < g * kCap) {
      const int vl = s * g + e % g;
      at = (off[vl >> 5] + e / g) * 32 + (vl & 31);
    } else {
      at = total * 32 + over[1 + s] + e - g * kCap;
    }
    entry[at] = (uint16_t)r;
    if ((same & below) == 0) cnt[c] = (uint16_t)(e + __popc(same));
  });
}

// Sums by code of one unit into stage [K][W]: get(row, acc) adds a row's W
// values.  Called by every thread of the block; the stage may be read after
// it, up to the next __syncthreads.  (Sums added to global memory code by code
// from here cost several times the gathers: every lane its own sector.  The
// stage lets them go out in code order, whole lines at a time.)
template <int W, int THREADS, typename Get>
__device__ __forceinline__ void unit_sums(const Unit &u, const IndexShape &x, float *stage,
                                          Get &&get) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = x.lanes;
  const int full = __ldg(u.over);
  for (int sl = warp; sl < x.slices; sl += THREADS / 32) {
    const int a = __ldg(u.off + sl), n = __ldg(u.off + sl + 1) - a;
    const uint16_t *e = u.entry + a * 32 + lane;
    const int s = (sl * 32 + lane) / g;
    const int c = s < x.K ? __ldg(u.code + s) : 0;
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    // eight entries at a time, those past the slice's end naming the zero row
    for (int i = 0; i < n; i += 8) {
      int r[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) r[q] = i + q < n ? __ldg(e + (i + q) * 32) : kGradRows;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i + q < n) get(r[q], acc);
    }
    for (int o = g / 2; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane % g == 0 && s < x.K) {
#pragma unroll
      for (int j = 0; j < W; ++j) stage[c * W + j] = acc[j];
    }
  }
  __syncthreads();
  if (full == 0) return;
  const uint16_t *rest = u.entry + __ldg(u.off + x.slices) * 32;
  for (int s = warp; s < full; s += THREADS / 32) {
    const int a = __ldg(u.over + 1 + s), b = __ldg(u.over + 2 + s);
    if (a == b) continue;
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    for (int i = a + lane; i < b; i += 32) get(__ldg(rest + i), acc);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane == 0) {
      const int c = __ldg(u.code + s);
#pragma unroll
      for (int j = 0; j < W; ++j) stage[c * W + j] += acc[j];
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------- rows of dE^T
//
// CTA (subspace m, slab of up to 3 dims[, level]): walks the piece's blocks,
// copies the slab's rows of dE^T (contiguous, kGradRows floats a dim) into
// shared memory and, per level, sums them by code into dC, whose part of this
// CTA nobody else touches.  Slabs of 3 dims leave room for two CTAs per SM, so
// one copies while the other gathers.
constexpr int kSlab = 3;
constexpr int kSlabPitch = kGradRows + 4;    // the row of zeros, vectors kept whole
constexpr int kGatherThreads = 512;

struct RowsArgs {
  const float *dwt;
  int64_t pitch;
  int block0, blocks;
  int64_t rows;         // of the piece
  const void *index;
  IndexShape x;
  int L, ds, slabs, accumulate, by_level;
  float *dC;
};

template <int W>
__device__ __forceinline__ void rows_block(const RowsArgs &a, const float *vals, float *stage,
                                           int b, int p, int j0) {
  unit_sums<W, kGatherThreads>(unit_at(a.index, a.x, a.block0 + b, p), a.x, stage,
                               [&](int r, float (&acc)[W]) {
#pragma unroll
                                 for (int j = 0; j < W; ++j) acc[j] += vals[j * kSlabPitch + r];
                               });
  float *dst = a.dC + (size_t)p * a.x.K * a.ds + j0;
  const bool old = a.accumulate || b > 0;
  const int n = a.x.K * W;
#pragma unroll 6
  for (int i = threadIdx.x; i < n; i += kGatherThreads) {
    const int c = i / W, j = i - c * W;
    float *d = dst + (size_t)c * a.ds + j;
    *d = old ? *d + stage[i] : stage[i];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kGatherThreads, 2) codebook_rows_kernel(const RowsArgs a) {
  extern __shared__ __align__(16) float vals[];     // [kSlab][kSlabPitch], stage [K][kSlab]
  float *stage = vals + kSlab * kSlabPitch;
  const int tid = threadIdx.x;
  const int m = blockIdx.x / a.slabs, j0 = blockIdx.x % a.slabs * kSlab;
  const int w = a.ds - j0 < kSlab ? a.ds - j0 : kSlab;
  const int l0 = a.by_level ? blockIdx.y : 0, l1 = a.by_level ? l0 + 1 : a.L;
  if (tid < kSlab) vals[tid * kSlabPitch + kGradRows] = 0.f;
  for (int b = 0; b < a.blocks; ++b) {
    const int64_t r0 = (int64_t)b * kGradRows;
    const int n = (int)(a.rows - r0 < kGradRows ? a.rows - r0 : kGradRows);
    __syncthreads();
    for (int j = 0; j < w; ++j) {
      const float *src = a.dwt + (int64_t)(m * a.ds + j0 + j) * a.pitch + r0;
#pragma unroll 5
      for (int i = tid * 4; i < n; i += kGatherThreads * 4)   // the pitch covers whole vectors
        *reinterpret_cast<float4 *>(vals + j * kSlabPitch + i) =
            __ldg(reinterpret_cast<const float4 *>(src + i));
    }
    __syncthreads();
    for (int l = l0; l < l1; ++l) {
      const int p = m * a.L + l;
      if (w == 3) rows_block<3>(a, vals, stage, b, p, j0);
      else if (w == 2) rows_block<2>(a, vals, stage, b, p, j0);
      else rows_block<1>(a, vals, stage, b, p, j0);
    }
  }
}

// ------------------------------------------------------------- sums of dz
//
// The (column, block) pairs, column by column, are dealt evenly to the CTAs; a
// CTA goes through the blocks, holds one block's dz [rows][W] in shared memory
// at a time and sums it for those of its columns whose share has the block.
// A column that spans CTAs has a slot of S for each.
struct SumsArgs {
  const float *dz;
  const void *index;
  IndexShape x;
  float *S;
};

constexpr int kSumsThreads = 1024;

// CTA that holds pair i of `total` dealt to `ctas`.
__host__ __device__ __forceinline__ int owner_of(int64_t i, int64_t total, int ctas) {
  return (int)(((i + 1) * ctas - 1) / total);
}
__host__ __device__ __forceinline__ int sum_ctas(int64_t total) {
  return (int)(total < 148 ? total : 148);
}

template <int W>
__global__ void __launch_bounds__(kSumsThreads) codebook_sums_kernel(const SumsArgs a) {
  extern __shared__ __align__(16) float vals[];     // [kGradRows + 1][W], stage [K][W]
  float *stage = vals + (kGradRows + 1) * W;
  const int tid = threadIdx.x, K = a.x.K, nb = a.x.blocks;
  const int64_t total = (int64_t)a.x.P * nb;
  const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
  const int p0 = (int)(lo / nb), p1 = (int)((hi - 1) / nb);
  if (tid < W) vals[kGradRows * W + tid] = 0.f;
  for (int b = 0; b < nb; ++b) {
    bool any = false;
    for (int p = p0; p <= p1 && !any; ++p) {
      const int64_t i = (int64_t)p * nb + b;
      any = i >= lo && i < hi;
    }
    if (!any) continue;
    const int64_t v0 = (int64_t)b * kGradRows;
    const int n = (int)((a.x.V - v0 < kGradRows ? a.x.V - v0 : kGradRows) * W);
    __syncthreads();
    const float *src = a.dz + v0 * W;
    for (int i = tid * 4; i + 3 < n; i += kSumsThreads * 4)
      *reinterpret_cast<float4 *>(vals + i) = __ldg(reinterpret_cast<const float4 *>(src + i));
    for (int i = n / 4 * 4 + tid; i < n; i += kSumsThreads) vals[i] = src[i];
    __syncthreads();
    for (int p = p0; p <= p1; ++p) {
      const int64_t i = (int64_t)p * nb + b;
      if (i < lo || i >= hi) continue;
      const int mine = owner_of((int64_t)p * nb, total, gridDim.x);
      float *S = a.S + ((size_t)(blockIdx.x - mine) * a.x.P + p) * K * W;
      const bool old = i > lo && b > 0;            // this CTA has been here before
      unit_sums<W, kSumsThreads>(
          unit_at(a.index, a.x, b, p), a.x, stage, [&](int r, float (&acc)[W]) {
            if (W == 4) {
              const float4 y = *reinterpret_cast<const float4 *>(vals + r * 4);
              acc[0] += y.x;
              acc[W > 1 ? 1 : 0] += y.y;
              acc[W > 2 ? 2 : 0] += y.z;
              acc[W > 3 ? 3 : 0] += y.w;
            } else if (W == 2) {
              const float2 y = *reinterpret_cast<const float2 *>(vals + r * 2);
              acc[0] += y.x;
              acc[W > 1 ? 1 : 0] += y.y;
            } else {
              acc[0] += vals[r];
            }
          });
#pragma unroll 4
      for (int j = tid; j < K * W; j += kSumsThreads) S[j] = old ? S[j] + stage[j] : stage[j];
      __syncthreads();
    }
  }
}

// One block per column p: S summed over its splits, dC (+)= S h and the
// column's share of dh.
template <int W>
__global__ void __launch_bounds__(256) codebook_finish_kernel(
    const float *__restrict__ S, int blocks, const void *h, int bf16, int t0, int nt,
    const float *__restrict__ C, int D, int L, int K, int P, int ds, int accumulate, float *dC,
    float *dhp) {
  extern __shared__ float fin[];                    // [W][ds] hidden slices, [8][W][ds] partials
  const int p = blockIdx.x, m = p / L, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t total = (int64_t)P * blocks, i0 = (int64_t)p * blocks;
  const int ctas = sum_ctas(total);
  const int slots = owner_of(i0 + blocks - 1, total, ctas) - owner_of(i0, total, ctas) + 1;
  for (int i = tid; i < W * ds; i += 256) {
    const int t = i / ds, j = i % ds;
    fin[i] = t < nt ? load_h(h, bf16, (int64_t)(t0 + t) * D + (int64_t)m * ds + j) : 0.f;
  }
  __syncthreads();
  // dims in steps of 2 so that their sums stay in registers
  for (int j0 = 0; j0 < ds; j0 += 2) {
    const int w = ds - j0 < 2 ? 1 : 2;
    float part[W][2];
#pragma unroll
    for (int t = 0; t < W; ++t) part[t][0] = part[t][1] = 0.f;
    for (int k = tid; k < K; k += 256) {
      float s[W];
#pragma unroll
      for (int t = 0; t < W; ++t) s[t] = 0.f;
      for (int x = 0; x < slots; ++x)
#pragma unroll
        for (int t = 0; t < W; ++t) s[t] += S[(((size_t)x * P + p) * K + k) * W + t];
      for (int j = 0; j < w; ++j) {
        const size_t at = ((size_t)p * K + k) * ds + j0 + j;
        if (dC) {
          float d = accumulate ? dC[at] : 0.f;
#pragma unroll
          for (int t = 0; t < W; ++t) d = fmaf(s[t], fin[t * ds + j0 + j], d);
          dC[at] = d;
        }
        if (dhp) {
          const float c = C[at];
#pragma unroll
          for (int t = 0; t < W; ++t) part[t][j] = fmaf(s[t], c, part[t][j]);
        }
      }
    }
    if (dhp) {
#pragma unroll
      for (int t = 0; t < W; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = part[t][j];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == 0 && j < w) fin[(1 + warp) * W * ds + t * ds + j0 + j] = x;
        }
    }
  }
  if (!dhp) return;
  __syncthreads();
  for (int i = tid; i < W * ds; i += 256) {
    float x = 0.f;
    for (int v = 0; v < 8; ++v) x += fin[(1 + v) * W * ds + i];
    dhp[(size_t)p * W * ds + i] = x;
  }
}

__global__ void __launch_bounds__(256) codebook_dh_kernel(const float *__restrict__ dhp, int W,
                                                          int t0, int nt, int D, int L, int ds,
                                                          int bf16, void *dh) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)nt * D) return;
  const int t = (int)(i / D), c = (int)(i % D), m = c / ds, j = c % ds;
  float x = 0.f;
  for (int l = 0; l < L; ++l) x += dhp[((size_t)(m * L + l) * W + t) * ds + j];
  const int64_t o = (int64_t)(t0 + t) * D + c;
  if (bf16) static_cast<__nv_bfloat16 *>(dh)[o] = __float2bfloat16_rn(x);
  else static_cast<float *>(dh)[o] = x;
}

}  // namespace

size_t grad_index_bytes(int64_t V, int P, int K) {
  const IndexShape x = index_shape(V, P, K);
  return (size_t)x.blocks * P * x.unit;
}

cudaError_t launch_prepare_grad(const CodeSrc &cs, void *index, const DevInfo &di, cudaStream_t s) {
  const IndexShape x = index_shape(cs.V, cs.P, cs.K);
  // as many columns a block as their counters leave room for
  int cols = 8;
  auto bytes = [&](int n) {
    return (size_t)n * (kStagePitch + 2 * cs.K + kCap + 32) * 2;
  };
  while (cols > 1 && bytes(cols) > 220 * 1024) cols /= 2;
  const void *fn = reinterpret_cast<const void *>(&prepare_grad_kernel);
  cudaError_t e = ensure_smem_limit(fn, di.device, bytes(cols));
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)x.blocks * ((cs.P + cols - 1) / cols);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  prepare_grad_kernel<<<(unsigned)grid, cols * 32, bytes(cols), s>>>(
      cs, x, cols, static_cast<unsigned char *>(index));
  return cudaGetLastError();
}

cudaError_t launch_codebook_rows(const float *dwt, int64_t pitch, int64_t v0, int64_t rows,
                                 const void *index, int64_t V, int M, int L, int K, int ds,
                                 bool accumulate, float *dC, const DevInfo &di, cudaStream_t s) {
  RowsArgs a;
  a.dwt = dwt;
  a.pitch = pitch;
  a.block0 = (int)(v0 / kGradRows);
  a.blocks = (int)((rows + kGradRows - 1) / kGradRows);
  a.rows = rows;
  a.index = index;
  a.x = index_shape(V, M * L, K);
  a.L = L;
  a.ds = ds;
  a.slabs = (ds + kSlab - 1) / kSlab;
  a.accumulate = accumulate ? 1 : 0;
  a.dC = dC;
  // few subspaces: a CTA per level, so that more SMs have work
  a.by_level = M * a.slabs < 2 * di.sms ? 1 : 0;
  const size_t smem = (size_t)kSlab * (kSlabPitch + K) * 4;
  const void *fn = reinterpret_cast<const void *>(&codebook_rows_kernel);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  codebook_rows_kernel<<<dim3((unsigned)(M * a.slabs), a.by_level ? L : 1), kGatherThreads, smem,
                         s>>>(a);
  return cudaGetLastError();
}

int codebook_sum_slots(int64_t V, int P) {
  const int blocks = (int)((V + kGradRows - 1) / kGradRows);
  const int ctas = sum_ctas((int64_t)P * blocks);
  return (ctas + P - 1) / P + 1;
}

cudaError_t launch_codebook_sums(const float *dz, int W, const void *index, int64_t V, int P, int K,
                                 float *S, const DevInfo &di, cudaStream_t s) {
  SumsArgs a;
  a.dz = dz;
  a.index = index;
  a.x = index_shape(V, P, K);
  a.S = S;
  const size_t smem = (size_t)(kGradRows + 1 + K) * W * 4;
  const void *fn = W == 1   ? reinterpret_cast<const void *>(&codebook_sums_kernel<1>)
                   : W == 2 ? reinterpret_cast<const void *>(&codebook_sums_kernel<2>)
                            : reinterpret_cast<const void *>(&codebook_sums_kernel<4>);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  void *args[] = {&a};
  return launch_maybe_pdl(fn, dim3((unsigned)sum_ctas((int64_t)P * a.x.blocks)), dim3(kSumsThreads),
                          smem, s, args, false);
}

cudaError_t launch_codebook_finish(const float *S, int64_t V, int W, const void *h, int bf16,
                                   int t0, int nt, const float *C, int D, int M, int L, int K,
                                   bool accumulate, float *dC, float *dhp, cudaStream_t s) {
  const int ds = D / M, P = M * L, acc = accumulate ? 1 : 0;
  const int blocks = (int)((V + kGradRows - 1) / kGradRows);
  const size_t smem = (size_t)9 * W * ds * 4;
  if (W == 1)
    codebook_finish_kernel<1><<<P, 256, smem, s>>>(S, blocks, h, bf16, t0, nt, C, D, L, K, P, ds,
                                                   acc, dC, dhp);
  else if (W == 2)
    codebook_finish_kernel<2><<<P, 256, smem, s>>>(S, blocks, h, bf16, t0, nt, C, D, L, K, P, ds,
                                                   acc, dC, dhp);
  else
    codebook_finish_kernel<4><<<P, 256, smem, s>>>(S, blocks, h, bf16, t0, nt, C, D, L, K, P, ds,
                                                   acc, dC, dhp);
  return cudaGetLastError();
}

cudaError_t launch_codebook_dh(const float *dhp, int W, int t0, int nt, int D, int M, int L,
                               int bf16, void *dh, cudaStream_t s) {
  const int64_t n = (int64_t)nt * D;
  codebook_dh_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(dhp, W, t0, nt, D, L, D / M, bf16,
                                                                dh);
  return cudaGetLastError();
}

}  // namespace rq
