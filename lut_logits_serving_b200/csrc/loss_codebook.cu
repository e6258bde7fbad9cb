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
// Index.  The vocabulary is cut into blocks of kGradRows rows.  Per (block,
// column p): uint16 list[kGradRows], the block's rows (local numbers) ordered
// by slot; uint16 off[K + 1], slot s owns list[off[s], off[s + 1]); uint16
// code[K], the code of slot s.  Slots are ordered by falling length, so that
// the lanes of a warp, one slot each, have lists of about one length: with
// K = 1024 a list has 8 rows on average and lanes in code order would wait
// for the longest of 32 (about 15).
//
// Two uses.  launch_codebook_rows sums the rows of a piece's dE^T [D][rows]
// (the tensor cores' h^T dz); launch_codebook_sums, for a few tokens, sums the
// logits' gradients themselves, S[p][k][t] = sum of dz[v][t], from which both
// gradients follow without the V x D matrix of either kind:
//   dC[m][l][k] = sum_t S[p][k][t] h_t (subspace m)
//   dh_t (subspace m) = sum_l sum_k S[p][k][t] C[m][l][k]
// Both keep the block's values in shared memory and gather them from there.
#include "loss_common.cuh"

namespace rq {

namespace {

struct IndexShape {
  int64_t V;
  int P, K, blocks;
  size_t off_at, code_at, unit;      // bytes
};

__host__ __device__ inline IndexShape index_shape(int64_t V, int P, int K) {
  IndexShape x;
  x.V = V;
  x.P = P;
  x.K = K;
  x.blocks = (int)((V + kGradRows - 1) / kGradRows);
  const int64_t rows = V < kGradRows ? V : kGradRows;
  x.off_at = (size_t)align_up(rows * 2, 16);
  x.code_at = x.off_at + (size_t)align_up((K + 1) * 2, 16);
  x.unit = x.code_at + (size_t)align_up(K * 2, 16);
  return x;
}

__device__ __forceinline__ const uint16_t *unit_at(const void *index, const IndexShape &x,
                                                   int block, int p) {
  return reinterpret_cast<const uint16_t *>(static_cast<const unsigned char *>(index) +
                                            ((size_t)block * x.P + p) * x.unit);
}

constexpr int kPrepWarps = 8;
constexpr int kLenBuckets = 256;     // lists of 255 rows and more share a bucket

// One warp per (block, column): rows in ascending order, 32 at a time; the
// lanes with one code take consecutive places (match_any), so no order of
// arrival enters.
__global__ void __launch_bounds__(kPrepWarps * 32) prepare_grad_kernel(const CodeSrc cs,
                                                                       const IndexShape x,
                                                                       unsigned char *index) {
  extern __shared__ uint16_t sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t u = (int64_t)blockIdx.x * kPrepWarps + warp;
  if (u >= (int64_t)x.blocks * x.P) return;
  const int block = (int)(u / x.P), p = (int)(u % x.P);
  uint16_t *cnt = sm + (size_t)warp * (x.K + kLenBuckets);   // rows per code, then next place
  uint16_t *bucket = cnt + x.K;
  const int64_t v0 = (int64_t)block * kGradRows;
  const int rows = (int)(x.V - v0 < kGradRows ? x.V - v0 : kGradRows);
  const unsigned below = (1u << lane) - 1u;
  unsigned char *unit = index + ((size_t)block * x.P + p) * x.unit;
  uint16_t *list = reinterpret_cast<uint16_t *>(unit);
  uint16_t *off = reinterpret_cast<uint16_t *>(unit + x.off_at);
  uint16_t *code = reinterpret_cast<uint16_t *>(unit + x.code_at);
  for (int i = lane; i < x.K; i += 32) cnt[i] = 0;
  for (int i = lane; i < kLenBuckets; i += 32) bucket[i] = 0;
  __syncwarp();
  constexpr int U = 8;                               // loads in flight
  auto sweep = [&](auto &&each) {
    for (int r0 = 0; r0 < rows; r0 += 32 * U) {
      uint32_t c[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * 32 + lane;
        c[i] = r < rows ? cs(v0 + r, p) : 0xFFFFFFFFu;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const unsigned same = __match_any_sync(0xffffffffu, c[i]);
        if (c[i] != 0xFFFFFFFFu) each(c[i], r0 + i * 32 + lane, same);
        __syncwarp();
      }
    }
  };
  sweep([&](uint32_t c, int, unsigned same) {
    if ((same & below) == 0) cnt[c] = (uint16_t)(cnt[c] + __popc(same));
  });
  // codes by falling length: bucket starts, then their places in code order
  auto key = [&](int c) { return kLenBuckets - 1 - (cnt[c] < kLenBuckets ? cnt[c] : kLenBuckets - 1); };
  for (int c0 = 0; c0 < x.K; c0 += 32) {
    const int c = c0 + lane;
    const int b = c < x.K ? key(c) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && (same & below) == 0) bucket[b] = (uint16_t)(bucket[b] + __popc(same));
    __syncwarp();
  }
  auto scan = [&](auto &&get, auto &&put, int n) {   // exclusive prefix sums; returns the total
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
  scan([&](int i) { return bucket[i]; }, [&](int i, int s) { bucket[i] = (uint16_t)s; },
       kLenBuckets);
  __syncwarp();
  for (int c0 = 0; c0 < x.K; c0 += 32) {
    const int c = c0 + lane;
    const int b = c < x.K ? key(c) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    int at = 0;
    if (b >= 0) at = bucket[b] + __popc(same & below);
    __syncwarp();
    if (b >= 0) {
      code[at] = (uint16_t)c;
      if ((same & below) == 0) bucket[b] = (uint16_t)(bucket[b] + __popc(same));
    }
    __syncwarp();
  }
  __threadfence_block();
  __syncwarp();
  // list starts; a code's counter becomes its next place
  const int total = scan([&](int s) { return cnt[code[s]]; },
                         [&](int s, int at) {
                           off[s] = (uint16_t)at;
                           cnt[code[s]] = (uint16_t)at;
                         },
                         x.K);
  if (lane == 0) off[x.K] = (uint16_t)total;
  __syncwarp();
  sweep([&](uint32_t c, int r, unsigned same) {
    const int at = cnt[c] + __popc(same & below);
    __syncwarp(same);
    list[at] = (uint16_t)r;
    if ((same & below) == 0) cnt[c] = (uint16_t)(cnt[c] + __popc(same));
  });
}

// The lanes that share this lane's slot.
__device__ __forceinline__ unsigned slot_mask(int g) {
  const int lane = threadIdx.x & 31;
  return g == 32 ? 0xffffffffu : ((1u << g) - 1u) << (lane / g * g);
}

// Lanes that share a slot: with few codes the lists are long and the slots few.
inline int lanes_per_slot(int K) {
  int g = 1;
  while (g < 32 && K * g < 512) g *= 2;
  return g;
}

// ------------------------------------------------------------- rows of dE^T
//
// CTA (subspace m, slab of up to 3 dims[, level]): walks the piece's blocks,
// copies the slab's rows of dE^T (contiguous, kGradRows floats a dim) into
// shared memory and, per level, gathers and adds each slot's rows; the sums go
// to dC, whose part of this CTA nobody else touches.  Slabs of 3 dims leave
// room for two CTAs per SM, so one copies while the other gathers.
constexpr int kSlab = 3;
constexpr int kGatherThreads = 512;

struct RowsArgs {
  const float *dwt;
  int64_t pitch;
  int block0, blocks;
  int64_t rows;         // of the piece
  const void *index;
  IndexShape x;
  int L, ds, slabs, lanes, accumulate, by_level;
  float *dC;
};

__global__ void __launch_bounds__(kGatherThreads) codebook_rows_kernel(const RowsArgs a) {
  extern __shared__ __align__(16) float vals[];     // [kSlab][kGradRows]
  const int tid = threadIdx.x;
  const int m = blockIdx.x / a.slabs, j0 = blockIdx.x % a.slabs * kSlab;
  const int w = a.ds - j0 < kSlab ? a.ds - j0 : kSlab;
  const int l0 = a.by_level ? blockIdx.y : 0, l1 = a.by_level ? l0 + 1 : a.L;
  const int g = a.lanes, sub = tid % g;
  const unsigned mask = slot_mask(g);
  for (int b = 0; b < a.blocks; ++b) {
    const int64_t r0 = (int64_t)b * kGradRows;
    const int n = (int)(a.rows - r0 < kGradRows ? a.rows - r0 : kGradRows);
    __syncthreads();
    for (int j = 0; j < w; ++j) {
      const float *src = a.dwt + (int64_t)(m * a.ds + j0 + j) * a.pitch + r0;
      for (int i = tid * 4; i < n; i += kGatherThreads * 4)   // the pitch covers whole vectors
        *reinterpret_cast<float4 *>(vals + j * kGradRows + i) =
            __ldg(reinterpret_cast<const float4 *>(src + i));
    }
    __syncthreads();
    for (int l = l0; l < l1; ++l) {
      const int p = m * a.L + l;
      const uint16_t *list = unit_at(a.index, a.x, a.block0 + b, p);
      const uint16_t *off = list + a.x.off_at / 2, *code = list + a.x.code_at / 2;
      float *dst = a.dC + (size_t)p * a.x.K * a.ds + j0;
      const bool add = a.accumulate || b > 0;
      for (int s = tid / g; s < a.x.K; s += kGatherThreads / g) {
        const int e = off[s + 1];
        float s0 = 0.f, s1 = 0.f, s2 = 0.f;
        for (int i = off[s] + sub; i < e; i += g) {
          const int r = list[i];
          s0 += vals[r];
          if (w > 1) s1 += vals[kGradRows + r];
          if (w > 2) s2 += vals[2 * kGradRows + r];
        }
        for (int o = g / 2; o > 0; o >>= 1) {
          s0 += __shfl_xor_sync(mask, s0, o);
          s1 += __shfl_xor_sync(mask, s1, o);
          s2 += __shfl_xor_sync(mask, s2, o);
        }
        if (sub == 0) {
          float *d = dst + (size_t)code[s] * a.ds;
          d[0] = add ? d[0] + s0 : s0;
          if (w > 1) d[1] = add ? d[1] + s1 : s1;
          if (w > 2) d[2] = add ? d[2] + s2 : s2;
        }
      }
    }
  }
}

// ------------------------------------------------------------- sums of dz
//
// CTA (columns [p0, p0 + np), split of the blocks): a block's dz [rows][W] in
// shared memory, used for np columns; sums over the split's blocks in shared
// memory, then S.
struct SumsArgs {
  const float *dz;
  const void *index;
  IndexShape x;
  int np, lanes, splits;
  float *S;
};

constexpr int kSumsThreads = 1024;

template <int W>
__global__ void __launch_bounds__(kSumsThreads) codebook_sums_kernel(const SumsArgs a) {
  extern __shared__ __align__(16) float vals[];     // [rows][W], then [np][K][W]
  const int tid = threadIdx.x, K = a.x.K;
  const int span = (int)(a.x.V < kGradRows ? a.x.V : kGradRows);
  float *sums = vals + (size_t)align_up((int64_t)span * W, 4);
  const int p0 = blockIdx.x * a.np, np = a.x.P - p0 < a.np ? a.x.P - p0 : a.np;
  const int b0 = (int)((int64_t)a.x.blocks * blockIdx.y / a.splits);
  const int b1 = (int)((int64_t)a.x.blocks * (blockIdx.y + 1) / a.splits);
  const int g = a.lanes, sub = tid % g;
  const unsigned mask = slot_mask(g);
  for (int i = tid; i < np * K * W; i += kSumsThreads) sums[i] = 0.f;
  for (int b = b0; b < b1; ++b) {
    const int64_t v0 = (int64_t)b * kGradRows;
    const int n = (int)((a.x.V - v0 < kGradRows ? a.x.V - v0 : kGradRows) * W);
    __syncthreads();
    const float *src = a.dz + v0 * W;
    for (int i = tid * 4; i + 3 < n; i += kSumsThreads * 4)
      *reinterpret_cast<float4 *>(vals + i) = __ldg(reinterpret_cast<const float4 *>(src + i));
    for (int i = n / 4 * 4 + tid; i < n; i += kSumsThreads) vals[i] = src[i];
    __syncthreads();
    for (int q = 0; q < np; ++q) {
      const uint16_t *list = unit_at(a.index, a.x, b, p0 + q);
      const uint16_t *off = list + a.x.off_at / 2, *code = list + a.x.code_at / 2;
      for (int s = tid / g; s < K; s += kSumsThreads / g) {
        const int e = off[s + 1];
        float acc[W];
#pragma unroll
        for (int t = 0; t < W; ++t) acc[t] = 0.f;
        for (int i = off[s] + sub; i < e; i += g) {
          const int r = list[i];
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
        }
        for (int o = g / 2; o > 0; o >>= 1) {
#pragma unroll
          for (int t = 0; t < W; ++t) acc[t] += __shfl_xor_sync(mask, acc[t], o);
        }
        if (sub == 0) {
          float *d = sums + ((size_t)q * K + code[s]) * W;
#pragma unroll
          for (int t = 0; t < W; ++t) d[t] += acc[t];
        }
      }
    }
  }
  __syncthreads();
  float *o = a.S + ((size_t)blockIdx.y * a.x.P + p0) * K * W;
  for (int i = tid; i < np * K * W; i += kSumsThreads) o[i] = sums[i];
}

// One block per column p: S summed over its splits, dC (+)= S h and the
// column's share of dh.
template <int W>
__global__ void __launch_bounds__(256) codebook_finish_kernel(
    const float *__restrict__ S, int splits, const void *h, int bf16, int t0, int nt,
    const float *__restrict__ C, int D, int L, int K, int P, int ds, int accumulate, float *dC,
    float *dhp) {
  extern __shared__ float fin[];                    // [W][ds] hidden slices, [8][W][ds] partials
  const int p = blockIdx.x, m = p / L, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
      for (int x = 0; x < splits; ++x)
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
  const size_t smem = (size_t)kPrepWarps * (cs.K + kLenBuckets) * 2;
  const void *fn = reinterpret_cast<const void *>(&prepare_grad_kernel);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)x.blocks * x.P, grid = (units + kPrepWarps - 1) / kPrepWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  prepare_grad_kernel<<<(unsigned)grid, kPrepWarps * 32, smem, s>>>(
      cs, x, static_cast<unsigned char *>(index));
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
  a.lanes = lanes_per_slot(K);
  a.accumulate = accumulate ? 1 : 0;
  a.dC = dC;
  // few subspaces: a CTA per level, so that more SMs have work
  a.by_level = M * a.slabs < 2 * di.sms ? 1 : 0;
  const size_t smem = (size_t)kSlab * kGradRows * 4;
  const void *fn = reinterpret_cast<const void *>(&codebook_rows_kernel);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  codebook_rows_kernel<<<dim3((unsigned)(M * a.slabs), a.by_level ? L : 1), kGatherThreads, smem,
                         s>>>(a);
  return cudaGetLastError();
}

namespace {
size_t sums_smem(int64_t V, int K, int W, int np) {
  const int64_t span = V < kGradRows ? V : kGradRows;
  return (size_t)(align_up(span * W, 4) + (int64_t)np * K * W) * 4;
}
constexpr size_t kSumsSmemMax = 225 * 1024;
int sums_columns(int64_t V, int P, int K, int W, int sms) {   // columns per CTA
  int np = (P + sms - 1) / sms;
  while (np > 1 && sums_smem(V, K, W, np) > kSumsSmemMax) --np;
  return np;
}
}  // namespace

int codebook_sum_splits(int64_t V, int P, int K, int W, const DevInfo &di) {
  const int np = sums_columns(V, P, K, W, di.sms), ctas = (P + np - 1) / np;
  const int blocks = (int)((V + kGradRows - 1) / kGradRows);
  int n = di.sms / ctas;
  if (n > blocks) n = blocks;
  return n < 1 ? 1 : n;
}

cudaError_t launch_codebook_sums(const float *dz, int W, const void *index, int64_t V, int P, int K,
                                 int splits, float *S, const DevInfo &di, cudaStream_t s) {
  SumsArgs a;
  a.dz = dz;
  a.index = index;
  a.x = index_shape(V, P, K);
  a.np = sums_columns(V, P, K, W, di.sms);
  a.lanes = lanes_per_slot(K);
  a.splits = splits;
  a.S = S;
  const size_t smem = sums_smem(V, K, W, a.np);
  if (smem > kSumsSmemMax) return cudaErrorInvalidValue;
  const void *fn = W == 1   ? reinterpret_cast<const void *>(&codebook_sums_kernel<1>)
                   : W == 2 ? reinterpret_cast<const void *>(&codebook_sums_kernel<2>)
                            : reinterpret_cast<const void *>(&codebook_sums_kernel<4>);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  void *args[] = {&a};
  return launch_maybe_pdl(fn, dim3((unsigned)((P + a.np - 1) / a.np), (unsigned)splits),
                          dim3(kSumsThreads), smem, s, args, false);
}

cudaError_t launch_codebook_finish(const float *S, int splits, int W, const void *h, int bf16,
                                   int t0, int nt, const float *C, int D, int M, int L, int K,
                                   bool accumulate, float *dC, float *dhp, cudaStream_t s) {
  const int ds = D / M, P = M * L, acc = accumulate ? 1 : 0;
  const size_t smem = (size_t)9 * W * ds * 4;
  if (W == 1)
    codebook_finish_kernel<1><<<P, 256, smem, s>>>(S, splits, h, bf16, t0, nt, C, D, L, K, P, ds,
                                                   acc, dC, dhp);
  else if (W == 2)
    codebook_finish_kernel<2><<<P, 256, smem, s>>>(S, splits, h, bf16, t0, nt, C, D, L, K, P, ds,
                                                   acc, dC, dhp);
  else
    codebook_finish_kernel<4><<<P, 256, smem, s>>>(S, splits, h, bf16, t0, nt, C, D, L, K, P, ds,
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
