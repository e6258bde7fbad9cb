// loss_rows.cu -- the row-wise kernels of the losses on the RQ-coded head:
// operand scales and fp16 splits, decoding a piece of the vocabulary for the
// tensor cores, log-sum-exp and losses, and the listed ids.
//
//   lse_n = log sum_v exp(y[n,v] / T)
//   cross entropy  loss_n = lse_n - y[n, t_n]
//   distillation   q = softmax(teacher / T) over the listed ids,
//                  loss_n = T^2 sum_j q_j (log q_j - y[n, id_j] / T + lse_n)
//   dy[n,v] = w_n T (exp(y[n,v] / T - lse_n) - q_n[v])
//
// The statistics are kept in fp32 as (maximum, sum of exp) parts that are
// joined in a fixed order, so every result is the same from run to run.
#include "loss_common.cuh"

namespace rq {

namespace {

// ------------------------------------------------------------- scales

__device__ __forceinline__ float block_max(float m, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.f;
  if (warp == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  return m;
}

// This thread's share of the largest |x[0 .. n)|: block b of `blocks`.
__device__ __forceinline__ float abs_max(const float *x, int64_t n, int b, int blocks) {
  const int64_t stride = (int64_t)blocks * blockDim.x;
  const int64_t i0 = (int64_t)b * blockDim.x + threadIdx.x;
  float m = 0.f;
  int64_t done = 0;
  if ((reinterpret_cast<uintptr_t>(x) & 15) == 0) {
    done = n / 4 * 4;
#pragma unroll 4
    for (int64_t i = i0; i < n / 4; i += stride) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(x) + i);
      m = fmaxf(fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
    }
  }
  for (int64_t i = done + i0; i < n; i += stride) m = fmaxf(m, fabsf(x[i]));
  return m;
}

__device__ float sparse_row(const BeginArgs &a, int64_t n, float *lists);

// The first kernel of a call.  With a.amax, blocks [0, kAmaxBlocks) take the
// partial maxima of |C|; the blocks after those a row each: its lists, and its
// hidden state as planes.
__global__ void __launch_bounds__(256) loss_begin_kernel(const BeginArgs a) {
  extern __shared__ float lists[];
  __shared__ float red[32];
  griddep_launch_dependents();
  griddep_wait();
  const int c_blocks = a.amax ? kAmaxBlocks : 0;
  if ((int)blockIdx.x < c_blocks) {
    const float m = block_max(abs_max(a.C, a.nc, blockIdx.x, kAmaxBlocks), red);
    if (threadIdx.x == 0) a.amax[blockIdx.x] = m;
    return;
  }
  const int64_t n = (int)blockIdx.x - c_blocks;
  float m = 0.f;
  if (a.hi && a.bf16) {
    for (int i = threadIdx.x; i < a.D; i += blockDim.x)
      m = fmaxf(m, fabsf(load_h(a.h, 1, n * a.D + i)));
  } else if (a.hi) {
    m = abs_max(static_cast<const float *>(a.h) + n * a.D, a.D, 0, 1);
  }
  const float f = sparse_row(a, n, lists);
  if (!a.hi) return;
  m = block_max(m, red);
  if (threadIdx.x == 0) {
    red[0] = a.sh[n] = pow2_scale(m);
    if (a.hw) a.hw[n] = f != 0.f ? m / scale_z(f) : 0.f;
  }
  __syncthreads();
  const float s = red[0];
  for (int i = threadIdx.x; i < a.D; i += blockDim.x) {
    __half x, y;
    split_f16(__fmul_rn(load_h(a.h, a.bf16, n * a.D + i), s), x, y);
    a.hi[n * a.pitch + i] = x;
    if (a.lo) a.lo[n * a.pitch + i] = y;
  }
}

// The scale of all rows of a.h as dz^T h takes them; the whole block calls it.
__device__ float dw_scale(const DwPlanes &a) {
  __shared__ float red[32];
  float m = 0.f;
  for (int i = threadIdx.x; i < a.N; i += blockDim.x) m = fmaxf(m, a.hw[i]);
  m = block_max(m, red);
  __syncthreads();
  if (threadIdx.x == 0) red[0] = m;
  __syncthreads();
  return pow2_scale(red[0]);
}

__device__ void dw_row(const DwPlanes &a, int64_t n, float sdw) {
  const float f = a.f[n], s = f != 0.f ? fminf(sdw / scale_z(f), FLT_MAX) : 0.f;
  if (n == 0 && threadIdx.x == 0) *a.sdw = sdw;
  const int even = (a.ds + 1) & ~1;
  for (int i = threadIdx.x; i < a.M * even; i += blockDim.x) {
    const int m = i / even, j = i - m * even;
    __half x, y;
    split_f16(s != 0.f && j < a.ds
                  ? __fmul_rn(load_h(a.h, a.bf16, (n * a.M + m) * a.ds + j), s)
                  : 0.f,
              x, y);
    a.hi[n * a.pitch + i] = x;
    if (a.lo) a.lo[n * a.pitch + i] = y;
  }
}

__global__ void __launch_bounds__(256) loss_widen_h_kernel(const __nv_bfloat16 *__restrict__ h,
                                                           int64_t n, float *__restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    out[i] = __bfloat162float(h[i]);
}

// ------------------------------------------------------------- row decode

// (x, y) as a word of the high plane and one of the low.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(__fsub_rn(x, f.x), __fsub_rn(y, f.y));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}
//
// Rows v0 .. v0 + rows of E as scaled fp16 hi / lo planes, in columns of 8 dims:
// element (row, dim) at ((dim / 8) pitch + row) 8 + dim % 8, zeros up to whole
// columns and to 8 rows.  Eight rows of a column are 128 bytes, the unit that
// the tensor cores take without a swizzle as either operand's rows, and a
// warp that decodes 32 rows stores whole lines.
//
// Two kernels.  loss_decode_rows_kernel (below) takes the sizes that it is
// compiled for; this one the others (many levels, odd or long subspaces, large
// codebooks): a CTA keeps the (scaled) codebooks of a group of gs subspaces in
// shared memory, if one fits, while it walks a chunk of rows.  A thread has one
// pair of dims of the group, the same for all its rows: it fetches the row's L
// codes (a few rows ahead), gathers and adds the pair's L codeword parts and
// stores one word to each plane; neighbouring lanes read neighbouring words of
// a codeword.  The items go chunk by chunk, all groups of a chunk at about the
// same time, so that the L2 joins their stores and codes.
struct DecodeArgs {
  CodeSrc cs;
  const float *C;
  int M, L, ds, gs, groups;
  int chunk, items;    // rows of an item, (chunk, group) items
  int64_t v0, rows, pitch;
  const float *amax;
  __half *hi, *lo;
  int64_t book;        // floats of one subspace's codebooks, L K ds
  DwPlanes dw;
  int quad;            // codebooks may be copied 16 bytes at a time
};

constexpr int kDecThreads = 1024;
constexpr int kDecU = 3;           // rows a thread has in flight

// Where the codes of subspace m start in a chunk's first row, and the bytes
// from one row to the next (uint16, bytes, and 10 bits at two levels; the other
// layouts go through CodeSrc).
struct CodeRow {
  const uint8_t *at;
  int step, shift;
  __device__ __forceinline__ CodeRow(const CodeSrc &cs, int64_t v, int m, int L) {
    const uint8_t *b = static_cast<const uint8_t *>(cs.codes);
    shift = 0;
    if (cs.fmt == RQ_CODES_U16) {
      step = cs.P * 2;
      at = b + v * step + m * L * 2;
    } else if (cs.fmt == RQ_CODES_U8) {
      step = cs.P;
      at = b + v * step + m * L;
    } else {      // bits [20 m, 20 m + 20) of the row, in three bytes
      step = (10 * cs.P + 7) / 8;
      at = b + v * step + (20 * m >> 3);
      shift = (m & 1) * 4;
    }
  }
};

// The codes of a subspace of a row, fetched ahead: load() only issues loads
// (an instruction on what they bring would wait for it), get() makes codes of
// them.  LL = 0 (many levels): nothing is kept, codes are fetched when used.
template <int LL>
struct RowCodes {
  uint32_t raw[LL == 0 ? 1 : LL == 2 ? 3 : LL];
  // row x of the chunk, row v of the vocabulary
  __device__ __forceinline__ void load(const CodeSrc &cs, const CodeRow &c, int x, int64_t v,
                                       int m) {
    const uint8_t *p = c.at + (int64_t)x * c.step;
    if (LL == 2 && cs.fmt == RQ_CODES_U16) {
      raw[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else if (LL == 2 && cs.fmt == RQ_CODES_PACKED10) {
#pragma unroll
      for (int i = 0; i < (LL == 2 ? 3 : 0); ++i) raw[i] = __ldg(p + i);
    } else if (cs.fmt == RQ_CODES_U16) {
#pragma unroll
      for (int l = 0; l < LL; ++l) raw[l] = __ldg(reinterpret_cast<const uint16_t *>(p) + l);
    } else if (cs.fmt == RQ_CODES_U8) {
#pragma unroll
      for (int l = 0; l < LL; ++l) raw[l] = __ldg(p + l);
    } else {
#pragma unroll
      for (int l = 0; l < LL; ++l) raw[l] = cs(v, m * LL + l);
    }
  }
  __device__ __forceinline__ uint32_t get(const CodeSrc &cs, const CodeRow &c, int l) const {
    if (LL == 2 && cs.fmt == RQ_CODES_U16) return cs.fix(l == 0 ? raw[0] & 0xFFFFu : raw[0] >> 16);
    if (LL == 2 && cs.fmt == RQ_CODES_PACKED10) {
      const uint32_t w =
          (raw[0] | raw[LL == 2 ? 1 : 0] << 8 | raw[LL == 2 ? 2 : 0] << 16) >> c.shift;
      return cs.fix(w >> (10 * l) & 1023u);
    }
    return cs.fix(raw[LL > 0 ? l : 0]);
  }
};

// EVEN: ds is even, so the pair lies in one subspace; else its dims may belong
// to two, and each fetches its own codes.
template <int LL, bool EVEN, bool SMEM>
__global__ void __launch_bounds__(kDecThreads) loss_decode_kernel(const DecodeArgs a) {
  extern __shared__ __align__(16) float books[];
  griddep_launch_dependents();
  griddep_wait();
  const int ds = a.ds, L = LL > 0 ? LL : a.L, K = a.cs.K, tid = threadIdx.x;
  const float se = scale_e(a.amax, a.L);
  const int words = (a.gs * ds + 1) / 2;            // pairs of a row's group
  const int span = words < kDecThreads ? words : kDecThreads;
  const int rstep = kDecThreads / span;             // rows the CTA takes at once
  const int lrow = tid / span;
  float sdw = 0.f;
  for (int64_t u = blockIdx.x; u < (int64_t)a.items + a.dw.N; u += gridDim.x) {
    if (u >= a.items) {
      if (sdw == 0.f) sdw = dw_scale(a.dw);
      dw_row(a.dw, u - a.items, sdw);
      continue;
    }
    const int g = (int)(u % a.groups);
    const int64_t r0 = (int64_t)(u / a.groups) * a.chunk;
    const int64_t r1 = r0 + a.chunk < a.rows ? r0 + a.chunk : a.rows;
    const int m0 = g * a.gs, ms = a.M - m0 < a.gs ? a.M - m0 : a.gs;
    if (SMEM) {
      __syncthreads();
      const float *src = a.C + m0 * a.book;
      const int n = (int)(ms * a.book);
      int i0 = 0;
      if (a.quad) {
        i0 = n / 4 * 4;
#pragma unroll 4
        for (int i = tid; i < n / 4; i += kDecThreads) {
          float4 x = __ldg(reinterpret_cast<const float4 *>(src) + i);
          x.x *= se;
          x.y *= se;
          x.z *= se;
          x.w *= se;
          reinterpret_cast<float4 *>(books)[i] = x;
        }
      }
      for (int i = i0 + tid; i < n; i += kDecThreads) books[i] = src[i] * se;
      __syncthreads();
    }
    // (wide subspaces have more pairs than the CTA threads)
    if (lrow >= rstep) continue;
#pragma unroll 1
    for (int w = tid % span; w < words; w += kDecThreads) {
      const int sub = 2 * w / ds, sub1 = EVEN ? sub : (2 * w + 1) / ds;
      const int j = 2 * w - sub * ds, j1 = 2 * w + 1 - sub1 * ds;
      if (sub >= ms) break;
      const bool second = EVEN || sub1 < ms;          // an odd last pair has one dim
      const float *b0 = (SMEM ? books + sub * a.book : a.C + (m0 + sub) * a.book) + j;
      const float *b1 = (SMEM ? books + sub1 * a.book : a.C + (m0 + sub1) * a.book) + j1;
      const int m = m0 + sub, m1 = m0 + sub1;
      const int64_t vc = a.v0 + r0;
      const int n = (int)(r1 - r0);
      const CodeRow ca(a.cs, vc, m, L), cb(a.cs, vc, EVEN ? m : m1, L);
      const int dim = m0 * ds + 2 * w;
      __half *oh = a.hi + ((dim >> 3) * a.pitch + r0) * 8 + (dim & 7);
      __half *ol = a.lo + ((dim >> 3) * a.pitch + r0) * 8 + (dim & 7);
      RowCodes<LL> cn[kDecU], dn[EVEN ? 1 : kDecU];
      auto fetch = [&](int r) {
#pragma unroll
        for (int i = 0; i < kDecU; ++i) {
          const int x = r + i * rstep;
          if (LL > 0 && x < n) {
            cn[i].load(a.cs, ca, x, vc + x, m);
            if (!EVEN && second) dn[EVEN ? 0 : i].load(a.cs, cb, x, vc + x, m1);
          }
        }
      };
      fetch(lrow);
      for (int r = lrow; r < n; r += kDecU * rstep) {
        RowCodes<LL> c[kDecU], d[EVEN ? 1 : kDecU];
#pragma unroll
        for (int i = 0; i < kDecU; ++i) {
          c[i] = cn[i];
          if (!EVEN) d[EVEN ? 0 : i] = dn[EVEN ? 0 : i];
        }
        fetch(r + kDecU * rstep);
#pragma unroll
        for (int i = 0; i < kDecU; ++i) {
          const int x = r + i * rstep;
          if (x >= n) break;
          float e0 = 0.f, e1 = 0.f;
#pragma unroll(LL > 0 ? LL : 1)
          for (int l = 0; l < L; ++l) {
            const uint32_t cl = LL > 0 ? c[i].get(a.cs, ca, l) : a.cs(vc + x, m * L + l);
            const float *p0 = b0 + (int64_t)(l * K + (int)cl) * ds;
            if (EVEN && SMEM) {
              const float2 y = *reinterpret_cast<const float2 *>(p0);
              e0 = __fadd_rn(e0, y.x);
              e1 = __fadd_rn(e1, y.y);
            } else {
              e0 = __fadd_rn(e0, *p0);
              if (EVEN) {
                e1 = __fadd_rn(e1, p0[1]);
              } else if (second) {
                const uint32_t dl = LL > 0 ? d[EVEN ? 0 : i].get(a.cs, cb, l)
                                           : a.cs(vc + x, m1 * L + l);
                e1 = __fadd_rn(e1, b1[(int64_t)(l * K + (int)dl) * ds]);
              }
            }
          }
          if (!SMEM) {
            e0 = __fmul_rn(e0, se);
            e1 = __fmul_rn(e1, se);
          }
          // columns are padded to 8 dims, so a pair past D has its place; a group
          // starts on a pair unless gs ds is odd (one group then)
          uint32_t hw, lw;
          split_pair(e0, e1, hw, lw);
          *reinterpret_cast<uint32_t *>(oh + (int64_t)x * 8) = hw;
          *reinterpret_cast<uint32_t *>(ol + (int64_t)x * 8) = lw;
        }
      }
    }
  }
  // zeros to a column of 8 dims and a row of 8
  const int D = a.M * ds, D8 = (D + 7) & ~7;
  const int64_t rows8 = (a.rows + 7) & ~7ll, threads = (int64_t)gridDim.x * kDecThreads;
  auto clear = [&](int dim, int64_t r) {
    const int64_t at = ((dim >> 3) * a.pitch + r) * 8 + (dim & 7);
    a.hi[at] = a.lo[at] = __ushort_as_half(0);
  };
  for (int64_t i = (int64_t)blockIdx.x * kDecThreads + tid; i < rows8 * (D8 - D); i += threads)
    clear(D + (int)(i / rows8), i % rows8);
  for (int64_t i = (int64_t)blockIdx.x * kDecThreads + tid; i < (rows8 - a.rows) * D8; i += threads)
    clear((int)(i % D8), a.rows + i / D8);
}

// Rows of E, a thread a row.  A CTA takes one unit of G subspaces, whose dims
// fill Q whole columns of the planes, and a chunk of rows.  The codebooks lie
// in shared memory split into parts of four, two and one dims, so that a
// codeword of six is one 16- and one 8-byte access: random codewords meet in a
// bank 2.6 times per 128 bytes so, 3.1 times in 8-byte accesses.  A row's codes
// come in wide words, rows ahead; a warp's stores are 32 neighbouring rows of a
// column, 512 bytes at once.  Bound by shared memory's data path and the stores
// (per 65536 rows of 2304 dims, two levels of 1024: 27 million passes of 128
// bytes for the gathers, 5 for the stores; without the stores 142 us): 182 us,
// 10-bit codes 238, where a thread per pair of dims and row-major planes take
// 272.  512 threads rather than 1024: a fifth faster on few rows.
struct DecodeRows {
  CodeSrc cs;
  const float *C;
  int M, units, items, chunk;
  int bits;            // of a code in the 32-bit words that hold a row's (VEC > 0)
  int64_t v0, rows, pitch;
  const float *amax;
  __half *hi, *lo;
  int cols;            // of the planes
  int pairs;           // codebooks may be copied two floats at a time
  int stages;          // VEC 16: rows that a thread has under way
  unsigned *err;
  DwPlanes dw;
};

constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;
constexpr int kRowStages = 4;

template <int DS>
struct RowUnit {
  static constexpr int G = DS % 8 == 0 ? 1 : DS % 4 == 0 ? 2 : DS % 2 == 0 ? 4 : 8;
  static constexpr int Q = G * DS / 8;
  static constexpr int V4 = DS / 4, V2 = DS % 4 / 2, V1 = DS % 2;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src),
               "n"(BYTES)
               : "memory");
}

// VEC: a row's codes of the unit come in the aligned words of 16 bytes (4) or 4
// (1) that hold them, or one by one (0; a last unit of fewer subspaces too).
// 16: a single word of 16 bytes, which comes by TMA, a box of 32 rows for each
// warp, up to four of them ahead, into a ring of its own: 32 rows' words lie in
// 32 lines, which as loads cost as many passes through the data path, and their
// latency behind the stores (65536 rows of uint16 codes 210 us so, 185 by TMA;
// with two boxes a row, 10-bit codes, 276, by loads 238).
template <int DS, int LL, int VEC>
__global__ void __launch_bounds__(kRowThreads)
    loss_decode_rows_kernel(const __grid_constant__ CUtensorMap map, const DecodeRows a) {
  using U = RowUnit<DS>;
  constexpr int N = U::G * LL;                       // codes of a row
  constexpr int S = VEC >= 4 ? 128 : 32;             // bits of a word as loaded
  constexpr int W10 = (N * 10 + 2 * S - 4) / S, W16 = (N * 16 + 2 * S - 18) / S;
  constexpr int W = VEC == 16 ? 4 : (W10 > W16 ? W10 : W16) * (S / 32);
  extern __shared__ __align__(16) float books[];
  __shared__ uint64_t bars[VEC == 16 ? kRowWarps * kRowStages : 1];
  const int K = a.cs.K, tid = threadIdx.x, P = a.cs.P, lane = tid & 31, warp = tid >> 5;
  if (VEC == 16) {
    if (tid == 0) {
      prefetch_tmap(&map);
      for (int i = 0; i < kRowWarps * a.stages; ++i) mbar_init(smem_addr(&bars[i]), 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  griddep_launch_dependents();
  griddep_wait();
  const float se = scale_e(a.amax, LL);
  const int book = (K * DS + 3) & ~3;                // a codebook's floats
  // where dim j of codeword k lies
  auto place = [&](int k, int j) {
    return j < U::V4 * 4             ? (j >> 2) * 4 * K + 4 * k + (j & 3)
           : j < U::V4 * 4 + U::V2 * 2 ? U::V4 * 4 * K + 2 * k + (j & 1)
                                       : (DS - 1) * K + k;
  };
  // the warp's ring of boxes, 16 bytes of 32 rows each: issued and used so far, and
  // the rows issued last, irow of item iu
  const uint32_t ring = ((smem_addr(books) + (uint32_t)(N * book) * 4 + 127u) & ~127u) +
                        (uint32_t)(warp * a.stages) * 512u;
  const uint32_t bar0 = smem_addr(bars) + 8u * (uint32_t)(warp * a.stages);
  const int64_t rows8 = (a.rows + 7) & ~7ll;
  int64_t iu = (int64_t)blockIdx.x - gridDim.x;
  int irow = 0, iend = 0, issued = 0, used = 0;
  bool lost = false;
  auto issue = [&]() {                               // by lane 0
    irow += kRowThreads;
    while (irow >= iend) {                           // the next item's rows
      iu += gridDim.x;
      if (iu >= a.items) {
        iu -= gridDim.x;                             // none left
        irow = iend;
        return;
      }
      const int64_t full = rows8 - iu / a.units * a.chunk;
      irow = warp * 32;
      iend = (int)(full < a.chunk ? full : a.chunk);
    }
    const uint32_t st = (uint32_t)(issued % a.stages);
    mbar_arrive_expect_tx(bar0 + 8u * st, 512u);
    tma_load_2d(ring + st * 512u, &map, a.bits * N * (int)(iu % a.units) / S * 8,
                (int)(a.v0 + iu / a.units * a.chunk + irow), bar0 + 8u * st, l2_policy_evict_last());
    ++issued;
  };
  if (VEC == 16 && lane == 0)
    for (int i = 0; i < a.stages; ++i) issue();
  float sdw = 0.f;
  for (int64_t u = blockIdx.x; u < (int64_t)a.items + a.dw.N; u += gridDim.x) {
    if (u >= a.items) {
      if (sdw == 0.f) sdw = dw_scale(a.dw);
      dw_row(a.dw, u - a.items, sdw);
      continue;
    }
    const int g = (int)(u % a.units), m0 = g * U::G, p0 = m0 * LL;
    const bool whole = m0 + U::G <= a.M;
    const int64_t r0 = (int64_t)(u / a.units) * a.chunk;
    const int64_t left = a.rows - r0, full = rows8 - r0;     // zeros to a row of 8
    const int n = (int)(left < a.chunk ? left : a.chunk);
    const int n8 = (int)(full < a.chunk ? full : a.chunk);
    // the words with the unit's codes in the chunk's first row, the first
    // code's place in them
    const int64_t step = ((int64_t)a.bits * P + 7) / 8;
    const int bit = a.bits * p0, sh = bit & (S - 1), nw = (sh + a.bits * N + S - 1) / S;
    const uint8_t *src =
        static_cast<const uint8_t *>(a.cs.codes) + (a.v0 + r0) * step + bit / S * (S / 8);
    const bool each = VEC == 0 || (VEC != 16 && !whole);
    uint32_t next[W];
    auto fetch = [&](int r) {
      if (VEC == 16 || each || r >= n) return;
      const uint8_t *p = src + r * step;
      if (VEC == 4) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          if (i < nw) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            next[4 * i] = x.x;
            next[4 * i + 1] = x.y;
            next[4 * i + 2] = x.z;
            next[4 * i + 3] = x.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (i < nw) next[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
      }
    };
    fetch(tid);
    __syncthreads();                                 // the last item's books are read
    const int have = whole ? N : (a.M - m0) * LL;    // codebooks; zeros for the rest
    const float *c0 = a.C + (int64_t)p0 * K * DS;
    for (int b = 0; b < N; ++b) {
      float *d = books + b * book;
      const float *c = c0 + (int64_t)b * K * DS;
      if (b >= have) {
        for (int i = tid; i < book; i += kRowThreads) d[i] = 0.f;
      } else if (DS % 2 == 0 && a.pairs) {
        for (int i = 2 * tid; i < K * DS; i += 2 * kRowThreads)
          copy_async<8>(d + place(i / DS, i % DS), c + i);
      } else {
        for (int i = tid; i < K * DS; i += kRowThreads) copy_async<4>(d + place(i / DS, i % DS), c + i);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (int base = warp * 32; base < n8; base += kRowThreads) {
      const int r = base + lane;
      uint32_t c[N];
      if (VEC == 16) {
        const uint32_t st = (uint32_t)(used % a.stages), bar = bar0 + 8u * st;
        const uint32_t parity = (uint32_t)(used / a.stages) & 1u;
        if (!lost && !mbar_try_wait(bar, parity) && !mbar_wait_bounded(bar, parity)) lost = true;
        lost = __any_sync(0xffffffffu, lost);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(next[0]), "=r"(next[1]), "=r"(next[2]), "=r"(next[3])
                     : "r"(ring + st * 512u + (uint32_t)lane * 16u)
                     : "memory");
        // The stage is free once every lane has its words: the vote needs them
        // (a barrier alone would let loads still under way meet the next copy,
        // which no order but this holds back)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %0, 0;\n\tvote.sync.any.pred q, p, "
            "0xffffffff;\n\tfence.proxy.async.shared::cta;\n\t}\n" ::"r"(next[0] ^ next[1] ^
                                                                         next[2] ^ next[3])
            : "memory");
        __syncwarp();
        if (!lost) {
          ++used;
          if (lane == 0) issue();
        }
      }
      if (each) {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = r < n && p0 + i < P ? a.cs.raw(a.v0 + r0 + r, p0 + i) : 0u;
      } else {
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = next[i];
        if (sh) {
          if (S > 32 && (sh & 64)) {
#pragma unroll
            for (int i = 0; i + 2 < W; ++i) w[i] = w[i + 2];
          }
          if (S > 32 && (sh & 32)) {
#pragma unroll
            for (int i = 0; i + 1 < W; ++i) w[i] = w[i + 1];
          }
#pragma unroll
          for (int i = 0; i + 1 < W; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], sh & 31);
          w[W - 1] >>= sh & 31;
        }
        if (a.bits == 16) {
#pragma unroll
          for (int i = 0; i < N; ++i) c[i] = w[i / 2] >> (16 * (i & 1)) & 0xFFFFu;
        } else if (a.bits == 8) {
#pragma unroll
          for (int i = 0; i < N; ++i) c[i] = w[i / 4] >> (8 * (i & 3)) & 0xFFu;
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            c[i] = __funnelshift_r(w[10 * i / 32], 10 * i / 32 + 1 < W ? w[10 * i / 32 + 1] : 0u,
                                   10 * i % 32) & 1023u;
        }
      }
      fetch(r + kRowThreads);
      float e[U::G * DS];
#pragma unroll
      for (int m = 0; m < U::G; ++m) {
#pragma unroll
        for (int l = 0; l < LL; ++l) {
          const int k = (int)a.cs.fix(c[m * LL + l]);
          const float *b = books + (m * LL + l) * book;
          float x[DS];
#pragma unroll
          for (int v = 0; v < U::V4; ++v) {
            const float4 y = *reinterpret_cast<const float4 *>(b + v * 4 * K + 4 * k);
            x[4 * v] = y.x;
            x[4 * v + 1] = y.y;
            x[4 * v + 2] = y.z;
            x[4 * v + 3] = y.w;
          }
          if (U::V2) {
            const float2 y = *reinterpret_cast<const float2 *>(b + U::V4 * 4 * K + 2 * k);
            x[U::V4 * 4] = y.x;
            x[U::V4 * 4 + (U::V2 ? 1 : 0)] = y.y;
          }
          if (U::V1) x[DS - 1] = b[(DS - 1) * K + k];
#pragma unroll
          for (int j = 0; j < DS; ++j)
            e[m * DS + j] = l == 0 ? x[j] : __fadd_rn(e[m * DS + j], x[j]);
        }
      }
      if (r >= n) {
#pragma unroll
        for (int i = 0; i < U::G * DS; ++i) e[i] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < U::Q; ++q) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          split_pair(__fmul_rn(e[8 * q + 2 * i], se), __fmul_rn(e[8 * q + 2 * i + 1], se), h[i],
                     l[i]);
        if (g * U::Q + q < a.cols && r < n8) {
          const int64_t at = ((g * U::Q + q) * a.pitch + r0 + r) * 8;
          *reinterpret_cast<uint4 *>(a.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(a.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    }
  }
  if (VEC == 16 && lost && lane == 0) {
    // the copies in flight land before the shared memory goes
    for (; used < issued; ++used)
      mbar_wait_bounded(bar0 + 8u * (uint32_t)(used % a.stages), (uint32_t)(used / a.stages) & 1u);
    atomicOr(a.err, RQ_DEVERR_TIMEOUT);
  }
}

// ------------------------------------------------------------- statistics

__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  if (!(m > -INFINITY)) return make_float2(m, a.y + b.y);
  return make_float2(m, a.y * expf(a.x - m) + b.y * expf(b.x - m));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// An id of the lists counts when it lies in [0, V) and, for a teacher, its
// logit is above -inf.  A teacher's logits are taken from their largest before
// the temperature divides them, which finite ones of any size survive.
__device__ __forceinline__ bool listed(int32_t id, int64_t V) { return id >= 0 && id < V; }

// A list's entry as its maximum takes it: fmaxf would pass over a NaN, and a list
// of nothing else would pass for an empty one.
__device__ __forceinline__ float list_top(float x) { return x != x ? INFINITY : x; }

// A row's loss and log-sum-exp from its statistics p, by one warp.
__device__ void finish_row(float2 p, int64_t n, int64_t V, const LossTargets &t,
                           const float *__restrict__ y, bool y_is_logits, float *__restrict__ loss,
                           float *__restrict__ lse, unsigned *err) {
  const int lane = threadIdx.x & 31;
  // lse = p.x + ls.  A loss takes p.x - y first: where a listed logit is the
  // maximum that is exactly 0, and a confident row's small loss keeps its bits
  // (the listed logits are those that the statistics were made of).
  const float ls = logf(p.y), l = p.x + ls;
  const int32_t *id = t.id + n * t.k;
  auto logit = [&](int j) { return y_is_logits ? y[n * V + id[j]] : y[n * t.k + j]; };
  float out = 0.f;
  if (t.val == nullptr) {
    if (lane == 0) {
      if (id[0] >= V) atomicOr(err, RQ_DEVERR_BAD_ID);
      if (listed(id[0], V)) out = (p.x - __fmul_rn(logit(0), t.beta)) + ls;
    }
  } else {
    const float *val = t.val + n * t.k;
    float m = -INFINITY;
    for (int j = lane; j < t.k; j += 32) {
      if (id[j] >= V) atomicOr(err, RQ_DEVERR_BAD_ID);
      if (listed(id[j], V)) m = fmaxf(m, list_top(val[j]));
    }
    m = warp_max(m);
    float z = 0.f, a = 0.f;
    if (m > -INFINITY) {
      for (int j = lane; j < t.k; j += 32)
        if (listed(id[j], V)) z += expf((val[j] - m) * t.beta);
      z = warp_sum(z);
      const float logz = logf(z);
      for (int j = lane; j < t.k; j += 32) {
        if (!listed(id[j], V)) continue;
        const float d = (val[j] - m) * t.beta, e = expf(d);
        if (e > 0.f || e != e)
          a = fmaf(e, (d - logz) + ((p.x - __fmul_rn(logit(j), t.beta)) + ls), a);
      }
      out = warp_sum(a) / z * t.T * t.T;
    }
  }
  if (lane == 0) {
    loss[n] = out;
    lse[n] = l;
  }
}

__device__ __forceinline__ float2 warp_join(float2 p) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    p = join(p, make_float2(__shfl_xor_sync(0xffffffffu, p.x, o),
                            __shfl_xor_sync(0xffffffffu, p.y, o)));
  return p;
}

// Few tokens' logits [N][V]: a cluster a row, each CTA a share of its columns,
// the shares joined in the first CTA's shared memory.  One launch for two (parts
// in global memory, joined by a second kernel) is 3 us of a small call's 28;
// with 256000 columns 32 rows take 16.6 us instead of 17.8, a single row 7.9
// instead of 6.
constexpr int kServeCtas = 8;

__global__ void __cluster_dims__(kServeCtas, 1, 1) __launch_bounds__(1024, 2)
    loss_logits_kernel(const float *__restrict__ logits, int64_t V, const LossTargets t,
                       float *__restrict__ loss, float *__restrict__ lse, unsigned *err) {
  __shared__ float2 red[32];
  __shared__ __align__(8) float2 shares[kServeCtas];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t n = blockIdx.y, share = ((V + kServeCtas - 1) / kServeCtas + 3) & ~3ll;
  const int rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = rank * share, c1 = c0 + share < V ? c0 + share : V;
  const float *row = logits + n * V;
  const bool quads = V % 4 == 0;                     // (the rows then start on 16 bytes)
  float2 p = make_float2(-INFINITY, 0.f);
  for (int64_t c = c0; c < c1; c += 16 * 1024) {
    float x[16], m = -INFINITY, s = 0.f;
    // all loads under way before the first use
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int64_t q = c + ((int64_t)i * 1024 + threadIdx.x * 4);
      if (quads) {
        const float4 v = q < c1 ? *reinterpret_cast<const float4 *>(row + q)
                                : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i + j] = q + j < c1 ? row[q + j] : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = __fmul_rn(x[i], t.beta);
      m = fmaxf(m, x[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s += m > -INFINITY ? expf(x[i] - m) : (x[i] != x[i] ? x[i] : 0.f);
    p = join(p, make_float2(m, s));
  }
  p = warp_join(p);
  if (lane == 0) red[warp] = p;
  __syncthreads();
  if (warp == 0) {
    p = warp_join(red[lane]);
    if (lane == 0) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(shares + rank)));
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(p.x), "f"(p.y)
                   : "memory");
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
  if (rank != 0 || warp != 0) return;
  p = warp_join(lane < kServeCtas ? shares[lane] : make_float2(-INFINITY, 0.f));
  finish_row(p, n, V, t, logits, true, loss, lse, err);
}

// Rows 8 b .. 8 b + 7: the parts joined by 128 threads a row, then one warp a
// row forms the loss.
constexpr int kFinishRows = 8;

__global__ void __launch_bounds__(1024) loss_finish_kernel(const float2 *__restrict__ stat,
                                                           int parts, int stat_ld, int64_t N,
                                                           int64_t V, const LossTargets t,
                                                           const float *__restrict__ y,
                                                           float *__restrict__ loss,
                                                           float *__restrict__ lse, unsigned *err) {
  constexpr int kLanes = 1024 / kFinishRows;
  __shared__ float2 red[kLanes][kFinishRows + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int r = threadIdx.x % kFinishRows, w = threadIdx.x / kFinishRows;
  const int64_t row = (int64_t)blockIdx.x * kFinishRows + r;
  float2 p = make_float2(-INFINITY, 0.f);
  if (row < N) {
#pragma unroll 8
    for (int i = w; i < parts; i += kLanes) p.x = fmaxf(p.x, stat[(int64_t)i * stat_ld + row].x);
#pragma unroll 8
    for (int i = w; i < parts; i += kLanes) {
      const float2 q = stat[(int64_t)i * stat_ld + row];
      p.y += p.x > -INFINITY ? q.y * expf(q.x - p.x) : q.y;
    }
  }
  red[w][r] = p;
  __syncthreads();
  const int lane = threadIdx.x & 31, v = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * kFinishRows + v;      // this warp's row
  if (v >= kFinishRows || n >= N) return;
  p = red[lane][v];
#pragma unroll
  for (int i = 32; i < kLanes; i += 32) p = join(p, red[lane + i][v]);
  finish_row(warp_join(p), n, V, t, y, false, loss, lse, err);
}

// ------------------------------------------------------------- gradient, sparse part

// One block per row: its listed ids in ascending order (kNoId after them), so
// that a tile of columns finds its own by bisection.  For a loss (sq null) sj
// keeps their places in the list; for a gradient an id listed twice is merged
// into one, with q_j, and f = w T, which is returned.
__device__ float sparse_row(const BeginArgs &a, int64_t n, float *lists) {
  __shared__ float red[8], red2[8];       // lists: [k] q, [k] id, [k] counts
  const LossTargets &t = a.t;
  const int tid = threadIdx.x, k = t.k, nt = blockDim.x, warps = nt / 32;
  float *q = lists;
  int *ids = reinterpret_cast<int *>(lists + k);
  const int32_t *id = t.id + n * k;
  const bool grad = a.sq != nullptr;
  float m = -INFINITY;
  for (int j = tid; j < k; j += nt) {
    int32_t v = id[j];
    float x = t.val ? t.val[n * k + j] : 0.f;
    if (grad && v >= a.V) atomicOr(a.err, RQ_DEVERR_BAD_ID);
    if (!listed(v, a.V)) {
      v = kNoId;
      x = -INFINITY;
    }
    ids[j] = v;
    q[j] = x;
    m = fmaxf(m, list_top(x));
  }
  bool some = true;
  float z = 0.f;
  if (grad) {
    m = warp_max(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
    for (int i = 1; i < warps; ++i) m = fmaxf(m, red[i]);
    some = m > -INFINITY;
    if (some)
      for (int j = tid; j < k; j += nt) {
        const float e = ids[j] != kNoId ? expf((q[j] - m) * t.beta) : 0.f;
        q[j] = e;
        z += e;
      }
    z = warp_sum(z);
    if ((tid & 31) == 0) red2[tid >> 5] = z;
    __syncthreads();
    z = red2[0];
    for (int i = 1; i < warps; ++i) z += red2[i];
  } else {
    __syncthreads();
  }
  // an entry counts if it is valid and, of a gradient, the first of its id
  int *counts = ids + k;
  int total = 0;
  for (int j0 = 0; j0 < k; j0 += nt) {
    const int j = j0 + tid, v = j < k && some ? ids[j] : kNoId;
    bool c = v != kNoId;
    if (grad)
      for (int i = 0; i < j && c; ++i) c = ids[i] != v;
    if (j < k) counts[j] = c;
    total += __syncthreads_count(c);
  }
  for (int j = tid; j < k; j += nt) {
    if (!counts[j]) continue;
    const int v = ids[j];
    int at = 0;
    float s = 0.f;
    for (int i = 0; i < k; ++i) {
      const int w = ids[i];
      at += counts[i] && (w < v || (w == v && i < j));
      if (grad && w == v) s += q[i];
    }
    a.sid[n * k + at] = v;
    if (grad) a.sq[n * k + at] = s / z;
    else a.sj[n * k + at] = j;
  }
  for (int j = total + tid; j < k; j += nt) {
    a.sid[n * k + j] = kNoId;
    if (grad) a.sq[n * k + j] = 0.f;
  }
  if (!grad) return 0.f;
  const float f = some ? (a.weight ? a.weight[n] : 1.f) * t.T : 0.f;
  if (tid == 0) a.f[n] = f;
  return f;
}

__device__ __forceinline__ float dz_at(float y, float q, float lse, float f, float beta,
                                       float cap) {
  const float th = cap > 0.f ? y / cap : 0.f;
  return f != 0.f ? (expf(fmaf(y, beta, -lse)) - q) * (1.f - th * th) * f : 0.f;
}

__global__ void __launch_bounds__(256) loss_dz_kernel(const float *__restrict__ logits, int64_t N,
                                                      int64_t V,
                                                      const float *__restrict__ lse,
                                                      const float *__restrict__ f, float beta,
                                                      float cap, float *__restrict__ dz,
                                                      int64_t pitch) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t n = 2 * (int64_t)blockIdx.y;
  const bool two = n + 1 < N;
  const float l0 = lse[n], w0 = f[n], l1 = two ? lse[n + 1] : 0.f, w1 = two ? f[n + 1] : 0.f;
  const float *y0 = logits + n * V, *y1 = y0 + (two ? V : 0);
  float2 *out = reinterpret_cast<float2 *>(dz) + blockIdx.y * pitch;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < pitch; v += (int64_t)gridDim.x * 256)
    out[v] = v < V ? make_float2(dz_at(y0[v], 0.f, l0, w0, beta, cap),
                                 dz_at(y1[v], 0.f, l1, w1, beta, cap))
                   : make_float2(0.f, 0.f);
}

__global__ void __launch_bounds__(256) loss_fix_kernel(
    const int32_t *__restrict__ sid, const float *__restrict__ sq, const float *__restrict__ logits,
    int k, int64_t count, int64_t V, const float *__restrict__ lse, const float *__restrict__ f,
    float beta, float cap, float *__restrict__ dz, int64_t pitch) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= count || sid[i] == kNoId) return;
  const int64_t n = i / k, v = sid[i];
  dz[(n / 2 * pitch + v) * 2 + n % 2] = dz_at(logits[n * V + v], sq[i], lse[n], f[n], beta, cap);
}

__global__ void __launch_bounds__(256) loss_dh_sum_kernel(const float *__restrict__ part,
                                                          int splits, int64_t stride,
                                                          int64_t pitch, int64_t N, int D,
                                                          int bf16, void *__restrict__ dh) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= N * D) return;
  const int64_t n = i / D, c = i - n * D;
  float s = 0.f;
  for (int p = 0; p < splits; ++p) s += part[p * stride + n * pitch + c];
  if (bf16) static_cast<__nv_bfloat16 *>(dh)[i] = __float2bfloat16_rn(s);
  else static_cast<float *>(dh)[i] = s;
}

unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

cudaError_t launch_loss_begin(const BeginArgs &a, cudaStream_t s) {
  return pdl_launch(loss_begin_kernel, dim3((unsigned)(a.rows + (a.amax ? kAmaxBlocks : 0))),
                    dim3(256), (size_t)a.t.k * 12, s, a);
}

cudaError_t launch_loss_widen_h(const void *h, int64_t n, float *out, cudaStream_t s) {
  return pdl_launch(loss_widen_h_kernel, dim3(blocks_of(n, 1024)), dim3(256), 0, s,
                    static_cast<const __nv_bfloat16 *>(h), n, out);
}

namespace {
template <bool EVEN, bool SMEM>
const void *decode_fn(int L) {
  switch (L) {
    case 1: return reinterpret_cast<const void *>(&loss_decode_kernel<1, EVEN, SMEM>);
    case 2: return reinterpret_cast<const void *>(&loss_decode_kernel<2, EVEN, SMEM>);
    case 3: return reinterpret_cast<const void *>(&loss_decode_kernel<3, EVEN, SMEM>);
  }
  return reinterpret_cast<const void *>(&loss_decode_kernel<0, EVEN, SMEM>);
}
}  // namespace

namespace {
template <int DS, int LL>
const void *rows_fn(int vec) {
  constexpr int N = RowUnit<DS>::G * LL;
  if (vec == 16 && N <= 16)      // (of a byte; 8 of two)
    return reinterpret_cast<const void *>(&loss_decode_rows_kernel<DS, LL, N <= 16 ? 16 : 4>);
  if (vec >= 4) return reinterpret_cast<const void *>(&loss_decode_rows_kernel<DS, LL, 4>);
  if (vec) return reinterpret_cast<const void *>(&loss_decode_rows_kernel<DS, LL, 1>);
  return reinterpret_cast<const void *>(&loss_decode_rows_kernel<DS, LL, 0>);
}
template <int DS>
const void *rows_fn(int L, int vec) {
  return L == 1 ? rows_fn<DS, 1>(vec) : L == 2 ? rows_fn<DS, 2>(vec) : L == 3 ? rows_fn<DS, 3>(vec)
                                                                            : nullptr;
}

// Rows per chunk: the shortest time of the last CTA, where an item costs its
// rows and `fill` more for its codebooks.
int64_t chunk_rows(int64_t rows, int64_t groups, int64_t ctas, int64_t step, int64_t fill,
                   int64_t most) {
  int64_t best = 0, chunk = step;
  for (int64_t c = step; c - step < rows && c <= most; c += step) {
    const int64_t waves = ((rows + c - 1) / c * groups + ctas - 1) / ctas;
    const int64_t cost = waves * (c + fill);
    if (best == 0 || cost < best) {
      best = cost;
      chunk = c;
    }
  }
  return chunk;
}
}  // namespace

// Subspaces whose dims fill whole columns of 8.
static int unit_subspaces(int ds) { return ds % 8 == 0 ? 1 : ds % 4 == 0 ? 2 : ds % 2 == 0 ? 4 : 8; }

static size_t unit_bytes(int K, int L, int ds) {
  return (size_t)unit_subspaces(ds) * L * (((size_t)K * ds + 3) & ~(size_t)3) * 4;
}

// A thread a row: dims and levels that it is compiled for, where a unit's
// codebooks fit in shared memory.
bool decode_rows_ok(int K, int L, int ds) {
  return (ds == 8 || (ds >= 2 && ds <= 6)) && L <= 3 && unit_bytes(K, L, ds) <= 220 * 1024;
}

static cudaError_t launch_decode_rows(const CodeSrc &cs, const float *C, int M, int L, int ds, int64_t v0,
                               int64_t rows, int64_t pitch, const float *amax, __half *hi,
                               __half *lo, const DwPlanes &dw, const DevInfo &di, cudaStream_t s) {
  size_t smem = unit_bytes(cs.K, L, ds);
  const int units = (M + unit_subspaces(ds) - 1) / unit_subspaces(ds);
  const int64_t bits = cs.fmt == RQ_CODES_U16       ? 16
                       : cs.fmt == RQ_CODES_U8       ? 8
                       : cs.fmt == RQ_CODES_PACKED10 ? 10
                                                     : 0;
  const int64_t row = (bits * cs.P + 7) / 8;
  int vec = bits == 0 ? 0 : row % 16 == 0 ? 4 : row % 4 == 0 ? 1 : 0;
  // by TMA where a unit's codes never cross a word (they start at multiples of
  // gcd(their bits, 128)), two stages fit beside the books and a thread has rows
  // enough (8192 rows of 96 units, 10 a thread: 39 us, 36 by loads; 32768 99, 104)
  const int64_t unit = bits * unit_subspaces(ds) * L, low = unit & -unit;
  const int64_t fit = (226 * 1024 - 128 - (int64_t)smem) / (kRowWarps * 512);
  if (vec == 4 && unit + 128 - (low < 128 ? low : 128) <= 128 && fit >= 2 &&
      M % unit_subspaces(ds) == 0 && rows * units >= 24 * (int64_t)di.sms * kRowThreads)
    vec = 16;
  const void *fn = ds == 2   ? rows_fn<2>(L, vec)
                   : ds == 3 ? rows_fn<3>(L, vec)
                   : ds == 4 ? rows_fn<4>(L, vec)
                   : ds == 5 ? rows_fn<5>(L, vec)
                   : ds == 6 ? rows_fn<6>(L, vec)
                   : ds == 8 ? rows_fn<8>(L, vec)
                             : nullptr;
  if (!fn) return cudaErrorInvalidValue;
  DecodeRows a;
  a.cs = cs;
  a.C = C;
  a.M = M;
  a.units = units;
  a.bits = (int)bits;
  a.v0 = v0;
  a.rows = rows;
  a.pitch = pitch;
  a.amax = amax;
  a.hi = hi;
  a.lo = lo;
  a.cols = (M * ds + 7) / 8;
  a.dw = dw;
  a.pairs = (reinterpret_cast<uintptr_t>(C) & 7) == 0 && cs.K * ds % 2 == 0;
  a.err = di.err;
  a.stages = fit < kRowStages ? (int)fit : kRowStages;
  CUtensorMap map = {};
  if (vec == 16) {
    smem += 128 + (size_t)a.stages * kRowWarps * 512;
    if (!encode_tmap_2d_u16(&map, cs.codes, (uint64_t)row / 2, (uint64_t)cs.V, (uint64_t)row, 8, 32,
                            CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  }
  const cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)di.sms * occupancy_cached(fn, di.device, kRowThreads, smem);
  a.chunk = (int)chunk_rows(rows, a.units, ctas, kRowThreads,
                            (int64_t)(650 * smem / (192 * 1024)) + 64, 16384);
  const int64_t items = (rows + a.chunk - 1) / a.chunk * a.units;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  a.items = (int)items;
  void *args[] = {&map, &a};
  const int64_t all = items + dw.N;
  return launch_maybe_pdl(fn, dim3((unsigned)(all < ctas ? all : ctas)), dim3(kRowThreads), smem,
                          s, args, true);
}

cudaError_t launch_loss_decode(const CodeSrc &cs, const float *C, int M, int L, int ds, int64_t v0,
                               int64_t rows, int64_t pitch, const float *amax, __half *hi,
                               __half *lo, const DwPlanes &dw, const DevInfo &di, cudaStream_t s) {
  if (decode_rows_ok(cs.K, L, ds))
    return launch_decode_rows(cs, C, M, L, ds, v0, rows, pitch, amax, hi, lo, dw, di, s);
  DecodeArgs a;
  a.cs = cs;
  a.C = C;
  a.M = M;
  a.L = L;
  a.ds = ds;
  a.v0 = v0;
  a.rows = rows;
  a.pitch = pitch;
  a.amax = amax;
  a.hi = hi;
  a.lo = lo;
  a.book = (int64_t)L * cs.K * ds;
  a.dw = dw;
  // as many subspaces as their codebooks fit in shared memory, a whole number of
  // pairs unless one group has them all, and at most a pair per thread unless
  // the fewest have more
  const int64_t fit = 220 * 1024 / 4 / a.book;
  const bool even = ds % 2 == 0;
  const int64_t fewest = even || M == 1 ? 1 : 2;
  const bool in_smem = fit >= fewest;
  int64_t gs = in_smem ? fit : M;
  if (gs > M) gs = M;
  if (gs * ds > 2 * kDecThreads) gs = 2 * kDecThreads / ds;
  if (gs < fewest) gs = fewest;
  if (!even && gs < M) gs -= gs % 2;
  a.gs = (int)gs;
  a.groups = (M + a.gs - 1) / a.gs;
  // even groups: fewer leftovers
  a.gs = (M + a.groups - 1) / a.groups;
  if (!even && a.gs < M) a.gs += a.gs % 2;
  a.groups = (M + a.gs - 1) / a.gs;
  const size_t smem = in_smem ? (size_t)a.gs * a.book * 4 : 0;
  a.quad = (reinterpret_cast<uintptr_t>(C) & 15) == 0 && a.gs * a.book % 4 == 0;
  const void *fn = even ? (in_smem ? decode_fn<true, true>(L) : decode_fn<true, false>(L))
                        : (in_smem ? decode_fn<false, true>(L) : decode_fn<false, false>(L));
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  const int occ = occupancy_cached(fn, di.device, kDecThreads, smem);
  const int words = (a.gs * ds + 1) / 2;
  const int rstep = words < kDecThreads ? kDecThreads / words : 1;
  const int64_t ctas = (int64_t)di.sms * occ;
  // rows per chunk: the shortest time of the last CTA, an item costing its rows
  // and the load of its books (as long as about 300 rows of 48 KB books a
  // subspace, less for smaller ones)
  const int64_t load = in_smem ? 300 * a.book / (2 * 1024 * 6) + 32 : 32;
  const int64_t chunk = chunk_rows(rows, a.groups, ctas, rstep, load, 4096);
  a.chunk = (int)chunk;
  const int64_t items = (rows + chunk - 1) / chunk * a.groups;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  a.items = (int)items;
  void *args[] = {&a};
  const int64_t all = items + dw.N;
  return launch_maybe_pdl(fn, dim3((unsigned)(all < ctas ? all : ctas)), dim3(kDecThreads), smem,
                          s, args, true);
}

cudaError_t launch_loss_logits(const float *logits, int64_t N, int64_t V, const LossTargets &t,
                               float *loss, float *lse, unsigned *err, cudaStream_t s) {
  return pdl_launch(loss_logits_kernel, dim3(kServeCtas, (unsigned)N), dim3(1024), (size_t)0, s,
                    logits, V, t, loss, lse, err);
}

cudaError_t launch_loss_finish(const float2 *stat, int parts, int stat_ld, int64_t N, int64_t V,
                               const LossTargets &t, const float *y, float *loss, float *lse,
                               unsigned *err, cudaStream_t s) {
  return pdl_launch(loss_finish_kernel, dim3(blocks_of(N, kFinishRows)), dim3(1024), (size_t)0, s,
                    stat, parts, stat_ld, N, V, t, y, loss, lse, err);
}

cudaError_t launch_loss_dz(const float *logits, int64_t N, int64_t V, const float *lse,
                           const float *f, float beta, float cap, float *dz, int64_t pitch,
                           cudaStream_t s) {
  return pdl_launch(loss_dz_kernel, dim3(blocks_of(pitch, 1024), (unsigned)((N + 1) / 2)), dim3(256),
                    (size_t)0, s, logits, N, V, lse, f, beta, cap, dz, pitch);
}

cudaError_t launch_loss_fix(const int32_t *sid, const float *sq, const float *logits, int k,
                            int64_t N, int64_t V, const float *lse, const float *f, float beta,
                            float cap, float *dz, int64_t pitch, cudaStream_t s) {
  return pdl_launch(loss_fix_kernel, dim3(blocks_of(N * k, 256)), dim3(256), (size_t)0, s, sid, sq,
                    logits, k, N * k, V, lse, f, beta, cap, dz, pitch);
}

cudaError_t launch_loss_dh_sum(const float *part, int splits, int64_t stride, int64_t pitch,
                               int64_t N, int D, int bf16, void *dh, cudaStream_t s) {
  return pdl_launch(loss_dh_sum_kernel, dim3(blocks_of(N * D, 256)), dim3(256), (size_t)0, s, part, splits, stride, pitch, N, D, bf16, dh);
}

}  // namespace rq
