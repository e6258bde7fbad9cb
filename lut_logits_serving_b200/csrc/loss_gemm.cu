// loss_gemm.cu -- the tensor-core products of the loss kernels, each fused
// with what it feeds:
//
//   kGemmStats  y = cap tanh(h E^T / cap); per row and 128 columns the
//               maximum of y / T and the sum of exp(y / T - max)
//   kGemmGrad   y again; dz = w T exp(y / T - lse) (1 - (y / cap)^2), as fp16
//               planes for the next two, or (kGemmGrad32) in fp32
//   kGemmDh     dz E       (contraction over the rows of the vocabulary)
//   kGemmDw     h^T dz     (contraction over the tokens)
//
// Mathematics.  Every operand is an fp16 hi / lo pair of planes scaled by a
// power of two (loss_common.cuh), so a product of two fp32 operands is three
// tensor-core products, a_hi b_hi + a_lo b_hi + a_hi b_lo (two where one
// operand is bf16, which a scaled fp16 plane holds exactly).  The tensor
// core's fp32 accumulator does not round to nearest and its error grows with
// the chain of MMAs, so a chain covers `chain` blocks of 64 of the
// contraction; a finished chain is added to fp32 registers, round to nearest,
// while the next one runs into the other half of tensor memory.
//
// One persistent CTA per SM: a copy warp (TMA tiles of 64 contraction
// elements, 128-byte swizzle), an MMA warp (128 x 256 x 16 tcgen05.mma, both
// operands in shared memory), eight warps that own the accumulators (a thread
// has one row and 128 columns) and run the epilogue.  Operands whose
// contraction runs down the rows of a row-major matrix are read as they lie
// (MN-major tiles), so nothing is stored twice.  Every wait is bounded; one
// that runs out raises RQ_DEVERR_TIMEOUT, lets copies and MMAs in flight
// land, frees tensor memory and ends the CTA.
#include "loss_common.cuh"

namespace rq {

namespace {

constexpr int kTM = 128, kTN = 256, kTK = 64;
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (kEpiWarps + 2) * 32;
constexpr int kMaxStages = 6;
constexpr int kABytes = kTM * kTK * 2, kBBytes = kTN * kTK * 2;
constexpr size_t kGemmSmemMax = 225 * 1024;   // 227 KB less the static part
constexpr size_t kGemmSmemTail = 1024 + 256;   // alignment slack, barriers

// Shared-memory matrix descriptor: 128-byte swizzle (layout type 2), version
// 1.  K-major tiles are rows of 64 elements (128 bytes), 8-row groups 1024
// bytes apart.  MN-major tiles are rows of 64 MN-elements, one row per
// contraction index: 8 KB from one 64-wide block to the next (leading byte
// offset), 1024 bytes between groups of 8 contraction indices (stride).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum));
}

__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void ld16(uint32_t t, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(t));
}

__device__ __forceinline__ void st16(uint32_t t, const float *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(t),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]),
      "f"(r[15]));
}

// 32 bytes, a whole sector, at once
__device__ __forceinline__ void stg32(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace

template <int MODE>
__global__ void __launch_bounds__(kGemmThreads, 1)
    loss_gemm_kernel(const __grid_constant__ CUtensorMap a_hi, const __grid_constant__ CUtensorMap a_lo,
                     const __grid_constant__ CUtensorMap b_hi, const __grid_constant__ CUtensorMap b_lo,
                     const GemmArgs g) {
  constexpr bool LOGITS = MODE == kGemmStats || MODE == kGemmGrad || MODE == kGemmGrad32;
  constexpr bool A_MN = MODE == kGemmDw;                        // contraction down the rows of A
  constexpr bool B_MN = MODE == kGemmDh || MODE == kGemmDw;     // and of B
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = (uint32_t)(g.a_planes * kABytes + g.b_planes * kBBytes);
  const uint32_t bars = base + (uint32_t)g.stages * stage_bytes;
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (kMaxStages + i); };
  auto tfull = [&](int i) { return bars + 8u * (2 * kMaxStages + i); };
  auto tempty = [&](int i) { return bars + 8u * (2 * kMaxStages + 2 + i); };
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    prefetch_tmap(&a_hi);
    prefetch_tmap(&b_hi);
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), kEpiWarps);
    }
    fence_mbar_init();
    abort_flag = 0;
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_launch_dependents();
  tc_before();
  __syncthreads();
  tc_after();
  griddep_wait();
  const uint32_t tmem = tmem_slot;

  const int mn = g.m_tiles * g.n_tiles, total = mn * g.splits;
  bool to = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!to && !mbar_try_wait(bar, parity) && !mbar_wait_bounded(bar, parity)) {
      to = true;
      abort_flag = 1;
    }
    return !to;
  };

  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_last();
      int it = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x) {
        const int sp = t / mn, r = t % mn, n0 = r / g.m_tiles * kTN, m0 = r % g.m_tiles * kTM;
        const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
        const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
        for (int k = k0; k < k1; ++k, ++it) {
          const int st = it % g.stages;
          if (!wait(empty(st), ((uint32_t)(it / g.stages) & 1u) ^ 1u)) break;
          mbar_arrive_expect_tx(full(st), stage_bytes);
          uint32_t dst = base + (uint32_t)st * stage_bytes;
          for (int p = 0; p < g.a_planes; ++p, dst += kABytes) {
            const CUtensorMap *map = p ? &a_lo : &a_hi;
            if (A_MN) {
              for (int i = 0; i < kTM / 64; ++i)
                tma_load_2d(dst + i * 8192, map, m0 + i * 64, k * kTK, full(st), pol);
            } else {
              tma_load_2d(dst, map, k * kTK, m0, full(st), pol);
            }
          }
          for (int p = 0; p < g.b_planes; ++p, dst += kBBytes) {
            const CUtensorMap *map = p ? &b_lo : &b_hi;
            if (B_MN) {
              for (int i = 0; i < kTN / 64; ++i)
                tma_load_2d(dst + i * 8192, map, n0 + i * 64, k * kTK, full(st), pol);
            } else {
              tma_load_2d(dst, map, k * kTK, n0, full(st), pol);
            }
          }
        }
        if (to) break;
      }
      if (abort_flag) {
        // the last copy into each stage lands before the shared memory goes
        for (int st = 0; st < g.stages; ++st) {
          const int last = it - 1 - ((it - 1 - st) % g.stages + g.stages) % g.stages;
          if (it > 0 && last >= 0) mbar_wait_bounded(full(st), (uint32_t)(last / g.stages) & 1u);
        }
        atomicOr(g.err, RQ_DEVERR_TIMEOUT);
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t idesc = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                             ((uint32_t)(kTN >> 3) << 17) | ((uint32_t)(kTM >> 4) << 24);
      // 16 contraction elements further: 32 bytes along a K-major row, 16
      // rows of 128 bytes in an MN-major tile (in descriptor units of 16 B)
      constexpr uint32_t a_step = A_MN ? 2048 / 16 : 32 / 16, b_step = B_MN ? 2048 / 16 : 32 / 16;
      int it = 0, c = 0;
      for (int t = blockIdx.x; t < total && !abort_flag; t += gridDim.x) {
        const int sp = t / mn;
        const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
        const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
        for (int ka = k0; ka < k1; ka += g.chain, ++c) {
          if (!wait(tempty(c & 1), ((uint32_t)(c >> 1) & 1u) ^ 1u)) break;
          tc_after();
          const uint32_t d = tmem + (uint32_t)(c & 1) * kTN;
          const int kb = ka + g.chain < k1 ? ka + g.chain : k1;
          for (int k = ka; k < kb; ++k, ++it) {
            const int st = it % g.stages;
            if (!wait(full(st), (uint32_t)(it / g.stages) & 1u)) break;
            tc_after();
            const uint32_t sa = base + (uint32_t)st * stage_bytes;
            const uint32_t sb = sa + (uint32_t)g.a_planes * kABytes;
            const uint64_t ah = sw128_desc(sa, A_MN ? 8192 : 16);
            const uint64_t bh = sw128_desc(sb, B_MN ? 8192 : 16);
            const uint64_t al = ah + kABytes / 16, bl = bh + kBBytes / 16;
#pragma unroll
            for (int j = 0; j < kTK / 16; ++j)
              mma_f16_ss(d, ah + j * a_step, bh + j * b_step, idesc, k > ka || j > 0);
            if (g.a_planes > 1) {
#pragma unroll
              for (int j = 0; j < kTK / 16; ++j)
                mma_f16_ss(d, al + j * a_step, bh + j * b_step, idesc, 1u);
            }
            if (g.b_planes > 1) {
#pragma unroll
              for (int j = 0; j < kTK / 16; ++j)
                mma_f16_ss(d, ah + j * a_step, bl + j * b_step, idesc, 1u);
            }
            tc_commit(empty(st));
          }
          if (to) break;
          tc_commit(tfull(c & 1));
        }
        if (to) break;
      }
      if (abort_flag) {
        // the MMAs in flight end before the tensor memory goes
        if (it > 0)
          mbar_wait_bounded(empty((it - 1) % g.stages), (uint32_t)((it - 1) / g.stages) & 1u);
        atomicOr(g.err, RQ_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------ accumulators
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)half * 128;
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      bool ok = to || mbar_try_wait(bar, parity) || mbar_wait_bounded(bar, parity);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && !to) {
        to = true;
        abort_flag = 1;
      }
      return !to;
    };
    const float sh = MODE != kGemmDh ? scale_h(g.amax) : 1.f;
    const float se = MODE != kGemmDw ? scale_e(g.amax, g.L) : 1.f;
    const float sz = MODE != kGemmStats && MODE != kGemmGrad32 ? scale_z(g.amax, g.T) : 1.f;
    const float inv = MODE == kGemmDh ? 1.f / (sz * se) : MODE == kGemmDw ? 1.f / (sz * sh)
                                                                          : 1.f / (sh * se);
    float acc[128];
    int c = 0;
    for (int t = blockIdx.x; t < total && !to; t += gridDim.x) {
      const int sp = t / mn, r = t % mn, nt = r / g.m_tiles;
      const int col0 = nt * kTN + half * 128, row = r % g.m_tiles * kTM + q * 32 + lane;
      const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
      const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      for (int ka = k0; ka < k1; ka += g.chain, ++c) {
        if (!wait_all(tfull(c & 1), (uint32_t)(c >> 1) & 1u)) break;
        tc_after();
        const uint32_t src = lanes + (uint32_t)(c & 1) * kTN;
#pragma unroll
        for (int j0 = 0; j0 < 128; j0 += 32) {
          float x[16], y[16];
          ld16(src + j0, x);
          ld16(src + j0 + 16, y);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            acc[j0 + j] = __fadd_rn(acc[j0 + j], x[j]);
            acc[j0 + 16 + j] = __fadd_rn(acc[j0 + 16 + j], y[j]);
          }
        }
        if (LOGITS && ka + g.chain >= k1) {
          // the tile's sums back into the chain's columns, from where the
          // epilogue takes them 16 at a time (the registers cannot be indexed
          // by a loop, and 128 unrolled tanh and exp would not fit the
          // instruction cache)
#pragma unroll
          for (int j0 = 0; j0 < 128; j0 += 16) st16(src + j0, acc + j0);
          wait_st();
          const float cap = g.cap, icap = g.inv_cap;
          if (MODE == kGemmStats) {
            float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
            for (int j0 = 0; j0 < 128; j0 += 16) {
              float x[16];
              ld16(src + j0, x);
              wait_ld();
              float cm = -INFINITY;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float z = x[j] * inv;
                const float y = cap > 0.f ? cap * tanhf(z * icap) : z;
                x[j] = col0 + j0 + j < g.cols ? y * g.beta : -INFINITY;
                cm = fmaxf(cm, x[j]);
              }
              const float nm = fmaxf(mx, cm);
              if (nm > -INFINITY) {
                sum *= expf(mx - nm);
#pragma unroll
                for (int j = 0; j < 16; ++j) sum += expf(x[j] - nm);
              } else {      // no column, or NaN in all of them
#pragma unroll
                for (int j = 0; j < 16; ++j) sum += x[j] != x[j] ? x[j] : 0.f;
              }
              mx = nm;
            }
            if (row < g.rows)
              g.stat[(int64_t)(g.stat_part0 + nt * 2 + half) * g.stat_ld + row] =
                  make_float2(mx, sum);
          } else {
            const bool in = row < g.rows;
            const float f = in ? g.f[row] : 0.f, lse = in ? g.lse[row] : 0.f, fs = f * sz;
            const int64_t at = (int64_t)row * g.dz_pitch + col0;
#pragma unroll 1
            for (int j0 = 0; j0 < 128; j0 += 16) {
              float x[16];
              ld16(src + j0, x);
              wait_ld();
              __half2 hi[8], lo[8];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float z = x[j] * inv;
                float y = z, slope = 1.f;
                if (cap > 0.f) {
                  const float th = tanhf(z * icap);
                  y = cap * th;
                  slope = 1.f - th * th;
                }
                const float d = f != 0.f ? expf(y * g.beta - lse) * slope * fs : 0.f;
                if (MODE == kGemmGrad32) {
                  x[j] = d;
                  continue;
                }
                __half dh, dl;
                split_f16(d, dh, dl);
                if (j & 1) {
                  hi[j / 2].y = dh;
                  lo[j / 2].y = dl;
                } else {
                  hi[j / 2].x = dh;
                  lo[j / 2].x = dl;
                }
              }
              if (in) {
                if (MODE == kGemmGrad32) {
                  if (col0 + j0 < g.cols) {        // the rows' pitch is 16 floats
                    stg32(g.dz + at + j0, reinterpret_cast<const uint32_t *>(x));
                    stg32(g.dz + at + j0 + 8, reinterpret_cast<const uint32_t *>(x + 8));
                  }
                } else if (col0 + j0 < g.dz_pitch) {   // the pitch is whole sectors
                  stg32(g.dz_hi + at + j0, reinterpret_cast<const uint32_t *>(hi));
                  stg32(g.dz_lo + at + j0, reinterpret_cast<const uint32_t *>(lo));
                }
              }
            }
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) arrive(tempty(c & 1));
      }
      if (to) break;
      if ((MODE == kGemmDh || MODE == kGemmDw) && row < g.rows) {
        float *o = g.out + (int64_t)sp * g.out_split + (int64_t)row * g.out_pitch + col0;
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
          if (col0 + j < g.out_pitch) {
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = acc[j + x] * inv;
            if (MODE == kGemmDh && g.accumulate) {
#pragma unroll
              for (int x = 0; x < 8; x += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(o + j + x);
                v[x] += w.x;
                v[x + 1] += w.y;
                v[x + 2] += w.z;
                v[x + 3] += w.w;
              }
            }
            stg32(o + j, reinterpret_cast<const uint32_t *>(v));
          }
        }
      }
    }
    if (to && lane == 0) atomicOr(g.err, RQ_DEVERR_TIMEOUT);
  }
  tc_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

namespace {

bool plane_map(CUtensorMap *m, const void *p, const GemmPlanes &x, bool mn, int tile) {
  return encode_tmap_2d_u16(m, p, (uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.pitch * 2, 64,
                            mn ? 64 : (uint32_t)tile, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE>
cudaError_t launch_gemm(const GemmPlanes &A, const GemmPlanes &B, GemmArgs a, const DevInfo &di,
                        cudaStream_t s) {
  constexpr bool A_MN = MODE == kGemmDw, B_MN = MODE == kGemmDh || MODE == kGemmDw;
  CUtensorMap ah, al, bh, bl;
  if (!plane_map(&ah, A.hi, A, A_MN, kTM) || !plane_map(&al, A.lo ? A.lo : A.hi, A, A_MN, kTM) ||
      !plane_map(&bh, B.hi, B, B_MN, kTN) || !plane_map(&bl, B.lo ? B.lo : B.hi, B, B_MN, kTN))
    return cudaErrorInvalidValue;
  const int64_t k = A_MN ? A.rows : A.cols;
  a.a_planes = A.lo ? 2 : 1;
  a.b_planes = B.lo ? 2 : 1;
  a.m_tiles = (int)(((A_MN ? A.cols : A.rows) + kTM - 1) / kTM);
  a.n_tiles = (int)(((B_MN ? B.cols : B.rows) + kTN - 1) / kTN);
  a.kblocks = (int)((k + kTK - 1) / kTK);
  if (a.splits < 1) a.splits = 1;
  if (a.splits > a.kblocks) a.splits = a.kblocks;
  const size_t stage = (size_t)a.a_planes * kABytes + (size_t)a.b_planes * kBBytes;
  int st = (int)((kGemmSmemMax - kGemmSmemTail) / stage);
  a.stages = st > kMaxStages ? kMaxStages : st;
  const size_t smem = kGemmSmemTail + a.stages * stage;
  const void *fn = reinterpret_cast<const void *>(&loss_gemm_kernel<MODE>);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  const int64_t total = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  if (total < 1 || total > 0x7fffffff) return cudaErrorInvalidValue;
  const int grid = (int)(total < di.sms ? total : di.sms);
  void *args[] = {&ah, &al, &bh, &bl, &a};
  return launch_maybe_pdl(fn, dim3(grid), dim3(kGemmThreads), smem, s, args, true);
}

}  // namespace

cudaError_t launch_loss_gemm(int mode, const GemmPlanes &A, const GemmPlanes &B, GemmArgs a,
                             const DevInfo &di, cudaStream_t s) {
  switch (mode) {
    case kGemmStats: return launch_gemm<kGemmStats>(A, B, a, di, s);
    case kGemmGrad: return launch_gemm<kGemmGrad>(A, B, a, di, s);
    case kGemmDh: return launch_gemm<kGemmDh>(A, B, a, di, s);
    case kGemmDw: return launch_gemm<kGemmDw>(A, B, a, di, s);
    case kGemmGrad32: return launch_gemm<kGemmGrad32>(A, B, a, di, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace rq
