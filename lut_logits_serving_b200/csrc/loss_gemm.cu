// loss_gemm.cu -- the tensor-core products of the loss kernels, each fused
// with what it feeds:
//
//   kGemmStats  y = cap tanh(h E^T / cap); per row and half a tile's columns
//               the maximum m of y / T and the sum of exp(y / T - m)
//   kGemmGrad   y again; dz = w T exp(y / T - lse) (1 - (y / cap)^2), as fp16
//               planes for the next two, or (kGemmGrad32) in fp32
//   kGemmDh     dz E       (contraction over the rows of the vocabulary)
//   kGemmDw     dz^T h     (contraction over the tokens)
//
// Mathematics.  Every operand is an fp16 hi / lo pair of planes scaled by a
// power of two (loss_common.cuh), so a product of two fp32 operands is three
// tensor-core products, a_hi b_hi + a_lo b_hi + a_hi b_lo (two where one
// operand is bf16, which a scaled fp16 plane holds exactly).  The tensor
// core's fp32 accumulator does not round to nearest and its error grows with
// the chain of MMAs, so a chain has 12 to 48 of them, the small products of each
// block first (each MMA costs the running sum half a unit in its last place;
// with a_hi b_hi first the errors are half as large again); a finished chain is
// added to fp32 registers, round to nearest, while the next one runs into the
// other half of tensor memory.
//
// Listed ids (targets, a teacher's lists) are served where their logits are: a
// tile's threads find those of their row and columns by bisection in the row's
// sorted list, write their logits (a loss) or subtract their probabilities.  A
// logit formed anew elsewhere would differ in its last bits from the one in
// the log-sum-exp, and 1 - p of a confident row with it (a loss of 61 such rows
// 1.6e-6 off instead of 3e-7, its gradients 8e-6).
//
// One persistent CTA per SM: a copy warp (TMA tiles of 64 contraction
// elements, 128-byte swizzle), an MMA warp (tcgen05.mma, both operands in
// shared memory), eight warps that own the accumulators (a thread has one row
// and half the tile's columns) and run the epilogue.  Operands whose
// contraction runs down the rows of their matrix are read as they lie (MN-major
// tiles), so nothing is stored twice; the decoded rows come in blocks of 8 x 8
// that serve either way without a swizzle.
//
// Tiles.  A CTA pair shares a 256 x 256 tile (cta_group::2: each SM holds its
// 128 rows of A and half of B): one SM alone on 128 x 256 would read
// (128 + 256) x 32 bytes of shared memory per MMA of 128 cycles and take in 64
// bytes a cycle of new tiles on top, more than the 128 bytes a cycle there
// are; a pair needs two thirds of that.  A single SM takes 128 x 256 where the
// rows fill no pair, and 128 x 64 where wider tiles would leave most SMs
// without one.
//
// Every wait is bounded; one that runs out raises RQ_DEVERR_TIMEOUT, lets
// copies and MMAs in flight land, frees tensor memory and ends the CTA.
#include <cudaTypedefs.h>

#include "loss_common.cuh"

namespace rq {

namespace {

constexpr int kTM = 128, kTK = 64;               // rows of a CTA, contraction block
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = (kEpiWarps + 4) * 32;   // + copy, MMA, two idle: whole warpgroups
constexpr int kMaxStages = 8;
constexpr int kABytes = kTM * kTK * 2;
// MMAs of one accumulation chain.  Errors of dC and dh against 64 bits (500
// fp32 tokens, 256000 rows): chains of 48 (dz^T h 36) 6.7e-7 and 7.1e-7, of 36
// (24) 4.7e-7 and 5.4e-7 for 2 to 8 % of a product's time; an fp32 library
// product leaves 8.4e-7 and 1.6e-6.  Short contractions (up to 4 blocks, where
// nothing is left to overlap) take short chains.  So do the logits of up to 128
// tokens, which the planes of E bound: 130 us per 65536 rows instead of 122, and
// a single confident row, whose logit all MMAs round in one direction, keeps a
// relative error of its loss of 1e-6 (3e-6 with longer ones).
constexpr int kChainMmas = 48, kChainMmasDw = 36, kChainMmasShort = 12;
constexpr size_t kGemmSmemMax = 226 * 1024;      // 227 KB less the static part
constexpr int kStoreBytes = 16384;               // a warpgroup's outgoing 128 rows x 128 bytes
constexpr size_t kGemmSmemTail = 1024 + 256;     // alignment slack, barriers

// Shared-memory matrix descriptor: 128-byte swizzle (layout type 2), version
// 1.  K-major tiles are rows of 64 elements (128 bytes), 8-row groups 1024
// bytes apart.  MN-major tiles are rows of 64 MN-elements, one row per
// contraction index: 8 KB from one 64-wide block to the next (leading byte
// offset), 1024 bytes between groups of 8 contraction indices (stride).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Descriptor of a tile without a swizzle, of blocks of 8 rows x 16 bytes that
// are 128 bytes in one piece.  `lead`: from one block to the next along the
// contraction; `stride`: along the other extent.
__device__ __forceinline__ uint64_t block_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(stride >> 4) << 32) | (1ull << 46);
}

template <int CG>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accum) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
}

// MMAs issued so far done: arrive at `bar`, in both CTAs of a pair.
template <int CG>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// 2-D tiled load into this CTA's shared memory; of a pair, completing on the
// first CTA's barrier (the shared-window address with the rank bit cleared).
template <int CG>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int x, int y,
                                          uint32_t bar, uint64_t pol) {
  if (CG == 1)
    tma_load_2d(dst, map, x, y, bar, pol);
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar & 0xFEFFFFFFu), "l"(pol)
        : "memory");
}

// The same of a tile of 8 x 8 blocks: block row y, column of blocks z.
template <int CG>
__device__ __forceinline__ void load_blocks(uint32_t dst, const CUtensorMap *map, int y, int z,
                                            uint32_t bar, uint64_t pol) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "l"(pol)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar & 0xFEFFFFFFu),
        "l"(pol)
        : "memory");
}

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Arrive at the barrier of the pair's first CTA.
__device__ __forceinline__ void arrive_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}\n" ::"r"(bar)
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

// 32 bytes, a whole sector, at once
__device__ __forceinline__ void stg32(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The gradients' planes leave through shared memory as TMA stores: a thread has
// a row, and stored directly a warp's words go to 32 rows, a sector each, which
// keeps the threads from the next tile's sums.
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void store_tile(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void async_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void group_sync(int id) {     // the 128 threads of a warpgroup
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_any(int id, bool x) {   // of them, whether any has x
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

// 2^x; results below the smallest normal number are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh without a branch, for an epilogue that evaluates many at once: below
// 0.6 x + x^3 P(x^2), P of degree 4 a least-maximum fit of (tanh x - x) / x^3
// (3e-9 of tanh x), above (1 - e) / (1 + e) with e = exp(-2 |x|).  At most 2.3
// units in the last place off over all floats (tanhf 1.8).  A function with a
// branch keeps a warp from having several columns under way: per 65536 rows,
// statistics of 500 fp32 tokens 354 us with tanhf and exp2f, 332 so, 322 with
// neither; gradients 395, 354, 345 (2048 bf16 tokens 1130, 1030, 880; 1386,
// 1110, 950).
__device__ __forceinline__ float tanh_flat(float x) {
  const float e = ex2(fabsf(x) * -2.885390082f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  const float u = x * x;
  float p = fmaf(u, -5.895151122e-3f, 2.079596527e-2f);
  p = fmaf(u, p, -5.378382821e-2f);
  p = fmaf(u, p, 1.333192410e-1f);
  p = fmaf(u, p, -3.333329800e-1f);
  const float s = fmaf(x * u, p, x), b = copysignf((1.f - e) * r, x);
  return fabsf(x) < 0.6f ? s : b;
}

__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
}  // namespace

template <int MODE, int CG, int TN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    loss_gemm_kernel(const __grid_constant__ CUtensorMap a_hi, const __grid_constant__ CUtensorMap a_lo,
                     const __grid_constant__ CUtensorMap b_hi, const __grid_constant__ CUtensorMap b_lo,
                     const __grid_constant__ CUtensorMap o_hi, const __grid_constant__ CUtensorMap o_lo,
                     const GemmArgs g) {
  constexpr bool STAGED = MODE == kGemmGrad;                    // output through TMA
  constexpr bool LOGITS = MODE == kGemmStats || MODE == kGemmGrad || MODE == kGemmGrad32;
  constexpr bool A_MN = MODE == kGemmDw;                        // contraction down the rows of A
  constexpr bool B_MN = MODE == kGemmDh || MODE == kGemmDw;     // and of B
  constexpr bool B_ROWS = MODE != kGemmDw;       // B is decoded rows, 8 x 8 blocks
  constexpr int BN = TN / CG;                    // columns of B in this CTA's shared memory
  constexpr int HALF = TN / 2;                   // columns of an accumulator thread
  constexpr int B_BYTES = BN * kTK * 2;
  constexpr uint32_t TMEM_COLS = 2 * TN;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = (uint32_t)(g.a_planes * kABytes + g.b_planes * B_BYTES);
  const uint32_t staging = base + (uint32_t)g.stages * stage_bytes;
  const uint32_t bars = staging + (STAGED ? 2 * kStoreBytes : 0);
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (kMaxStages + i); };
  auto tfull = [&](int i) { return bars + 8u * (2 * kMaxStages + i); };
  auto tempty = [&](int i) { return bars + 8u * (2 * kMaxStages + 2 + i); };
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CG == 2 ? (int)cta_rank() : 0;
  if (tid == 0) {
    prefetch_tmap(&a_hi);
    prefetch_tmap(&b_hi);
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull(i), 1);
      mbar_init(tempty(i), kEpiWarps * CG);
    }
    fence_mbar_init();
    abort_flag = 0;
  }
  if (CG == 2) cluster_sync_all();               // the pair's barriers exist
  if (warp == kEpiWarps + 1) {
    if (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmem_slot)),
                   "r"(TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmem_slot)),
                   "r"(TMEM_COLS));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  griddep_launch_dependents();
  tc_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();               // and its tensor memory
  tc_after();
  griddep_wait();
  const uint32_t tmem = tmem_slot;

  // CTA (or pair) `unit` of `units` takes every units-th tile
  const int unit = blockIdx.x / CG, units = gridDim.x / CG;
  const int mn = g.m_tiles * g.n_tiles, total = mn * g.splits;
  // the operand with fewer tiles stays in the L2, so its tiles change fastest
  auto m_tile = [&](int r) { return MODE == kGemmDw ? r / g.n_tiles : r % g.m_tiles; };
  auto n_tile = [&](int r) { return MODE == kGemmDw ? r % g.n_tiles : r / g.m_tiles; };
  bool to = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!to && !mbar_try_wait(bar, parity) && !mbar_wait_bounded(bar, parity)) {
      to = true;
      abort_flag = 1;
    }
    return !to;
  };

  // the accumulating warpgroups take over registers that the third does not
  // need: 8 x 232 + 4 x 40 = 12 x 168, the launch's total
  if (warp >= kEpiWarps) {
    if (TN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kEpiWarps) {
      // ------------------------------------------------------------ copies
      if (lane == 0) {
        const uint64_t pol = l2_policy_evict_last();
        int it = 0;
        for (int t = unit; t < total && !abort_flag; t += units) {
          const int sp = t / mn, r = t % mn;
          const int n0 = n_tile(r) * TN + rank * BN;
          const int m0 = (m_tile(r) * CG + rank) * kTM;
          const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
          const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
          for (int k = k0; k < k1; ++k, ++it) {
            const int st = it % g.stages;
            if (!wait(empty(st), ((uint32_t)(it / g.stages) & 1u) ^ 1u)) break;
            // a pair's first CTA expects both CTAs' bytes
            if (rank == 0) mbar_arrive_expect_tx(full(st), stage_bytes * CG);
            uint32_t dst = base + (uint32_t)st * stage_bytes;
            for (int p = 0; p < g.a_planes; ++p, dst += kABytes) {
              const CUtensorMap *map = p ? &a_lo : &a_hi;
              if (A_MN) {
#pragma unroll
                for (int i = 0; i < kTM / 64; ++i)
                  load_tile<CG>(dst + i * 8192, map, m0 + i * 64, k * kTK, full(st), pol);
              } else {
                load_tile<CG>(dst, map, k * kTK, m0, full(st), pol);
              }
            }
            for (int p = 0; p < g.b_planes; ++p, dst += B_BYTES) {
              const CUtensorMap *map = p ? &b_lo : &b_hi;
              if (B_ROWS) {
                if (B_MN) load_blocks<CG>(dst, map, k * (kTK / 8), n0 / 8, full(st), pol);
                else load_blocks<CG>(dst, map, n0 / 8, k * (kTK / 8), full(st), pol);
              } else {
#pragma unroll
                for (int i = 0; i < BN / 64; ++i)
                  load_tile<CG>(dst + i * 8192, map, n0 + i * 64, k * kTK, full(st), pol);
              }
            }
          }
          if (to) break;
        }
        if (abort_flag) {
          // the copies in flight land before the shared memory goes: a
          // millisecond, as a pair's second CTA has no barrier to wait on
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000) {
          }
          atomicOr(g.err, RQ_DEVERR_TIMEOUT);
        }
      }
    } else if (warp == kEpiWarps + 1) {
      // ------------------------------------------------------------ MMA issue
      if (lane == 0 && rank == 0) {
        const uint32_t idesc = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
                               ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(kTM * CG >> 4) << 24);
        // 16 contraction elements further: 32 bytes along a K-major row, 16
        // rows of 128 bytes in an MN-major tile (in descriptor units of 16 B)
        // (and two blocks of 8 x 8)
        constexpr uint32_t a_step = A_MN ? 2048 / 16 : 32 / 16;
        constexpr uint32_t b_step = !B_ROWS ? 2048 / 16 : B_MN ? 256 / 16 : BN * 32 / 16;
        int it = 0, c = 0;
        for (int t = unit; t < total && !abort_flag; t += units) {
          const int sp = t / mn;
          const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
          const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
          for (int ka = k0; ka < k1; ka += g.chain, ++c) {
            if (!wait(tempty(c & 1), ((uint32_t)(c >> 1) & 1u) ^ 1u)) break;
            tc_after();
            const uint32_t d = tmem + (uint32_t)(c & 1) * TN;
            const int kb = ka + g.chain < k1 ? ka + g.chain : k1;
            for (int k = ka; k < kb; ++k, ++it) {
              const int st = it % g.stages;
              if (!wait(full(st), (uint32_t)(it / g.stages) & 1u)) break;
              tc_after();
              const uint32_t sa = base + (uint32_t)st * stage_bytes;
              const uint32_t sb = sa + (uint32_t)g.a_planes * kABytes;
              const uint64_t ah = sw128_desc(sa, A_MN ? 8192 : 16);
              const uint64_t bh = !B_ROWS ? sw128_desc(sb, 8192)
                                  : B_MN  ? block_desc(sb, 128, 1024)
                                          : block_desc(sb, BN * 16, 128);
              const uint64_t al = ah + kABytes / 16, bl = bh + B_BYTES / 16;
              // the small products first
              uint32_t on = k > ka;
              if (g.b_planes > 1) {
#pragma unroll
                for (int j = 0; j < kTK / 16; ++j, on = 1u)
                  mma_f16_ss<CG>(d, ah + j * a_step, bl + j * b_step, idesc, on);
              }
              if (g.a_planes > 1) {
#pragma unroll
                for (int j = 0; j < kTK / 16; ++j, on = 1u)
                  mma_f16_ss<CG>(d, al + j * a_step, bh + j * b_step, idesc, on);
              }
#pragma unroll
              for (int j = 0; j < kTK / 16; ++j, on = 1u)
                mma_f16_ss<CG>(d, ah + j * a_step, bh + j * b_step, idesc, on);
              tc_commit<CG>(empty(st));
            }
            if (to) break;
            tc_commit<CG>(tfull(c & 1));
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
    }
  } else {
    // ------------------------------------------------------------ accumulators
    if (TN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * HALF);
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      bool ok = to || mbar_try_wait(bar, parity) || mbar_wait_bounded(bar, parity);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && !to) {
        to = true;
        abort_flag = 1;
      }
      return !to;
    };
    const float se = MODE != kGemmDw ? scale_e(g.amax, g.L) : 1.f;
    const float cap = g.cap, icap = g.inv_cap, beta = g.beta;
    float acc[HALF];
    int c = 0;
    for (int t = unit; t < total && !to; t += units) {
      const int sp = t / mn, r = t % mn, nt = n_tile(r);
      const int col0 = nt * TN + half * HALF;
      const int row = (m_tile(r) * CG + rank) * kTM + q * 32 + lane;
      const int k0 = (int)((int64_t)g.kblocks * sp / g.splits);
      const int k1 = (int)((int64_t)g.kblocks * (sp + 1) / g.splits);
      // what the epilogue needs of the row, on its way while the MMAs run: the
      // next listed id at or after col0, its weight and log-sum-exp
      const bool in = row < g.rows;
      int li = 0, next = kNoId;
      float f = 0.f, lse = 0.f, inv = 1.f, inv2 = 1.f;
      if (MODE == kGemmDw) inv = 1.f / __ldg(g.amax + kAmaxBlocks);
      if (MODE == kGemmDh && in) {         // one after the other, the smaller first
        const float a = 1.f / scale_z(g.f[row]), b = 1.f / se;
        inv = fminf(a, b);
        inv2 = fmaxf(a, b);
      }
      if (LOGITS && in) inv = fminf(1.f / (g.sh[row] * se), FLT_MAX);
      if (LOGITS && in) {
        const int32_t *list = g.sid + (int64_t)row * g.k;
        const int want = g.v0 + col0;
        if (g.k > 1) {
          for (int hi = g.k; li < hi;) {
            const int mid = (li + hi) >> 1;
            if (__ldg(list + mid) < want) li = mid + 1;
            else hi = mid;
          }
        }
        if (li < g.k) next = __ldg(list + li);
        if (MODE != kGemmStats) {
          f = g.f[row];
          lse = g.lse[row];
        }
      }
      auto step = [&]() {
        next = ++li < g.k ? __ldg(g.sid + (int64_t)row * g.k + li) : kNoId;
        if (next != kNoId) next -= g.v0;
      };
#pragma unroll
      for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
      for (int ka = k0; ka < k1; ka += g.chain, ++c) {
        if (!wait_all(tfull(c & 1), (uint32_t)(c >> 1) & 1u)) break;
        tc_after();
        const uint32_t src = lanes + (uint32_t)(c & 1) * TN;
#pragma unroll
        for (int j0 = 0; j0 < HALF; j0 += 32) {
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
        tc_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) arrive_first(tempty(c & 1));
          else arrive(tempty(c & 1));
        }
      }
      // a warp that gave up would leave the others waiting at the group's barriers
      if (STAGED) to = group_any(1 + half, to);
      if (to) break;
      if (LOGITS && next != kNoId) {       // as a column (a single one may lie before col0)
        next -= g.v0;
        if (next < col0) next = kNoId;
      }
      if (MODE == kGemmStats) {
        // The epilogues take 32 columns at a time from the front of the sums,
        // which then move up: registers cannot be indexed by a loop, and 128
        // unrolled tanh and exp would not fit the instruction cache.
        float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int j0 = 0; j0 < HALF; j0 += 32) {
          float cm = -INFINITY;
          for (; next < col0 + j0 + 32; step()) {      // listed here
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = col0 + j0 + j == next ? acc[j] : z;
            z *= inv;
            const int64_t at = (int64_t)row * g.k;
            g.y[at + __ldg(g.sj + at + li)] = cap > 0.f ? cap * tanh_flat(z * icap) : z;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float z = acc[j] * inv;
            const float y = cap > 0.f ? cap * tanh_flat(z * icap) : z;
            acc[j] = col0 + j0 + j < g.cols ? __fmul_rn(y, beta) : -INFINITY;
            cm = fmaxf(cm, acc[j]);
          }
          const float nm = fmaxf(mx, cm);
          if (nm > -INFINITY) {
            sum *= ex2((mx - nm) * kLog2e);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum += ex2((acc[j] - nm) * kLog2e);
          } else {      // no column, or NaN in all of them
#pragma unroll
            for (int j = 0; j < 32; ++j) sum += acc[j] != acc[j] ? acc[j] : 0.f;
          }
          mx = nm;
#pragma unroll
          for (int j = 0; j + 32 < HALF; ++j) acc[j] = acc[j + 32];
        }
        if (in)
          g.stat[(int64_t)(g.stat_part0 + nt * 2 + half) * g.stat_ld + row] = make_float2(mx, sum);
      } else if (LOGITS) {
        const float fs = MODE == kGemmGrad ? f * scale_z(f) : f;
        const int64_t at = ((int64_t)(row >> 1) * g.dz_pitch + col0) * 2 + (row & 1);   // fp32
#pragma unroll 1
        for (int j0 = 0; j0 < HALF; j0 += 32) {
          if (STAGED) {
            if (q == 0 && lane == 0) store_wait_read();   // the last chunk is read out
            group_sync(1 + half);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float z = acc[16 * k + j] * inv;
              float y = z, slope = 1.f;
              if (cap > 0.f) {
                const float th = tanh_flat(z * icap);
                y = cap * th;
                slope = 1.f - th * th;
              }
              x[j] = f != 0.f ? ex2(fmaf(y, beta, -lse) * kLog2e) * slope * fs : 0.f;
            }
            if (MODE == kGemmGrad32) {
              if (in && col0 + j0 + 16 * k < g.cols) {          // the pitch is 16 columns
#pragma unroll
                for (int j = 0; j < 16; ++j) g.dz[at + 2 * (j0 + 16 * k + j)] = x[j];
              }
            } else {
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                const float2 y = __half22float2(h);
                const __half2 l =
                    __floats2half2_rn(__fsub_rn(x[2 * j], y.x), __fsub_rn(x[2 * j + 1], y.y));
                hi[j] = *reinterpret_cast<const uint32_t *>(&h);
                lo[j] = *reinterpret_cast<const uint32_t *>(&l);
              }
              // rows of 64 bytes, 16-byte pieces swizzled by row / 2
              const uint32_t r = staging + (uint32_t)(half * kStoreBytes + (q * 32 + lane) * 64);
              const uint32_t sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t o = r + (((uint32_t)(2 * k + p) ^ sw) << 4);
                sts16(o, hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
                sts16(o + kStoreBytes / 2, lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
              }
            }
          }
          for (; next < col0 + j0 + 32; step()) {      // listed here: p - q instead
            const int c = next - col0 - j0;
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = c == j ? acc[j] : z;
            z *= inv;
            const float th = cap > 0.f ? tanh_flat(z * icap) : 0.f;
            const float p = ex2(fmaf(cap > 0.f ? cap * th : z, beta, -lse) * kLog2e);
            const float d =
                f != 0.f ? (p - __ldg(g.sq + (int64_t)row * g.k + li)) * (1.f - th * th) * fs : 0.f;
            if (MODE == kGemmGrad32) {
              g.dz[at + 2 * (j0 + c)] = d;
            } else {
              __half dh, dl;
              split_f16(d, dh, dl);
              const uint32_t o = staging + (uint32_t)(half * kStoreBytes + (q * 32 + lane) * 64) +
                                 ((((uint32_t)c >> 3) ^ ((uint32_t)(lane >> 1) & 3u)) << 4) +
                                 ((uint32_t)c & 7u) * 2;
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(o), "h"(__half_as_ushort(dh)) : "memory");
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(o + kStoreBytes / 2),
                           "h"(__half_as_ushort(dl))
                           : "memory");
            }
          }
          if (STAGED) {
            async_fence();
            group_sync(1 + half);
            if (q == 0 && lane == 0) {
              const int x = col0 + j0, y = row;           // (row of the group's first thread)
              if (x < g.cols && y < g.rows) {
                store_tile(&o_hi, staging + half * kStoreBytes, x, y);
                store_tile(&o_lo, staging + half * kStoreBytes + kStoreBytes / 2, x, y);
              }
              store_commit();
            }
          }
#pragma unroll
          for (int j = 0; j + 32 < HALF; ++j) acc[j] = acc[j + 32];
        }
      } else if (MODE == kGemmDw) {
        // a thread has a row of the vocabulary and stores pairs of dims, a warp
        // 32 neighbouring rows of a pair
        if (in) {
          float2 *o = reinterpret_cast<float2 *>(g.out) + (int64_t)(col0 / 2) * g.out_pitch + row;
#pragma unroll
          for (int j = 0; j < HALF; j += 2, o += g.out_pitch)
            if (col0 + j < g.cols) *o = make_float2(acc[j] * inv, acc[j + 1] * inv);
        }
      } else if (in) {
        float *o = g.out + (int64_t)sp * g.out_split + (int64_t)row * g.out_pitch + col0;
#pragma unroll
        for (int j = 0; j < HALF; j += 8) {
          if (col0 + j < g.out_pitch) {
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = acc[j + x] * inv * inv2;
            if (g.accumulate) {
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
    if (STAGED && q == 0 && lane == 0) store_wait_all();
    if (to && lane == 0) atomicOr(g.err, RQ_DEVERR_TIMEOUT);
  }
  tc_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();      // nothing of the pair still on its way here
  if (warp == kEpiWarps + 1) {
    __syncwarp();
    tc_after();
    if (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TMEM_COLS));
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TMEM_COLS));
  }
}

namespace {

// Tile of a product with `m` rows, `n` columns and `splits` shares of the
// contraction; see the comment at the top of the file.  Measured, 256000 rows
// of 2304: a training step of 2048 bf16 tokens 21.9 ms on single SMs, 18.1 ms
// on pairs; 4096 rows of 192, 33 tokens: the gradients of the logits 23 us with
// 256 columns a tile, 11 us with 64.
struct Tile {
  int cg, tn;
};

Tile tile_of(int64_t m, int64_t n, int splits) {
  const int64_t mt = (m + kTM - 1) / kTM, nt = (n + 255) / 256;
  if (mt * nt * splits < 74) return {1, 64};
  // a pair's last tile may be half empty: worth it from 7 row tiles on
  if (mt % 2 == 0 || mt >= 7) return {2, 256};
  return {1, 256};
}

bool plane_map(CUtensorMap *m, const void *p, const GemmPlanes &x, bool mn, int tile) {
  return encode_tmap_2d_u16(m, p, (uint64_t)x.cols, (uint64_t)x.rows, (uint64_t)x.pitch * 2, 64,
                            mn ? 64 : (uint32_t)tile, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Decoded rows: boxes of `brows` x `bcols` blocks of 8 x 8.
bool rows_map(CUtensorMap *m, const void *p, const GemmPlanes &x, int brows, int bcols) {
  static const PFN_cuTensorMapEncodeTiled encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled>(f)
               : nullptr;
  }();
  if (!encode) return false;
  const cuuint64_t dim[3] = {64, (cuuint64_t)(x.rows + 7) / 8, (cuuint64_t)(x.cols + 7) / 8};
  const cuuint64_t stride[2] = {128, (cuuint64_t)x.pitch * 16};
  const cuuint32_t box[3] = {64, (cuuint32_t)brows, (cuuint32_t)bcols}, one[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(p), dim, stride, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int CG, int TN>
cudaError_t launch_tile(const GemmPlanes &A, const GemmPlanes &B, GemmArgs a, const DevInfo &di,
                        cudaStream_t s) {
  constexpr bool A_MN = MODE == kGemmDw, B_MN = MODE == kGemmDh || MODE == kGemmDw;
  constexpr int BN = TN / CG;
  CUtensorMap ah, al, bh, bl;
  auto b_map = [&](CUtensorMap *m, const void *p) {
    return MODE == kGemmDw ? plane_map(m, p, B, true, BN)
           : B_MN          ? rows_map(m, p, B, kTK / 8, BN / 8)
                           : rows_map(m, p, B, BN / 8, kTK / 8);
  };
  if (!plane_map(&ah, A.hi, A, A_MN, kTM) || !b_map(&bh, B.hi)) return cudaErrorInvalidValue;
  al = ah;
  bl = bh;
  if ((A.lo && !plane_map(&al, A.lo, A, A_MN, kTM)) || (B.lo && !b_map(&bl, B.lo)))
    return cudaErrorInvalidValue;
  const int64_t k = A_MN ? A.rows : A.cols;
  a.a_planes = A.lo ? 2 : 1;
  a.b_planes = B.lo ? 2 : 1;
  a.m_tiles = (int)(((A_MN ? A.cols : A.rows) + kTM * CG - 1) / (kTM * CG));
  a.n_tiles = (int)(((B_MN ? B.cols : B.rows) + TN - 1) / TN);
  a.kblocks = (int)((k + kTK - 1) / kTK);
  const bool few = (MODE != kGemmDh && MODE != kGemmDw && a.rows <= kTM) || a.kblocks <= 4;
  const int mmas = few ? kChainMmasShort : MODE == kGemmDw ? kChainMmasDw : kChainMmas;
  a.chain = mmas / (kTK / 16 * (a.a_planes + a.b_planes - 1));
  if (a.splits > a.kblocks) a.splits = a.kblocks;
  CUtensorMap oh = ah, ol = ah;
  if (MODE == kGemmGrad &&
      (!encode_tmap_2d_u16(&oh, a.dz_hi, (uint64_t)a.cols, (uint64_t)a.rows,
                           (uint64_t)a.dz_pitch * 2, 32, kTM, CU_TENSOR_MAP_SWIZZLE_64B) ||
       !encode_tmap_2d_u16(&ol, a.dz_lo, (uint64_t)a.cols, (uint64_t)a.rows,
                           (uint64_t)a.dz_pitch * 2, 32, kTM, CU_TENSOR_MAP_SWIZZLE_64B)))
    return cudaErrorInvalidValue;
  const size_t stage = (size_t)a.a_planes * kABytes + (size_t)a.b_planes * (BN * kTK * 2);
  const size_t tail = kGemmSmemTail + (MODE == kGemmGrad ? 2 * kStoreBytes : 0);
  int st = (int)((kGemmSmemMax - tail) / stage);
  a.stages = st > kMaxStages ? kMaxStages : st;
  const size_t smem = tail + a.stages * stage;
  const void *fn = reinterpret_cast<const void *>(&loss_gemm_kernel<MODE, CG, TN>);
  cudaError_t e = ensure_smem_limit(fn, di.device, smem);
  if (e != cudaSuccess) return e;
  const int64_t total = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  if (total < 1 || total > 0x7fffffff) return cudaErrorInvalidValue;
  const int units = di.sms / CG;
  void *args[] = {&ah, &al, &bh, &bl, &oh, &ol, &a};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((total < units ? total : units) * CG));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int MODE>
cudaError_t launch_gemm(const GemmPlanes &A, const GemmPlanes &B, GemmArgs a, const DevInfo &di,
                        cudaStream_t s) {
  constexpr bool A_MN = MODE == kGemmDw, B_MN = MODE == kGemmDh || MODE == kGemmDw;
  if (a.splits < 1) a.splits = 1;
  const Tile t = tile_of(A_MN ? A.cols : A.rows, B_MN ? B.cols : B.rows, a.splits);
  if (t.cg == 2) return launch_tile<MODE, 2, 256>(A, B, a, di, s);
  if (t.tn == 64) return launch_tile<MODE, 1, 64>(A, B, a, di, s);
  return launch_tile<MODE, 1, 256>(A, B, a, di, s);
}

}  // namespace

int loss_stats_parts(int64_t tokens, int64_t rows) {
  const int tn = tile_of(tokens, rows, 1).tn;
  return 2 * (int)((rows + tn - 1) / tn);
}

cudaError_t launch_loss_gemm(int mode, const GemmPlanes &A, const GemmPlanes &B, const GemmArgs &a,
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
