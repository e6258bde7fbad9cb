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
// power of two, so that K g fills a block's lanes), the lanes are ordered by
// falling length and cut into slices of 32, one per warp, and a slice is
// stored step by step: entries 2 i and 2 i + 1 of its 32 lanes side by side as
// 32-bit words, a lane without a row there naming row kGradRows, which holds
// zeros.  So a warp reads two entries a lane with one access and no conflict,
// no lane waits for a longer one (with K = 1024 a list has 8 rows on average;
// in code order the longest of 32 would have 16), and there is no branch.  A lane holds at most
// kCap entries; what a code has beyond its g kCap (skewed codes) follows as a
// plain list that one warp adds at the end.
//   uint16 off[slices + 1]   in rows of 64 entries
//   uint16 code[K]           slot s = lanes [s g, (s + 1) g)
//   uint16 over[1 + n + 1]   over[0] = n codes (the first n slots) may have
//                            more; theirs are [over[1 + s], over[2 + s]) of the
//                            entries that follow the slices
//   uint16 entry[]           4 x the rows' local numbers, ascending per lane
//                            (half the distance between rows' pairs of values)
//
// Two uses of one kernel.  launch_codebook_rows sums the rows of a piece's
// dE in pairs of dims (the tensor cores' dz^T h); launch_codebook_sums, for a few
// tokens, sums the logits' gradients themselves, S[p][k][t] = sum of dz[t][v],
// from which both gradients follow without the V x D matrix of either kind:
//   dC[m][l][k] = sum_t S[p][k][t] h_t (subspace m)
//   dh_t (subspace m) = sum_l sum_k S[p][k][t] C[m][l][k]
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
  while (x.lanes < 32 && K * x.lanes < 1024) x.lanes *= 2;
  x.slices = (K * x.lanes + 31) / 32;
  const int rows = (int)(V < kGradRows ? V : kGradRows);
  x.most = rows / (x.lanes * (kCap - 1) + 1);
  x.code_at = (size_t)align_up((x.slices + 1) * 2, 16);
  x.over_at = x.code_at + (size_t)align_up(K * 2, 16);
  x.entry_at = (size_t)align_up((int64_t)x.over_at + (x.most + 2) * 2, 128);
  // a slice is as long as its first lane, no longer than the lanes of the slice
  // before, give or take one where codes share lanes, and even: rows + the
  // first slice's padding + 32 per slice, or 64
  x.unit = x.entry_at +
           (size_t)align_up((rows + 32 * kCap + (x.lanes > 1 ? 64 : 32) * x.slices) * 2, 128);
  return x;
}

// One block takes `cols` adjacent columns of a block of rows, staged column by
// column in shared memory; a warp per column.  Rows go in ascending order, 32
// at a time; lanes with one code take consecutive places, so no order of
// arrival enters.
constexpr int kStagePitch = kGradRows + 8;   // columns 4 banks apart

// A warp's counters: rows per code, slots, buckets, starts of the slices, and
// the lane that last wrote a code's mark.
__host__ __device__ __forceinline__ int prep_words(const IndexShape &x) {
  return 2 * x.K + kCap + 2 + x.slices + 1 + (x.K + 1) / 2;
}

__global__ void __launch_bounds__(256) prepare_grad_kernel(const CodeSrc cs, const IndexShape x,
                                                           int cols, unsigned char *index) {
  extern __shared__ uint16_t sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (x.P + cols - 1) / cols;
  const int block = blockIdx.x / groups, p0 = blockIdx.x % groups * cols;
  const int nc = x.P - p0 < cols ? x.P - p0 : cols;
  const int64_t v0 = (int64_t)block * kGradRows;
  const int rows = (int)(x.V - v0 < kGradRows ? x.V - v0 : kGradRows);
  // eight codes of a thread on their way at a time
  const int csh = __ffs(cols) - 1, c = threadIdx.x & (cols - 1);
  if (c < nc) {
    for (int r0 = threadIdx.x >> csh; r0 < rows; r0 += 8 * (blockDim.x >> csh)) {
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + i * (blockDim.x >> csh);
        if (r < rows) x[i] = cs.raw(v0 + r, p0 + c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + i * (blockDim.x >> csh);
        if (r < rows) sm[c * kStagePitch + r] = (uint16_t)cs.fix(x[i]);
      }
    }
  }
  __syncthreads();
  if (warp >= nc) return;
  const int p = p0 + warp, g = x.lanes, gsh = __ffs(g) - 1;
  const uint16_t *col = sm + warp * kStagePitch;
  uint16_t *cnt = sm + cols * kStagePitch + (size_t)warp * prep_words(x);
  uint16_t *slot = cnt + x.K, *bucket = slot + x.K, *start = bucket + kCap + 2;
  unsigned char *mark = reinterpret_cast<unsigned char *>(start + x.slices + 1);
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
      const int c = r < rows ? col[r] : -1;
      // lanes with this lane's code: mostly itself alone.  Each marks its code;
      // who finds another's mark shares it, and only those are looked up
      // (match_any takes several times as long on 32 different codes)
      if (c >= 0) mark[c] = (unsigned char)lane;
      __syncwarp();
      unsigned lost = __ballot_sync(0xffffffffu, c >= 0 && mark[c] != lane), same = 1u << lane;
      while (lost) {
        const unsigned m =
            __ballot_sync(0xffffffffu, c == __shfl_sync(0xffffffffu, c, __ffs(lost) - 1));
        if (m >> lane & 1u) same = m;
        lost &= ~m;
      }
      if (c >= 0) each(c, r, same);
      __syncwarp();
    }
  };
  sweep([&](int c, int, unsigned same) {
    if ((same & below) == 0) cnt[c] = (uint16_t)(cnt[c] + __popc(same));
  });
  // codes by falling number of rounds: bucket starts, then places in code order
  auto key = [&](int c) {
    const int n = (cnt[c] + g - 1) >> gsh;
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
  const int total = scan(x.slices, [&](int s) { return (kCap - key(code[s * 32 >> gsh]) + 1) >> 1; },
                         [&](int s, int at) { off[s] = start[s] = (uint16_t)at; });
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
  for (int i = lane; i < total * 64; i += 32) entry[i] = (uint16_t)(4 * kGradRows);
  for (int i = lane; i < x.K; i += 32) cnt[i] = 0;
  __threadfence_block();
  __syncwarp();
  sweep([&](int c, int r, unsigned same) {
    const int e = cnt[c] + __popc(same & below), s = slot[c];
    __syncwarp(same);
    int at;
    if (e < g * kCap) {
      const int vl = (s << gsh) + (e & (g - 1)), i = e >> gsh;
      at = ((start[vl >> 5] + (i >> 1)) * 32 + (vl & 31)) * 2 + (i & 1);
    } else {
      at = total * 64 + over[1 + s] + e - g * kCap;
    }
    entry[at] = (uint16_t)(4 * r);
    if ((same & below) == 0) cnt[c] = (uint16_t)(e + __popc(same));
  });
}

// ------------------------------------------------------------- sums by code
//
// A CTA takes values in pairs [V][2] (two dims of a subspace, or two tokens)
// and the subspace's L columns, and walks the blocks: per block the values (64
// KB) and per column the unit (21 KB at K = 1024) arrive by bulk copies, each
// into the buffer that the step before last left, so that the copies run under
// the gathers.  A warp has a slice, a lane a list; the sums of all blocks are
// kept in shared memory and leave once.  A last dim or token without a partner
// is summed beside whatever its other half holds, which is not stored.
//
// Bound by the random 8-byte reads of shared memory (half a warp's meet in a
// bank 3.1 times).  256000 rows, 768 columns of 1024 codes: 660 us for four
// tokens (a value row of its own for either of a pair, read 4 bytes at a time:
// 720), 1000 us for 2304 dims, where the first version, which added its sums in
// global memory list by list, took 3.8 ms, and one without the pipeline 2.3 ms.
constexpr int kPairFloats = 2 * kGradRows + 4;    // and the row of zeros, vectors kept whole
constexpr int kGatherThreads = 1024;
constexpr size_t kGatherSmemMax = 226 * 1024;     // 227 KB less the static part

struct GatherArgs {
  const float *vals;        // values in pairs of value rows, [pair][pitch][2]
  int64_t pitch;
  const void *index;
  IndexShape x;
  int64_t rows;             // of the values
  int block0, blocks;       // index blocks they cover
  int ds, pairs;            // value rows of one source, pairs of them
  int L, by_level, splits;  // columns of a subspace, a unit per column, shares of the blocks
  int per_subspace;         // value rows belong to the subspace (dims), else to all (tokens)
  int units;
  float *out;
  int64_t out_p, out_k, out_split;   // strides: column, code, share
  int64_t out_pair;                  // pair (0: its two columns lie at 2 pair)
  int accumulate;
  int buffers;              // for units: 2, or 3 (see the kernel)
  int value_buffers;        // for values: 2, or 1 where codebooks are largest
  unsigned *err;
};

// Shared memory by 32-bit address, an immediate offset apart.
__device__ __forceinline__ float2 lds_f32x2(uint32_t a) {
  float2 x;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(a));
  return x;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_b32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(x) : "r"(a), "n"(OFF));
  return x;
}

struct GatherUnit {         // subspace, pair, levels, share of the blocks
  int m, j, l0, l1, b0, b1, share;
  __device__ __forceinline__ bool set(const GatherArgs &a, int u) {   // false: an empty share
    share = u % a.splits;
    int r = u / a.splits;
    l0 = 0;
    l1 = a.L;
    if (a.by_level) {
      l0 = r % a.L;
      l1 = l0 + 1;
      r /= a.L;
    }
    j = r % a.pairs * 2;
    m = r / a.pairs;
    b0 = a.blocks * share / a.splits;
    b1 = a.blocks * (share + 1) / a.splits;
    return b0 < b1;
  }
};

// The issuing thread's place in the same walk.
struct GatherAhead {
  GatherUnit q;
  int u, b, l;
  __device__ __forceinline__ void unit(const GatherArgs &a, int from) {
    for (u = from; u < a.units; u += gridDim.x)
      if (q.set(a, u)) break;      // a short last piece leaves shares empty
    b = q.b0;
    l = q.l0;
  }
  __device__ __forceinline__ void block(const GatherArgs &a) {
    l = q.l0;
    if (++b == q.b1) unit(a, u + gridDim.x);
  }
  __device__ __forceinline__ void step(const GatherArgs &a) {
    if (++l == q.l1) block(a);
  }
};

__global__ void __launch_bounds__(kGatherThreads, 1) codebook_gather_kernel(const GatherArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kWarps = kGatherThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = a.x.K, g = a.x.lanes, gsh = __ffs(g) - 1, nb = a.buffers, nv = a.value_buffers;
  float *vals = reinterpret_cast<float *>(smem);                   // [nv][kPairFloats]
  unsigned char *units = smem + nv * kPairFloats * 4;              // [nb] units
  float2 *stage = reinterpret_cast<float2 *>(units + nb * a.x.unit);  // [levels][K]
  __shared__ uint64_t bars[3 + 2 + 2];        // units, values, steps done (all warps)
  __shared__ volatile int abort_flag;
  auto ubar = [&](int i) { return smem_addr(&bars[i]); };
  auto vbar = [&](int i) { return smem_addr(&bars[3 + i]); };
  auto dbar = [&](int i) { return smem_addr(&bars[5 + i]); };
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(smem_addr(&bars[i]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(dbar(i), kWarps);
    fence_mbar_init();
    abort_flag = 0;
  }
  if (tid < 2 * nv) vals[(tid >> 1) * kPairFloats + 2 * kGradRows + (tid & 1)] = 0.f;
  griddep_launch_dependents();
  __syncthreads();
  griddep_wait();
  // The last warp, whose lists are the shortest, issues the copies: a step
  // (units) and a block (values) ahead.  With three unit buffers the warps may
  // be a step apart (`lag` 2: a step starts when all have finished the last but
  // one), so that nobody waits for the longest list of every step.  With one
  // value buffer (lag 1) a block's values come once the last block is done.
  const int lag = nb - 1;
  const uint32_t vals_at = smem_addr(vals);
  const bool issuer = tid == kGatherThreads - 32;
  GatherAhead au{}, av{};
  int it = 0, iv = 0;        // copies issued
  auto issue_unit = [&]() {
    if (au.u >= a.units) return;
    const int i = it % nb;
    mbar_arrive_expect_tx(ubar(i), (uint32_t)a.x.unit);
    bulk_g2s(smem_addr(units + i * a.x.unit),
             static_cast<const unsigned char *>(a.index) +
                 ((size_t)(a.block0 + au.b) * a.x.P + au.q.m * a.L + au.l) * a.x.unit,
             (uint32_t)a.x.unit, ubar(i));
    ++it;
    au.step(a);
  };
  auto issue_vals = [&]() {
    if (av.u >= a.units) return;
    const int64_t r0 = (int64_t)av.b * kGradRows, left = a.rows - r0;
    const uint32_t bytes = (uint32_t)align_up(left < kGradRows ? left : kGradRows, 2) * 8;
    const int i = iv & (nv - 1);
    const int64_t pair = (a.per_subspace ? (int64_t)av.q.m * a.pairs : 0) + av.q.j / 2;
    mbar_arrive_expect_tx(vbar(i), bytes);
    bulk_g2s(smem_addr(vals + i * kPairFloats), a.vals + (pair * a.pitch + r0) * 2, bytes, vbar(i));
    ++iv;
    av.block(a);
  };
  if (issuer) {
    au.unit(a, blockIdx.x);
    av = au;
    issue_unit();
    issue_vals();
  }
  int t = 0, vt = 0, ub = 0;     // steps and blocks so far; the step's unit buffer
  uint32_t uphase = 0;           // and its phase
  // What the index names is held to its places, so that one that rq_prepare_grad
  // did not write for these sizes gives wrong sums and mostly an error, but no
  // access out of bounds.  An entry's two low bits do not count, and the values
  // come first in shared memory that goes on as far as 16 bits reach (a minimum
  // per entry took 2 % of a step); a slice's end is one compare (a minimum there,
  // in the way of the loop's length, 8 % of this kernel; so 1 % or less).
  const int steps = (int)((a.x.unit - a.x.entry_at) / 128);   // rows of 64 entries
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok && !mbar_try_wait(bar, parity) && !mbar_wait_bounded(bar, parity)) {
      ok = false;
      abort_flag = 1;
    }
    ok = __all_sync(0xffffffffu, ok);      // a warp works as a whole or not at all
  };
  for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
    GatherUnit q;
    if (!q.set(a, u)) continue;
    const bool two = a.ds - q.j > 1;
    for (int b = q.b0; b < q.b1; ++b, ++vt) {
      for (int l = q.l0; l < q.l1; ++l, ++t) {
        if (abort_flag) ok = false;      // (the loops go on, without work, to meet at their ends)
        // everyone has finished step t - lag: its unit buffer takes the next
        // unit, its lists' sums are in the stage, and, a step into a block (at
        // lag 1 at once), nobody reads the last block's values any more, in
        // whose place go the next block's (of one buffer, this block's)
        if (t >= lag) wait(dbar((t - lag) & 1), (uint32_t)((t - lag) >> 1) & 1u);
        if (issuer && ok) {
          issue_unit();
          if (l == q.l0 + (lag > 1 ? 1 : 0) && (nv > 1 || vt > 0)) issue_vals();
        }
        wait(ubar(ub), uphase);
        if (l == q.l0) wait(vbar(vt & (nv - 1)), (uint32_t)(vt >> (nv - 1)) & 1u);
        if (ok) {
          const unsigned char *un = units + ub * a.x.unit;
          const uint16_t *off = reinterpret_cast<const uint16_t *>(un);
          const uint16_t *code = reinterpret_cast<const uint16_t *>(un + a.x.code_at);
          const uint16_t *over = reinterpret_cast<const uint16_t *>(un + a.x.over_at);
          const uint32_t entry = smem_addr(un) + (uint32_t)a.x.entry_at + (uint32_t)lane * 4;
          const uint32_t v0 = vals_at + (uint32_t)(vt & (nv - 1)) * (kPairFloats * 4);
          float2 *st = stage + (size_t)(l - q.l0) * K;
          // one word of entries: two rows of either value row
          auto add = [&](uint32_t w, float &s0, float &s1) {
            const float2 x = lds_f32x2(v0 + (w & 0xFFFCu) * 2), y = lds_f32x2(v0 + (w >> 18) * 8);
            s0 += x.x;
            s1 += x.y;
            s0 += y.x;
            s1 += y.y;
          };
          const int full = min((int)over[0], a.x.most);
          for (int sl = warp; sl < a.x.slices; sl += kWarps) {
            const int e0 = off[sl], e1 = off[sl + 1], n = e1 - e0;
            if (e1 > steps) {
              if (lane == 0) atomicOr(a.err, RQ_DEVERR_BAD_INDEX);
              break;
            }
            uint32_t e = entry + (uint32_t)e0 * 128;
            const int s = (sl * 32 + lane) >> gsh;
            float s0 = 0.f, s1 = 0.f;
            int i = 0;
            for (; i + 4 <= n; i += 4, e += 512) {
              const uint32_t w0 = lds_b32<0>(e), w1 = lds_b32<128>(e), w2 = lds_b32<256>(e),
                             w3 = lds_b32<384>(e);
              add(w0, s0, s1);
              add(w1, s0, s1);
              add(w2, s0, s1);
              add(w3, s0, s1);
            }
            if (i + 2 <= n) {
              const uint32_t w0 = lds_b32<0>(e), w1 = lds_b32<128>(e);
              add(w0, s0, s1);
              add(w1, s0, s1);
              i += 2;
              e += 256;
            }
            if (i < n) add(lds_b32<0>(e), s0, s1);
            for (int o = g >> 1; o > 0; o >>= 1) {
              s0 += __shfl_xor_sync(0xffffffffu, s0, o);
              s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            }
            if ((lane & (g - 1)) == 0 && s < K) {
              const int c = min((int)code[s], K - 1);
              if (b > q.b0) {
                const float2 d = st[c];
                s0 += d.x;
                s1 += d.y;
              }
              st[c] = make_float2(s0, s1);
            }
            // what this slice's codes have beyond their lanes' kCap entries
            const int f1 = (sl + 1) * 32 >> gsh;
            for (int f = sl * 32 >> gsh; f < f1 && f < full; ++f) {
              __syncwarp();
              const int at = min((int)off[a.x.slices], steps) * 64;
              const uint16_t *rest = reinterpret_cast<const uint16_t *>(un + a.x.entry_at) + at;
              const int end = min((int)over[2 + f], steps * 64 - at);
              float r0 = 0.f, r1 = 0.f;
              for (int k = over[1 + f] + lane; k < end; k += 32) {
                const float2 x = lds_f32x2(v0 + (rest[k] & 0xFFFCu) * 2);
                r0 += x.x;
                r1 += x.y;
              }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) {
                r0 += __shfl_xor_sync(0xffffffffu, r0, o);
                r1 += __shfl_xor_sync(0xffffffffu, r1, o);
              }
              if (lane == 0) {
                const int c = min((int)code[f], K - 1);
                const float2 d = st[c];
                st[c] = make_float2(d.x + r0, d.y + r1);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(dbar(t & 1)) : "memory");
        if (++ub == nb) {
          ub = 0;
          uphase ^= 1u;
        }
      }
    }
    __syncthreads();
    // the unit's sums out, in code order
    const int w = two ? 2 : 1;
    for (int l = q.l0; l < q.l1; ++l) {
      float *o = a.out + q.share * a.out_split + (int64_t)(q.m * a.L + l) * a.out_p +
                 (a.out_pair > 0 ? q.j / 2 * a.out_pair : q.j);
      const float *src = reinterpret_cast<const float *>(stage + (size_t)(l - q.l0) * K);
#pragma unroll 2
      for (int i = tid; i < K * w; i += kGatherThreads) {
        const int c = w == 2 ? i >> 1 : i, j = w == 2 ? i & 1 : 0;
        float *d = o + (int64_t)c * a.out_k + j;
        *d = a.accumulate ? *d + src[c * 2 + j] : src[c * 2 + j];
      }
    }
    __syncthreads();
  }
  if (issuer && abort_flag) {
    // the copies in flight land before the shared memory goes
    for (int i = 1; i <= nb; ++i)
      if (it >= i) mbar_wait_bounded(ubar((it - i) % nb), (uint32_t)((it - i) / nb) & 1u);
    for (int i = 1; i <= nv; ++i)
      if (iv >= i) mbar_wait_bounded(vbar((iv - i) & (nv - 1)), (uint32_t)((iv - i) >> (nv - 1)) & 1u);
    atomicOr(a.err, RQ_DEVERR_TIMEOUT);
  }
}

// out[i] (+)= sum over the shares of part[share][i]
__global__ void __launch_bounds__(256) codebook_join_kernel(const float *__restrict__ part,
                                                            int splits, int64_t n,
                                                            float *__restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = part[i];
  for (int x = 1; x < splits; ++x) s += part[x * n + i];
  out[i] = s;
}

// One block per column p, for tokens [0, nt) in pairs: S [pair][split][p][K][2]
// summed over its splits; dC = S h and the column's share of dh,
// dhp[p][t][ds].
constexpr int kFinThreads = 256;
constexpr int kFinTokens = 4;        // tokens whose sums a thread holds at once

__global__ void __launch_bounds__(kFinThreads) codebook_finish_kernel(
    const float *__restrict__ S, int splits, const void *h, int bf16, int nt,
    const float *__restrict__ f, const float *__restrict__ C, int D, int L, int K, int P, int ds, float *dC, float *dhp) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ float fin[];     // [nt][ds] hidden slices, [8][kFinTokens][ds] partials
  const int p = blockIdx.x, m = p / L, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *part = fin + nt * ds;
  for (int i = tid; i < nt * ds; i += kFinThreads)      // (padding may hold anything)
    fin[i] = f[i / ds] != 0.f ? load_h(h, bf16, (int64_t)(i / ds) * D + (int64_t)m * ds + i % ds)
                              : 0.f;
  __syncthreads();
  const int64_t pair = (int64_t)splits * P * K * 2;
  for (int t0 = 0; t0 < nt; t0 += kFinTokens) {
    const int n = nt - t0 < kFinTokens ? nt - t0 : kFinTokens;
    // dims in steps of 2 so that their sums stay in registers
    for (int j0 = 0; j0 < ds; j0 += 2) {
      const int w = ds - j0 < 2 ? 1 : 2;
      float dh[kFinTokens][2];
#pragma unroll
      for (int t = 0; t < kFinTokens; ++t) dh[t][0] = dh[t][1] = 0.f;
      for (int k = tid; k < K; k += kFinThreads) {
        float s[kFinTokens];
#pragma unroll
        for (int t = 0; t < kFinTokens; t += 2) {
          float2 y = make_float2(0.f, 0.f);
          if (t < n) {
            const float *src = S + (t0 + t) / 2 * pair + ((int64_t)p * K + k) * 2;
            for (int x = 0; x < splits; ++x) {
              const float2 z = *reinterpret_cast<const float2 *>(src + (int64_t)x * P * K * 2);
              y.x += z.x;
              y.y += z.y;
            }
          }
          s[t] = y.x;
          s[t + 1] = t + 1 < n ? y.y : 0.f;
        }
        for (int j = 0; j < w; ++j) {
          const int64_t at = ((int64_t)p * K + k) * ds + j0 + j;
          if (dC) {
            float d = t0 > 0 ? dC[at] : 0.f;
#pragma unroll
            for (int t = 0; t < kFinTokens; ++t)
              if (t < n) d = fmaf(s[t], fin[(t0 + t) * ds + j0 + j], d);
            dC[at] = d;
          }
          if (dhp) {
            const float c = C[at];
#pragma unroll
            for (int t = 0; t < kFinTokens; ++t) dh[t][j] = fmaf(s[t], c, dh[t][j]);
          }
        }
      }
      if (dhp) {
#pragma unroll
        for (int t = 0; t < kFinTokens; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = dh[t][j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0 && j < w) part[(warp * kFinTokens + t) * ds + j0 + j] = x;
          }
      }
    }
    if (!dhp) continue;
    __syncthreads();
    for (int i = tid; i < n * ds; i += kFinThreads) {
      float x = 0.f;
      for (int v = 0; v < kFinThreads / 32; ++v) x += part[v * kFinTokens * ds + i];
      dhp[((int64_t)p * nt + t0) * ds + i] = x;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) codebook_dh_kernel(const float *__restrict__ dhp, int nt,
                                                          int D, int L, int ds, int bf16,
                                                          void *dh) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)nt * D) return;
  const int t = (int)(i / D), c = (int)(i % D), m = c / ds, j = c % ds;
  float x = 0.f;
  for (int l = 0; l < L; ++l) x += dhp[((int64_t)(m * L + l) * nt + t) * ds + j];
  if (bf16) static_cast<__nv_bfloat16 *>(dh)[i] = __float2bfloat16_rn(x);
  else static_cast<float *>(dh)[i] = x;
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
    return (size_t)n * (kStagePitch + prep_words(x)) * 2;
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

namespace {

// Units of a gather and how they split: a column of its own where a subspace's
// L sums do not fit, or where whole subspaces would leave SMs idle; then
// shares of the blocks.  From 3841 codewords on (8192 rows or more) two blocks'
// values no longer fit beside a column's sums, and one does up to kMaxGradK:
// 2 x 35712 bytes of units, 65552 of values and 32768 of sums.  The copies then
// wait for the sums: 131072 rows of 384 subspaces of six dims, two levels, 791 us
// at 3840 codewords and 1055 at 3841 (four tokens' sums 540 and 685).
struct GatherPlan {
  bool by_level;
  int splits, buffers, value_buffers;
  int64_t units;
  size_t smem;
};

GatherPlan gather_plan(const IndexShape &x, int blocks, int sources, int pairs, int L) {
  GatherPlan p;
  const auto bytes = [&](int levels, int buffers = 2, int value_buffers = 2) {
    return buffers * x.unit + (size_t)value_buffers * kPairFloats * 4 + (size_t)levels * x.K * 8;
  };
  p.units = (int64_t)sources * pairs;
  p.by_level = L > 1 && (bytes(L) > 225 * 1024 || p.units < 148);
  if (p.by_level) p.units *= L;
  // warps a step apart need a third unit buffer, and two levels: a step's sums
  // and values are then not those of the step before
  const int levels = p.by_level ? 1 : L;
  p.buffers = levels > 1 && bytes(levels, 3) <= kGatherSmemMax ? 3 : 2;
  p.value_buffers = bytes(levels, p.buffers) <= kGatherSmemMax ? 2 : 1;
  p.smem = bytes(levels, p.buffers, p.value_buffers);
  const size_t reach = (size_t)(p.value_buffers - 1) * kPairFloats * 4 + 65536 * 2;
  if (p.smem < reach) p.smem = reach;      // (of any 16-bit entry in the last buffer)
  p.splits = 1;
  if (p.units < 148) {
    const int64_t n = 148 / p.units;
    p.splits = (int)(n < blocks ? n : blocks);
  }
  p.units *= p.splits;
  return p;
}

cudaError_t launch_gather(GatherArgs a, const GatherPlan &p, const DevInfo &di, cudaStream_t s) {
  if (p.units > 0x7fffffff || p.smem > kGatherSmemMax) return cudaErrorInvalidValue;
  a.by_level = p.by_level ? 1 : 0;
  a.splits = p.splits;
  a.buffers = p.buffers;
  a.value_buffers = p.value_buffers;
  a.units = (int)p.units;
  a.err = di.err;
  const void *fn = reinterpret_cast<const void *>(&codebook_gather_kernel);
  cudaError_t e = ensure_smem_limit(fn, di.device, p.smem);
  if (e != cudaSuccess) return e;
  void *args[] = {&a};
  return launch_maybe_pdl(fn, dim3((unsigned)(p.units < di.sms ? p.units : di.sms)),
                          dim3(kGatherThreads), p.smem, s, args, true);
}

int blocks_of(int64_t rows) { return (int)((rows + kGradRows - 1) / kGradRows); }

}  // namespace

int codebook_rows_splits(int64_t V, int64_t rows, int M, int L, int K, int ds) {
  return gather_plan(index_shape(V, M * L, K), blocks_of(rows), M, (ds + 1) / 2, L).splits;
}

cudaError_t launch_codebook_rows(const float *dw, int64_t pitch, int64_t v0, int64_t rows,
                                 const void *index, int64_t V, int M, int L, int K, int ds,
                                 int splits, bool accumulate, float *out, const DevInfo &di,
                                 cudaStream_t s) {
  GatherArgs a = {};
  a.vals = dw;
  a.pitch = pitch;
  a.index = index;
  a.x = index_shape(V, M * L, K);
  a.rows = rows;
  a.block0 = (int)(v0 / kGradRows);
  a.blocks = blocks_of(rows);
  a.ds = ds;
  a.pairs = (ds + 1) / 2;
  a.L = L;
  a.per_subspace = 1;
  a.out = out;
  a.out_p = (int64_t)K * ds;
  a.out_k = ds;
  a.out_split = (int64_t)M * L * K * ds;
  a.accumulate = accumulate ? 1 : 0;
  GatherPlan p = gather_plan(a.x, a.blocks, M, a.pairs, L);
  // a last piece of fewer blocks keeps the first piece's shares, some empty
  p.units = p.units / p.splits * splits;
  p.splits = splits;
  return launch_gather(a, p, di, s);
}

cudaError_t launch_codebook_join(const float *part, int splits, int64_t n, float *dC,
                                 cudaStream_t s) {
  return pdl_launch(codebook_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), (size_t)0, s, part, splits, n, dC);
}

int codebook_sum_splits(int64_t V, int M, int L, int K, int N) {
  return gather_plan(index_shape(V, M * L, K), blocks_of(V), M, (N + 1) / 2, L).splits;
}

cudaError_t launch_codebook_sums(const float *dz, int64_t pitch, int N, const void *index, int64_t V,
                                 int M, int L, int K, float *S, const DevInfo &di, cudaStream_t s) {
  GatherArgs a = {};
  a.vals = dz;
  a.pitch = pitch;
  a.index = index;
  a.x = index_shape(V, M * L, K);
  a.rows = V;
  a.blocks = blocks_of(V);
  a.ds = N;
  a.pairs = (N + 1) / 2;
  a.L = L;
  a.out = S;
  const GatherPlan p = gather_plan(a.x, a.blocks, M, a.pairs, L);
  a.out_k = 2;
  a.out_p = (int64_t)K * 2;
  a.out_split = (int64_t)M * L * K * 2;
  a.out_pair = p.splits * a.out_split;
  return launch_gather(a, p, di, s);
}

cudaError_t launch_codebook_finish(const float *S, int splits, const void *h, int bf16, int N,
                                   const float *f, const float *C, int D, int M, int L, int K,
                                   float *dC, float *dhp, cudaStream_t s) {
  const int ds = D / M, P = M * L;
  const size_t smem = (size_t)(N + kFinThreads / 32 * kFinTokens) * ds * 4;
  return pdl_launch(codebook_finish_kernel, dim3(P), dim3(kFinThreads), smem, s, S,
                    splits, h, bf16, N, f, C, D, L, K, P, ds, dC, dhp);
}

cudaError_t launch_codebook_dh(const float *dhp, int N, int D, int M, int L, int bf16, void *dh,
                               cudaStream_t s) {
  const int64_t n = (int64_t)N * D;
  return pdl_launch(codebook_dh_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), (size_t)0, s, dhp, N, D, L, D / M, bf16, dh);
}

}  // namespace rq
