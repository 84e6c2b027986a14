// Attention over the 8-bit key/value cache for more than a few rows of a
// sequence, on the 5th-gen tensor cores. Formulas in include/exl3.h.
//
// One CTA per SM. A segment is a (sequence, key/value head, 256 rows of its group
// in token order: two tiles of 128); its units are 128 cached tokens. All units of
// all segments lie one behind the other, and each CTA takes one equal, contiguous
// range of them; segments that several CTAs share are joined by a second kernel.
// Per unit:
//   * warps 9..16 (converters): the unit's keys and values from global memory, one
//     operand ahead in registers, to fp16 in the two-stage operand buffers
//     (128-byte swizzle; the same layout serves keys as the K-major operand of
//     Q K^T and values as the MN-major operand of P V). Each block's scale goes in
//     as a power of two relative to the largest of the CTA's part of the segment, so
//     one factor serves all its scores and outputs: exact, but for codes of blocks 2^15
//     and more below the largest, which lose 2^-25 of its largest code at most;
//   * warp 8 (one lane): for each tile tcgen05.mma S = Q K^T into TMEM, then, when
//     the tile's probabilities are there, O += P V with P read from TMEM, where it
//     has taken the place of S;
//   * warps 0..3 / 4..7 (tile 0 / 1; thread = row = TMEM lane): the row's 128
//     scores, 32 at a time: maximum first, then mask, exp2, sum, probabilities as
//     fp16 back to TMEM. While one tile's softmax runs, the tensor core works on the other's
//     products. O is rescaled only when the maximum grows by more than 2^3.75 over the
//     one that the reference in use was set by (the result is the same: the sum uses
//     that reference), so rarely after the first units.
// TMEM: S0 S1 O0 O1, 128 columns each.
//
// Measured: 2048 rows of 40 heads on 8 over 8192 cached tokens, D = 128: 329 us (301
// GFLOP, 915 TFLOP/s, the join 15 to 20 us of it). The softmax binds it: a chain of
// TMEM reads, maximum, exponentials and TMEM writes per tile and unit, 2 row warps a
// scheduler; the tensor pipe is busy 42 % of the time. Not bound by the operands: Q
// from TMEM (half the shared-memory reads of Q K^T) took 321 us of then 326. Slower
// were two threads a row (72 registers, 452 us), a register split by role (419 us and
// more), one pass over the scores with a guessed maximum (345 us).
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kTile = 128, kPair = 2 * kTile;  // rows
constexpr int kTokens = 128;                   // of a unit
constexpr int kConvWarps = 8;
constexpr int kChunkThreads = (9 + kConvWarps) * 32;  // 96 registers a thread
constexpr int kChunkSeqs = 1024;               // sequences of one launch
// Entering a segment (queries, the blocks' largest scales, the output), in units.
constexpr int kChunkEntry = 3;
// A row's reference is set 2^12 below its maximum (kHeadroom), and set anew when a maximum
// passes it by more than 2^15.75 (kLazy; fp16 ends at 2^16): a row is rescaled a few times
// at most, and the many small probabilities of a long sequence keep their bits (one of
// 2^-26 of the largest has all 11; fp16 ends 2^-37 below it). 2048 rows over 8192 tokens:
// 329 us, 327 with 2^7 and 2^15, 324 with 1 and 2^14, where what is below 2^-25 of the
// largest is lost (65536 tokens there have up to 2^-9 of the weight); 337 with the exact
// product by 2^12 in place of the sum, which rounds exponents to 2^-21.
constexpr float kHeadroom = 12.0f, kLazy = 15.75f;
// With the reference back at the maximum first: a logarithm near 12 would be 2^-20 off.
__device__ __forceinline__ float row_lse(float ref, float sum) { return log_sum(ref + kHeadroom, sum * 0x1p-12f); }

template <int D>
struct ChunkCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kOperand = kHalves * 128 * 128;   // 128 rows (or tokens) x D fp16
  static constexpr int kOffK = 2 * kOperand;             // two query tiles before it
  static constexpr int kOffV = kOffK + 2 * kOperand;
  static constexpr int kOffPlan = kOffV + 2 * kOperand;  // int64 prefix, scratch, int2 sequences
  static constexpr int kOffBar = kOffPlan + (kChunkSeqs + 32) * 8 + (kChunkSeqs + 8) * 8;
  static constexpr int kSmem = 1024 + kOffBar + 256;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};
enum { kBarQ = 0, kBarKFull = 2, kBarKEmpty = 4, kBarVFull = 6, kBarVEmpty = 8, kBarS = 10, kBarP = 12, kBarO = 14,
       kBarDone = 16, kNumBars = 17 };

struct ChunkParams {
  KvAttention a;
  int group, ctas;
  int join_rows;  // of a CTA of the join: kJoinRows or a multiple that divides 256
  // Workspace: partial results of the CTAs (slot 0: a segment that began before
  // the CTA's range, slot 1: one that began in it and goes on after it) and the plan.
  float *part_o;      // CTAs x 2 x 256 x D
  float *part_ml;     // CTAs x 2 x 256 x 2
  int64_t *plan;
  int64_t part_rows;  // 2 * CTAs * 256
};

// Units of the pair of tiles rt of a sequence: as far as its last row sees.
__device__ __forceinline__ int pair_units(const KvSeq &q, int group, int causal, int rt) {
  const int last = min((rt + 1) * kPair, q.rows * group) - 1;
  const int seen = causal ? q.len - q.rows + last / group + 1 : q.len;
  return seen > 0 ? (seen + kTokens - 1) / kTokens : 0;
}
__device__ __forceinline__ int pair_cost(const KvSeq &q, int group, int causal, int rt) {
  const int u = pair_units(q, group, causal, rt);
  return u > 0 ? u + kChunkEntry : 0;
}
__device__ __forceinline__ int pairs_of(const KvSeq &q, int group) { return (q.rows * group + kPair - 1) / kPair; }

struct ChunkPlan {
  int64_t *prefix;  // kChunkSeqs + 1, then scratch
  int2 *seq;
  __device__ __forceinline__ KvSeq at(int s) const {
    const int2 a = seq[s];
    return KvSeq{a.x, a.y < 0 ? 0 : seq[s + 1].x - a.x, a.y < 0 ? 0 : a.y};
  }
};

// Ends with a barrier.
__device__ __forceinline__ void build_chunk_plan(const KvView &kv, int group, int causal, const ChunkPlan &plan) {
  int64_t *warp_sum = plan.prefix + kChunkSeqs + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  int64_t carry = 0;
  if (threadIdx.x == 0) plan.prefix[0] = 0;
  for (int c = 0; c < kv.n_seqs; c += blockDim.x) {
    const int s = c + (int)threadIdx.x;
    int64_t n = 0;
    if (s < kv.n_seqs) {
      const KvSeq q = kv_sequence(kv, s);
      for (int rt = 0; rt < pairs_of(q, group); ++rt) n += pair_cost(q, group, causal, rt);
      n *= kv.n_kv_heads;
      plan.seq[s] = make_int2(kv.q_start[s], q.rows > 0 ? q.len : -1);
      if (s + 1 == kv.n_seqs) plan.seq[s + 1] = make_int2(kv.q_start[s + 1], -1);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += o;
    }
    if (lane == 31) warp_sum[warp] = n;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < nwarps; ++w) {
      const int64_t x = warp_sum[w];
      if (w < warp) n += x;
      total += x;
    }
    if (s < kv.n_seqs) plan.prefix[s + 1] = carry + n;
    carry += total;
    __syncthreads();
  }
  __syncthreads();
}

// A CTA's part of a segment: units u0 .. u1 - 1 of `units`.
struct Segment {
  KvSeq q;
  int s, h, rt, rows;  // rows of the pair that exist
  int units, u0, u1;
};
struct Walk {
  int64_t z0, z1, zs;  // the CTA's range; where the segment (s, h, rt) begins
  KvSeq q;
  int s, h, rt;
  __device__ __forceinline__ void begin(const KvView &kv, int group, int causal, const ChunkPlan &plan, int64_t a, int64_t b) {
    z0 = a;
    z1 = b;
    int lo = 0, hi = kv.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (plan.prefix[mid + 1] > a) hi = mid;
      else lo = mid + 1;
    }
    s = lo;
    q = plan.at(s);
    const int64_t head = (plan.prefix[s + 1] - plan.prefix[s]) / kv.n_kv_heads;
    h = (int)((a - plan.prefix[s]) / head);
    zs = plan.prefix[s] + h * head;
    rt = 0;
    for (int c; zs + (c = pair_cost(q, group, causal, rt)) <= a; ++rt) zs += c;
  }
  __device__ __forceinline__ bool next(const KvView &kv, int group, int causal, const ChunkPlan &plan, Segment &g) {
    while (zs < z1) {
      g.units = pair_units(q, group, causal, rt);
      const int64_t first = zs + kChunkEntry;
      g.u0 = (int)max(z0 - first, (int64_t)0);
      g.u1 = (int)min((int64_t)g.units, z1 - first);
      g.q = q;
      g.s = s;
      g.h = h;
      g.rt = rt;
      g.rows = min(kPair, q.rows * group - rt * kPair);
      zs += g.units > 0 ? g.units + kChunkEntry : 0;
      if (++rt == pairs_of(q, group)) {
        rt = 0;
        if (++h == kv.n_kv_heads) {
          h = 0;
          do ++s;
          while (s < kv.n_seqs && plan.prefix[s + 1] == plan.prefix[s]);
          if (s < kv.n_seqs) q = plan.at(s);
          else zs = z1;
        }
      }
      if (g.units > 0 && g.u1 > g.u0) return true;
    }
    return false;
  }
};

// The largest exponents of the key and value scales of the CTA's blocks of a
// segment (partial results carry them, so the CTAs need not agree: with the whole
// segment's, 20 rows over 60000 tokens took 183 us). The whole warp takes part.
__device__ __forceinline__ int2 largest_scales(const KvView &kv, const Segment &g, int lane) {
  constexpr int kBlocks = kTokens / kKvBlock;
  const int end = min(g.u1 * kBlocks, (g.q.len + kKvBlock - 1) / kKvBlock);
  int ek = -127, ev = -127;
#pragma unroll 4
  for (int b = g.u0 * kBlocks + lane; b < end; b += 32) {
    const int page = kv_page(kv, g.s, b);
    if (page < 0) continue;
    const int64_t slab = (int64_t)page * kv.n_kv_heads + g.h;
    ek = max(ek, pow2_exponent(kv.k_scale[slab]));
    ev = max(ev, pow2_exponent(kv.v_scale[slab]));
  }
  return make_int2(__reduce_max_sync(0xffffffffu, ek), __reduce_max_sync(0xffffffffu, ev));
}

// 16 codes to two 16-byte pieces of fp16, times a power of two (one: none).
__device__ __forceinline__ void convert_16(uint4 w, bool times, __half2 factor, uint32_t (&o)[8]) {
  codes_to_half(w, o);
  if (times) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&o[i]), factor);
      o[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
  }
}

// One lane's share of a unit's operand: 16 codes of each of kMine tokens. A warp
// has kPerToken lanes for each of 32 / kPerToken tokens; lanes of the dimension's
// second half take the token next to it, so that eight lanes that store together
// hit eight different bank groups (the swizzle differs between the two tokens).
template <int D>
struct Operand {
  static constexpr int kPerToken = D / 16;
  static constexpr int kStep = kConvWarps * 32 / kPerToken;  // tokens between a lane's
  static constexpr int kMine = kTokens / kStep;
  static_assert(kKvBlock % kStep == 0 && kStep % 8 == 0, "one block and one swizzle row a piece");
  uint4 w[kMine];
  __device__ static __forceinline__ int first(int cw, int lane) {
    return cw * (32 / kPerToken) + (lane / kPerToken ^ (lane % kPerToken >> 2));
  }
  __device__ __forceinline__ void load(const uint8_t *codes, const int64_t (&slab)[2], int tokens, int cw, int lane, int64_t size) {
    const int tok0 = first(cw, lane), c = lane % kPerToken;
#pragma unroll
    for (int it = 0; it < kMine; ++it) {
      constexpr int kHalf = kMine / 2;  // pieces of a block
      const int tok = tok0 + (it % kHalf) * kStep;
      w[it] = make_uint4(0, 0, 0, 0);  // tokens past the sequence, and pages that the table does not name
      const int64_t at = slab[it / kHalf];
      if (tok + (it / kHalf) * kKvBlock < tokens && at >= 0) {
        const int64_t off = (at * kKvBlock + tok) * D + c * 16;
        if (EXL3_SPAN(off, 16, size)) w[it] = *reinterpret_cast<const uint4 *>(codes + off);
      }
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, const float (&factor)[2], int cw, int lane) const {
    const int tok0 = first(cw, lane), c = lane % kPerToken;
    const uint32_t half = dst + (c >> 2) * (128 * 128);
    const uint32_t lo = half + swizzled(tok0, 2 * (c & 3)), hi = half + swizzled(tok0, 2 * (c & 3) + 1);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bool times = factor[b] != 1.0f;
      const __half2 f = __float2half2_rn(factor[b]);
#pragma unroll
      for (int it = b * (kMine / 2); it < (b + 1) * (kMine / 2); ++it) {
        uint32_t o[8];
        convert_16(w[it], times, f, o);
        sts16(lo + it * kStep * 128, o[0], o[1], o[2], o[3]);
        sts16(hi + it * kStep * 128, o[4], o[5], o[6], o[7]);
      }
    }
  }
};

template <int D, bool CAP>
__global__ void __launch_bounds__(kChunkThreads, 1) kv8_chunk_kernel(const ChunkParams p) {
  using Cfg = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(smem);
  const KvView &kv = p.a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ChunkPlan plan{reinterpret_cast<int64_t *>(smem + Cfg::kOffPlan),
                       reinterpret_cast<int2 *>(smem + Cfg::kOffPlan + (kChunkSeqs + 32) * 8)};
  const uint32_t bars = base + Cfg::kOffBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kOffBar + 8 * kNumBars);
  int *status = kv.status;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBarQ + t), 4);
      mbar_init(bar(kBarKFull + t), kConvWarps);
      mbar_init(bar(kBarKEmpty + t), 1);
      mbar_init(bar(kBarVFull + t), kConvWarps);
      mbar_init(bar(kBarVEmpty + t), 1);
      mbar_init(bar(kBarS + t), 1);
      mbar_init(bar(kBarP + t), 4);
      mbar_init(bar(kBarO + t), 1);
    }
    mbar_init(bar(kBarDone), 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  build_chunk_plan(kv, p.group, p.a.causal, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t T = plan.prefix[kv.n_seqs], W = min((int64_t)p.ctas, T);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= kv.n_seqs; i += kChunkThreads) p.plan[i] = plan.prefix[i];

  if (blockIdx.x < W) {
    Walk walk;
    walk.begin(kv, p.group, p.a.causal, plan, range_start(blockIdx.x, W, T), range_start(blockIdx.x + 1, W, T));
    Segment g;
    if (warp == 8) {
      // ---------------- tensor core (one lane) ----------------
      if (lane == 0) {
        constexpr uint32_t kIdescS = f16_idesc(kTile, kTokens), kIdescO = f16_idesc(kTile, D) | kIdescBTransposed;
        uint32_t unit = 0, seg_of[2] = {0, 0}, done_of[2] = {0, 0};  // units of the CTA; segments and units of a tile
        bool ok = true;
        auto scores = [&](int t, uint32_t n) {
          const uint32_t q = base + t * Cfg::kOperand, k = base + Cfg::kOffK + (n & 1) * Cfg::kOperand;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t off = (j >> 2) * (128 * 128) + (j & 3) * 32;
            tc_mma(tmem + 128 * t, sw128_desc(q + off), sw128_desc(k + off), kIdescS, j > 0);
          }
          tc_commit(bar(kBarS + t));
        };
        while (ok && walk.next(kv, p.group, p.a.causal, plan, g)) {
          const int tiles = g.rows > kTile ? 2 : 1, n = g.u1 - g.u0;
          ok = mbar_wait(bar(kBarKFull + (unit & 1)), (unit >> 1) & 1, status);
          for (int t = 0; ok && t < tiles; ++t) {
            ok = mbar_wait(bar(kBarQ + t), seg_of[t]++ & 1, status);
            if (!ok) break;
            tc_fence_after();
            scores(t, unit);
          }
          if (ok) tc_commit(bar(kBarKEmpty + (unit & 1)));
          for (int j = 0; ok && j < n; ++j, ++unit) {
            for (int t = 0; ok && t < tiles; ++t) {
              if (t == 0) ok = mbar_wait(bar(kBarVFull + (unit & 1)), (unit >> 1) & 1, status);
              ok = ok && mbar_wait(bar(kBarP + t), done_of[t]++ & 1, status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t v = base + Cfg::kOffV + (unit & 1) * Cfg::kOperand;
#pragma unroll
              for (int k = 0; k < kTokens / 16; ++k)
                tc_mma_ta(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, sw128_mn_desc(v + k * 2048, 128 * 128, 1024), kIdescO,
                          (j | k) > 0);
              tc_commit(bar(kBarO + t));
              if (j + 1 < n) {
                if (t == 0) ok = mbar_wait(bar(kBarKFull + ((unit + 1) & 1)), ((unit + 1) >> 1) & 1, status);
                if (!ok) break;
                tc_fence_after();
                scores(t, unit + 1);
              }
            }
            if (!ok) break;
            tc_commit(bar(kBarVEmpty + (unit & 1)));
            if (j + 1 < n) tc_commit(bar(kBarKEmpty + ((unit + 1) & 1)));
          }
        }
        tc_commit(bar(kBarDone));  // every issued product ends before the TMEM is released
        mbar_wait_short(bar(kBarDone), 0);
      }
    } else if (warp > 8) {
      // ---------------- converters ----------------
      const int cw = warp - 9;
      const int64_t size = kv.n_pages * kv.n_kv_heads * kKvBlock * (int64_t)D;
      const float sign = p.a.scale < 0.f ? -1.f : 1.f;
      // Powers of two below fp16's range are 0 (see above). A block that is not there
      // (past the sequence, or a page that the table does not name) has zero codes and
      // the scale 1, which may be far above `top`: a factor past fp16's range would make
      // NaN of the zeros, and no block that is there has a factor above 1.
      auto factor = [&](float scale, int top) {
        const int d = min(pow2_exponent(scale) - top, 0);
        return d >= -24 ? pow2i(d) : 0.f;
      };
      uint32_t unit = 0;
      bool more = walk.next(kv, p.group, p.a.causal, plan, g);
      int u = g.u0;
      int2 top = make_int2(0, 0);
      int64_t slab[2] = {-1, -1}, slab_n[2] = {-1, -1};
      float fk[2], fv[2], ks[2], vs[2];
      auto find = [&](const Segment &s, int at, int64_t (&to)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int block = 2 * at + b;
          const int page = block * kKvBlock < s.q.len ? kv_page(kv, s.s, block) : -1;
          to[b] = page < 0 ? -1 : (int64_t)page * kv.n_kv_heads + s.h;
        }
      };
      auto scales = [&](const int64_t (&at)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          ks[b] = at[b] < 0 ? 1.f : kv.k_scale[at[b]];
          vs[b] = at[b] < 0 ? 1.f : kv.v_scale[at[b]];
        }
      };
      auto factors = [&]() {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          fk[b] = sign * factor(ks[b], top.x);
          fv[b] = factor(vs[b], top.y);
        }
      };
      Operand<D> keys, values;
      if (more) {
        top = largest_scales(kv, g, lane);
        find(g, u, slab);
        keys.load(kv.k, slab, g.q.len - u * kTokens, cw, lane, size);
        scales(slab);
        factors();
      }
      while (more) {
        // the unit after this one
        Segment gn = g;
        int un = u + 1;
        bool more_n = true;
        if (un == g.u1) {
          more_n = walk.next(kv, p.group, p.a.causal, plan, gn);
          un = gn.u0;
        }
        if (more_n) find(gn, un, slab_n);
        values.load(kv.v, slab, g.q.len - u * kTokens, cw, lane, size);
        const uint32_t st = unit & 1, ph = (unit >> 1) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarKEmpty + st), ph ^ 1, status))) break;
        keys.store(base + Cfg::kOffK + st * Cfg::kOperand, fk, cw, lane);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarKFull + st));
        if (more_n) {
          keys.load(kv.k, slab_n, gn.q.len - un * kTokens, cw, lane, size);
          scales(slab_n);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarVEmpty + st), ph ^ 1, status))) break;
        values.store(base + Cfg::kOffV + st * Cfg::kOperand, fv, cw, lane);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarVFull + st));
        ++unit;
        if (more_n) {
          if (un != u + 1 || gn.s != g.s || gn.h != g.h || gn.rt != g.rt) top = largest_scales(kv, gn, lane);
          slab[0] = slab_n[0];
          slab[1] = slab_n[1];
          factors();
        }
        g = gn;
        u = un;
        more = more_n;
      }
    } else {
      // ---------------- softmax: thread = row of tile t ----------------
      const int t = warp >> 2, row = threadIdx.x & 127;
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_tmem = lane_base + 128 * t, o_tmem = lane_base + 256 + 128 * t;
      const SoftCap cap(p.a.softcap, kLog2e);
      uint32_t count = 0;  // units of this tile so far
      bool ok = true;
      while (ok && walk.next(kv, p.group, p.a.causal, plan, g)) {
        if (t * kTile >= g.rows) continue;  // the pair has no second tile
        const int j = g.rt * kPair + t * kTile + row, i = j / p.group;
        const bool real = i < g.q.rows;
        const int head = g.h * p.group + j - i * p.group;
        const int limit = !real ? 0 : p.a.causal ? g.q.len - g.q.rows + i + 1 : g.q.len;
        const int least = __reduce_min_sync(0xffffffffu, limit);
        {  // the query row; the products that read the last segment's are done (its scores have been read)
          const int64_t off = (int64_t)(g.q.row0 + i) * p.a.ldq + (int64_t)head * D;
          const __half *q = static_cast<const __half *>(p.a.q) + off;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real && EXL3_SPAN(off + 8 * c, 8, (int64_t)(kv.rows - 1) * p.a.ldq + (int64_t)p.a.n_heads * D))
              v = reinterpret_cast<const uint4 *>(q)[c];
            sts16(base + t * Cfg::kOperand + (c >> 3) * (128 * 128) + swizzled(row, c & 7), v.x, v.y, v.z, v.w);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarQ + t));
        }
        const int2 top_scale = largest_scales(kv, g, lane);
        // scores in log2 units are the products times c, then capped
        const float c = fmaxf(fabsf(p.a.scale) * pow2i(top_scale.x) * Raised<D>::kLog2e, 1e-37f);
        float ref = -INFINITY, sum = 0.f;
        for (int u = g.u0; u < g.u1; ++u, ++count) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarS + t), count & 1, status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int pos0 = u * kTokens;
          const bool masked = pos0 + kTokens > least;
          const float scale = CAP ? 1.0f : c;
          float top = -INFINITY;
          auto mask = [&](int q, float (&s)[32]) {
            if (masked) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (pos0 + 32 * q + k >= limit) s[k] = -INFINITY;
            }
          };
          // not unrolled, here and below: instruction fetch is part of the bound
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float s[32];
            tmem_ld32(s_tmem + 32 * q, s);
            mask(q, s);
            float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k < 28; k += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], fmaxf(s[k + e], s[k + 4 + e]));
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], s[28 + e]);
            top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
          }
          if constexpr (CAP) top = top == -INFINITY ? top : cap(make_float2(top * c, 0.f)).x;  // as the cap is monotonic
          else top *= scale;
          const float now = top > ref + kLazy || ref == -INFINITY ? top - kHeadroom : ref;
          const float keep = now == ref || ref == -INFINITY ? 1.0f : ex2(ref - now);
          if (u > g.u0 && __any_sync(0xffffffffu, keep != 1.0f)) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarO + t), (count - 1) & 1, status))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              float o[32];
              tmem_ld32(o_tmem + 32 * k, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= keep;
              tmem_st32(o_tmem + 32 * k, o);
            }
            sum *= keep;
          }
          ref = now;
          const float shift = now == -INFINITY ? 0.f : -now;
          const float2 scale2 = make_float2(scale, scale), shift2 = make_float2(shift, shift);
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float s[32];
            uint32_t packed[16];  // fp16 probabilities: 2^-12 on average (see kHeadroom), the size of the result's own rounding
            tmem_ld32(s_tmem + 32 * q, s);
            if constexpr (CAP) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 x = cap(mul2(make_float2(s[k], s[k + 1]), make_float2(c, c)));
                s[k] = x.x;
                s[k + 1] = x.y;
              }
            }
            mask(q, s);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 x = fma2(make_float2(s[2 * k], s[2 * k + 1]), scale2, shift2);
              x = make_float2(ex2(x.x), ex2(x.y));
              part[k & 1] = add2(part[k & 1], x);
              const __half2 h2 = __floats2half2_rn(x.x, x.y);
              packed[k] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            tmem_st16(s_tmem + 16 * q, packed);
          }
          part[0] = add2(part[0], part[1]);
          sum += part[0].x + part[0].y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarP + t));
        }
        if (!ok || !__all_sync(0xffffffffu, mbar_wait(bar(kBarO + t), (count - 1) & 1, status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool whole = g.u0 == 0 && g.u1 == g.units;
        const float unit = pow2i(min(max(top_scale.y, -126), 127));
        const float f = whole ? (sum == 0.f ? 0.f : unit / sum) : unit;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (g.u0 == 0 ? 1 : 0)) * kPair + t * kTile + row;
        const int64_t off = (int64_t)(g.q.row0 + i) * p.a.ldo + (int64_t)head * D;
        const bool fits = whole ? EXL3_SPAN(real ? off : 0, D, (int64_t)(kv.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D)
                                : EXL3_SPAN(slot, 1, p.part_rows);
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          float o[32];
          tmem_ld32(o_tmem + 32 * k, o);
          if (!real || !fits) continue;
          if (whole) {
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(p.a.out) + off + 32 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __half2 h2 = __floats2half2_rn(o[8 * e + 2 * x] * f, o[8 * e + 2 * x + 1] * f);
                w[x] = *reinterpret_cast<const uint32_t *>(&h2);
              }
              out[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4 *out = reinterpret_cast<float4 *>(p.part_o + slot * D + 32 * k);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              out[e] = make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
          }
        }
        if (real && fits) {
          if (!whole) reinterpret_cast<float2 *>(p.part_ml)[slot] = make_float2(ref, sum);
          else if (p.a.lse) p.a.lse[(int64_t)(g.q.row0 + i) * p.a.n_heads + head] = row_lse(ref, sum);
        }
        tc_fence_before();  // the output has been read: before the next segment's first products
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the partials of the segments that several CTAs worked on, in the order of
// the CTAs, and writes the rows that see no token. All latency, so a warp has two
// rows and the loads of four partials in flight: 65 rows over 777 tokens, 10 partials
// each, took 38 us in ncu with 64 rows a CTA and one partial after the other.
constexpr int kJoinRows = 16, kJoinThreads = 256;

// SPLIT warps share two rows' partials.
template <int D, int SPLIT>
__global__ void __launch_bounds__(kJoinThreads) kv8_chunk_join_kernel(const ChunkParams p) {
  const KvView &kv = p.a.kv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.y, h = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const KvSeq q = kv_sequence(kv, s);
  const int j0 = blockIdx.x * p.join_rows, rt = j0 / kPair;
  if (j0 >= q.rows * p.group) return;
  const int units = pair_units(q, p.group, p.a.causal, rt);
  int64_t c0 = 0, c1 = -1;
  if (units > 0) {
    int before = 0;
    for (int r = lane; r < rt; r += 32) before += pair_cost(q, p.group, p.a.causal, r);
    before = __reduce_add_sync(0xffffffffu, before);
    const int64_t T = p.plan[kv.n_seqs], W = min((int64_t)p.ctas, T);
    const int64_t z = p.plan[s] + (p.plan[s + 1] - p.plan[s]) / kv.n_kv_heads * h + before + kChunkEntry;
    c0 = range_owner(z, W, T);
    c1 = range_owner(z + units - 1, W, T);
    if (c0 == c1) return;  // the CTA wrote the result
  }
  constexpr int E = D / 32, kAtOnce = kJoinRows / (kJoinThreads / 32), kAhead = 4;
  const int64_t share = (c1 - c0 + SPLIT) / SPLIT, a0 = c0 + warp % SPLIT * share, a1 = min(c1, a0 + share - 1);
  for (int first = j0 + warp / SPLIT * kAtOnce; first < j0 + p.join_rows; first += kJoinRows / SPLIT) {
    float m[kAtOnce], l[kAtOnce], o[kAtOnce][E];
#pragma unroll
    for (int r = 0; r < kAtOnce; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    for (int64_t c = a0; c <= a1; c += kAhead) {
      float2 ml[kAhead][kAtOnce];
      float x[kAhead][kAtOnce][E];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t at = (2 * (c + i) + (c + i == c0 ? 1 : 0)) * kPair + first % kPair;
        const bool there = c + i <= a1 && EXL3_SPAN(at, kAtOnce, p.part_rows);
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {  // rows past the sequence's last hold nothing and are not written
          ml[i][r] = there ? reinterpret_cast<const float2 *>(p.part_ml)[at + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < E; ++e) x[i][r][e] = there ? p.part_o[(at + r) * D + 32 * e + lane] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (c + i > a1) continue;
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
          const float top = fmaxf(m[r], ml[i][r].x), ref = top == -INFINITY ? 0.f : top;
          const float a = ex2(m[r] - ref), b = ex2(ml[i][r].x - ref);
          l[r] = l[r] * a + ml[i][r].y * b;
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = o[r][e] * a + x[i][r][e] * b;
          m[r] = top;
        }
      }
    }
    if constexpr (SPLIT > 1) {  // the warps' results, in their order; a CTA has one pass then
      __shared__ float so[SPLIT][kAtOnce][D];
      __shared__ float2 sml[SPLIT][kAtOnce];
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r) {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][r][32 * e + lane] = o[r][e];
        if (lane == 0) sml[warp][r] = make_float2(m[r], l[r]);
      }
      __syncthreads();
      if (warp > 0) return;
#pragma unroll
      for (int w = 1; w < SPLIT; ++w)
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
          const float2 ml = sml[w][r];
          const float top = fmaxf(m[r], ml.x), ref = top == -INFINITY ? 0.f : top;
          const float a = ex2(m[r] - ref), b = ex2(ml.x - ref);
          l[r] = l[r] * a + ml.y * b;
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = o[r][e] * a + so[w][r][32 * e + lane] * b;
          m[r] = top;
        }
    }
#pragma unroll
    for (int r = 0; r < kAtOnce; ++r) {
      const int j = first + r, i = j / p.group;
      if (i >= q.rows) return;
      const int head = h * p.group + j - i * p.group;
      const int64_t row = q.row0 + i, off = row * p.a.ldo + (int64_t)head * D;
      if (EXL3_SPAN(off, D, (int64_t)(kv.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D))
#pragma unroll
        for (int e = 0; e < E; ++e)
          static_cast<__half *>(p.a.out)[off + 32 * e + lane] = __float2half_rn(l[r] == 0.f ? 0.f : o[r][e] / l[r]);
      if (p.a.lse && lane == 0) p.a.lse[row * p.a.n_heads + head] = row_lse(m[r], l[r]);
    }
  }
}

struct ChunkWorkspace {  // in floats; the plan first
  int64_t part_rows, o, ml, total;
};
ChunkWorkspace chunk_workspace(int D, int num_sms) {
  ChunkWorkspace w;
  w.part_rows = (int64_t)num_sms * 2 * kPair;
  w.o = 2 * (kChunkSeqs + 8);
  w.ml = w.o + w.part_rows * D;
  w.total = w.ml + w.part_rows * 2;
  return w;
}

template <int D>
cudaError_t chunk_attention(const KvAttention &a, cudaStream_t st) {
  ChunkParams p;
  p.a = a;
  p.group = a.n_heads / a.kv.n_kv_heads;
  p.ctas = a.num_sms;
  const ChunkWorkspace w = chunk_workspace(D, a.num_sms);
  float *ws = static_cast<float *>(a.workspace);
  p.plan = reinterpret_cast<int64_t *>(ws);
  p.part_o = ws + w.o;
  p.part_ml = ws + w.ml;
  p.part_rows = w.part_rows;
  for (int s0 = 0; s0 < a.kv.n_seqs; s0 += kChunkSeqs) {
    p.a.kv = kv_slice(a.kv, s0, a.kv.n_seqs - s0 < kChunkSeqs ? a.kv.n_seqs - s0 : kChunkSeqs);
    cudaError_t e = launch_overlapped(a.softcap > 0.f ? kv8_chunk_kernel<D, true> : kv8_chunk_kernel<D, false>, p.ctas,
                                      kChunkThreads, ChunkCfg<D>::kSmem, st, 1, p);
    if (e != cudaSuccess) return e;
    // With many rows what a CTA does before its first load counts, so it has more of
    // them: 10240 rows of 8 heads over 8192 tokens take 7 us less with 64 than with 16;
    // 255 rows over 777 tokens 34 with 64, 23.4 with 16, over 60000 tokens 130 and 105.
    const int64_t joins = ceil_div((int64_t)a.kv.max_rows * p.group, kJoinRows) * p.a.kv.n_seqs * a.kv.n_kv_heads;
    p.join_rows = joins > 16 * a.num_sms ? 4 * kJoinRows : kJoinRows;
    // A long sequence's segments are spread over all CTAs: where it has few, and there are
    // few rows, the warps of a CTA share two rows' many partials. 1 head, 800 rows over
    // 6000 tokens: 29 us so, 38 without; 8 such sequences of 600 tokens: 46 and 26.
    constexpr int kSplit = kJoinThreads / 32;
    const int64_t segments = ceil_div((int64_t)a.kv.max_rows * p.group, kPair) * a.kv.n_kv_heads;
    const bool split = segments * 24 < a.num_sms && joins * kSplit <= 4 * a.num_sms;
    if (split) p.join_rows = kJoinRows / kSplit;
    const dim3 join((unsigned)ceil_div((int64_t)a.kv.max_rows * p.group, p.join_rows), p.a.kv.n_seqs, a.kv.n_kv_heads);
    e = launch_overlapped(split ? kv8_chunk_join_kernel<D, kSplit> : kv8_chunk_join_kernel<D, 1>, join, kJoinThreads, 0, st, 1, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t kv8_chunk_workspace_bytes(int head_dim, int num_sms) {
  return (size_t)chunk_workspace(head_dim, num_sms).total * sizeof(float);
}

cudaError_t launch_kv8_chunk_attention(const KvAttention &a, cudaStream_t st) {
  return a.kv.head_dim == 64 ? chunk_attention<64>(a, st) : chunk_attention<128>(a, st);
}

cudaError_t init_kv8_chunk_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  for (const void *f : {(const void *)kv8_chunk_kernel<64, false>, (const void *)kv8_chunk_kernel<64, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<64>::kSmem);
  for (const void *f : {(const void *)kv8_chunk_kernel<128, false>, (const void *)kv8_chunk_kernel<128, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<128>::kSmem);
  cudaFuncAttributes attr;
  for (const void *f : {(const void *)kv8_chunk_join_kernel<64, 1>, (const void *)kv8_chunk_join_kernel<128, 1>,
                        (const void *)kv8_chunk_join_kernel<64, 8>, (const void *)kv8_chunk_join_kernel<128, 8>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, f);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_chunk(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
