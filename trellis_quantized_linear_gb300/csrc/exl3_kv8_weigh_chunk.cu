// Accumulated attention weight of cached tokens under many query rows, on the
// 5th-gen tensor cores. Formula in include/exl3.h.
//
// An item is 128 cached tokens of a (sequence, key/value head). Its keys come to
// fp16 (exact) in shared memory once; the query rows that see it stream past, up
// to 128 columns (rows x heads of the group) a step: S^T = K Q^T into one of two
// TMEM buffers, thread = token = TMEM lane, and each thread adds up
// exp2(s - lse) over the step's columns. No maximum, no second product: 128 x 128
// exponentials a step against 512 cycles of tensor work, so two CTAs share an SM and
// take turns.
//   * warps 0..7: the item's keys, then per step the columns' lse, the exponentials
//     and the sums; warps 0..3 have the first 64 columns and warps 4..7 the others
//     (eight warps hide the latency of a dependent chain that four leave bare: 287 us
//     with four). Each warp brings its own 64 lse, a step ahead in registers, then in
//     shared memory of its own: with one copy for all, a barrier a step, 224 us;
//   * warp 8 (one lane): tcgen05.mma;
//   * warp 9 (one lane): TMA of the queries, a box of 64 dimensions x heads x rows,
//     so a step is the group's heads of consecutive rows without a copy.
// The items go to pairs of CTAs (clusters) in turn, the ones that most rows see
// first, and a pair shares an item's steps: the first half of them and the second,
// whose sums the other CTA's shared memory receives. So sums are formed in a fixed
// order, and there are twice the pieces to deal out (2048 rows of 40 heads over 8192
// tokens are 512 items of up to 82 steps for 304 CTAs: 206 us with an item a CTA,
// 170 us so: 150 GFLOP, 885 TFLOP/s, and 0.6 G exponentials). Bound by a step's chain
// of TMEM read, difference, exponential and sum, which two CTAs of eight warps an SM
// hide in part: of an earlier 225 us the exponentials themselves were 19 us and the
// broadcast reads of the lse 42.
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kItem = 128;         // tokens
constexpr int kCols = 128;         // of a step
constexpr int kExpWarps = 8;
constexpr int kWeighThreads = (kExpWarps + 2) * 32;
constexpr int kWeighSeqs = 512;    // sequences of one launch

template <int D>
struct WeighCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kOperand = kHalves * 128 * 128;
  static constexpr int kOffQ = kOperand;                    // two stages
  static constexpr int kOffCol = kOffQ + 2 * kOperand;      // (lse, limit) x 64 a warp, then sums: two of the other half, two of the other CTA
  static constexpr int kOffPlan = kOffCol + kExpWarps * (kCols / 2) * 8 + 4 * kItem * 4;  // int prefix, then int2 sequences
  static constexpr int kOffBar = kOffPlan + (kWeighSeqs + 8) * 4 + (kWeighSeqs + 8) * 8;
  static constexpr int kSmem = 1024 + kOffBar + 256;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
};
enum { kWQFull = 0, kWQEmpty = 2, kWSFull = 4, kWSEmpty = 6, kWKeys = 8, kWDone = 9, kWPeer = 10, kWTaken = 12, kWBars = 14 };

struct WeighParams {
  KvAttention a;
  int group;
  int heads, rows;  // of a step: heads * rows <= 128 columns
};

struct Item {
  KvSeq q;
  int s, h, tile;
  int first;     // first row that sees the item
  int chunks;    // steps of heads
  int step0, steps;  // of this CTA: the first, how many
};

// Items (128-token tiles x heads) of all sequences before each; ends with a barrier.
struct WeighPlan {
  int *prefix;
  int2 *seq;
  __device__ __forceinline__ KvSeq at(int s) const {
    const int2 a = seq[s];
    return KvSeq{a.x, a.y < 0 ? 0 : seq[s + 1].x - a.x, a.y < 0 ? 0 : a.y};
  }
};
__device__ __forceinline__ void build_weigh_plan(const KvView &kv, const WeighPlan &plan) {
  for (int s = threadIdx.x; s < kv.n_seqs; s += blockDim.x) {
    const KvSeq q = kv_sequence(kv, s);
    plan.seq[s] = make_int2(kv.q_start[s], q.rows > 0 ? q.len : -1);
    plan.prefix[s + 1] = q.rows > 0 ? (q.len + kItem - 1) / kItem * kv.n_kv_heads : 0;
    if (s + 1 == kv.n_seqs) plan.seq[s + 1] = make_int2(kv.q_start[s + 1], -1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // one warp: 32 at a time
    const int lane = threadIdx.x;
    int carry = 0;
    if (lane == 0) plan.prefix[0] = 0;
    for (int c = 0; c < kv.n_seqs; c += 32) {
      int n = c + lane < kv.n_seqs ? plan.prefix[c + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
      }
      if (c + lane < kv.n_seqs) plan.prefix[c + lane + 1] = carry + n;
      carry += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  __syncthreads();
}

// Item k of this CTA pair, false past the last. Heads vary fastest: tiles of the
// sequence's front, which most rows see, come first. Every other round goes the
// other way, so that the pairs with the shorter items of a round get the longer of
// the next. The first CTA of the pair has the first half of an item's steps.
__device__ __forceinline__ bool get_item(const WeighParams &p, const WeighPlan &plan, int k, Item &it) {
  const KvView &kv = p.a.kv;
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1, rank = blockIdx.x & 1;
  const int z = k * pairs + (k & 1 ? pairs - 1 - pair : pair);
  if (z >= plan.prefix[kv.n_seqs]) return false;
  int lo = 0, hi = kv.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (plan.prefix[mid + 1] > z) hi = mid;
    else lo = mid + 1;
  }
  it.s = lo;
  it.q = plan.at(lo);
  const int i = z - plan.prefix[lo];
  it.h = i % kv.n_kv_heads;
  it.tile = i / kv.n_kv_heads;
  it.first = p.a.causal ? max(0, it.tile * kItem - (it.q.len - it.q.rows)) : 0;
  it.chunks = (p.group + p.heads - 1) / p.heads;
  const int steps = max(0, (it.q.rows - it.first + p.rows - 1) / p.rows) * it.chunks;
  it.step0 = rank ? (steps + 1) / 2 : 0;
  it.steps = rank ? steps / 2 : (steps + 1) / 2;
  return true;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// A barrier of the exponential warps that is true when every thread's `ok` is.
__device__ __forceinline__ bool all_agree(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.red.and.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "n"(kExpWarps * 32)
      : "memory");
  return all != 0;
}

template <int D, bool CAP>
__global__ void __launch_bounds__(kWeighThreads, 2)
    kv8_weigh_chunk_kernel(const __grid_constant__ CUtensorMap tq, const WeighParams p) {
  using Cfg = WeighCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(smem);
  const KvView &kv = p.a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WeighPlan plan{reinterpret_cast<int *>(smem + Cfg::kOffPlan),
                       reinterpret_cast<int2 *>(smem + Cfg::kOffPlan + (kWeighSeqs + 8) * 4)};
  const uint32_t bars = base + Cfg::kOffBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kOffBar + 8 * kWBars);
  int *status = kv.status;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kWQFull + t), 1);
      mbar_init(bar(kWQEmpty + t), 1);
      mbar_init(bar(kWSFull + t), 1);
      mbar_init(bar(kWSEmpty + t), kExpWarps);
    }
    mbar_init(bar(kWKeys), kExpWarps);
    mbar_init(bar(kWDone), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kWPeer + t), 4);
      mbar_init(bar(kWTaken + t), 4);
    }
    fence_barrier_init();
  }
  if (warp == kExpWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(256)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  cluster_sync_all();  // the other CTA's barriers are there
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  build_weigh_plan(kv, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int step_cols = p.heads * p.rows;
  // rows of the query stages that no copy fills
  for (int i = threadIdx.x; i < (kCols - step_cols) * 8 * 2 * Cfg::kHalves; i += kWeighThreads)
    sts16(base + Cfg::kOffQ + i / ((kCols - step_cols) * 8) * (128 * 128) + step_cols * 128 + i % ((kCols - step_cols) * 8) * 16, 0, 0, 0, 0);
  fence_proxy_async_shared();
  __syncthreads();
  Item it;

  if (warp == kExpWarps + 1) {
    // ---------------- queries (one lane) ----------------
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int k = 0; ok && get_item(p, plan, k, it); ++k)
        for (int st = 0, chunk = it.step0 % it.chunks, row = it.q.row0 + it.first + it.step0 / it.chunks * p.rows;
             ok && st < it.steps; ++st, ++n) {
          const uint32_t b = n & 1;
          ok = mbar_wait(bar(kWQEmpty + b), ((n >> 1) & 1) ^ 1, status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kWQFull + b), (uint32_t)(Cfg::kHalves * step_cols * 128));
          const int head = it.h * p.group + chunk * p.heads;
#pragma unroll
          for (int hf = 0; hf < Cfg::kHalves; ++hf)
            if (EXL3_RANGE(head, 0, p.a.n_heads) && EXL3_RANGE(row, 0, kv.rows))
              tma_load_3d(base + Cfg::kOffQ + b * Cfg::kOperand + hf * (128 * 128), &tq, bar(kWQFull + b), 64 * hf, head, row);
          if (++chunk == it.chunks) {
            chunk = 0;
            row += p.rows;
          }
        }
      // the copies in flight land before the CTA leaves
      for (uint32_t u = n > 2 ? n - 2 : 0; u < n; ++u) mbar_wait_short(bar(kWQFull + (u & 1)), (u >> 1) & 1);
    }
  } else if (warp == kExpWarps) {
    // ---------------- tensor core (one lane) ----------------
    if (lane == 0) {
      constexpr uint32_t kIdesc = f16_idesc(kItem, kCols);
      uint32_t n = 0, held = 0;  // steps; items with steps, whose keys are brought
      bool ok = true;
      for (int k = 0; ok && get_item(p, plan, k, it); ++k) {
        if (it.steps == 0) continue;
        ok = mbar_wait(bar(kWKeys), held++ & 1, status);
        for (int st = 0; ok && st < it.steps; ++st, ++n) {
          const uint32_t b = n & 1, ph = (n >> 1) & 1;
          ok = mbar_wait(bar(kWQFull + b), ph, status) && mbar_wait(bar(kWSEmpty + b), ph ^ 1, status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t q = base + Cfg::kOffQ + b * Cfg::kOperand;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t off = (j >> 2) * (128 * 128) + (j & 3) * 32;
            tc_mma(tmem + 128 * b, sw128_desc(base + off), sw128_desc(q + off), kIdesc, j > 0);
          }
          tc_commit(bar(kWQEmpty + b));
          tc_commit(bar(kWSFull + b));
        }
      }
      tc_commit(bar(kWDone));
      mbar_wait_short(bar(kWDone), 0);
    }
  } else {
    // ---------------- exponentials: thread = token ----------------
    const int tid = threadIdx.x, row = tid & 127, half = tid >> 7;  // token of the item, half of the columns
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 64 * half;
    const SoftCap cap(p.a.softcap, 1.0f);
    constexpr int kHalf = kCols / 2;
    float *col_lse = reinterpret_cast<float *>(smem + Cfg::kOffCol) + warp * 2 * kHalf;  // the warp's own
    int *col_limit = reinterpret_cast<int *>(col_lse + kHalf);
    float *half_sum = reinterpret_cast<float *>(smem + Cfg::kOffCol) + kExpWarps * 2 * kHalf;
    float *peer_sum = half_sum + 2 * kItem;
    const int rank = blockIdx.x & 1;
    const uint32_t peer_smem = map_to_rank(base, 1 - rank);
    [[maybe_unused]] const int64_t size = kv.n_pages * kv.n_kv_heads * kKvBlock * (int64_t)D;
    // a lane brings two of its warp's columns
    const int col0 = half * kHalf + lane, col1 = col0 + 32;
    const int row_0 = col0 / p.heads, head_0 = col0 % p.heads, row_1 = col1 / p.heads, head_1 = col1 % p.heads;
    uint32_t n = 0;
    bool ok = true;
    for (int k = 0; get_item(p, plan, k, it); ++k) {
      const int pos0 = it.tile * kItem, pos = pos0 + row;
      int page = -1;
      float ks = 0.f;
      if (pos < it.q.len) page = kv_page(kv, it.s, pos / kKvBlock);
      const int64_t slab = (int64_t)max(page, 0) * kv.n_kv_heads + it.h;
      if (page >= 0) ks = kv.k_scale[slab] * p.a.scale * Raised<D>::kOne;
      // The keys, where this CTA has a step of the item: a product that reads them, and the wait for
      // its scores, are what keeps these warps within one item of the tensor core's lane (without
      // them the barrier could pass two phases between its looks). A token has D / 16 lanes; lanes
      // of the second half of the dimension take the token next to theirs.
      if (it.steps > 0) {
        constexpr int kPerToken = D / 16, kStep = kExpWarps * 32 / kPerToken;
        const int c = tid % kPerToken, tok0 = tid / kPerToken ^ (c >> 2);
        uint4 w[kItem / kStep];
#pragma unroll
        for (int i = 0; i < kItem / kStep; ++i) {
          const int t = tok0 + i * kStep;
          w[i] = make_uint4(0, 0, 0, 0);
          if (pos0 + t >= it.q.len) continue;
          const int page = kv_page(kv, it.s, (pos0 + t) / kKvBlock);
          if (page < 0) continue;
          const int64_t off = (((int64_t)page * kv.n_kv_heads + it.h) * kKvBlock + (pos0 + t) % kKvBlock) * D + c * 16;
          if (EXL3_SPAN(off, 16, size)) w[i] = *reinterpret_cast<const uint4 *>(kv.k + off);
        }
#pragma unroll
        for (int i = 0; i < kItem / kStep; ++i) {
          uint32_t o[8];
          codes_to_half(w[i], o);
          const uint32_t at = base + (c >> 2) * (128 * 128);
          sts16(at + swizzled(tok0 + i * kStep, 2 * (c & 3)), o[0], o[1], o[2], o[3]);
          sts16(at + swizzled(tok0 + i * kStep, 2 * (c & 3) + 1), o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kWKeys));
      }

      // a column of the steps in order: its row's lse, and how many tokens the row sees
      int step_row = it.first + it.step0 / it.chunks * p.rows, chunk = it.step0 % it.chunks;
      auto column = [&](int col, int r, int hd, float &lse, int &limit) {
        const int g = chunk * p.heads + hd;
        r += step_row;
        limit = 0;
        lse = 0.f;
        if (col < step_cols && g < p.group && r < it.q.rows) {
          const int64_t at = (int64_t)(it.q.row0 + r) * p.a.n_heads + it.h * p.group + g;
          if (EXL3_SPAN(at, 1, (int64_t)kv.rows * p.a.n_heads)) lse = p.a.lse[at];
          limit = p.a.causal ? it.q.len - it.q.rows + r + 1 : it.q.len;
        }
      };
      float lse0 = 0.f, lse1 = 0.f, total = 0.f;
      int limit0 = 0, limit1 = 0;
      auto columns = [&]() {
        column(col0, row_0, head_0, lse0, limit0);
        column(col1, row_1, head_1, lse1, limit1);
        if (++chunk == it.chunks) {
          chunk = 0;
          step_row += p.rows;
        }
      };
      if (it.steps > 0) columns();
      const int end = min(pos0 + kItem, it.q.len);
      for (int st = 0; ok && st < it.steps; ++st, ++n) {
        const uint32_t b = n & 1;
        if (lse0 == -INFINITY) limit0 = 0;  // a row that saw nothing (here, so that the load has had a step's time)
        if (lse1 == -INFINITY) limit1 = 0;
        // (a column that no step has: its query row is zero and its lse infinite)
        const bool full = __all_sync(0xffffffffu, (limit0 >= end || col0 >= step_cols) && (limit1 >= end || col1 >= step_cols));
        col_lse[lane] = col0 < step_cols ? -lse0 : -INFINITY;
        col_lse[lane + 32] = col1 < step_cols ? -lse1 : -INFINITY;
        if (!full) {
          col_limit[lane] = limit0;
          col_limit[lane + 32] = limit1;
        }
        if (st + 1 < it.steps) columns();
        __syncwarp();
        ok = mbar_wait(bar(kWSFull + b), (n >> 1) & 1, status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // exp(s - lse): the difference in natural units first, one rounding of a number
        // that is small where the weight is not, so that the factor log2 e costs no bits
        auto weight = [&](float a0, float a1, float2 minus) {
          const float2 acc = make_float2(a0, a1);
          float2 d;
          if constexpr (CAP)
            d = add2(cap(mul2(acc, make_float2(ks, ks))), minus);
          else
            d = fma2(acc, make_float2(ks, ks), minus);
          d = mul2(d, make_float2(kLog2e, kLog2e));
          return make_float2(ex2(d.x), ex2(d.y));
        };
        auto release = [&]() {  // the buffer is free for the step after the next
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kWSEmpty + b));
        };
        if (full) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float s[32];
            tmem_ld32(lane_base + 128 * b + 32 * i, s);
            if (i == 1) release();
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 m = *reinterpret_cast<const float4 *>(col_lse + 32 * i + k);
              part[0] = add2(part[0], weight(s[k], s[k + 1], make_float2(m.x, m.y)));
              part[1] = add2(part[1], weight(s[k + 2], s[k + 3], make_float2(m.z, m.w)));
            }
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            float s[32];
            tmem_ld32(lane_base + 128 * b + 32 * i, s);
            if (i == 1) release();
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 m = *reinterpret_cast<const float2 *>(col_lse + 32 * i + k);
              const int2 l = *reinterpret_cast<const int2 *>(col_limit + 32 * i + k);
              const float2 x = weight(s[k], s[k + 1], m);
              part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], make_float2(pos < l.x ? x.x : 0.f, pos < l.y ? x.y : 0.f));
            }
          }
        }
        __syncwarp();  // all lanes are past the columns
        part[0] = add2(part[0], part[1]);
        total += part[0].x + part[0].y;  // a sum of sums: 82 steps of 10240 rows lose no bits that matter
      }
      // the other half's sum; all warps are past the item's last step then (its scores
      // come from the last product that reads the keys), and a wait that ran out in one,
      // here or in the join of the item before, ends the loop in all
      const int slot = (k & 1) * kItem + row;
      if (half == 1) half_sum[slot] = total;
      ok = all_agree(ok);
      if (!ok) break;
      if (half == 1) continue;
      total += half_sum[slot];
      // the other CTA's sum, through two slots
      const uint32_t full = bar(kWPeer + (k & 1)), taken = bar(kWTaken + (k & 1)), ph = (k >> 1) & 1;
      if (rank == 1) {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(taken, ph ^ 1, status, kWaitLimitNs));
        if (!ok) continue;
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_smem + (smem_u32(peer_sum + slot) - base)), "f"(total) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(peer_smem + (full - base));
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(full, ph, status, kWaitLimitNs));
        if (!ok) continue;
        total += peer_sum[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(peer_smem + (taken - base));
        const int64_t at = slab * kKvBlock + pos % kKvBlock;
        if (page >= 0 && EXL3_SPAN(at, 1, kv.n_pages * kv.n_kv_heads * kKvBlock))
          atomicAdd(&kv.weight[at], total);  // alone but for sequences that share the block
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // nothing of the other CTA is on its way here
  if (warp == kExpWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
  }
}

template <int D>
cudaError_t weigh_chunk(const KvAttention &a, cudaStream_t st) {
  WeighParams p;
  p.a = a;
  p.group = a.n_heads / a.kv.n_kv_heads;
  p.heads = p.group < kCols ? p.group : kCols;
  p.rows = kCols / p.heads;
  CUtensorMap tq;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.n_heads, (uint64_t)a.kv.rows};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.ldq * 2};
  const uint32_t box[3] = {64, (uint32_t)p.heads, (uint32_t)p.rows};
  if (!encode_tensor_map_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  for (int s0 = 0; s0 < a.kv.n_seqs; s0 += kWeighSeqs) {
    p.a.kv = kv_slice(a.kv, s0, a.kv.n_seqs - s0 < kWeighSeqs ? a.kv.n_seqs - s0 : kWeighSeqs);
    const cudaError_t e = launch_overlapped(a.softcap > 0.f ? kv8_weigh_chunk_kernel<D, true> : kv8_weigh_chunk_kernel<D, false>,
                                            2 * a.num_sms, kWeighThreads, WeighCfg<D>::kSmem, st, 2, tq, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv8_weigh_chunk(const KvAttention &a, cudaStream_t st) {
  return a.kv.head_dim == 64 ? weigh_chunk<64>(a, st) : weigh_chunk<128>(a, st);
}

cudaError_t init_kv8_weigh_chunk_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  for (const void *f : {(const void *)kv8_weigh_chunk_kernel<64, false>, (const void *)kv8_weigh_chunk_kernel<64, true>,
                        (const void *)kv8_weigh_chunk_kernel<128, false>, (const void *)kv8_weigh_chunk_kernel<128, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, WeighCfg<128>::kSmem);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_weigh_chunk(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
