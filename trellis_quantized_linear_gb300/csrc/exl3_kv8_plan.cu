// Block tables, lengths, positions and slots of a step from its requests' lengths.
// Contract in include/exl3.h.
//
// The prefix sums of rows and of pages over the sequences say everything: who is served, whose
// pages are whose, where a row lies. One cluster: its CTAs have a contiguous part of the
// sequences each (four a thread), join their sums through shared memory of the cluster, then
// hand out the pages, a thread each, and after a last barrier the rows' positions and slots,
// four rows a thread, which finds the first one's sequence by a binary search in shared memory.
// Few sequences are one CTA's, and many rows are still shared by the cluster.
//
// All latency: the bytes are some hundred KB at most, and a few dependent loads stand one after
// the other, with the barriers between them. Measured (in a graph): 16 sequences of one token
// 4.9 us; 64 with 16 prompts, 16K rows 8.5; 4096 sequences, 18K rows 12.7 (15.9 by one CTA; a fence at
// each of the cluster's barriers 13.2).
#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;  // at most
constexpr int kEach = 4;               // sequences of a thread, one behind the other
constexpr int kMaxRanks = 8;
constexpr int kHeldSeqs = 11 * 1024;   // sequences whose row starts are held in shared memory
constexpr uint32_t kFull = 1u << 30;   // sums stop here: above every bound that they are compared with

__device__ __forceinline__ uint32_t sum_to_full(uint32_t a, uint32_t b) { return min(a + b, kFull); }

// Three sums at once: rows, pages that are needed, pages that come back.
struct Sums {
  uint32_t rows, need, give;
  __device__ __forceinline__ Sums plus(const Sums &o) const {
    return {sum_to_full(rows, o.rows), sum_to_full(need, o.need), sum_to_full(give, o.give)};
  }
  __device__ __forceinline__ Sums from(int lane) const {
    return {__shfl_sync(0xffffffffu, rows, lane), __shfl_sync(0xffffffffu, need, lane), __shfl_sync(0xffffffffu, give, lane)};
  }
  __device__ __forceinline__ Sums inclusive() const {  // over the warp's lanes up to this one
    Sums v = *this;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o{__shfl_up_sync(0xffffffffu, v.rows, d), __shfl_up_sync(0xffffffffu, v.need, d), __shfl_up_sync(0xffffffffu, v.give, d)};
      if (lane >= d) v = v.plus(o);
    }
    return v;
  }
};
// Over the threads before this one, and over all of them. Two barriers.
__device__ __forceinline__ Sums scan_before(Sums v, Sums *warp_sum, Sums &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Sums up = v.inclusive();
  if (lane == 31) warp_sum[warp] = up;
  __syncthreads();
  static_assert(kPlanWarps == 32, "a warp's lane for each warp");
  Sums w{0, 0, 0};
  if (lane < (int)(blockDim.x >> 5)) w = warp_sum[lane];
  w = w.inclusive();
  const Sums before_warp = w.from(max(warp - 1, 0)), before_lane = up.from(max(lane - 1, 0));
  total = w.from(31);
  __syncthreads();
  Sums b{0, 0, 0};
  if (warp > 0) b = before_warp;
  return lane > 0 ? b.plus(before_lane) : b;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (int)(((uint32_t)tokens + kKvBlock - 1) / kKvBlock); }

// The last of n numbers, not decreasing, that is at most x (the first is).
__device__ __forceinline__ int last_at_most(const uint32_t *v, int n, uint32_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// What the CTAs of the cluster tell each other.
struct Told {
  Sums all;        // of its sequences
  int first_left;  // the first of them that is not served
  Sums before;     // what comes before it
};

__global__ void __launch_bounds__(kPlanThreads) kv8_plan_kernel(const KvPlan p, int ranks, int sharing) {
  extern __shared__ int2 held[];  // where the rows of a sequence end, and a row's distance to its position, where there is room
  __shared__ uint32_t page_at[kPlanThreads * kEach];  // pages before each sequence of a pass
  __shared__ int block_at[kPlanThreads * kEach];      // and its first block that one of them is for
  __shared__ Sums warp_sum[kPlanWarps];
  __shared__ Told told[kMaxRanks];
  __shared__ int first_left;      // of this CTA's sequences
  __shared__ Sums at_left;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rank = ranks > 1 ? (int)cluster_ctarank() : 0;
  const int threads = blockDim.x, at_once = threads * kEach;
  const bool holds = p.n_seqs <= kHeldSeqs;
  [[maybe_unused]] const int64_t table_size = (int64_t)p.n_seqs * p.max_pages;
  const int64_t room = (int64_t)p.max_pages * kKvBlock;
  const int part = (p.n_seqs + sharing - 1) / sharing, part0 = min(rank * part, p.n_seqs), part1 = min(part0 + part, p.n_seqs);
  const bool once = part <= at_once;  // a thread's sequences stay in registers
  auto everyone = [&](int ctas) {  // the CTAs' threads; releases what they wrote before, memory included
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
  };
  // thread r of the first warp stores to CTA r; `at` in words of Told
  auto tell = [&](int at, const uint32_t *v, int n) {
    if (threadIdx.x < (uint32_t)sharing)
      for (int i = 0; i < n; ++i) {
        const uint32_t dst = smem_u32(reinterpret_cast<uint32_t *>(told + rank) + at + i);
        if (sharing > 1) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(dst, threadIdx.x)), "r"(v[i]) : "memory");
        else reinterpret_cast<uint32_t *>(told + rank)[at + i] = v[i];
      }
  };

  if (rank < sharing) {
    int count = *p.free_count;
    if (threadIdx.x == 0) first_left = INT32_MAX;
    // of the thread's sequences: tokens after the step, blocks before it, and what they add to the sums
    int len[kEach], blocks[kEach];
    bool valid[kEach], fits[kEach];
    Sums adds[kEach], mine, total, before;
    auto load = [&](int c) {
      const int s0 = c + (int)threadIdx.x * kEach;
      mine = {0, 0, 0};
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        valid[k] = fits[k] = true;
        len[k] = blocks[k] = 0;
        adds[k] = mine;
      }
      if (s0 < part1) {  // whole warps have none, where rows need more threads than sequences
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int s = s0 + k, tokens = s < part1 ? p.tokens[s] : 0, have = s < part1 ? p.cached[s] : 0, add = max(tokens, 0);
          valid[k] = have >= 0 && have <= room;
          fits[k] = valid[k] && add <= p.max_rows && have + (int64_t)add <= room;
          blocks[k] = valid[k] ? blocks_of(have) : 0;
          len[k] = tokens < 0 || !valid[k] ? 0 : have;
          adds[k] = {(uint32_t)min(add, (int)kFull), fits[k] && add > 0 ? (uint32_t)(blocks_of(have + add) - blocks[k]) : 0u,
                     tokens < 0 ? (uint32_t)blocks[k] : 0u};
          mine = mine.plus(adds[k]);
        }
      }
      before = scan_before(mine, warp_sum, total);
    };
    if (count < 0 || count > p.free_capacity) {
      if (rank == 0 && threadIdx.x == 0) report_index(p.status);
      count = min(max(count, 0), p.free_capacity);
    }
    // 1. sums of the part
    Sums sum{0, 0, 0};
    for (int c = part0; c < part1; c += at_once) {
      load(c);
      sum = sum.plus(total);
    }
    if (sharing > 1) cluster_sync_all();  // every CTA runs before another stores to it
    {
      const uint32_t v[3] = {sum.rows, sum.need, sum.give};
      tell(0, v, 3);
    }
    everyone(sharing);
    Sums base{0, 0, 0}, whole{0, 0, 0};
    for (int r = 0; r < sharing; ++r) {
      if (r == rank) base = whole;
      whole = whole.plus(told[r].all);
    }
    // 2. pages come back, and the first sequence of the part that does not fit
    const int after = (int)min((uint32_t)count + whole.give, (uint32_t)p.free_capacity);
    Sums carry = base;
    for (int c = part0; c < part1; c += at_once) {
      if (!once) load(c);
      if (total.give > 0) {  // the same in all threads
        uint32_t at = before.give;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          page_at[threadIdx.x * kEach + k] = at;
          at = sum_to_full(at, adds[k].give);
        }
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < total.give; j += threads) {
          const int i = last_at_most(page_at, at_once, j);
          const int64_t from = (int64_t)(c + i) * p.max_pages + (j - page_at[i]);
          const uint32_t to = (uint32_t)count + sum_to_full(carry.give, j);
          if (to >= (uint32_t)p.free_capacity) report_index(p.status);  // more pages than there are
          else if (EXL3_SPAN(from, 1, table_size)) p.free_pages[to] = p.page_table[from];
        }
      }
      Sums upto = carry.plus(before);
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int s = c + (int)threadIdx.x * kEach + k;
        upto = upto.plus(adds[k]);
        if (s < part1) {
          if (!valid[k]) report_index(p.status);
          if (!(fits[k] && upto.rows <= (uint32_t)p.rows && upto.need <= (uint32_t)after)) atomicMin(&first_left, s);
        }
      }
      __syncthreads();
      upto = carry.plus(before);
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (c + (int)threadIdx.x * kEach + k == first_left) at_left = upto;
        upto = upto.plus(adds[k]);
      }
      carry = carry.plus(total);
    }
    __syncthreads();
    {
      const uint32_t v[4] = {(uint32_t)first_left, at_left.rows, at_left.need, 0};
      tell(3, v, 4);
    }
    everyone(sharing);  // and the pages that came back are there
    int left = INT32_MAX;  // of all
    Sums ends = whole;     // the served ones' sums
    for (int r = 0; r < sharing; ++r)
      if (told[r].first_left < left) {
        left = told[r].first_left;
        ends = told[r].before;
      }
    // 3. lengths, row ranges, and pages from the top
    carry = base;
    for (int c = part0; c < part1; c += at_once) {
      if (!once) load(c);
      Sums upto = before;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        page_at[threadIdx.x * kEach + k] = upto.need;
        block_at[threadIdx.x * kEach + k] = blocks[k];
        upto.need = sum_to_full(upto.need, adds[k].need);
      }
      upto = carry.plus(before);
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int s = c + (int)threadIdx.x * kEach + k;
        const bool served = s < left;
        upto = upto.plus(adds[k]);
        if (s < part1) {
          const int end = (int)(served ? upto.rows : ends.rows), now = len[k] + (served ? (int)adds[k].rows : 0);
          p.kv_len[s] = now;
          p.q_start[s + 1] = end;
          if (holds) held[s] = make_int2(end, now - end);
        }
      }
      __syncthreads();
      const uint32_t all = left < c ? 0u : left < min(c + at_once, part1) ? ends.need - carry.need : total.need;
      for (uint32_t j = threadIdx.x; j < all; j += threads) {
        const int i = last_at_most(page_at, at_once, j), from = after - 1 - (int)(carry.need + j);
        const int64_t to = (int64_t)(c + i) * p.max_pages + block_at[i] + (j - page_at[i]);
        int page = EXL3_SPAN(from, 1, p.free_capacity) ? p.free_pages[from] : -1;
        if (page < 0 || page >= p.n_pages) {
          report_index(p.status);
          page = -1;
        }
        if (EXL3_SPAN(to, 1, table_size)) p.page_table[to] = page;
      }
      carry = carry.plus(total);
    }
    if (rank == 0 && threadIdx.x == 0) {
      p.q_start[0] = 0;
      *p.free_left = after - (int)ends.need;
      *p.served = min(left, p.n_seqs);
    }
  }
  everyone(ranks);
  // 4. the rows
  if (ranks > 1 && holds) {
    for (int s = threadIdx.x; s < p.n_seqs; s += threads) {
      if (s >= part0 && s < part1) continue;
      const int end = __ldcg(p.q_start + s + 1);
      held[s] = make_int2(end, __ldcg(p.kv_len + s) - end);
    }
    __syncthreads();
  }
  auto end_of = [&](int s) { return holds ? held[s].x : __ldcg(p.q_start + s + 1); };
  const int used = p.n_seqs > 0 ? end_of(p.n_seqs - 1) : 0;
  constexpr int kRows = 4;  // of a thread
  const bool by_four = ((reinterpret_cast<uintptr_t>(p.position) | reinterpret_cast<uintptr_t>(p.slot)) & 15) == 0;
  for (int64_t r0 = ((int64_t)rank * threads + threadIdx.x) * kRows; r0 < p.rows; r0 += (int64_t)ranks * threads * kRows) {
    int pos[kRows], slot[kRows], page[kRows];
    int lo = 0;
    if (r0 < used) {  // the first row's sequence: the first one that ends after it
      int hi = p.n_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end_of(mid) > r0) hi = mid;
        else lo = mid + 1;
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = (int)r0 + k;
      pos[k] = page[k] = -1;
      if (r < used) {
        while (end_of(lo) <= r) ++lo;
        pos[k] = r + (holds ? held[lo].y : __ldcg(p.kv_len + lo) - end_of(lo));
        slot[k] = lo;
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (pos[k] < 0) continue;
      const int64_t at = (int64_t)slot[k] * p.max_pages + pos[k] / kKvBlock;
      if (EXL3_SPAN(at, 1, table_size)) page[k] = __ldcg(p.page_table + at);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const bool ok = page[k] >= 0 && page[k] < p.n_pages;
      if (pos[k] >= 0 && !ok) report_index(p.status);
      slot[k] = pos[k] >= 0 && ok ? page[k] * kKvBlock + pos[k] % kKvBlock : -1;
    }
    if (by_four && r0 + kRows <= p.rows) {
      *reinterpret_cast<int4 *>(p.position + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4 *>(p.slot + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (r0 + k < p.rows) {
          p.position[r0 + k] = pos[k];
          p.slot[r0 + k] = slot[k];
        }
    }
  }
}

}  // namespace

cudaError_t launch_kv8_plan(const KvPlan &p, cudaStream_t st) {
  const int ranks = p.rows > 4 * kPlanThreads || p.n_seqs > kPlanThreads ? kMaxRanks : 1;
  // No more threads than sequences and rows give work to: with 1024, 16 sequences take 7.6 us, with 64 of them 5.
  // Up to 1024 sequences are one CTA's: shared by 8, 64 of them with prompts take 9.9 us for 8.5,
  // 4096 sequences 12.7 for 15.9.
  const int sharing = p.n_seqs > kPlanThreads ? ranks : 1;
  const int64_t rows = ceil_div(p.rows, ranks), seqs = ceil_div(p.n_seqs, sharing);
  const int64_t work = ceil_div(rows > seqs ? rows : seqs, kEach);
  const int threads = work >= kPlanThreads ? kPlanThreads : work <= 64 ? 64 : (int)(ceil_div(work, 32) * 32);
  const size_t smem = p.n_seqs <= kHeldSeqs ? (size_t)p.n_seqs * sizeof(int2) : 0;
  return launch_overlapped(kv8_plan_kernel, dim3((unsigned)ranks), threads, smem, st, ranks, p, ranks, sharing);
}

cudaError_t init_kv8_plan_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  return e == cudaSuccess ? cudaFuncSetAttribute(kv8_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldSeqs * (int)sizeof(int2))
                          : e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_plan(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
