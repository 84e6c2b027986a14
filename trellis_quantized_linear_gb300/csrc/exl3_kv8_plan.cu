// Block tables, lengths, positions and slots of a step from its requests' lengths.
// Contract in include/exl3.h.
//
// One cluster. Its first CTA takes the pages of ended sequences back, then goes over the
// sequences (a prefix sum of rows and of new pages) and hands pages out; after the
// cluster's barrier all its CTAs write the rows' positions and slots, each row finding
// its sequence by a binary search in shared memory. All latency: a few dependent loads.
#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kHeldSeqs = 11 * 1024;  // sequences whose row starts are held in shared memory
constexpr uint32_t kFull = 1u << 30;  // sums stop here: above every bound that they are compared with

__device__ __forceinline__ uint32_t sum_to_full(uint32_t a, uint32_t b) { return min(a + b, kFull); }

// Sum over the threads up to this one, and over all of them; of two numbers at once.
struct Two {
  uint32_t a, b;
  __device__ __forceinline__ Two plus(const Two &o) const { return {sum_to_full(a, o.a), sum_to_full(b, o.b)}; }
};
__device__ __forceinline__ Two scan(Two v, Two *warp_sum, Two &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two o{__shfl_up_sync(0xffffffffu, v.a, d), __shfl_up_sync(0xffffffffu, v.b, d)};
    if (lane >= d) v = v.plus(o);
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  Two w = warp_sum[lane];
  static_assert(kPlanWarps == 32, "a warp's lane for each warp");
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Two o{__shfl_up_sync(0xffffffffu, w.a, d), __shfl_up_sync(0xffffffffu, w.b, d)};
    if (lane >= d) w = w.plus(o);
  }
  total = {__shfl_sync(0xffffffffu, w.a, 31), __shfl_sync(0xffffffffu, w.b, 31)};
  const Two before{__shfl_sync(0xffffffffu, w.a, max(warp - 1, 0)), __shfl_sync(0xffffffffu, w.b, max(warp - 1, 0))};
  if (warp > 0) v = v.plus(before);
  __syncthreads();
  return v;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (int)(((uint32_t)tokens + kKvBlock - 1) / kKvBlock); }

// Hands the warp's lanes' pages out or takes them back: f(sequence, block of it, place in
// the lane's order), `n` pages from block `first` of sequence `s` of each lane.
template <typename F>
__device__ __forceinline__ void for_pages(int s, int first, int n, uint32_t place, F &&f) {
  const int lane = threadIdx.x & 31;
  if (n == 1) f(s, first, place);
  for (uint32_t many = __ballot_sync(0xffffffffu, n > 1); many; many &= many - 1) {
    const int from = __ffs(many) - 1;
    const int s1 = __shfl_sync(0xffffffffu, s, from), first1 = __shfl_sync(0xffffffffu, first, from),
              n1 = __shfl_sync(0xffffffffu, n, from);
    const uint32_t place1 = __shfl_sync(0xffffffffu, place, from);
    for (int i = lane; i < n1; i += 32) f(s1, first1 + i, place1 + i);
  }
}

__global__ void __launch_bounds__(kPlanThreads) kv8_plan_kernel(const KvPlan p, int ranks) {
  extern __shared__ int held[];  // row starts, where there is room for them
  __shared__ Two warp_sum[kPlanWarps];
  __shared__ int first_left;     // the first sequence that is not served
  __shared__ Two at_left;        // rows and pages of those before it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t rank = ranks > 1 ? cluster_ctarank() : 0;
  const bool holds = p.n_seqs <= kHeldSeqs;
  [[maybe_unused]] const int64_t table_size = (int64_t)p.n_seqs * p.max_pages;
  const int64_t room = (int64_t)p.max_pages * kKvBlock;
  if (rank == 0) {
    if (threadIdx.x == 0) first_left = INT32_MAX;
    int count = *p.free_count;
    if (count < 0 || count > p.free_capacity) {
      if (threadIdx.x == 0) report_index(p.status);
      count = min(max(count, 0), p.free_capacity);
    }
    Two total;
    uint32_t given = 0;
    for (int c = 0; c < p.n_seqs; c += kPlanThreads) {
      const int s = c + (int)threadIdx.x;
      int n = 0;
      if (s < p.n_seqs && p.tokens[s] < 0) {
        const int have = p.cached[s];
        if (have >= 0 && have <= room) n = blocks_of(have);
      }
      if (!__syncthreads_or(n > 0)) continue;
      const uint32_t end = sum_to_full(given, scan({(uint32_t)n, 0}, warp_sum, total).a);
      for_pages(s, 0, n, (uint32_t)count + end - n, [&](int seq, int block, uint32_t place) {
        const int64_t from = (int64_t)seq * p.max_pages + block;
        if (place >= (uint32_t)p.free_capacity) report_index(p.status);  // more pages than there are
        else if (EXL3_SPAN(from, 1, table_size)) p.free_pages[place] = p.page_table[from];
      });
      given = sum_to_full(given, total.a);
    }
    count = (int)min((uint32_t)count + given, (uint32_t)p.free_capacity);
    __syncthreads();  // the pages that came back
    Two carry{0, 0};
    if (threadIdx.x == 0) {
      p.q_start[0] = 0;
      if (holds) held[0] = 0;
    }
    for (int c = 0; c < p.n_seqs; c += kPlanThreads) {
      const int s = c + (int)threadIdx.x;
      int tokens = 0, have = 0;
      bool fits = true;
      if (s < p.n_seqs) {
        tokens = p.tokens[s];
        have = p.cached[s];
        if (have < 0 || have > room) {
          report_index(p.status);
          fits = false;
          have = 0;
        }
      }
      const int add = max(tokens, 0);
      fits = fits && add <= p.max_rows && have + (int64_t)add <= room;
      const int held_blocks = blocks_of(have), need = fits && add > 0 ? blocks_of(have + add) - held_blocks : 0;
      const Two upto = carry.plus(scan({(uint32_t)min(add, (int)kFull), (uint32_t)need}, warp_sum, total));
      fits = fits && upto.a <= (uint32_t)p.rows && upto.b <= (uint32_t)count;
      if (s < p.n_seqs && !fits) atomicMin(&first_left, s);
      __syncthreads();
      // a sequence that does not fit has its own sums in `upto`; those before it end where it begins
      if (s == first_left && threadIdx.x == 0) at_left = carry;
      if (s + 1 == first_left && threadIdx.x + 1 < kPlanThreads) at_left = upto;
      __syncthreads();
      const bool served = s < first_left;
      if (s < p.n_seqs) {
        p.kv_len[s] = tokens < 0 ? 0 : served ? have + add : have;
        const int end = (int)(served ? upto.a : at_left.a);
        p.q_start[s + 1] = end;
        if (holds) held[s + 1] = end;
      }
      for_pages(s, held_blocks, s < p.n_seqs && served ? need : 0, upto.b - need, [&](int seq, int block, uint32_t place) {
        const int64_t to = (int64_t)seq * p.max_pages + block;
        const int from = count - 1 - (int)place;
        int page = EXL3_SPAN(from, 1, p.free_capacity) ? p.free_pages[from] : -1;
        if (page < 0 || page >= p.n_pages) {
          report_index(p.status);
          page = -1;
        }
        if (EXL3_SPAN(to, 1, table_size)) p.page_table[to] = page;
      });
      carry = carry.plus(total);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      const bool all = first_left >= p.n_seqs;
      *p.free_left = count - (int)(all ? carry.b : at_left.b);
      *p.served = all ? p.n_seqs : first_left;
    }
    __threadfence();
  }
  if (ranks > 1) cluster_sync_all();
  else __syncthreads();
  if (rank > 0 && holds) {
    for (int s = threadIdx.x; s <= p.n_seqs; s += kPlanThreads) held[s] = __ldcg(p.q_start + s);
    __syncthreads();
  }
  const int *start = holds ? held : p.q_start;
  const int used = start[p.n_seqs];
  for (int r = rank * kPlanThreads + threadIdx.x; r < p.rows; r += ranks * kPlanThreads) {
    int pos = -1, slot = -1;
    if (r < used) {
      int lo = 0, hi = p.n_seqs - 1;  // the sequence with start[s] <= r < start[s + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid + 1] > r) hi = mid;
        else lo = mid + 1;
      }
      pos = __ldcg(p.kv_len + lo) - (start[lo + 1] - r);
      const int64_t at = (int64_t)lo * p.max_pages + pos / kKvBlock;
      const int page = EXL3_SPAN(at, 1, table_size) ? __ldcg(p.page_table + at) : -1;
      if (page < 0 || page >= p.n_pages) report_index(p.status);
      else slot = page * kKvBlock + pos % kKvBlock;
    }
    p.position[r] = pos;
    p.slot[r] = slot;
  }
}

}  // namespace

cudaError_t launch_kv8_plan(const KvPlan &p, cudaStream_t st) {
  const int ranks = p.rows > 2 * kPlanThreads ? 8 : 1;
  const size_t smem = p.n_seqs <= kHeldSeqs ? ((size_t)p.n_seqs + 1) * sizeof(int) : 0;
  return launch_overlapped(kv8_plan_kernel, dim3((unsigned)ranks), kPlanThreads, smem, st, ranks, p, ranks);
}

cudaError_t init_kv8_plan_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes attr;
  return e == cudaSuccess ? cudaFuncGetAttributes(&attr, kv8_plan_kernel) : e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_plan(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
