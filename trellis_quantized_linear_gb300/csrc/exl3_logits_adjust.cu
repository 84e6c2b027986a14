// Penalties, biases and a grammar mask on logits, and the greedy choice from
// what is left. Formula in include/exl3.h.
//
// A cluster of up to 16 CTAs per row, each with a contiguous range of the
// vocabulary. A CTA counts the row's history into one 32-bit word for each of
// its tokens in shared memory (integer adds: any order gives the same counts),
// while its logits are already on their way into registers; each logit is read
// and written once. The row's greedy choice is joined through the cluster's
// shared memory. Biases are few: their tokens are marked, left out of the
// stream and done one by one after it.
#include <limits.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kAdjustVecs = 8;   // 4-token pieces that a thread holds at a time
constexpr int kMaxCluster = 16;
// A token's word: in the history at all, has a bias, times generated.
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3FFFFFFFu;

struct AdjustParams {
  const float *logits;
  float *out;
  int32_t *argmax;
  int *status;
  int64_t ldl, ldo, M;
  int n, range;  // tokens, tokens of a CTA (a multiple of 128)
  exl3_logits_rules r;
};

struct RowRules {
  float rep, pres, freq;
};

__device__ __forceinline__ float penalized(float x, uint32_t word, const RowRules &r) {
  if (word & (kSeen | kCount)) {
    x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
    const uint32_t made = word & kCount;
    if (made) x = __fsub_rn(x, __fadd_rn(__fmul_rn(r.freq, (float)made), r.pres));
  }
  return x;
}

// Start and end of row m in a list of `size` entries; an impossible range is
// reported and empty.
__device__ __forceinline__ int2 row_range(const int32_t *start, int64_t m, int size, int *status) {
  if (!start) return make_int2(0, 0);
  const int2 v = make_int2(start[m], start[m + 1]);
  if (v.x >= 0 && v.y >= v.x && v.y <= size) return v;
  report_index(status);
  return make_int2(0, 0);
}

struct Best {
  float x = -INFINITY;
  int t = INT_MAX;
  __device__ __forceinline__ void take(float y, int i) {
    if (y > x || (y == x && i < t)) {
      x = y;
      t = i;
    }
  }
  // Only the first maximum above -inf counts, so INT_MAX stays with -inf.
  __device__ __forceinline__ void see(float y, int i) {
    if (y > x) {
      x = y;
      t = i;
    }
  }
};

template <int kAdjustThreads>
__global__ void __launch_bounds__(kAdjustThreads, 768 / kAdjustThreads) logits_adjust_kernel(const AdjustParams p) {
  extern __shared__ __align__(16) uint32_t words[];  // one of each token of the range
  __shared__ float sb[kAdjustThreads / 32], cb[kMaxCluster];
  __shared__ int si[kAdjustThreads / 32], ci[kMaxCluster], duplicates;
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  const int64_t m = blockIdx.x / ranks;
  const int t0 = (int)rank * p.range, t1 = min(t0 + p.range, p.n);  // this CTA's tokens
  for (int i = tid * 4; i < p.range; i += kAdjustThreads * 4)
    if (EXL3_SPAN(i, 4, p.range)) *reinterpret_cast<uint4 *>(words + i) = make_uint4(0, 0, 0, 0);
  if (tid == 0) duplicates = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const float *logits = p.logits + m * p.ldl;
  float *out = p.out + m * p.ldo;
  const uint32_t *allowed = p.r.allowed ? p.r.allowed + m * ((p.n + 31) / 32) : nullptr;
  float4 x[kAdjustVecs];
  uint32_t bits[kAdjustVecs];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < kAdjustVecs; ++k) {
      const int t = base + (k * kAdjustThreads + tid) * 4;
      if (t >= t1) continue;
      if (t + 4 <= p.n) {
        x[k] = *reinterpret_cast<const float4 *>(logits + t);
      } else {  // what lies past the last token is not read
        x[k].x = logits[t];
        x[k].y = t + 1 < p.n ? logits[t + 1] : 0.f;
        x[k].z = t + 2 < p.n ? logits[t + 2] : 0.f;
        x[k].w = 0.f;
      }
      bits[k] = allowed ? allowed[t >> 5] >> (t & 31) : 0xFu;
    }
  };
  load(t0);  // in flight while the history is counted

  const RowRules r{p.r.repetition ? p.r.repetition[m] : 1.f, p.r.presence ? p.r.presence[m] : 0.f,
                   p.r.frequency ? p.r.frequency[m] : 0.f};
  const int2 h = row_range(p.r.history_start, m, p.r.history_size, p.status);
  const int2 b = row_range(p.r.bias_start, m, p.r.bias_size, p.status);
  const int made_from = p.r.generated_from ? p.r.generated_from[m] : 0;
  __syncthreads();
  constexpr int kAhead = 8;
  for (int i = h.x + tid; i < h.y; i += kAdjustThreads * kAhead) {
    uint32_t t[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      t[k] = i + k * kAdjustThreads < h.y ? (uint32_t)p.r.history[i + k * kAdjustThreads] - (uint32_t)t0 : ~0u;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t[k] < (uint32_t)(t1 - t0) && t0 < t1) {
        if (i + k * kAdjustThreads - h.x >= made_from) atomicAdd(&words[t[k]], 1u);
        else atomicOr(&words[t[k]], kSeen);
      }
  }
  for (int i = b.x + tid; i < b.y; i += kAdjustThreads) {
    const uint32_t t = (uint32_t)p.r.bias_id[i] - (uint32_t)t0;
    if (t0 < t1 && t < (uint32_t)(t1 - t0) && (atomicOr(&words[t], kBiased) & kBiased)) duplicates = 1;
  }
  __syncthreads();

  Best best;
  for (int base = t0; base < t1; base += kAdjustThreads * kAdjustVecs * 4) {
    if (base != t0) load(base);
#pragma unroll
    for (int k = 0; k < kAdjustVecs; ++k) {
      const int t = base + (k * kAdjustThreads + tid) * 4;
      if (t >= t1 || !EXL3_SPAN(t - t0, 4, p.range)) continue;
      const uint4 w = *reinterpret_cast<const uint4 *>(words + t - t0);
      float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      if (w.x | w.y | w.z | w.w) {
        v[0] = penalized(v[0], w.x, r);
        v[1] = penalized(v[1], w.y, r);
        v[2] = penalized(v[2], w.z, r);
        v[3] = penalized(v[3], w.w, r);
      }
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!((bits[k] >> e) & 1u)) v[e] = -INFINITY;
        if (!(ww[e] & kBiased) && t + e < p.n) best.see(v[e], t + e);
      }
      if (t + 4 <= p.n) {
        *reinterpret_cast<float4 *>(out + t) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (t + e < p.n) out[t + e] = v[e];
      }
    }
  }
  if (b.y > b.x) {
    // The stream has written l before the bias (or -inf) for the marked tokens;
    // whoever clears a token's mark adds its bias: its entry, or all of them in
    // their order where some token has several.
    __syncthreads();
    for (int i = b.x + tid; i < b.y; i += kAdjustThreads) {
      const int id = p.r.bias_id[i];
      if (id < t0 || id >= t1 || !(atomicAnd(&words[id - t0], ~kBiased) & kBiased)) continue;
      float sum = p.r.bias_value[i];
      if (duplicates) {
        sum = 0.f;
        for (int j = b.x; j < b.y; ++j)
          if (p.r.bias_id[j] == id) sum = __fadd_rn(sum, p.r.bias_value[j]);
      }
      float v = out[id];
      if (!allowed || ((allowed[id >> 5] >> (id & 31)) & 1u)) {
        v = __fadd_rn(v, sum);
        out[id] = v;
      }
      if (v > -INFINITY) best.take(v, id);
    }
  }

#pragma unroll
  for (int k = 16; k > 0; k >>= 1) best.take(__shfl_xor_sync(0xffffffffu, best.x, k), __shfl_xor_sync(0xffffffffu, best.t, k));
  if (lane == 0) {
    sb[tid >> 5] = best.x;
    si[tid >> 5] = best.t;
  }
  __syncthreads();
  if (tid < 32) {
    best = Best();
    if (lane < kAdjustThreads / 32) best.take(sb[lane], si[lane]);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) best.take(__shfl_xor_sync(0xffffffffu, best.x, k), __shfl_xor_sync(0xffffffffu, best.t, k));
    if (lane == 0) {  // to the first CTA of the cluster
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&cb[rank]), 0)), "f"(best.x) : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&ci[rank]), 0)), "r"(best.t) : "memory");
    }
  }
  __syncwarp();
  cluster_sync_all();
  if (rank == 0 && tid == 0) {
    best = Best();
    for (uint32_t c = 0; c < ranks; ++c) best.take(cb[c], ci[c]);
    p.argmax[m] = best.t == INT_MAX ? -1 : best.t;
  }
}

}  // namespace

cudaError_t launch_logits_adjust(const float *logits, int64_t ldl, int64_t M, int64_t n, const exl3_logits_rules &r,
                                 float *out, int64_t ldo, int32_t *argmax, int *status, int num_sms, cudaStream_t st) {
  if (M == 0) return cudaSuccess;
  // 2048 tokens (one piece a thread) to a CTA at least, up to 16 CTAs
  int ranks = 1;
  while (ranks < kMaxCluster && n > (int64_t)ranks * 2048) ranks *= 2;
  AdjustParams p{logits, out, argmax, status, ldl, ldo, M, (int)n, (int)(ceil_div(n, 128 * ranks) * 128), r};
  // Few rows: every CTA has an SM to itself and 512 threads hold its whole range;
  // many rows: three CTAs of 256 threads an SM, so that one streams while another counts.
  const bool few = M * ranks <= num_sms;
  const auto kernel = few ? logits_adjust_kernel<512> : logits_adjust_kernel<256>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * ranks));
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.dynamicSmemBytes = (size_t)p.range * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t init_logits_adjust_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  for (const void *f : {(const void *)logits_adjust_kernel<256>, (const void *)logits_adjust_kernel<512>}) {
    // the widest range: 2^19 tokens over 16 CTAs
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (1 << 19) / kMaxCluster * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  }
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_logits_adjust(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
