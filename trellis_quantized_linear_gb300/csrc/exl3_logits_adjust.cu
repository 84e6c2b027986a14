// Penalties, biases and a grammar mask on logits, and the greedy choice from
// what is left. Formula in include/exl3.h.
#include <limits.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

constexpr int kAdjustThreads = 1024;
constexpr int kAdjustChunk = 4096;  // tokens whose counts and biases are held in shared memory at a time
constexpr uint32_t kSeen = 0x80000000u;

// One CTA per row, a chunk of the vocabulary at a time: the row's history is
// counted into shared memory (integers: any order gives the same counts), its
// biases are added up by one warp in their order, then the chunk's logits go
// through once.
__global__ void __launch_bounds__(kAdjustThreads) logits_adjust_kernel(const float *logits, int64_t ldl, int n,
                                                                       exl3_logits_rules r, float *out, int64_t ldo,
                                                                       int32_t *argmax, int *status) {
  __shared__ uint32_t count[kAdjustChunk];
  __shared__ float bias[kAdjustChunk];
  const int m = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  int h0 = 0, h1 = 0, g0 = 0, b0 = 0, b1 = 0;
  if (r.history) {
    h0 = r.history_start[m];
    h1 = r.history_start[m + 1];
    if (h0 < 0 || h1 < h0 || h1 > r.history_size) {
      if (tid == 0) report_index(status);
      h0 = h1 = 0;
    }
    g0 = r.generated_from ? r.generated_from[m] : 0;
  }
  if (r.bias_id) {
    b0 = r.bias_start[m];
    b1 = r.bias_start[m + 1];
    if (b0 < 0 || b1 < b0 || b1 > r.bias_size) {
      if (tid == 0) report_index(status);
      b0 = b1 = 0;
    }
  }
  const float rep = r.repetition ? r.repetition[m] : 1.f;
  const float pres = r.presence ? r.presence[m] : 0.f, freq = r.frequency ? r.frequency[m] : 0.f;
  const uint32_t *allowed = r.allowed ? r.allowed + (int64_t)m * ((n + 31) / 32) : nullptr;
  float best = -INFINITY;
  int index = INT_MAX;
  for (int c0 = 0; c0 < n; c0 += kAdjustChunk) {
    for (int i = tid; i < kAdjustChunk; i += kAdjustThreads) {
      count[i] = 0;
      bias[i] = 0.f;
    }
    __syncthreads();
    for (int i = h0 + tid; i < h1; i += kAdjustThreads) {
      const uint32_t t = (uint32_t)r.history[i] - (uint32_t)c0;
      if (t < (uint32_t)kAdjustChunk) {
        if (i - h0 >= g0) atomicAdd(&count[t], 1u);
        else atomicOr(&count[t], kSeen);
      }
    }
    if (tid < 32)
      for (int i = b0; i < b1; i += 32) {
        const uint32_t t = i + lane < b1 ? (uint32_t)r.bias_id[i + lane] - (uint32_t)c0 : ~0u;
        const float v = i + lane < b1 ? r.bias_value[i + lane] : 0.f;
        for (int l = 0; l < 32; ++l) {
          if (lane == l && t < (uint32_t)kAdjustChunk) bias[t] += v;
          __syncwarp();
        }
      }
    __syncthreads();
    for (int i = tid; i < kAdjustChunk && c0 + i < n; i += kAdjustThreads) {
      const int t = c0 + i;
      float x = logits[m * ldl + t];
      const uint32_t c = count[i];
      if (c) {
        x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        const uint32_t made = c & ~kSeen;
        if (made) x = __fsub_rn(x, __fadd_rn(__fmul_rn(freq, (float)made), pres));
      }
      x = __fadd_rn(x, bias[i]);
      if (allowed && !((allowed[t >> 5] >> (t & 31)) & 1u)) x = -INFINITY;
      out[m * ldo + t] = x;
      if (x > best) {
        best = x;
        index = t;
      }
    }
    __syncthreads();
  }
  __shared__ float sb[32];
  __shared__ int si[32];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) {
    const float ob = __shfl_xor_sync(0xffffffffu, best, k);
    const int oi = __shfl_xor_sync(0xffffffffu, index, k);
    if (ob > best || (ob == best && oi < index)) {
      best = ob;
      index = oi;
    }
  }
  if (lane == 0) {
    sb[tid >> 5] = best;
    si[tid >> 5] = index;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kAdjustThreads / 32; ++w)
      if (sb[w] > best || (sb[w] == best && si[w] < index)) {
        best = sb[w];
        index = si[w];
      }
    argmax[m] = index == INT_MAX ? -1 : index;
  }
}

}  // namespace

cudaError_t launch_logits_adjust(const float *logits, int64_t ldl, int64_t M, int64_t n, const exl3_logits_rules &r,
                                 float *out, int64_t ldo, int32_t *argmax, int *status, cudaStream_t st) {
  if (M == 0) return cudaSuccess;
  logits_adjust_kernel<<<(unsigned)M, kAdjustThreads, 0, st>>>(logits, ldl, (int)n, r, out, ldo, argmax, status);
  return cudaGetLastError();
}

cudaError_t init_logits_adjust_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes a;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, logits_adjust_kernel);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_logits_adjust(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
