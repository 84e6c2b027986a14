// Attention over the 8-bit key/value cache, and the accumulated attention weight
// of its tokens. Formulas in include/exl3.h.
#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

// Sequence of row r: the last s with q_start[s] <= r.
__device__ __forceinline__ int sequence_of_row(const KvView &kv, int r) {
  int lo = 0, hi = kv.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (kv.q_start[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// This lane's D / 32 elements of a token's codes.
template <int D>
__device__ __forceinline__ void load_codes(const uint8_t *p, int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const uint32_t h = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(p + lane * E + 2 * i));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <int D>
__device__ __forceinline__ float warp_dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) r = fmaf(a[i], b[i], r);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
  return r;
}

template <int D>
__device__ __forceinline__ void load_row(const __half *q, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = __half2float(q[lane * (D / 32) + i]);
}

// One warp per (row, query head), one token at a time: running maximum, sum and
// output, all fp32.
template <int D>
__global__ void __launch_bounds__(128) kv8_attention_kernel(KvAttention p) {
  const KvView &kv = p.kv;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= (int64_t)kv.rows * p.n_heads) return;
  const int r = (int)(w / p.n_heads), head = (int)(w % p.n_heads);
  const int s = sequence_of_row(kv, r), h = head / (p.n_heads / kv.n_kv_heads);
  const KvSeq q = kv_sequence(kv, s);
  const int limit = min(q.len, p.causal ? q.len - q.rows + (r - q.row0) + 1 : q.len);
  constexpr int E = D / 32;
  float qx[E], o[E] = {};
  load_row<D>(static_cast<const __half *>(p.q) + r * p.ldq + (int64_t)head * D, lane, qx);
  float top = -INFINITY, total = 0.f;
  for (int b = 0; b * kKvBlock < limit; ++b) {
    const int page = kv_page(kv, s, b);
    if (page < 0) continue;
    const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
    const float ks = kv.k_scale[slab] * p.scale, vs = kv.v_scale[slab];
    for (int t = 0; t < kKvBlock && b * kKvBlock + t < limit; ++t) {
      float kx[E], vx[E];
      load_codes<D>(kv.k + (slab * kKvBlock + t) * D, lane, kx);
      load_codes<D>(kv.v + (slab * kKvBlock + t) * D, lane, vx);
      float x = warp_dot<D>(qx, kx) * ks;
      if (p.softcap > 0.f) x = soft_cap(x, p.softcap, 1.0f / p.softcap);
      const float now = fmaxf(top, x);
      const float keep = exp2f((top - now) * kLog2e), e = exp2f((x - now) * kLog2e);
      total = total * keep + e;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = o[i] * keep + e * vs * vx[i];
      top = now;
    }
  }
  const float inv = total > 0.f ? 1.0f / total : (total == total ? 0.f : total);
  __half *out = static_cast<__half *>(p.out) + r * p.ldo + (int64_t)head * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) out[i] = __float2half_rn(o[i] * inv);
  if (p.lse && lane == 0) p.lse[(int64_t)r * p.n_heads + head] = total == 0.f ? -INFINITY : top + logf(total);
}

// One warp per (cached token, sequence, key/value head): all rows of the
// sequence in order.
template <int D>
__global__ void __launch_bounds__(128) kv8_weigh_kernel(KvAttention p) {
  const KvView &kv = p.kv;
  const int lane = threadIdx.x & 31, s = blockIdx.y, h = blockIdx.z;
  const int t = blockIdx.x * (int)(blockDim.x >> 5) + (threadIdx.x >> 5);
  const KvSeq q = kv_sequence(kv, s);
  if (t >= q.len || q.rows == 0) return;
  const int page = kv_page(kv, s, t / kKvBlock);
  if (page < 0) return;
  const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
  const int64_t at = slab * kKvBlock + t % kKvBlock;
  const float ks = kv.k_scale[slab] * p.scale;
  float kx[D / 32], qx[D / 32], add = 0.f;
  load_codes<D>(kv.k + at * D, lane, kx);
  const int group = p.n_heads / kv.n_kv_heads;
  const int from = p.causal ? max(0, t - (q.len - q.rows)) : 0;
  for (int i = from; i < q.rows; ++i)
    for (int g = 0; g < group; ++g) {
      const int head = h * group + g;
      const int64_t r = q.row0 + i;
      const float lse = p.lse[r * p.n_heads + head];
      load_row<D>(static_cast<const __half *>(p.q) + r * p.ldq + (int64_t)head * D, lane, qx);
      float x = warp_dot<D>(qx, kx) * ks;
      if (p.softcap > 0.f) x = soft_cap(x, p.softcap, 1.0f / p.softcap);
      if (lse != -INFINITY) add += exp2f((x - lse) * kLog2e);
    }
  if (lane == 0) kv.weight[at] += add;
}

}  // namespace

size_t kv8_attention_workspace_bytes(const exl3_kv8_cache &, const exl3_kv8_batch &, int, int) { return 16; }

cudaError_t launch_kv8_attention(const KvAttention &p, cudaStream_t st) {
  const int64_t warps = (int64_t)p.kv.rows * p.n_heads;
  if (warps == 0 || p.kv.n_seqs == 0) return cudaSuccess;
  const unsigned grid = (unsigned)ceil_div(warps, 4);
  if (p.kv.head_dim == 64) kv8_attention_kernel<64><<<grid, 128, 0, st>>>(p);
  else kv8_attention_kernel<128><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_weigh(const KvAttention &p, cudaStream_t st) {
  if (p.kv.rows == 0 || p.kv.n_seqs == 0) return cudaSuccess;
  const dim3 grid((unsigned)(p.kv.max_pages * (kKvBlock / 4)), p.kv.n_seqs, p.kv.n_kv_heads);
  if (p.kv.head_dim == 64) kv8_weigh_kernel<64><<<grid, 128, 0, st>>>(p);
  else kv8_weigh_kernel<128><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t init_kv8_attention_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes a;
  for (const void *f : {(const void *)kv8_attention_kernel<64>, (const void *)kv8_attention_kernel<128>,
                        (const void *)kv8_weigh_kernel<64>, (const void *)kv8_weigh_kernel<128>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_attention(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
