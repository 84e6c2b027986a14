// Writing the 8-bit key/value cache: append (quantize new tokens into their
// blocks) and evict (choose what a sequence keeps, move it to new blocks).
#include <limits.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

// One CTA per (block that receives tokens, sequence, head, keys or values). The
// block's new values stay in registers between the maximum and the conversion:
// 2 bytes read and 1 written per value, the older codes touched only when the
// scale grows.
constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(KvView kv, const __half *__restrict__ xk, int64_t ldk,
                                                                    const __half *__restrict__ xv, int64_t ldv) {
  constexpr int kVecs = D / 8;                       // 8-element pieces of a token
  constexpr int kTokens = kAppendThreads / kVecs;    // tokens per pass
  constexpr int kPasses = kKvBlock / kTokens;
  const int s = blockIdx.y, h = blockIdx.z >> 1;
  const bool is_k = (blockIdx.z & 1) == 0;
  const KvSeq q = kv_sequence(kv, s);
  const int first = q.len - q.rows;                  // position of the first new token; < 0: the row has no place
  const int b = max(first, 0) / kKvBlock + (int)blockIdx.x;
  if (q.rows == 0 || b * (int64_t)kKvBlock >= q.len) return;
  if (first < 0 && threadIdx.x == 0) report_index(kv.status);
  const int page = kv_page(kv, s, b);
  if (page < 0) return;

  const __half *x = is_k ? xk : xv;
  const int64_t ld = is_k ? ldk : ldv;
  const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
  uint8_t *codes = (is_k ? kv.k : kv.v) + slab * (kKvBlock * D);
  float *scale = (is_k ? kv.k_scale : kv.v_scale) + slab;

  const int c = threadIdx.x % kVecs, t0 = threadIdx.x / kVecs;
  uint4 raw[kPasses];
  uint32_t amax = 0;                                 // fp16 magnitudes order like their bits
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int pos = b * kKvBlock + i * kTokens + t0;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (pos >= first && pos < q.len) {
      const int64_t off = (int64_t)(q.row0 + pos - first) * ld + h * D + c * 8;
      if (EXL3_SPAN(off, 8, (int64_t)(kv.rows - 1) * ld + (int64_t)kv.n_kv_heads * D))
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(x + off));
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
        if (lo < 0x7C00u) amax = max(amax, lo);
        if (hi < 0x7C00u) amax = max(amax, hi);
      }
    }
  }
  __shared__ uint32_t warp_max[kAppendThreads / 32];
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  // every thread reads the old scale before thread 0 may replace it
  const int e_old = pow2_exponent(*scale);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = max(amax, warp_max[w]);
  int e = block_exponent(__half2float(__ushort_as_half((unsigned short)amax)));
  const bool has_old = first > b * kKvBlock;
  if (has_old) e = max(e, e_old);
  if (threadIdx.x == 0) *scale = pow2i(e);

  const float to_code = pow2i(-e);
  const bool rescale = has_old && e != e_old;
  const float grow = rescale ? pow2i(max(e_old - e, -126)) : 1.0f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kTokens + t0, pos = b * kKvBlock + t;
    uint2 *at = reinterpret_cast<uint2 *>(codes + t * D + c * 8);
    if (pos >= first && pos < q.len) {
      const __half *v = reinterpret_cast<const __half *>(&raw[i]);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = to_e4m3x2(__half2float(v[2 * j]) * to_code, __half2float(v[2 * j + 1]) * to_code);
      *at = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
      if (is_k && c == 0 && kv.weight) kv.weight[slab * kKvBlock + t] = 0.f;
    } else if (rescale && pos < first) {
      *at = rescale_codes(*at, grow);
    }
  }
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------

// Weights as unsigned keys of the same order: -0 is 0, NaN the lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0x007FFFFFu;  // with -inf
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float token_weight(const KvView &kv, int s, int h, int pos) {
  const int page = kv_page(kv, s, pos / kKvBlock);
  return page < 0 ? 0.f : kv.weight[((int64_t)page * kv.n_kv_heads + h) * kKvBlock + pos % kKvBlock];
}

// One CTA per (sequence, head): a radix selection (8 bits a pass, from the top)
// of the key of the last token that is kept, then one pass in position order
// that writes the kept positions; ties take the lower positions.
constexpr int kSelectThreads = 1024;

__global__ void __launch_bounds__(kSelectThreads) kv8_select_kernel(KvView kv, int budget, int recent, int32_t *kept,
                                                                    int32_t *new_len) {
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const int len = kv_length(kv, s);
  const int keep = min(len, budget);
  if (h == 0 && tid == 0) new_len[s] = keep;
  int32_t *out = kept + ((int64_t)s * kv.n_kv_heads + h) * budget;
  for (int i = keep + tid; i < budget; i += kSelectThreads) out[i] = -1;
  const int early = len - min(recent, len);   // tokens that are kept by weight
  const int want = keep - (len - early);      // how many of them
  for (int i = early + tid; i < len; i += kSelectThreads) out[want + i - early] = i;

  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  if (tid == 0) {
    s_prefix = 0;
    s_left = want;
  }
  if (want > 0 && want < early) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, above = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int i = tid; i < early; i += kSelectThreads) {
        const uint32_t key = weight_key(token_weight(kv, s, h, i));
        if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = s_left, d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_prefix = prefix | ((uint32_t)d << shift);
        s_left = left;
      }
      __syncthreads();
    }
  }
  __syncthreads();
  const uint32_t threshold = want >= early ? 0u : s_prefix;  // want >= early: all of them
  int ties = want >= early ? INT_MAX : s_left;               // tokens of the threshold's key that are kept
  if (want == 0) return;
  __shared__ int warp_gt[kSelectThreads / 32], warp_eq[kSelectThreads / 32];
  int done = 0;
  for (int base = 0; base < early; base += kSelectThreads) {
    const int i = base + tid;
    const uint32_t key = i < early ? weight_key(token_weight(kv, s, h, i)) : 0u;
    const bool gt = i < early && key > threshold, eq = i < early && key == threshold;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const int w = tid >> 5;
    if ((tid & 31) == 0) {
      warp_gt[w] = __popc(mg);
      warp_eq[w] = __popc(me);
    }
    __syncthreads();
    int g = __popc(mg & ((1u << (tid & 31)) - 1)), e = __popc(me & ((1u << (tid & 31)) - 1)), tg = 0, te = 0;
    for (int j = 0; j < kSelectThreads / 32; ++j) {
      if (j < w) {
        g += warp_gt[j];
        e += warp_eq[j];
      }
      tg += warp_gt[j];
      te += warp_eq[j];
    }
    __syncthreads();
    if (gt || (eq && e < ties)) out[done + g + min(e, ties)] = i;
    done += tg + min(te, ties);
    ties -= min(te, ties);
  }
}

// One CTA per (new block, sequence, head, keys or values): the block's scale is
// the largest of its tokens' scales, so codes only ever shrink.
constexpr int kMoveThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(KvView kv, const int32_t *__restrict__ dst_pages,
                                                                int dst_blocks, int budget,
                                                                const int32_t *__restrict__ kept) {
  const int b = blockIdx.x, s = blockIdx.y, h = blockIdx.z >> 1, tid = threadIdx.x;
  const bool is_k = (blockIdx.z & 1) == 0;
  const int len = kv_length(kv, s);
  const int n = min(min(len, budget) - b * kKvBlock, kKvBlock);
  if (n <= 0) return;
  const int dst = dst_pages[(int64_t)s * dst_blocks + b];
  if (dst < 0 || dst >= kv.n_pages) {
    if (tid == 0) report_index(kv.status);
    return;
  }
  uint8_t *codes = is_k ? kv.k : kv.v;
  float *scales = is_k ? kv.k_scale : kv.v_scale;
  __shared__ int64_t src[kKvBlock];  // slab * 64 + token, -1 where there is none
  __shared__ int exps[kKvBlock], top[2];
  if (tid < kKvBlock) {
    int64_t at = -1;
    int e = INT_MIN;
    if (tid < n) {
      const int pos = kept[((int64_t)s * kv.n_kv_heads + h) * budget + b * kKvBlock + tid];
      const int page = EXL3_RANGE(pos, 0, len) ? kv_page(kv, s, pos / kKvBlock) : -1;
      if (page >= 0) {
        const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
        at = slab * kKvBlock + pos % kKvBlock;
        e = pow2_exponent(scales[slab]);
      }
    }
    src[tid] = at;
    exps[tid] = e;
    const int m = __reduce_max_sync(0xffffffffu, e);
    if ((tid & 31) == 0) top[tid >> 5] = m;
  }
  __syncthreads();
  const int e = max(top[0], top[1]);
  const int64_t to = (int64_t)dst * kv.n_kv_heads + h;
  if (tid == 0 && e != INT_MIN) scales[to] = pow2i(e);
  constexpr int kVecs = D / 8;
#pragma unroll
  for (int i = tid; i < kKvBlock * kVecs; i += kMoveThreads) {
    const int t = i / kVecs, c = i % kVecs;
    if (src[t] < 0) continue;
    uint2 v = __ldg(reinterpret_cast<const uint2 *>(codes + src[t] * D) + c);
    if (exps[t] != e) v = rescale_codes(v, pow2i(max(exps[t] - e, -126)));
    reinterpret_cast<uint2 *>(codes + (to * kKvBlock + t) * D)[c] = v;
    if (is_k && c == 0) kv.weight[to * kKvBlock + t] = kv.weight[src[t]];
  }
}

}  // namespace

cudaError_t launch_kv8_append(const KvView &kv, const void *k, int64_t ldk, const void *v, int64_t ldv, cudaStream_t st) {
  if (kv.n_seqs == 0 || kv.rows == 0 || kv.max_rows == 0) return cudaSuccess;
  // the most blocks that max_rows consecutive tokens touch
  const dim3 grid((unsigned)((kv.max_rows + (int64_t)2 * kKvBlock - 2) / kKvBlock), kv.n_seqs, 2 * kv.n_kv_heads);
  const __half *xk = static_cast<const __half *>(k), *xv = static_cast<const __half *>(v);
  if (kv.head_dim == 64) kv8_append_kernel<64><<<grid, kAppendThreads, 0, st>>>(kv, xk, ldk, xv, ldv);
  else kv8_append_kernel<128><<<grid, kAppendThreads, 0, st>>>(kv, xk, ldk, xv, ldv);
  return cudaGetLastError();
}

cudaError_t launch_kv8_evict(const KvView &kv, const int32_t *dst_pages, int budget, int recent, int32_t *kept,
                             int32_t *new_len, cudaStream_t st) {
  if (kv.n_seqs == 0) return cudaSuccess;
  kv8_select_kernel<<<dim3(kv.n_kv_heads, kv.n_seqs), kSelectThreads, 0, st>>>(kv, budget, recent, kept, new_len);
  const int blocks = (int)(((int64_t)budget + kKvBlock - 1) / kKvBlock);
  const dim3 grid(blocks, kv.n_seqs, 2 * kv.n_kv_heads);
  if (kv.head_dim == 64) kv8_move_kernel<64><<<grid, kMoveThreads, 0, st>>>(kv, dst_pages, blocks, budget, kept);
  else kv8_move_kernel<128><<<grid, kMoveThreads, 0, st>>>(kv, dst_pages, blocks, budget, kept);
  return cudaGetLastError();
}

cudaError_t init_kv8_cache_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes a;
  for (const void *f : {(const void *)kv8_append_kernel<64>, (const void *)kv8_append_kernel<128>,
                        (const void *)kv8_select_kernel, (const void *)kv8_move_kernel<64>,
                        (const void *)kv8_move_kernel<128>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_cache(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
