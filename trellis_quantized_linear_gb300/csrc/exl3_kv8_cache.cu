// Writing the 8-bit key/value cache: append (quantize new tokens into their
// blocks) and evict (choose what a sequence keeps, move it to new blocks).
#include <limits.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

// One CTA per (block that receives tokens, sequence, head, keys or values). The
// block's new values stay in registers between the maximum and the conversion:
// 2 bytes read and 1 written per value, the older codes touched only when the
// scale grows. Bound by those bytes and, until they fill the chip, by the chain
// length - page - values - store: 6.8K tokens of 8 heads, D = 128, keys and values (42
// MB) 10.3 us, 4.1 TB/s; 16 tokens 2.6 us, less than the launch takes the host.
constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(KvView kv, const __half *xk, int64_t ldk,
                                                                    const __half *xv, int64_t ldv) {
  constexpr int kVecs = D / 8;                       // 8-element pieces of a token
  constexpr int kTokens = kAppendThreads / kVecs;    // tokens per pass
  constexpr int kPasses = kKvBlock / kTokens;
  const int s = blockIdx.y, h = blockIdx.z >> 1;
  const bool is_k = (blockIdx.z & 1) == 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  __half2 top = __half2half2(__ushort_as_half(0));   // a NaN never wins a maximum
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int pos = b * kKvBlock + i * kTokens + t0;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (pos >= first && pos < q.len) {
      const int64_t off = (int64_t)(q.row0 + pos - first) * ld + h * D + c * 8;
      if (EXL3_SPAN(off, 8, (int64_t)(kv.rows - 1) * ld + (int64_t)kv.n_kv_heads * D))
        raw[i] = *reinterpret_cast<const uint4 *>(x + off);
      const __half2 *w = reinterpret_cast<const __half2 *>(&raw[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = __hmax2(top, __habs2(w[j]));
    }
  }
  // fp16 magnitudes order like their bits
  uint32_t amax = __half_as_ushort(__hmax(__low2half(top), __high2half(top)));
  if (amax == 0x7C00u) {  // an infinity: the largest finite value instead
    amax = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
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

// One CTA per (sequence, head), or a cluster of them, each with a contiguous part
// of the tokens, where the keys of the tokens to choose among do not fit one's
// shared memory. The keys are read once (those past what a cluster of eight holds
// are read again from memory); a radix selection, 11 bits a pass from the top over
// the sums of the CTAs' bins, finds the key of the last token that is kept, and
// each warp then writes the kept positions of its part, ties to the lower
// positions. The first pass's bins hold the sign, the exponent and two bits:
// weights fill few of them, so each bin has four copies, one for every fourth lane.
// Eight sequences of 9K to 32K tokens, 8 heads: 18.6 us on 64 CTAs, bound by their
// instructions (2.5 a cycle): 4 us reading the weights, 2.5 each pass, 4 writing what
// is kept.
constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectKeys = 44 * 1024;  // held in shared memory
constexpr int kBins = 2048, kCopies = 4;
constexpr int kSelectMaxCluster = 8;

__global__ void __launch_bounds__(kSelectThreads, 1) kv8_select_kernel(KvView kv, int budget, int recent, int held_max,
                                                                       int32_t *kept, int32_t *new_len) {
  extern __shared__ __align__(16) uint32_t select_smem[];
  int *hist = reinterpret_cast<int *>(select_smem);            // kBins x kCopies, then the sums
  uint32_t *keys = select_smem + kBins * kCopies;
  __shared__ int sums[kBins];
  __shared__ int warp_count[kSelectWarps], warp_tie[kSelectWarps], cta_count[2], s_bin, s_left;
  const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x, ranks = gridDim.x;         // the cluster is one row of the grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = kv_length(kv, s);
  const int keep = min(len, budget);
  if (rank == 0 && h == 0 && tid == 0) new_len[s] = keep;
  int32_t *out = kept + ((int64_t)s * kv.n_kv_heads + h) * budget;
  const int every = (int)ranks * kSelectThreads, me = (int)rank * kSelectThreads + tid;
  for (int i = keep + me; i < budget; i += every) out[i] = -1;
  const int early = len - min(recent, len);   // tokens that are kept by weight
  const int want = keep - (len - early);      // how many of them
  for (int i = early + me; i < len; i += every) out[want + i - early] = i;
  if (want == 0) return;                      // the same in every CTA of the cluster
  if (want == early) {
    for (int i = me; i < early; i += every) out[i] = i;
    return;
  }

  const int share = ((early + (int)ranks - 1) / (int)ranks + kKvBlock - 1) / kKvBlock * kKvBlock;
  const int first = min((int)rank * share, early), n = min(share, early - first);  // this CTA's tokens
  auto read_key = [&](int i) {
    const int page = kv_page(kv, s, i / kKvBlock);
    return page < 0 ? 0u : weight_key(kv.weight[((int64_t)page * kv.n_kv_heads + h) * kKvBlock + i % kKvBlock]);
  };
  const int held = min(n, held_max);
  // Keys i .. i + 3 (i a multiple of 4), 0 past the last: no weight has that key, so
  // it is never counted on (the tokens wanted have higher ones) nor chosen.
  auto four = [&](int i) {
    if (i < held) return *reinterpret_cast<const uint4 *>(keys + i);
    uint32_t k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = i + e < n ? read_key(first + i + e) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  // a warp takes whole blocks, two tokens a lane; `first` is a multiple of a block
  for (int b0 = warp; b0 * kKvBlock < held; b0 += kSelectWarps * 32) {
    // page numbers of the warp's next 32 blocks, one a lane
    const int mine = (b0 + lane * kSelectWarps) * kKvBlock;
    const int page = mine < held ? kv_page(kv, s, (first + mine) / kKvBlock) : -1;
    constexpr int kAhead = 8;
    for (int j0 = 0; j0 < 32 && (b0 + j0 * kSelectWarps) * kKvBlock < held; j0 += kAhead) {
      float2 w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int p = __shfl_sync(0xffffffffu, page, j0 + j);
        w[j] = make_float2(NAN, NAN);
        if (p >= 0) w[j] = reinterpret_cast<const float2 *>(kv.weight + ((int64_t)p * kv.n_kv_heads + h) * kKvBlock)[lane];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = (b0 + (j0 + j) * kSelectWarps) * kKvBlock + 2 * lane;
        if (i < ((held + 3) & ~3))
          *reinterpret_cast<uint2 *>(keys + i) = make_uint2(i < held ? weight_key(w[j].x) : 0u, i + 1 < held ? weight_key(w[j].y) : 0u);
      }
    }
  }

  uint32_t threshold = 0;  // the bits of the threshold's key found so far
  int left = want;         // tokens still to keep among those that share them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u, above = pass == 0 ? 0u : ~0u << (shift + (pass == 2 ? 10 : 11));
    for (int i = tid; i < kBins * kCopies / 4; i += kSelectThreads) reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid * 4; i < n; i += kSelectThreads * 4) {
      const uint4 k = four(i);
      const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((key[e] & above) == threshold) atomicAdd(&hist[((key[e] >> shift) & mask) * kCopies + lane % kCopies], 1);
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kSelectThreads) {
      const int4 x = reinterpret_cast<const int4 *>(hist)[i];
      sums[i] = x.x + x.y + x.z + x.w;
    }
    // from the top: thread tid has bins 2047 - 2 tid and the one below, of all CTAs
    const int hi = kBins - 1 - 2 * tid;
    int c1 = 0, c0 = 0;
    if (ranks > 1) {
      cluster_sync_all();
      const uint32_t at = smem_u32(&sums[hi - 1]);
#pragma unroll
      for (uint32_t r = 0; r < kSelectMaxCluster; ++r)
        if (r < ranks) {
          int a, b;
          asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(map_to_rank(at, r)) : "memory");
          c0 += a;
          c1 += b;
        }
    } else {
      __syncthreads();
      c0 = sums[hi - 1];
      c1 = sums[hi];
    }
    int sum = c1 + c0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) warp_count[warp] = sum;
    __syncthreads();
    int base = lane < warp ? warp_count[lane] : 0;
    base = __reduce_add_sync(0xffffffffu, base);
    const int before = base + sum - c1 - c0;  // tokens in the bins above
    if (before < left && left <= before + c1) {
      s_bin = hi;
      s_left = left - before;
    } else if (before + c1 < left && left <= before + c1 + c0) {
      s_bin = hi - 1;
      s_left = left - before - c1;
    }
    if (ranks > 1) cluster_sync_all();  // no CTA reads this pass's sums any more
    else __syncthreads();
    threshold |= (uint32_t)s_bin << shift;
    left = s_left;
  }

  // `left` tokens of the threshold's key are kept, the first ones.
  const int part = ((n + kSelectWarps - 1) / kSelectWarps + 127) & ~127;
  const int i0 = min(warp * part, n), i1 = min(i0 + part, n);
  int gt = 0, eq = 0;
  for (int i = i0 + 4 * lane; i < i1; i += 128) {
    const uint4 k = four(i);
    gt += (k.x > threshold) + (k.y > threshold) + (k.z > threshold) + (k.w > threshold);
    eq += (k.x == threshold) + (k.y == threshold) + (k.z == threshold) + (k.w == threshold);
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_count[warp] = gt;
    warp_tie[warp] = eq;
  }
  __syncthreads();
  int g = __reduce_add_sync(0xffffffffu, lane < warp ? warp_count[lane] : 0);
  int e = __reduce_add_sync(0xffffffffu, lane < warp ? warp_tie[lane] : 0);
  if (ranks > 1) {
    if (tid == kSelectThreads - 1) {
      cta_count[0] = g + gt;
      cta_count[1] = e + eq;
    }
    __syncwarp();
    cluster_sync_all();
#pragma unroll
    for (uint32_t r = 0; r < kSelectMaxCluster; ++r)
      if (r < rank) {
        int a, b;
        const uint32_t at = map_to_rank(smem_u32(cta_count), r);
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(a) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(b) : "r"(at + 4) : "memory");
        g += a;
        e += b;
      }
    cluster_sync_all();  // a CTA stays until its counts have been read
  }
  for (int b = i0; b < i1; b += 128) {
    const int i = b + 4 * lane;
    const uint4 k = i < i1 ? four(i) : make_uint4(0, 0, 0, 0);
    const uint32_t key[4] = {k.x, k.y, k.z, k.w};
    if (!__any_sync(0xffffffffu, k.x == threshold || k.y == threshold || k.z == threshold || k.w == threshold)) {
      // no tie among the 128: the lanes before from ballots
      int at = g + min(e, left), all = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t who = __ballot_sync(0xffffffffu, key[x] > threshold);
        at += __popc(who & ((1u << lane) - 1));
        all += __popc(who);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (key[x] > threshold) {
          if (EXL3_RANGE(at, 0, want)) out[at] = first + i + x;
          ++at;
        }
      g += all;
      continue;
    }
    // above the threshold in the low half, at it in the high half: one sum over the lanes before
    int mine = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) mine += key[e] > threshold ? 1 : key[e] == threshold ? 0x10000 : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    int above = g + ((sum - mine) & 0xFFFF), ties = e + ((sum - mine) >> 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool is_gt = key[x] > threshold, is_eq = key[x] == threshold;
      const int at = above + min(ties, left);
      if ((is_gt || (is_eq && ties < left)) && EXL3_RANGE(at, 0, want)) out[at] = first + i + x;
      above += is_gt;
      ties += is_eq;
    }
    g += all & 0xFFFF;
    e += all >> 16;
  }
}

// One CTA per (new block, sequence, head): its keys and values. The block's scale
// is the largest of its tokens' scales, so codes only ever shrink. Bound by the
// bytes moved; all of a thread's loads are in flight before its first store. Eight
// sequences, 8 heads, 4096 tokens of D = 128 each: 22 us for 137 MB, 6.2 TB/s (with the
// codes' loads before the scales are compared no faster: it is not the chain that binds).
constexpr int kMoveThreads = 128;

__device__ __forceinline__ uint4 rescale_16(uint4 c, float factor) {
  const uint2 a = rescale_codes(make_uint2(c.x, c.y), factor), b = rescale_codes(make_uint2(c.z, c.w), factor);
  return make_uint4(a.x, a.y, b.x, b.y);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(KvView kv, const int32_t *dst_pages,
                                                                int dst_blocks, int budget, const int32_t *kept) {
  const int b = blockIdx.x, s = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
  __shared__ int64_t src[kKvBlock];  // slab * 64 + token, -1 where there is none
  __shared__ int exps[2][kKvBlock], top[2][2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = kv_length(kv, s);
  const int n = min(min(len, budget) - b * kKvBlock, kKvBlock);
  if (n <= 0) return;
  const int dst = dst_pages[(int64_t)s * dst_blocks + b];
  if (dst < 0 || dst >= kv.n_pages) {
    if (tid == 0) report_index(kv.status);
    return;
  }
  const int64_t to = (int64_t)dst * kv.n_kv_heads + h;
  if (tid < kKvBlock) {
    int64_t at = -1;
    int ek = INT_MIN, ev = INT_MIN;
    if (tid < n) {
      const int pos = kept[((int64_t)s * kv.n_kv_heads + h) * budget + b * kKvBlock + tid];
      const int page = EXL3_RANGE(pos, 0, len) ? kv_page(kv, s, pos / kKvBlock) : -1;
      if (page >= 0) {
        const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
        at = slab * kKvBlock + pos % kKvBlock;
        ek = pow2_exponent(kv.k_scale[slab]);
        ev = pow2_exponent(kv.v_scale[slab]);
        kv.weight[to * kKvBlock + tid] = kv.weight[at];
      }
    }
    src[tid] = at;
    exps[0][tid] = ek;
    exps[1][tid] = ev;
    const int mk = __reduce_max_sync(0xffffffffu, ek), mv = __reduce_max_sync(0xffffffffu, ev);
    if ((tid & 31) == 0) {
      top[0][tid >> 5] = mk;
      top[1][tid >> 5] = mv;
    }
  }
  __syncthreads();
  constexpr int kVecs = D / 16, kPasses = kKvBlock * kVecs / kMoveThreads;
  uint4 v[2][kPasses];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int64_t at = src[(i * kMoveThreads + tid) / kVecs];
      if (at >= 0) v[x][i] = reinterpret_cast<const uint4 *>((x ? kv.v : kv.k) + at * D)[tid % kVecs];
    }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int e = max(top[x][0], top[x][1]);
    if (tid == 0 && e != INT_MIN) (x ? kv.v_scale : kv.k_scale)[to] = pow2i(e);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int t = (i * kMoveThreads + tid) / kVecs;
      if (src[t] < 0) continue;
      if (exps[x][t] != e) v[x][i] = rescale_16(v[x][i], pow2i(max(exps[x][t] - e, -126)));
      reinterpret_cast<uint4 *>((x ? kv.v : kv.k) + (to * kKvBlock + t) * D)[tid % kVecs] = v[x][i];
    }
  }
}

}  // namespace

cudaError_t launch_kv8_append(const KvView &kv, const void *k, int64_t ldk, const void *v, int64_t ldv, cudaStream_t st) {
  if (kv.n_seqs == 0 || kv.rows == 0 || kv.max_rows == 0) return cudaSuccess;
  // the most blocks that max_rows consecutive tokens touch
  const dim3 grid((unsigned)((kv.max_rows + (int64_t)2 * kKvBlock - 2) / kKvBlock), kv.n_seqs, 2 * kv.n_kv_heads);
  const __half *xk = static_cast<const __half *>(k), *xv = static_cast<const __half *>(v);
  return launch_overlapped(kv.head_dim == 64 ? kv8_append_kernel<64> : kv8_append_kernel<128>, grid, kAppendThreads, 0, st, 1, kv,
                           xk, ldk, xv, ldv);
}

cudaError_t launch_kv8_evict(const KvView &kv, const int32_t *dst_pages, int budget, int recent, int32_t *kept,
                             int32_t *new_len, cudaStream_t st) {
  if (kv.n_seqs == 0) return cudaSuccess;
  // As many CTAs to a (sequence, head) as hold its keys. A pass over a cluster's
  // bins costs 5 us in barriers and remote reads, whatever the length: 8 sequences
  // of up to 32K tokens, 8 heads, take 23 us with one CTA each and 26 us with four.
  const int64_t most = (int64_t)kv.max_pages * kKvBlock;
  int ranks = 1;
  while (ranks < kSelectMaxCluster && most > (int64_t)ranks * kSelectKeys) ranks *= 2;
  const int64_t share = ceil_div(most, ranks * kKvBlock) * kKvBlock;
  const int held = (int)(share < kSelectKeys ? share : kSelectKeys);
  cudaError_t e = launch_overlapped(kv8_select_kernel, dim3(ranks, kv.n_kv_heads, kv.n_seqs), kSelectThreads,
                                    (size_t)(kBins * kCopies + held) * 4, st, ranks, kv, budget, recent, held, kept, new_len);
  if (e != cudaSuccess) return e;
  const int blocks = (int)(((int64_t)budget + kKvBlock - 1) / kKvBlock);
  const dim3 grid(blocks, kv.n_seqs, kv.n_kv_heads);
  return launch_overlapped(kv.head_dim == 64 ? kv8_move_kernel<64> : kv8_move_kernel<128>, grid, kMoveThreads, 0, st, 1, kv,
                           dst_pages, blocks, budget, kept);
}

cudaError_t init_kv8_cache_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes a;
  for (const void *f : {(const void *)kv8_append_kernel<64>, (const void *)kv8_append_kernel<128>,
                        (const void *)kv8_move_kernel<64>, (const void *)kv8_move_kernel<128>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kBins * kCopies + kSelectKeys) * 4);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_cache(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
