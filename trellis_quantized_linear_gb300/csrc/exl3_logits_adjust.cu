// Penalties, biases and a grammar mask on logits, and the greedy choice from
// what is left. Formula in include/exl3.h.
//
// A cluster of CTAs per row; the row's tiles of 128 tokens go to them in turn (a
// vocabulary has its common tokens together: contiguous ranges took half as long
// again). Each CTA counts the row's history into a word for each of its tokens in
// shared memory (integer adds: any order gives the same counts); a long history
// is first dealt out, each CTA reading a share of it and handing every entry to
// the CTA that has the token. Then one stream reads and writes each logit once.
// The few tokens with a word (2 % at a history of 8192) are listed as they are
// first counted and done after the stream, so that their divisions do not hold up
// the rest, and so are the biases. The row's greedy choice is joined through the
// cluster's shared memory.
//
// Measured, 248077 tokens: 64 rows with histories of 8192, 300 biases and a mask 55 us
// (131 MB, 2.4 TB/s). Without rules the stream takes 29 us; the mask adds 4, the biases
// 6, handing out, counting and penalizing the history 15: latencies that all CTAs meet
// at the same time, as they are all resident. One row with a history of 700 and 20
// biases 10.2 us in a graph, 5.2 without rules.
#include <limits.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kMaxCluster = 16;
// A token's word: in the history at all, has a bias, times generated.
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3FFFFFFFu;

struct AdjustParams {
  const float *logits;
  float *out;
  int32_t *argmax;
  int *status;
  int64_t ldl, ldo, M;
  int n, lg;  // tokens, log2 of a cluster's CTAs
  int held;   // tokens of a CTA, rounded up (16-bit words in shared memory)
  exl3_logits_rules r;
};

struct RowRules {
  float rep, pres, freq;
};

__device__ __forceinline__ float penalized(float x, uint32_t word, const RowRules &r) {
  if ((word & (kSeen | kCount)) == 0) return x;
  x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  const uint32_t made = word & kCount;
  return made ? __fsub_rn(x, __fadd_rn(__fmul_rn(r.freq, (float)made), r.pres)) : x;
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
};

// The tokens' words: 16 bits each (seen, biased, 14 bits of count) where the
// row's history is short enough to count in them, else 32 bits and half as many
// tokens at a time.
constexpr int kShortHistory = 1 << 14;
struct Words {
  uint32_t *at;
  bool wide;
  // Each of these returns the word as it was.
  __device__ __forceinline__ uint32_t count(int i) const {
    if (wide) return atomicAdd(&at[i], 1u);
    return unpack(atomicAdd(&at[i >> 1], 1u << (16 * (i & 1))) >> (16 * (i & 1)));
  }
  __device__ __forceinline__ uint32_t set(int i, uint32_t flag) const {
    if (wide) return atomicOr(&at[i], flag);
    return unpack(atomicOr(&at[i >> 1], pack(flag) << (16 * (i & 1))) >> (16 * (i & 1)));
  }
  __device__ __forceinline__ uint32_t one(int i) const { return wide ? at[i] : unpack(at[i >> 1] >> (16 * (i & 1))); }
  __device__ __forceinline__ uint4 four(int i) const {
    if (wide) return *reinterpret_cast<const uint4 *>(at + i);
    const uint2 w = *reinterpret_cast<const uint2 *>(at + (i >> 1));
    if ((w.x | w.y) == 0) return make_uint4(0, 0, 0, 0);
    return make_uint4(unpack(w.x), unpack(w.x >> 16), unpack(w.y), unpack(w.y >> 16));
  }
  __device__ static __forceinline__ uint32_t pack(uint32_t w) { return (w & kCount) | ((w & ~kCount) >> 16); }
  __device__ static __forceinline__ uint32_t unpack(uint32_t w) { return (w & 0x3FFFu) | ((w & 0xC000u) << 16); }
};

constexpr int kList = 2048;               // history entries that are handed to a CTA
constexpr uint32_t kMade = 0x80000000u;   // in a list: generated
constexpr int kHeld = 16384;              // tokens that have words at a time, where there are many rows
constexpr int kSpecial = 2048;            // tokens with a word that are listed
struct AdjustSmem {
  uint32_t list[kList];
  uint32_t special[kSpecial];
  uint32_t words[1];  // as many as the launch asks for
};

template <int T, int V, int CTAS>
__global__ void __launch_bounds__(T, CTAS) logits_adjust_kernel(const AdjustParams p) {
  extern __shared__ __align__(16) uint8_t adjust_smem[];
  AdjustSmem &sm = *reinterpret_cast<AdjustSmem *>(adjust_smem);
  __shared__ int special_n, list_n;
  __shared__ uint32_t duplicates;  // a bit for each kSpecial tokens of the chunk: some of them have several biases
  __shared__ float sb[T / 32], cb[kMaxCluster];
  __shared__ int si[T / 32], ci[kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  const int64_t m = blockIdx.x / ranks;
  if (tid == 0) list_n = 0;
  __syncwarp();
  cluster_arrive_all();  // awaited before the first access to another CTA's shared memory: that CTA has started then
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const float *logits = p.logits + m * p.ldl;
  float *out = p.out + m * p.ldo;
  const uint32_t *allowed = p.r.allowed ? p.r.allowed + m * ((p.n + 31) / 32) : nullptr;
  // This CTA's tokens in order, local index to token and back.
  const int mine = ((p.n + 127) / 128 + (int)ranks - 1 - (int)rank) / (int)ranks * 128;
  auto token = [&](int i) { return ((((i >> 7) << p.lg) | (int)rank) << 7) | (i & 127); };
  auto owner = [&](uint32_t t) { return (t >> 7) & (ranks - 1); };
  auto local = [&](uint32_t t) { return ((t >> 7 >> p.lg) << 7) | (t & 127); };
  auto permits = [&](int t) { return !allowed || ((allowed[t >> 5] >> (t & 31)) & 1u); };
  const int2 h = row_range(p.r.history_start, m, p.r.history_size, p.status);
  const int2 b = row_range(p.r.bias_start, m, p.r.bias_size, p.status);
  const int made_from = p.r.generated_from ? p.r.generated_from[m] : 0;
  const RowRules r{p.r.repetition ? p.r.repetition[m] : 1.f, p.r.presence ? p.r.presence[m] : 0.f,
                   p.r.frequency ? p.r.frequency[m] : 0.f};
  const Words words{sm.words, h.y - h.x >= kShortHistory};
  const int step = words.wide ? p.held / 2 : p.held;  // tokens that have words at a time
  const bool rules = h.y > h.x || b.y > b.x;

  float4 x[V];
  uint32_t bits[V];
  auto load = [&](int base, int end) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = base + (k * T + tid) * 4, t = token(i);
      x[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      bits[k] = 0xFu;
      if (i >= end || t >= p.n) continue;
      if (t + 4 <= p.n) {
        x[k] = *reinterpret_cast<const float4 *>(logits + t);
      } else {  // what lies past the last token is not read
        x[k].x = logits[t];
        if (t + 1 < p.n) x[k].y = logits[t + 1];
        if (t + 2 < p.n) x[k].z = logits[t + 2];
      }
      if (allowed) bits[k] = allowed[t >> 5] >> (t & 31);
    }
  };

  // Long histories are handed out: 64 rows of 1500 / 3000 / 8192 entries 43 / 45 / 53 us,
  // 44 / 49 / 64 with every CTA reading all; below 4 entries a thread the two cluster
  // barriers cost a single row 1 us.
  bool listed = false;
  const bool handed_out = h.y - h.x > 4 * T;  // the same in every CTA of the cluster
  if (handed_out) {
    cluster_wait_all();
    const int every = T * (int)ranks;
    constexpr int kAhead = 4;
    for (int i0 = h.x + (int)rank * T; i0 < h.y; i0 += every * kAhead) {  // the same for every thread
      uint32_t t[kAhead], at[kAhead], to_cta[kAhead], peers[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + tid + k * every;
        t[k] = i < h.y ? (uint32_t)p.r.history[i] : ~0u;
      }
      // one add for all of a warp's entries of the same owner: adds to one address wait for one another
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        to_cta[k] = t[k] < (uint32_t)p.n ? owner(t[k]) : ~0u;
        peers[k] = __match_any_sync(0xffffffffu, to_cta[k]);
        at[k] = 0;
        if (to_cta[k] != ~0u && lane == __ffs(peers[k]) - 1)
          asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;"
                       : "=r"(at[k])
                       : "r"(map_to_rank(smem_u32(&list_n), to_cta[k])), "r"(__popc(peers[k]))
                       : "memory");
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t to = __shfl_sync(0xffffffffu, at[k], __ffs(peers[k]) - 1) + __popc(peers[k] & ((1u << lane) - 1));
        if (to_cta[k] != ~0u && to < (uint32_t)kList)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&sm.list[to]), to_cta[k])),
                       "r"(local(t[k]) | (i0 + tid + k * every - h.x >= made_from ? kMade : 0u))
                       : "memory");
      }
    }
    cluster_sync_all();
    listed = list_n <= kList;  // else this CTA reads the history itself
  }

  Best best;
  for (int c0 = 0; c0 < mine; c0 += step) {
    const int n = min(step, mine - c0);
    // where token t has its word in this chunk, or something past the last
    auto word_of = [&](uint32_t t) { return t < (uint32_t)p.n && owner(t) == rank ? local(t) - (uint32_t)c0 : ~0u; };
    if (rules) {
      const int used = words.wide ? n : (n + 1) / 2;
      for (int i = tid * 4; i < used; i += T * 4)
        if (EXL3_SPAN(i, 4, p.held / 2)) *reinterpret_cast<uint4 *>(sm.words + i) = make_uint4(0, 0, 0, 0);
      if (tid == 0) {
        special_n = 0;
        duplicates = 0;
      }
      __syncthreads();
      // i: a token with a word, or anything else; every lane of the warp takes part
      auto note = [&](uint32_t i, auto mark) {
        const bool fresh = i < (uint32_t)n && mark((int)i) == 0;
        const uint32_t all = __ballot_sync(0xffffffffu, fresh);
        if (all == 0) return;
        int at = 0;
        if (lane == __ffs(all) - 1) at = atomicAdd(&special_n, __popc(all));
        at = __shfl_sync(0xffffffffu, at, __ffs(all) - 1) + __popc(all & ((1u << lane) - 1));
        if (fresh && at < kSpecial) sm.special[at] = i;
      };
      auto count = [&](uint32_t i, bool made) {
        note(i, [&](int j) { return made ? words.count(j) : words.set(j, kSeen); });
      };
      if (listed) {
        for (int i0 = 0; i0 < list_n; i0 += T) {
          const uint32_t e = i0 + tid < list_n ? sm.list[i0 + tid] : ~0u;
          count((e & ~kMade) - (uint32_t)c0, e & kMade);
        }
      } else {
        constexpr int kAhead = 8;
        for (int i0 = h.x; i0 < h.y; i0 += T * kAhead) {
          uint32_t t[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + tid + k * T;
            t[k] = i < h.y ? (uint32_t)p.r.history[i] : ~0u;
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) count(word_of(t[k]), i0 + tid + k * T - h.x >= made_from);
        }
      }
      for (int i0 = b.x; i0 < b.y; i0 += T) {
        const uint32_t t = i0 + tid < b.y ? (uint32_t)p.r.bias_id[i0 + tid] : ~0u;
        note(word_of(t), [&](int j) {
          const uint32_t was = words.set(j, kBiased);
          if (was & kBiased) atomicOr(&duplicates, 1u << (j / kSpecial));
          return was;
        });
      }
      __syncthreads();
    }

    int piece = INT_MAX;  // of the best token without a word
    float top = best.x;
    for (int base = 0; base < n; base += T * V * 4) {
      load(c0 + base, c0 + n);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int i = base + (k * T + tid) * 4, t = token(c0 + i);
        const bool real = i < n && t < p.n;
        float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (bits[k] >> e) & 1u ? v[e] : -INFINITY;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (rules && real && EXL3_SPAN(i, 4, step)) w = words.four(i);
        if (real) {
          if (t + 4 <= p.n) {
            *reinterpret_cast<float4 *>(out + t) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (t + e < p.n) out[t + e] = v[e];
          }
        }
        if ((w.x | w.y | w.z | w.w) != 0) {  // those with a word: not by the stream
          v[0] = w.x ? -INFINITY : v[0];
          v[1] = w.y ? -INFINITY : v[1];
          v[2] = w.z ? -INFINITY : v[2];
          v[3] = w.w ? -INFINITY : v[3];
        }
        const float four = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        if (four > top) {
          top = four;
          piece = i;
        }
      }
    }
    if (piece != INT_MAX) {  // its first token of that value: the thread wrote it itself
      const uint4 w = rules ? words.four(piece) : make_uint4(0, 0, 0, 0);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      const int t = token(c0 + piece);
      for (int e = 0; e < 4; ++e)
        if (t + e < p.n && ww[e] == 0 && out[t + e] == top) {
          best.take(top, t + e);
          break;
        }
    }
    if (!rules) continue;
    __syncthreads();  // the stream has written the tokens with a word as well: masked, not yet penalized
    // four at a time: their logits come from L2
    constexpr int kAhead = 4;
    auto penalize = [&](int count, auto entry) {
      for (int i0 = tid; i0 < count; i0 += T * kAhead) {
        uint32_t word[kAhead];
        int t[kAhead];
        float y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int at = i0 + k * T < count ? entry(i0 + k * T) : -1;
          word[k] = at < 0 ? 0u : words.one(at);
          if (word[k] & kBiased) word[k] = 0u;
          t[k] = token(c0 + at);
          y[k] = word[k] ? out[t[k]] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (word[k] == 0) continue;
          const float was = y[k];
          y[k] = penalized(was, word[k], r);
          // a penalty that is not finite would bring back what the mask forbids
          if (was == -INFINITY && y[k] != -INFINITY && !permits(t[k])) continue;
          out[t[k]] = y[k];
          if (y[k] > -INFINITY) best.take(y[k], t[k]);
        }
      }
    };
    if (special_n <= kSpecial) penalize(special_n, [&](int i) { return (int)sm.special[i]; });
    else penalize(n, [](int i) { return i; });  // too many to list: look at every word
    // A biased token is done by its entry, unless some token near it has several.
    for (int i0 = b.x + tid; i0 < b.y; i0 += T * 2) {
      int id[2];
      float sum[2], y[2];
      uint32_t at[2];
      bool may[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        id[k] = i0 + k * T < b.y ? p.r.bias_id[i0 + k * T] : -1;
        sum[k] = i0 + k * T < b.y ? p.r.bias_value[i0 + k * T] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        at[k] = word_of((uint32_t)id[k]);
        const bool here = at[k] < (uint32_t)n;
        y[k] = here ? out[id[k]] : 0.f;
        may[k] = !here || permits(id[k]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (at[k] >= (uint32_t)n || ((duplicates >> (at[k] / kSpecial)) & 1u)) continue;
        if (may[k]) {
          y[k] = __fadd_rn(penalized(y[k], words.one((int)at[k]), r), sum[k]);
          out[id[k]] = y[k];
        }
        if (y[k] > -INFINITY) best.take(y[k], id[k]);
      }
    }
    // Tokens with several biases, kSpecial at a time with a sum each (where the list of
    // special tokens was): every warp reads the row's entries in order and adds those of
    // its share of the tokens. One row of 250000 entries, each token twice: 3.7 ms.
    float *sums = reinterpret_cast<float *>(sm.special);
    for (uint32_t windows = duplicates; windows; windows &= windows - 1) {
      const int w0 = (__ffs(windows) - 1) * kSpecial;
      constexpr int kShare = kSpecial / (T / 32);
      __syncthreads();  // the list, or the sums before, have been read
      for (int i = tid; i < kSpecial; i += T) sums[i] = -0.0f;
      __syncthreads();
      constexpr int kAhead = 4;
      for (int i0 = b.x; i0 < b.y; i0 += 32 * kAhead) {  // the same for every lane
        uint32_t at[kAhead];
        float value[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + 32 * k + lane;
          at[k] = word_of(i < b.y ? (uint32_t)p.r.bias_id[i] : ~0u) - (uint32_t)w0;
          value[k] = i < b.y ? p.r.bias_value[i] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const bool here = at[k] / kShare == (uint32_t)(tid >> 5);
          if (!__any_sync(0xffffffffu, here)) continue;
          // entries of one token one after the other
          const uint32_t peers = __match_any_sync(0xffffffffu, here ? at[k] : ~0u);
          const int before = __popc(peers & ((1u << lane) - 1)), most = __reduce_max_sync(0xffffffffu, here ? before : 0);
          for (int turn = 0; turn <= most; ++turn) {
            if (here && before == turn && EXL3_RANGE((int)at[k], 0, kSpecial)) sums[at[k]] = __fadd_rn(sums[at[k]], value[k]);
            __syncwarp();
          }
        }
      }
      __syncthreads();
      for (int i = tid; i < kSpecial && w0 + i < n; i += T) {
        const uint32_t word = words.one(w0 + i);
        const int t = token(c0 + w0 + i);
        if (!(word & kBiased) || !permits(t)) continue;  // a word is only of a token below p.n
        const float y = __fadd_rn(penalized(out[t], word, r), sums[i]);
        out[t] = y;
        if (y > -INFINITY) best.take(y, t);
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int k = 16; k > 0; k >>= 1) best.take(__shfl_xor_sync(0xffffffffu, best.x, k), __shfl_xor_sync(0xffffffffu, best.t, k));
  if (lane == 0) {
    sb[tid >> 5] = best.x;
    si[tid >> 5] = best.t;
  }
  __syncwarp();
  if (!handed_out) cluster_wait_all();
  __syncthreads();
  if (tid < 32) {
    best = Best();
    if (lane < T / 32) best.take(sb[lane], si[lane]);
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
  // Few rows: clusters of up to 16 CTAs of 512 threads. Many rows: up to 8 of 256
  // (clusters of 16 leave a quarter of the SMs without work), four an SM, so that
  // one streams while another counts. 248K tokens, histories of 700, 9 / 16 / 32 / 64
  // rows: 20 / 35 / 62 / 121 us in the first form, 23 / 33 / 38 / 43 in the second.
  // (Three CTAs an SM with twice the loads in flight 101 us where four took 64, words
  // for 8192 tokens at a time 81.) At least 2048 tokens to a CTA.
  const bool few = M * kMaxCluster <= num_sms;
  const int most = few ? kMaxCluster : kMaxCluster / 2;
  int lg = 0;
  while ((1 << lg) < most && n > (int64_t)2048 << lg) ++lg;
  const int ranks = 1 << lg;
  const int64_t share = ceil_div(ceil_div(n, 128), ranks) * 128;
  const int held = (int)(few || share < kHeld ? share : kHeld);
  AdjustParams p{logits, out, argmax, status, ldl, ldo, M, (int)n, lg, held, r};
  const auto kernel = few ? logits_adjust_kernel<512, 8, 1> : logits_adjust_kernel<256, 4, 4>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * ranks));
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.dynamicSmemBytes = sizeof(AdjustSmem) + (size_t)held * 2;
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
  for (const void *f : {(const void *)logits_adjust_kernel<256, 4, 4>, (const void *)logits_adjust_kernel<512, 8, 1>}) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AdjustSmem) + (1 << 19) / 8 * 2);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  }
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_logits_adjust(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
