// Attention over whole prompts, packed one behind the other, on the 5th-gen tensor
// cores. Formulas in include/exl3.h.
//
// One CTA per SM. An item is a (sequence, key/value head, pair of tiles); a tile is
// 128 rows: floor(128 / group) tokens with the group's query heads, so that keys and
// values are read once for all of them. Items are worked on from the longest to the
// shortest, dealt to the CTAs to and fro, so that each gets about the same number of
// units (128 keys) without a counter that would have to be cleared and without results
// that depend on who was first. Per unit:
//   * warp 9 (one lane): queries, keys and values by TMA into 128-byte swizzled operand
//     buffers, keys and values in rings;
//   * warp 8 (one lane): for each tile tcgen05.mma S = Q K^T into TMEM, then, when the
//     tile's probabilities are there, O += P V with P read from TMEM, where it has taken
//     the place of S; the first half of P V starts when half of P is there;
//   * warps 0..3 / 4..7 (tile 0 / 1; thread = row = TMEM lane): the row's 128 scores in
//     registers, maximum, exp2, sum, probabilities as fp16 back to TMEM. While one tile's
//     softmax runs, the tensor core works on the other's products. O is rescaled only
//     when the maximum grows by more than 2^3.75 over the one that the reference in use
//     was set by (the result is the same: the sum uses that reference);
//   * warps 10, 11: in units that not all rows see whole, values past the sequence become
//     zero, and so do infinities and NaN, which times a probability of zero would reach
//     rows that do not see them. Rows that do see one get it back at the end.
// TMEM: S0 S1 O0 O1, 128 columns each.
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kTile = 128;         // rows
constexpr int kTokens = 128;       // of a unit
constexpr int kMmaWarp = 8 /* after the softmax warps */, kLoadWarp = 9, kCleanWarp = 10, kCleanWarps = 2;
constexpr int kPromptThreads = 12 * 32;  // 168 registers a thread
constexpr int kPromptSeqs = 1024;  // sequences of one launch
constexpr int kFlags = 8;          // items whose flag is kept; more than a ring can be ahead
// A row's reference is set 2^12 below its maximum, and set anew when a maximum passes it
// by more than 2^15.75 (fp16 ends at 2^16): the many small probabilities of a long
// sequence keep their bits (one of 2^-26 of the largest has all 11).
constexpr float kHeadroom = 12.0f, kLazy = 15.75f;

template <int D>
struct PromptCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = D == 64 ? 4 : 2;        // of keys, and of values
  static constexpr int kOperand = kHalves * 128 * 128;   // 128 rows (or tokens) x D fp16
  static constexpr int kOffK = 2 * kOperand;             // two query tiles before it
  static constexpr int kOffV = kOffK + kStages * kOperand;
  static constexpr int kOffSeq = kOffV + kStages * kOperand;
  static constexpr int kOffLen = kOffSeq + kPromptSeqs * 8;
  static constexpr int kOffBar = kOffLen + kPromptSeqs * 4;
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};
constexpr int kMaxStages = 4;
enum { kPQFull = 0, kPQEmpty = 2, kPKFull = 4, kPKEmpty = kPKFull + kMaxStages, kPVFull = kPKEmpty + kMaxStages,
       kPVEmpty = kPVFull + kMaxStages, kPClean = kPVEmpty + kMaxStages, kPS = kPClean + kMaxStages, kPP = kPS + 2 /* tile x half */,
       kPO = kPP + 4, kPDone = kPO + 2, kPBars = kPDone + 1 };

struct PromptParams {
  PromptAttention a;
  int group, tile_tokens;
};

// The launch's sequences from the longest to the shortest (equal ones in their order):
// first row and tokens. Returns how many have any. All threads; ends with a barrier.
__device__ __forceinline__ int sort_prompts(const PromptAttention &a, int2 *seq, int *len) {
  const int n4 = (a.n_seqs + 3) & ~3;
  for (int s = threadIdx.x; s < n4; s += kPromptThreads) {
    int n = 0;
    if (s < a.n_seqs) {
      const int row0 = a.q_start[s];
      n = a.q_start[s + 1] - row0;
      if (row0 < 0 || n < 0 || row0 + (int64_t)n > a.rows) {
        report_index(a.status);
        n = 0;
      }
    }
    len[s] = n;
  }
  __syncthreads();
  int some = 0;
  for (int s = threadIdx.x; s < a.n_seqs; s += kPromptThreads) {
    const int n = len[s];
    int before = 0;
    for (int t = 0; t < n4; t += 4) {
      const int4 o = *reinterpret_cast<const int4 *>(len + t);
      before += (o.x > n || (o.x == n && t < s)) + (o.y > n || (o.y == n && t + 1 < s)) + (o.z > n || (o.z == n && t + 2 < s)) +
                (o.w > n || (o.w == n && t + 3 < s));
    }
    if (n > 0) seq[before] = make_int2(a.q_start[s], n);
    some += n > 0;
  }
  // the number of sequences with tokens: a vote a pass, as each thread has at most three
  int total = 0;
#pragma unroll
  for (int k = 0; k < (kPromptSeqs + kPromptThreads - 1) / kPromptThreads; ++k) total += __syncthreads_count(some > k);
  return total;
}

struct Item {
  int row0, n;     // the sequence
  int h;           // key/value head
  int token0;      // first token of the pair
  int units[2];    // of each tile; 0: the pair has no second tile
  int all;         // of the pair
  int first_masked;  // from this unit on, not every row sees all keys
};

// The items of a CTA: number k of them is item k * CTAs + c or, every second time, from
// the other end. Causal items are ordered by the pair's place in its sequence, the last
// ones first (which is by length but for sequences' last pairs), others by sequence.
struct PromptWalk {
  uint32_t round, base;
  int level, count;  // causal: place of the pair, and sequences that have it; else the sequence
  __device__ __forceinline__ void begin(const int2 *seq, int n_seqs, int pair, int causal) {
    round = base = 0;
    level = causal ? (n_seqs > 0 ? (seq[0].y + pair - 1) / pair - 1 : -1) : 0;
    count = 0;
    if (causal) widen(seq, n_seqs, pair);
  }
  __device__ __forceinline__ void widen(const int2 *seq, int n_seqs, int pair) {
    while (count < n_seqs && seq[count].y > level * pair) ++count;
  }
  __device__ __forceinline__ bool next(const int2 *seq, int n_seqs, const PromptParams &p, Item &it) {
    const uint32_t c = blockIdx.x, C = gridDim.x, heads = p.a.n_kv_heads;
    const int pair = 2 * p.tile_tokens;
    const uint32_t idx = round * C + (round & 1 ? C - 1 - c : c);
    ++round;
    int s, place;
    if (p.a.causal) {
      while (level >= 0 && idx - base >= count * heads) {
        base += count * heads;
        --level;
        widen(seq, n_seqs, pair);
      }
      if (level < 0) return false;
      s = (idx - base) / heads;
      place = level;
    } else {
      uint32_t mine = 0;
      while (level < n_seqs && idx - base >= (mine = (uint32_t)((seq[level].y + pair - 1) / pair) * heads)) {
        base += mine;
        ++level;
      }
      if (level >= n_seqs) return false;
      s = level;
      place = (idx - base) / heads;
    }
    it.h = (idx - base) % heads;
    it.row0 = seq[s].x;
    it.n = seq[s].y;
    it.token0 = place * pair;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = it.token0 + t * p.tile_tokens;
      const int seen = p.a.causal ? min(first + p.tile_tokens, it.n) : it.n;
      it.units[t] = first < it.n ? (seen + kTokens - 1) / kTokens : 0;
    }
    it.all = max(it.units[0], it.units[1]);
    it.first_masked = (p.a.causal ? it.token0 + 1 : it.n) / kTokens;
    return true;
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Loads 128 consecutive TMEM columns of this thread's lane and waits for them inside the
// same asm statement, so no use can be scheduled before the wait.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]),
        "=f"(v[64]), "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
        "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]),
        "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]),
        "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]),
        "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]),
        "=f"(v[104]), "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
        "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]),
        "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]), "=f"(v[126]), "=f"(v[127])
      : "r"(taddr));
}

// Bits of the fp16 pair w whose exponent is all ones (infinity, NaN): 0x8000 for each.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

template <int D, bool CAP>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv, const PromptParams p) {
  using Cfg = PromptCfg<D>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2 *seq = reinterpret_cast<int2 *>(smem + Cfg::kOffSeq);
  const uint32_t bars = base + Cfg::kOffBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kOffBar + 8 * kPBars);
  volatile uint32_t *flags = tmem_slot + 1;  // number + 1 of the last item of each slot that has an infinity or NaN to give back
  int *status = p.a.status;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kPQFull + t), 1);
      mbar_init(bar(kPQEmpty + t), 1);
      mbar_init(bar(kPS + t), 1);
      mbar_init(bar(kPP + 2 * t), 4);
      mbar_init(bar(kPP + 2 * t + 1), 4);
      mbar_init(bar(kPO + t), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kPKFull + i), 1);
      mbar_init(bar(kPKEmpty + i), 1);
      mbar_init(bar(kPVFull + i), 1);
      mbar_init(bar(kPVEmpty + i), 1);
      mbar_init(bar(kPClean + i), kCleanWarps);
    }
    mbar_init(bar(kPDone), 1);
    for (int i = 0; i < kFlags; ++i) flags[i] = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == kLoadWarp * 32) {
    prefetch_tensor_map(&tq);
    prefetch_tensor_map(&tk);
    prefetch_tensor_map(&tv);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  const int n_seqs = sort_prompts(p.a, seq, reinterpret_cast<int *>(smem + Cfg::kOffLen));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PromptWalk walk;
  walk.begin(seq, n_seqs, 2 * p.tile_tokens, p.a.causal);
  Item it;

  if (warp == kMmaWarp) {
    // ---------------- tensor core (one lane) ----------------
    if (lane == 0) {
      // bit 13: A negated, for a negative scale
      const uint32_t idesc_s = f16_idesc(kTile, kTokens) | (p.a.scale < 0.f ? 1u << 13 : 0u);
      constexpr uint32_t kIdescO = f16_idesc(kTile, D) | kIdescBTransposed;
      uint32_t unit = 0, items_of[2] = {0, 0}, units_of[2] = {0, 0};
      bool ok = true;
      auto wait_k = [&](uint32_t u) { return mbar_wait(bar(kPKFull + u % kStages), (u / kStages) & 1, status); };
      auto scores = [&](int t, uint32_t u) {
        const uint32_t q = base + t * Cfg::kOperand, k = base + Cfg::kOffK + (u % kStages) * Cfg::kOperand;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t off = (j >> 2) * (128 * 128) + (j & 3) * 32;
          tc_mma(tmem + 128 * t, sw128_desc(q + off), sw128_desc(k + off), idesc_s, j > 0);
        }
        tc_commit(bar(kPS + t));
      };
      while (ok && walk.next(seq, n_seqs, p, it)) {
        ok = wait_k(unit);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok) break;
          if (it.units[t] == 0) continue;
          ok = mbar_wait(bar(kPQFull + t), items_of[t]++ & 1, status);
          if (!ok) break;
          tc_fence_after();
          scores(t, unit);
          if (it.units[t] == 1) tc_commit(bar(kPQEmpty + t));
        }
        if (ok) tc_commit(bar(kPKEmpty + unit % kStages));
        for (int j = 0; ok && j < it.all; ++j, ++unit) {
          ok = mbar_wait(bar(kPVFull + unit % kStages), (unit / kStages) & 1, status);
          ok = ok && mbar_wait(bar(kPClean + unit % kStages), (unit / kStages) & 1, status);
          const uint32_t v = base + Cfg::kOffV + (unit % kStages) * Cfg::kOperand;
          bool next_k = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) break;
            if (j >= it.units[t]) continue;
            const uint32_t ph = units_of[t]++ & 1;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && mbar_wait(bar(kPP + 2 * t + half), ph, status);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                tc_mma_ta(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, sw128_mn_desc(v + k * 2048, 128 * 128, 1024), kIdescO,
                          (j | k) > 0);
            }
            if (!ok) break;
            if (j + 1 < it.units[t]) {
              if (!next_k) ok = wait_k(unit + 1);
              if (!ok) break;
              next_k = true;
              tc_fence_after();
              scores(t, unit + 1);
              if (j + 2 == it.units[t]) tc_commit(bar(kPQEmpty + t));
            } else {
              tc_commit(bar(kPO + t));
            }
          }
          if (!ok) break;
          tc_commit(bar(kPVEmpty + unit % kStages));
          if (next_k) tc_commit(bar(kPKEmpty + (unit + 1) % kStages));
        }
      }
      tc_commit(bar(kPDone));  // every issued product ends before the TMEM is released
      mbar_wait_short(bar(kPDone), 0);
    }
  } else if (warp == kLoadWarp) {
    // ---------------- loads (one lane) ----------------
    if (lane == 0) {
      uint32_t unit = 0, units_k = 0, units_v = 0, items_of[2] = {0, 0};
      bool ok = true;
      const uint32_t q_bytes = (uint32_t)(Cfg::kHalves * 128) * p.group * p.tile_tokens;
      auto operand = [&](const CUtensorMap *map, uint32_t dst, uint32_t b, int head, int row) {
#pragma unroll
        for (int hf = 0; hf < Cfg::kHalves; ++hf)
          if (EXL3_RANGE(row, 0, p.a.rows) && EXL3_SMEM(dst + hf * (128 * 128), 128 * 128))
            tma_load_3d(dst + hf * (128 * 128), map, b, 64 * hf, head, row);
      };
      while (ok && walk.next(seq, n_seqs, p, it)) {
        for (int j = 0; ok && j < it.all; ++j, ++unit) {
          const uint32_t st = unit % kStages, ph = (unit / kStages) & 1;
          const int row = it.row0 + j * kTokens;
          ok = mbar_wait(bar(kPKEmpty + st), ph ^ 1, status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kPKFull + st), Cfg::kOperand);
          operand(&tk, base + Cfg::kOffK + st * Cfg::kOperand, bar(kPKFull + st), it.h, row);
          ++units_k;
          if (j == 0) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok) break;
              if (it.units[t] == 0) continue;
              ok = mbar_wait(bar(kPQEmpty + t), (items_of[t] & 1) ^ 1, status);
              if (!ok) break;
              ++items_of[t];
              mbar_arrive_expect_tx(bar(kPQFull + t), q_bytes);
              operand(&tq, base + t * Cfg::kOperand, bar(kPQFull + t), it.h * p.group, it.row0 + it.token0 + t * p.tile_tokens);
            }
            if (!ok) break;
          }
          ok = mbar_wait(bar(kPVEmpty + st), ph ^ 1, status);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(kPVFull + st), Cfg::kOperand);
          operand(&tv, base + Cfg::kOffV + st * Cfg::kOperand, bar(kPVFull + st), it.h, row);
          ++units_v;
        }
      }
      // nothing is on its way into this CTA's memory when it ends (at once, unless a wait ran out)
      for (uint32_t i = 0; i < kStages; ++i) {
        if (units_k > i) mbar_wait_short(bar(kPKFull + i), ((units_k - 1 - i) / kStages) & 1);
        if (units_v > i) mbar_wait_short(bar(kPVFull + i), ((units_v - 1 - i) / kStages) & 1);
      }
      for (int t = 0; t < 2; ++t)
        if (items_of[t] > 0) mbar_wait_short(bar(kPQFull + t), (items_of[t] - 1) & 1);
    }
  } else if (warp >= kCleanWarp) {
    // ---------------- values that not every row may use ----------------
    uint32_t unit = 0, number = 0;
    bool ok = true;
    for (; ok && walk.next(seq, n_seqs, p, it); ++number) {
      for (int j = 0; ok && j < it.all; ++j, ++unit) {
        const uint32_t st = unit % kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kPVFull + st), (unit / kStages) & 1, status));
        if (!ok) break;
        if (j >= it.first_masked) {
          const uint32_t v = base + Cfg::kOffV + st * Cfg::kOperand;
          const int left = it.n - j * kTokens;  // tokens of the sequence from here
          bool found = false;
#pragma unroll 4
          for (int i = (warp - kCleanWarp) * 32 + lane; i < Cfg::kHalves * 128 * 8; i += kCleanWarps * 32) {
            const uint32_t addr = v + i * 16;
            const bool there = ((i >> 3) & 127) < left;
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
            const uint32_t bad = not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
            if (!there || bad) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t b = not_finite(w[e]);
                w[e] = there ? w[e] & ~((b & 0x8000u ? 0xFFFFu : 0u) | (b & 0x80000000u ? 0xFFFF0000u : 0u)) : 0u;
              }
              sts16(addr, w[0], w[1], w[2], w[3]);
              found = found || (there && bad);
            }
          }
          if (found) flags[number % kFlags] = number + 1;
          fence_proxy_async_shared();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar(kPClean + st));  // of every unit: the ring cannot get ahead of this warp
      }
    }
  } else {
    // ---------------- softmax: thread = row of tile t ----------------
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_tmem = lane_base + 128 * t, o_tmem = lane_base + 256 + 128 * t;
    const SoftCap cap(p.a.softcap, kLog2e);
    const float c = fmaxf(fabsf(p.a.scale) * Raised<D>::kLog2e, 1e-37f);  // scores in log2 units are the products times c
    const int token = row / p.group, head_in = row - token * p.group;
    uint32_t count = 0, items = 0, number = 0;  // units and items of this tile, items of the CTA
    bool ok = true;
    for (; ok && walk.next(seq, n_seqs, p, it); ++number) {
      const int units = t == 0 ? it.units[0] : it.units[1];
      if (units == 0) continue;
      const int pos = it.token0 + t * p.tile_tokens + token;
      const bool real = token < p.tile_tokens && pos < it.n;
      const int limit = !real ? 0 : p.a.causal ? pos + 1 : it.n;
      const int least = __reduce_min_sync(0xffffffffu, real ? limit : INT32_MAX);
      const bool live = __any_sync(0xffffffffu, real);
      float ref = -INFINITY, sum = 0.f;
      for (int u = 0; u < units; ++u, ++count) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kPS + t), count & 1, status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
          float s[128];
          tmem_ld128(s_tmem, s);
          const int pos0 = u * kTokens;
          if constexpr (CAP) {
#pragma unroll
            for (int k = 0; k < 128; k += 2) {
              const float2 x = cap(mul2(make_float2(s[k], s[k + 1]), make_float2(c, c)));
              s[k] = x.x;
              s[k + 1] = x.y;
            }
          }
          if (pos0 + kTokens > least) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (pos0 + k >= limit) s[k] = -INFINITY;
          }
          float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < 124; k += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(s[k + e], s[k + 4 + e]));
#pragma unroll
          for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], s[124 + e]);
          float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
          if constexpr (!CAP) top *= c;
          const float now = top > ref + kLazy || ref == -INFINITY ? top - kHeadroom : ref;
          const float keep = now == ref || ref == -INFINITY || !real ? 1.0f : ex2(ref - now);
          // the scores' product came after the output's, which is therefore done
          if (u > 0 && __any_sync(0xffffffffu, keep != 1.0f)) {
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
          const float scale = CAP ? 1.0f : c, shift = now == -INFINITY ? 0.f : -now;
          const float2 scale2 = make_float2(scale, scale), shift2 = make_float2(shift, shift);
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t packed[16];  // fp16 probabilities: 2^-12 on average, the size of the result's own rounding
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 x = make_float2(s[32 * q + 2 * k], s[32 * q + 2 * k + 1]);
              x = fma2(x, scale2, shift2);
              x = make_float2(ex2(x.x), ex2(x.y));
              part[k & 1] = add2(part[k & 1], x);
              const __half2 h2 = __floats2half2_rn(x.x, x.y);
              packed[k] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            tmem_st16(s_tmem + 16 * q, packed);
            if (q & 1) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(kPP + 2 * t + (q >> 1)));
            }
          }
          part[0] = add2(part[0], part[1]);
          sum += part[0].x + part[0].y;
        } else {  // rows past the sequence: whatever the products make of them is not used
          tc_fence_before();
          if (lane == 0) {
            mbar_arrive(bar(kPP + 2 * t));
            mbar_arrive(bar(kPP + 2 * t + 1));
          }
        }
      }
      if (!ok || !__all_sync(0xffffffffu, mbar_wait(bar(kPO + t), items++ & 1, status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (live) {
        const float f = sum == 0.f ? 0.f : 1.0f / sum;
        const int head = it.h * p.group + head_in;
        const int64_t off = (int64_t)(it.row0 + pos) * p.a.ldo + (int64_t)head * D;
        const bool fits = real && EXL3_SPAN(off, D, (int64_t)(p.a.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D);
        const bool back = fits && flags[number % kFlags] == number + 1;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          float o[32];
          __syncwarp();
          tmem_ld32(o_tmem + 32 * k, o);
          if (!fits) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          if (back) {  // infinities and NaN that this row sees, of the units where they were taken out
            for (int at = it.first_masked * kTokens; at < limit; ++at) {
              const int64_t from = (int64_t)(it.row0 + at) * p.a.ldv + (int64_t)it.h * D + 32 * k;
              if (!EXL3_SPAN(from, 32, (int64_t)(p.a.rows - 1) * p.a.ldv + (int64_t)p.a.n_kv_heads * D)) continue;
              const __half *v = static_cast<const __half *>(p.a.v) + from;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __half2float(v[e]);
                if (!isfinite(x)) o[e] += x;
              }
            }
          }
          uint4 *out = reinterpret_cast<uint4 *>(static_cast<__half *>(p.a.out) + off + 32 * k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __half2 h2 = __floats2half2_rn(o[8 * e + 2 * x], o[8 * e + 2 * x + 1]);
              w[x] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            out[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        // a logarithm near 12 would be 2^-20 off: with the reference back at the maximum first
        if (fits && p.a.lse) p.a.lse[(int64_t)(it.row0 + pos) * p.a.n_heads + head] = log_sum(ref + kHeadroom, sum * 0x1p-12f);
      }
      tc_fence_before();  // the output has been read: before the next item's first products
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D>
cudaError_t prompt_attention(const PromptAttention &a, int num_sms, cudaStream_t st) {
  PromptParams p;
  p.a = a;
  p.group = a.n_heads / a.n_kv_heads;
  p.tile_tokens = kTile / p.group;
  CUtensorMap tq, tk, tv;
  auto encode = [&](CUtensorMap *m, const void *ptr, int heads, int64_t ld, uint32_t box_heads, uint32_t box_rows) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)a.rows};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)ld * 2};
    const uint32_t box[3] = {64, box_heads, box_rows};
    return encode_tensor_map_3d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!encode(&tq, a.q, a.n_heads, a.ldq, (uint32_t)p.group, (uint32_t)p.tile_tokens) ||
      !encode(&tk, a.k, a.n_kv_heads, a.ldk, 1, kTokens) || !encode(&tv, a.v, a.n_kv_heads, a.ldv, 1, kTokens))
    return cudaErrorInvalidValue;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kPromptSeqs) {
    p.a.q_start = a.q_start + s0;
    p.a.n_seqs = a.n_seqs - s0 < kPromptSeqs ? a.n_seqs - s0 : kPromptSeqs;
    // no more items than this
    const int64_t most = (ceil_div(a.rows, 2 * p.tile_tokens) + p.a.n_seqs) * a.n_kv_heads;
    const cudaError_t e =
        launch_overlapped(a.softcap > 0.f ? prompt_attention_kernel<D, true> : prompt_attention_kernel<D, false>,
                          dim3((unsigned)(most < num_sms ? most : num_sms)), kPromptThreads, PromptCfg<D>::kSmem, st, 1, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptAttention &a, int num_sms, cudaStream_t st) {
  return a.head_dim == 64 ? prompt_attention<64>(a, num_sms, st) : prompt_attention<128>(a, num_sms, st);
}

cudaError_t init_prompt_attention_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  for (const void *f : {(const void *)prompt_attention_kernel<64, false>, (const void *)prompt_attention_kernel<64, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<64>::kSmem);
  for (const void *f : {(const void *)prompt_attention_kernel<128, false>, (const void *)prompt_attention_kernel<128, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<128>::kSmem);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_prompt_attention(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
