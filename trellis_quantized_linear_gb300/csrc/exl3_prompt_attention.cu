// Attention over whole prompts, packed one behind the other, on the 5th-gen tensor
// cores. Formulas in include/exl3.h.
//
// One CTA per SM. An item is a (sequence, key/value head, pair of tiles); a tile is
// 128 rows: floor(128 / group) tokens with the group's query heads, so that keys and
// values are read once for all of them. Items are worked on from the longest to the
// shortest, dealt to the CTAs to and fro, so that each gets about the same number of
// units (128 keys; 8192 tokens of 40 heads: 280 to 285) without a counter that would have
// to be cleared and without results that depend on who was first. Per unit:
//   * warp 9 (one lane): announces the items; queries, keys and values by TMA into 128-byte
//     swizzled operand buffers, keys and values in rings;
//   * warp 8 (one lane): for each tile tcgen05.mma S = Q K^T into TMEM, then, when the
//     tile's probabilities are there, O += P V with P read from TMEM, where it has taken
//     the place of S; the first half of P V starts when half of P is there;
//   * warps 0..3 / 4..7 (tile 0 / 1; thread = row = TMEM lane): the row's 128 scores in
//     registers, exp2, sum, probabilities as fp16 back to TMEM. While one tile's softmax
//     runs, the tensor core works on the other's products. O is rescaled only where the
//     probabilities would leave fp16 with the reference in use (see kHeadroom);
//   * warps 10, 11: in units that not all rows see whole, values past the sequence become
//     zero, and so do infinities and NaN, which times a probability of zero would reach
//     rows that do not see them. Rows that do see one get it back at the end.
// TMEM: S0 S1 O0 O1, 128 columns each.
//
// Where there are fewer items than SMs can take (few heads, few sequences), the longest one's
// units, one after the other, are what a call takes. Then a cluster of 2 or 4 CTAs has an item
// together: each a range of its keys, and in the end references, sums and outputs go from CTA
// to CTA through shared memory of the cluster (`join`), each CTA joining and storing its share of the
// columns: no workspace, and the same result each time. By st.async, which counts its bytes at
// the receiver: a released arrival waits for the stores to memory too, and took 20 us an item;
// what it takes now is about 2. prompt_ranks has the rule and both sides.
//
// Measured (in a graph): one prompt of 8192 tokens, 40 heads on 8, D = 128: 453 to 460 us (687
// GFLOP, up to 1517 TFLOP/s; 500 among other calls in a long run, in which the clock falls: 1374),
// one of 2048: 47 us; D = 64: 386 us; scores capped: 697 and 650 us; 4096 tokens, not causal: 250
// us (1373 TFLOP/s), D = 64: 225. What binds it is the chain of a tile's unit: about
// 1550 cycles of softmax (of them 512 for 128 exponentials a row at 4 cycles a warp)
// and 1300 from the last probability to the next scores (768 of products, the rest the ways
// through barriers), with TMEM full, so that the next scores cannot be formed meanwhile; the
// tensor core is busy 2048 of the 2850 cycles that a pair of units takes. Steps on the way
// (8192 tokens): the issuing lane by elect.sync, not lane 0, 644 -> 479 us; no maximum before
// the exponentials, items' places without a loop over all, stores by rows 479 -> 454. Slower:
// two threads a row (531), two issuing lanes (606), 168 registers for the softmax (782); at D
// = 64, where TMEM has room, P apart from S and the next scores ahead of it (414 for 388).
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_prompt_ranks.h"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kTile = 128;         // rows
constexpr int kTokens = 128;       // of a unit
constexpr int kMmaWarp = 8 /* after the softmax warps */, kLoadWarp = 9, kCleanWarp = 10, kCleanWarps = 2;
constexpr int kPromptThreads = 12 * 32;  // 168 registers a thread
constexpr int kPromptSeqs = 1024;  // sequences of one launch
constexpr int kMaxParts = 4;       // CTAs that share an item's keys
constexpr int kItems = 4;          // items announced at a time
constexpr int kFlags = 8;          // items whose flag is kept; more than a ring can be ahead
// Probabilities are taken relative to a reference: 2^kHeadroom below the row's maximum over
// its first unit, and set anew only when one of a unit's could leave fp16: when those of the
// first 64 keys add up to more than kMostSum (a sum that is formed anyway), or one of the
// others, whose scores are looked at while the first ones' exponentials run, is above 2^kMost.
// The result is the same, as the row's sum goes by the same reference. A row's largest
// probability is then 2^8 to 2^16: one of 2^-22 of it has all 11 bits, one of 2^-33 counts.
constexpr float kHeadroom = 8.0f, kMostSum = 65504.0f, kMost = 15.9f;
// The exponent is one fused operation, product * c - reference, which does not round the score
// as the reference was rounded. Below kLarge the two are 2^-4 apart at most; at 2^28 they would be
// 16 apart, which leaves fp16. Where a row's reference is past kLarge, every unit of the
// item from there on sets references anew and then puts rounded scores less the reference in
// the products' place (`less_reference`).
constexpr float kLarge = 0x1p20f;

template <int D, bool SPLIT>
struct PromptCfg {
  static constexpr int kSeqs = SPLIT ? kSplitSeqs : kPromptSeqs;
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = D == 64 ? 4 : 2;        // of keys, and of values
  static constexpr int kOperand = kHalves * 128 * 128;   // 128 rows (or tokens) x D fp16
  static constexpr int kOffK = 2 * kOperand;             // two query tiles before it
  static constexpr int kOffV = kOffK + kStages * kOperand;
  static constexpr int kOffSeq = kOffV + kStages * kOperand;
  static constexpr int kOffLen = kOffSeq + kSeqs * 8;
  static constexpr int kOffStage = kOffLen + kSeqs * 4;
  // of each softmax warp: 32 rows x 32 columns fp16 of the output, or what the other CTAs send: slabs of 32 rows x 8 columns
  // fp32, and references and sums
  static constexpr int kSlab = 32 * 8 * 4, kStats = 32 * 8, kSlabs = D == 64 ? 6 : 3;
  static constexpr int kStage = SPLIT ? kSlabs * kSlab + (kMaxParts - 1) * kStats : 2048;
  static constexpr int kOffItem = kOffStage + 8 * kStage;
  static constexpr int kOffBar = kOffItem + kItems * 32;
  static constexpr int kOffJoin = kOffBar + 512;  // a warp's barriers with those of the other CTAs: kGates for each
  static constexpr int kSmem = 1024 + kOffJoin + (SPLIT ? 8 * (kMaxParts - 1) * 3 * 8 : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};
constexpr int kMaxStages = 4;
// kPReady: values of a unit fit for use, and the next unit's keys.
// kPPassed: all that uses a unit's scores has them, so its keys and the values of the unit
// before are not needed any more.
enum { kPQFull = 0, kPFirst = 2, kPPassed = 3, kPVFull = kPPassed + kMaxStages, kPReady = kPVFull + kMaxStages,
       kPS = kPReady + kMaxStages, kPP = kPS + 2 /* tile x half */, kPO = kPP + 4, kPItemFull = kPO + 2,
       kPItemEmpty = kPItemFull + kItems, kPDone = kPItemEmpty + kItems, kPBars = kPDone + 1 };

// Of a warp with the same one of another CTA: its slab and its references and sums are here; what was sent there has been read.
enum { kSlabHere = 0, kStatsHere = 1, kSlabRead = 2, kGates = 3 };

struct PromptParams {
  PromptAttention a;
  int group, tile_tokens;
  int ranks;  // CTAs of a cluster, which share the keys of their items
  uint32_t nothing;  // 0, which the compiler does not know
};

// The launch's sequences from the longest to the shortest (equal ones in their order):
// first row and tokens, and pairs of tiles. Returns how many have any tokens. All threads;
// ends with a barrier.
template <int SEQS>
__device__ __forceinline__ int sort_prompts(const PromptAttention &a, int pair, int2 *seq, int *pairs) {
  const int n4 = (a.n_seqs + 3) & ~3;
  int *len = pairs;  // by sequence, until the sorted ones take its place
  constexpr int kEach = (SEQS + kPromptThreads - 1) / kPromptThreads;
  int row0[kEach], n[kEach], before[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int s = threadIdx.x + k * kPromptThreads;
    row0[k] = n[k] = 0;
    if (s < a.n_seqs) {
      row0[k] = a.q_start[s];
      n[k] = a.q_start[s + 1] - row0[k];
      if (row0[k] < 0 || n[k] < 0 || row0[k] + (int64_t)n[k] > a.rows) {
        report_index(a.status);
        n[k] = 0;
      }
    }
    if (s < n4) len[s] = n[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int s = threadIdx.x + k * kPromptThreads;
    before[k] = 0;
    if (n[k] > 0)
      for (int t = 0; t < n4; t += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(len + t);
        before[k] += (o.x > n[k] || (o.x == n[k] && t < s)) + (o.y > n[k] || (o.y == n[k] && t + 1 < s)) +
                     (o.z > n[k] || (o.z == n[k] && t + 2 < s)) + (o.w > n[k] || (o.w == n[k] && t + 3 < s));
      }
  }
  int total = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) total += __syncthreads_count(n[k] > 0);  // all are past the lengths
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (n[k] > 0) {
      seq[before[k]] = make_int2(row0[k], n[k]);
      pairs[before[k]] = (n[k] + pair - 1) / pair;
    }
  __syncthreads();
  return total;
}

struct Item {
  int row0, n;       // the sequence
  int h;             // key/value head
  int token0;        // first token of the pair
  int units0, units1;// of each tile; 0: the pair has no second tile
  int first_masked;  // from this unit on, not every row sees all keys
  int there;         // 0: there are no more items
  // Where CTAs share an item: units0 and units1 are this one's of total0 and total1, from `from` on, `share` of them at most.
  int from, share, total0, total1;
  __device__ __forceinline__ int all() const { return max(units0, units1); }
  template <bool SPLIT>
  __device__ __forceinline__ void take_part(int rank, int ranks) {
    from = 0;
    if constexpr (SPLIT) {
      total0 = units0;
      total1 = units1;
      share = (all() + ranks - 1) / ranks;
      from = rank * share;
      units0 = min(max(units0 - from, 0), share);
      units1 = min(max(units1 - from, 0), share);
    }
  }
};

// The items of a CTA (or a cluster): number k of them is item k * CTAs + c or, every second
// time, from the other end. Causal items are ordered by the pair's place in its sequence, the last
// ones first (which is by length but for sequences' last pairs), others by sequence.
struct PromptWalk {
  const int2 *seq;
  const int *pairs;
  int n_seqs;
  uint32_t round, base;
  int level, count;  // causal: place of the pair, and sequences that have it; else the sequence
  __device__ __forceinline__ void begin(int causal) {
    round = base = 0;
    level = causal && n_seqs > 0 ? pairs[0] - 1 : 0;
    count = 0;
  }
  __device__ __forceinline__ bool next(const PromptParams &p, Item &it, int ranks) {
    const uint32_t c = blockIdx.x / ranks, C = gridDim.x / ranks, heads = p.a.n_kv_heads;
    const uint32_t idx = round * C + (round & 1 ? C - 1 - c : c);
    ++round;
    int s, place;
    if (p.a.causal) {
      // places that the same sequences have are passed over at once
      for (;;) {
        while (count < n_seqs && pairs[count] > level) ++count;
        const uint32_t size = count * heads, same = level + 1 - (count < n_seqs ? pairs[count] : 0);
        if (size == 0) return false;
        const uint32_t skip = min((idx - base) / size, same);
        base += skip * size;
        level -= skip;
        if (skip < same) break;
        if (level < 0) return false;
      }
      s = (idx - base) / heads;
      place = level;
    } else {
      uint32_t mine = 0;
      while (level < n_seqs && idx - base >= (mine = pairs[level] * heads)) {
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
    it.token0 = place * 2 * p.tile_tokens;
    auto units = [&](int first) {
      const int seen = p.a.causal ? min(first + p.tile_tokens, it.n) : it.n;
      return first < it.n ? (seen + kTokens - 1) / kTokens : 0;
    };
    it.units0 = units(it.token0);
    it.units1 = units(it.token0 + p.tile_tokens);
    it.first_masked = (p.a.causal ? it.token0 + 1 : it.n) / kTokens;
    it.there = 1;
    return true;
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// True in one lane of the warp. What it guards needs no loop over lanes around each
// tensor-core instruction, which `lane == 0` gets from the compiler (46 cycles an
// instruction and more, where 32 or 64 are the tensor core's own time).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Loads 64 consecutive TMEM columns of this thread's lane and waits for them inside the
// same asm statement, so no use can be scheduled before the wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr), "r"(taddr + 32));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(taddr));
}
// tmem_ld64 in two parts: nothing may use v between them, and what comes after goes through
// the second.
__device__ __forceinline__ void tmem_ld64_begin(uint32_t taddr, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr), "r"(taddr + 32));
}
__device__ __forceinline__ void tmem_ld64_end(float (&v)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" :
      "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
      "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
      "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
      "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]),
      "+f"(v[32]), "+f"(v[33]), "+f"(v[34]), "+f"(v[35]), "+f"(v[36]), "+f"(v[37]), "+f"(v[38]), "+f"(v[39]),
      "+f"(v[40]), "+f"(v[41]), "+f"(v[42]), "+f"(v[43]), "+f"(v[44]), "+f"(v[45]), "+f"(v[46]), "+f"(v[47]),
      "+f"(v[48]), "+f"(v[49]), "+f"(v[50]), "+f"(v[51]), "+f"(v[52]), "+f"(v[53]), "+f"(v[54]), "+f"(v[55]),
      "+f"(v[56]), "+f"(v[57]), "+f"(v[58]), "+f"(v[59]), "+f"(v[60]), "+f"(v[61]), "+f"(v[62]), "+f"(v[63]));
}

// tmem_st32 of 32-bit words.
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  float f[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
  tmem_st32(taddr, f);
}

// A cap of the scores, in log2 units. Where x^2 < 1/4, x = score / cap, cap * tanh(x) is
// score * p(x^2) with the polynomial p of degree 3, p(0) = 1, that is nearest to tanh(x) / x
// there (to 6.5e-7, found by minimising the largest relative error): no exponential and no
// reciprocal, which would cost three times the softmax's own. It is of the product's square,
// with coefficients that bring that to x^2, where they stay in fp32's range (`ready`). Scores
// beyond go through 1 - 2 / (exp(2 x) + 1), an absolute error near cap * 2^-22, in a pass of
// their own over TMEM: in line with the softmax it would be too much code for the instruction
// cache. The others have the same value there, so that a score's does not depend on its
// neighbours.
struct PromptCap {
  bool ready;               // else all scores take the pass over TMEM
  float k, unit, cap, edge; // x = product * k; edge: what (product * unit)^2 is below, of those near
  float p[4];               // of (product * unit)^2, times what brings a product to log2 units
  // A cap whose double leaves fp32 is lowered: no score comes near it. So is k, which times 0 has to be 0.
  __device__ __forceinline__ PromptCap(float softcap, float c)
      : k(fminf(c / fmaxf(softcap * kLog2e, 1e-30f), 0x1p127f)), cap(fminf(softcap * kLog2e, 1.5e38f)) {
    ready = k > 0x1p-18f && k < 0x1p14f && c > 0x1p-10f && c < 0x1p14f;
    unit = ready ? 1.0f : k;
    const float k2 = ready ? k * k : 1.0f;
    edge = 0.25f / k2;
    p[0] = c;
    p[1] = c * -0.333281593f * k2;
    p[2] = c * 0.132053586f * (k2 * k2);
    p[3] = c * -0.0447506050f * (k2 * k2 * k2);
  }
  // N products to capped scores, those with x^2 < 1/4; `most` becomes the largest (product * unit)^2.
  template <bool READY, int N>
  __device__ __forceinline__ void near(float (&s)[N], float &most) const {
    auto both = [](float v) { return make_float2(v, v); };
    float m[4] = {most, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = make_float2(s[i], s[i + 1]), x = READY ? v : mul2(v, both(unit)), y = mul2(x, x);
      m[i / 2 % 4] = fmaxf(m[i / 2 % 4], fmaxf(y.x, y.y));
      float2 t = fma2(y, both(p[3]), both(p[2]));
      t = fma2(y, t, both(p[1]));
      t = mul2(v, fma2(y, t, both(p[0])));
      s[i] = t.x;
      s[i + 1] = t.y;
    }
    most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  }
  // A row's 128 products in TMEM, in place. Rows that are not real hold anything.
  __device__ __forceinline__ void all(uint32_t scores, bool real) const {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float s[32], most = 0.f;
      tmem_ld32(scores + 32 * q, s);
      near<false>(s, most);
      if (__any_sync(0xffffffffu, real && most >= edge)) {
        float raw[32];
        tmem_ld32(scores + 32 * q, raw);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = raw[i] * k, u = raw[i] * unit, f = fmaf(-2.0f * cap, rcp(ex2(x * (2.0f * kLog2e)) + 1.0f), cap);
          s[i] = u * u < edge ? s[i] : f;
        }
      }
      tmem_st32(scores + 32 * q, s);
    }
    tmem_wait_st();
  }
};

// A row's 128 products in TMEM, in place: (score - ref) / c for rows that want it.
__device__ __forceinline__ void less_reference(uint32_t scores, bool wanted, float c, float ref) {
  const float back = 1.0f / c;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    float s[32];
    tmem_ld32(scores + 32 * q, s);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = wanted ? (__fmul_rn(s[i], c) - ref) * back : s[i];
    tmem_st32(scores + 32 * q, s);
  }
  tmem_wait_st();
}

// Stores to another CTA of the cluster, whose bytes are counted on its barrier (both addresses
// from map_to_rank): nothing has to be waited for here, as a release would, for stores to memory too.
__device__ __forceinline__ void store_there(uint32_t dst, uint32_t bar, float a, float b, float c, float d) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst), "f"(a), "f"(b),
               "f"(c), "f"(d), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void store_there(uint32_t dst, uint32_t bar, float a, float b) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst), "f"(a), "f"(b), "r"(bar)
               : "memory");
}

// Bits of the fp16 pair w whose exponent is all ones (infinity, NaN): 0x8000 for each.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

template <int D, bool CAP, bool SPLIT>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv, const PromptParams p) {
  using Cfg = PromptCfg<D, SPLIT>;
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
  const int ranks = SPLIT ? p.ranks : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kPQFull + t), 1);
      mbar_init(bar(kPS + t), 1);
      mbar_init(bar(kPP + 2 * t), 4);
      mbar_init(bar(kPP + 2 * t + 1), 4);
      mbar_init(bar(kPO + t), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(kPPassed + i), 4);
      mbar_init(bar(kPVFull + i), 1);
      mbar_init(bar(kPReady + i), 1 + kCleanWarps);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(kPItemFull + i), 1);
      mbar_init(bar(kPItemEmpty + i), 8 + 1 + kCleanWarps);
    }
    mbar_init(bar(kPFirst), 1);
    mbar_init(bar(kPDone), 1);
    for (int i = 0; i < kFlags; ++i) flags[i] = 0;
    if constexpr (SPLIT)
      for (int i = 0; i < 8 * (kMaxParts - 1) * kGates; ++i) mbar_init(base + Cfg::kOffJoin + 8 * i, 1);
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
  if constexpr (SPLIT) {  // every CTA runs, with its barriers, before another stores to it
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_before();
  PromptWalk walk{seq, reinterpret_cast<int *>(smem + Cfg::kOffLen),
                  sort_prompts<Cfg::kSeqs>(p.a, 2 * p.tile_tokens, seq, reinterpret_cast<int *>(smem + Cfg::kOffLen))};
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int4 *items = reinterpret_cast<int4 *>(smem + Cfg::kOffItem);
  // Item number n, as the loading lane announces it.
  auto item_there = [&](uint32_t n) { return mbar_wait(bar(kPItemFull + n % kItems), (n / kItems) & 1, status); };
  auto read_item = [&](uint32_t n, Item &it) {
    const int4 a = items[2 * (n % kItems)], b = items[2 * (n % kItems) + 1];
    it = Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    it.take_part<SPLIT>(rank, ranks);
  };
  auto item_read = [&](uint32_t n) { mbar_arrive(bar(kPItemEmpty + n % kItems)); };

  // 168 registers a thread at launch: the last four warps give 12288 of theirs to the others
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kMmaWarp) {
      // ---------------- tensor core (one lane) ----------------
      if (elect_one()) {
        // bit 13: A negated, for a negative scale
        const uint32_t idesc_s = f16_idesc(kTile, kTokens) | (p.a.scale < 0.f ? 1u << 13 : 0u);
        constexpr uint32_t kIdescO = f16_idesc(kTile, D) | kIdescBTransposed;
        uint32_t unit = 0, number = 0, items_of[2] = {0, 0}, units_of[2] = {0, 0};
        auto ready = [&](uint32_t u) { return mbar_wait(bar(kPReady + u % kStages), (u / kStages) & 1, status); };
        auto scores = [&](int t, uint32_t u) {
          const uint32_t q = base + t * Cfg::kOperand, k = base + Cfg::kOffK + (u % kStages) * Cfg::kOperand;
  #pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t off = (j >> 2) * (128 * 128) + (j & 3) * 32;
            tc_mma(tmem + 128 * t, sw128_desc(q + off), sw128_desc(k + off), idesc_s, j > 0);
          }
          tc_commit(bar(kPS + t));
        };
        bool ok = item_there(0);
        Item it;
        read_item(0, it);
        if (ok && it.there) ok = mbar_wait(bar(kPFirst), 0, status);
        while (ok && it.there) {
          const int units[2] = {it.units0, it.units1}, all = it.all();
          item_read(number++);
  #pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || units[t] == 0) continue;
            ok = mbar_wait(bar(kPQFull + t), items_of[t]++ & 1, status);
            if (!ok) break;
            tc_fence_after();
            scores(t, unit);
          }
          for (int j = 0; ok && j < all; ++j, ++unit) {
            ok = ready(unit);
            const uint32_t v = base + Cfg::kOffV + (unit % kStages) * Cfg::kOperand;
  #pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || j >= units[t]) continue;
              const uint32_t ph = units_of[t]++ & 1;
  #pragma unroll
              for (int half = 0; half < 2; ++half) {
                ok = ok && mbar_wait(bar(kPP + 2 * t + half), ph, status);
                if (!ok) break;
                tc_fence_after();
  #pragma unroll
                for (int k = 4 * half; k < 4 * half + 4; ++k)
                  tc_mma_ta(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, sw128_mn_desc(v + k * 2048, 128 * 128, 1024), kIdescO, (j | k) > 0);
              }
              if (!ok) break;
              if (j + 1 < units[t]) scores(t, unit + 1);
              else tc_commit(bar(kPO + t));
            }
          }
          ok = ok && item_there(number);
          read_item(number, it);
        }
        tc_commit(bar(kPDone));  // every issued product ends before the TMEM is released
        mbar_wait_short(bar(kPDone), 0);
      }
    } else if (warp == kLoadWarp) {
      // ---------------- items and loads (one lane) ----------------
      if (elect_one()) {
        uint32_t unit = 0, number = 0, items_of[2] = {0, 0};
        bool ok = true;
        const uint32_t q_bytes = (uint32_t)(Cfg::kHalves * 128) * p.group * p.tile_tokens;
        auto operand = [&](const CUtensorMap *map, uint32_t dst, uint32_t b, int head, int row) {
  #pragma unroll
          for (int hf = 0; hf < Cfg::kHalves; ++hf)
            if (EXL3_RANGE(row, 0, p.a.rows) && EXL3_SMEM(dst + hf * (128 * 128), 128 * 128))
              tma_load_3d(dst + hf * (128 * 128), map, b, 64 * hf, head, row);
        };
        auto announce = [&](const Item &it) {
          ok = ok && mbar_wait(bar(kPItemEmpty + number % kItems), ((number / kItems) & 1) ^ 1, status);
          if (!ok) return;
          items[2 * (number % kItems)] = make_int4(it.row0, it.n, it.h, it.token0);
          items[2 * (number % kItems) + 1] = make_int4(SPLIT ? it.total0 : it.units0, SPLIT ? it.total1 : it.units1, it.first_masked, it.there);
          mbar_arrive(bar(kPItemFull + number % kItems));
          ++number;
        };
        // In any order, but each unit's before the next one with its slot is loaded.
        auto passed = [&](uint32_t u) { return mbar_wait(bar(kPPassed + u % kStages), (u / kStages) & 1, status); };
        auto keys = [&](uint32_t u, uint32_t b, const Item &it, int j) {
          mbar_arrive_expect_tx(b, Cfg::kOperand);
          operand(&tk, base + Cfg::kOffK + (u % kStages) * Cfg::kOperand, b, it.h, it.row0 + (it.from + j) * kTokens);
        };
        auto walk_on = [&](Item &it) {  // to the next item that this CTA has units of
          do {
            it.there = walk.next(p, it, ranks);
            it.take_part<SPLIT>(rank, ranks);
          } while (SPLIT && it.there && it.all() == 0);
        };
        walk.begin(p.a.causal);
        Item it, next;
        walk_on(it);
        announce(it);
        const bool any = it.there;
        if (any) keys(0, bar(kPFirst), it, 0);
        while (ok && it.there) {
          ok = unit == 0 || passed(unit - 1);  // the last item's scores: its queries are not needed any more
          if (!ok) break;
  #pragma unroll
          for (int t = 0; t < 2; ++t) {
            if ((t == 0 ? it.units0 : it.units1) == 0) continue;
            ++items_of[t];
            mbar_arrive_expect_tx(bar(kPQFull + t), q_bytes);
            operand(&tq, base + t * Cfg::kOperand, bar(kPQFull + t), it.h * p.group, it.row0 + it.token0 + t * p.tile_tokens);
          }
          walk_on(next);
          const int all = it.all();
          for (int j = 0; ok && j < all; ++j, ++unit) {
            const uint32_t st = unit % kStages;
            ok = unit + 1 < kStages || passed(unit + 1 - kStages);
            if (!ok) break;
            mbar_arrive_expect_tx(bar(kPVFull + st), Cfg::kOperand);
            operand(&tv, base + Cfg::kOffV + st * Cfg::kOperand, bar(kPVFull + st), it.h, it.row0 + (it.from + j) * kTokens);
            if (j == 0) announce(next);
            if (j + 1 < all) keys(unit + 1, bar(kPReady + st), it, j + 1);
            else if (next.there) keys(unit + 1, bar(kPReady + st), next, 0);
            else mbar_arrive(bar(kPReady + st));
          }
          it = next;
        }
        // nothing is on its way into this CTA's memory when it ends (at once, unless a wait ran out)
        if (any) mbar_wait_short(bar(kPFirst), 0);
        for (uint32_t i = 0; i < kStages; ++i)
          if (unit > i) {
            mbar_wait_short(bar(kPVFull + i), ((unit - 1 - i) / kStages) & 1);
            mbar_wait_short(bar(kPReady + i), ((unit - 1 - i) / kStages) & 1);
          }
        for (int t = 0; t < 2; ++t)
          if (items_of[t] > 0) mbar_wait_short(bar(kPQFull + t), (items_of[t] - 1) & 1);
      }
    } else {
      // ---------------- values that not every row may use ----------------
      uint32_t unit = 0, number = 0;
      Item it;
      for (bool ok = true;; ++number) {
        ok = __all_sync(0xffffffffu, ok && item_there(number));
        if (!ok) break;
        read_item(number, it);
        __syncwarp();
        if (lane == 0) item_read(number);
        if (!it.there) break;
        const int all = it.all();
        for (int j = 0; j < all; ++j, ++unit) {
          const uint32_t st = unit % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kPVFull + st), (unit / kStages) & 1, status));
          if (!ok) break;
          if (it.from + j >= it.first_masked) {
            const uint32_t v = base + Cfg::kOffV + st * Cfg::kOperand;
            const int left = it.n - (it.from + j) * kTokens;  // tokens of the sequence from here
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
          if (lane == 0) mbar_arrive(bar(kPReady + st));  // of every unit: the ring cannot get ahead of this warp
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---------------- softmax: thread = row of tile t ----------------
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_tmem = lane_base + 128 * t, o_tmem = lane_base + 256 + 128 * t;
    const float c = fminf(fmaxf(fabsf(p.a.scale) * Raised<D>::kLog2e, 1e-37f), 0x1.fffffep127f);  // scores in log2 units are the products times c
    const PromptCap cap(p.a.softcap, c);
    const int token = row / p.group, head_in = row - token * p.group;
    uint32_t count = 0, items = 0, number = 0, unit = 0;  // units and items of this tile, items and units of the CTA
    [[maybe_unused]] uint32_t stats_got = 0, got = 0, sent = 0;  // phases of the barriers with the other CTAs, a bit each
    bool ok = true;
    auto hand_over = [&](int half) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPP + 2 * t + half));
    };
    Item it, next;
    auto next_item = [&](uint32_t n) {
      ok = __all_sync(0xffffffffu, ok && item_there(n));
      read_item(n, next);
      __syncwarp();
      if (lane == 0) item_read(n);
    };
    next_item(0);
    for (; ok && next.there; ++number, unit += it.all()) {
      it = next;
      const int units = t == 0 ? it.units0 : it.units1;
      if (units == 0) {
        next_item(number + 1);
        continue;
      }
      // the last tile that uses a unit's keys and values: this one from here on (the products of tile 1 come after those of tile 0)
      const int last_from = t == 0 ? it.units1 : 0;
      const int pos = it.token0 + t * p.tile_tokens + token;
      const bool real = token < p.tile_tokens && pos < it.n;
      const int limit = !real ? 0 : p.a.causal ? pos + 1 : it.n;
      const int least = __reduce_min_sync(0xffffffffu, real ? limit : INT32_MAX);
      const bool live = __any_sync(0xffffffffu, real);
      float ref = -INFINITY, sum = 0.f;
      bool far = !cap.ready;  // scores beyond half the cap were seen
      bool large = false;     // a reference past kLarge was
      for (int u = 0; u < units; ++u, ++count) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kPS + t), count & 1, status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // The scores are there, so their keys are not needed any more, nor the values of the unit
        // before (its product came first), nor, with the item's last scores, the queries. Said from
        // here: a commit for it would stop the lane that issues the products (64 to 200 cycles).
        if (u >= last_from && lane == 0) mbar_arrive(bar(kPPassed + (unit + u) % kStages));
        if (live) {
          const int pos0 = (it.from + u) * kTokens;
          const float scale = CAP ? 1.0f : c;
          const float2 scale2 = make_float2(scale, scale);
          bool renew = u == 0 || large || __any_sync(0xffffffffu, real && ref == -INFINITY);
          bool less = false;  // TMEM holds scores less the reference, of rows past kLarge
          float s[64], s2[64];  // of the unit's first and second 64 keys
          uint32_t packed[32];  // fp16 probabilities: 2^-12 on average, the size of the result's own rounding
          float2 part[2], shift2;
          auto exponentials = [&](const float (&x64)[64], int from, int to) {
#pragma unroll
            for (int k = from; k < to; ++k) {
              float2 x = fma2(make_float2(x64[2 * k], x64[2 * k + 1]), scale2, shift2);
              x = make_float2(ex2(x.x), ex2(x.y));
              part[k & 1] = add2(part[k & 1], x);
              const __half2 h2 = __floats2half2_rn(x.x, x.y);
              packed[k] = *reinterpret_cast<const uint32_t *>(&h2);
            }
          };
          auto most = [&](const float (&x)[64]) {
            float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int k = 4; k < 60; k += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], fmaxf(x[k + e], x[k + 4 + e]));
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], x[60 + e]);
            return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * scale;
          };
          auto mask = [&](float (&x64)[64], int first) {
            if (first + 64 > least) {
              const int n = min(max(limit - first, 0), 64);  // keys that the row sees; as bits, whose tests take an instruction for several
              const uint64_t seen = n == 64 ? ~0ull : (1ull << n) - 1;
              const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (!(lo & 1u << k)) x64[k] = -INFINITY;
                if (!(hi & 1u << k)) x64[32 + k] = -INFINITY;
              }
            }
          };
          bool capped = !CAP;  // the scores in TMEM
          if (CAP && (renew || far)) {
            cap.all(s_tmem, real);
            capped = true;
          }
          // A second round is rare; the scores are still in TMEM then.
#pragma unroll 1
          for (;;) {
            tmem_ld64(s_tmem, s);
            tmem_ld64_begin(s_tmem + 64, s2);
            float most_x = 0.f;
            if (CAP && !capped) cap.near<true>(s, most_x);
            mask(s, pos0);
            if (renew) {
              tmem_ld64_end(s2);
              mask(s2, pos0 + 64);
              const float now = fmaxf(__fsub_ru(fmaxf(most(s), most(s2)), kHeadroom), ref);  // up: 16 below would leave fp16
              if (u > 0) {
                const float keep = now == ref || ref == -INFINITY ? 1.0f : ex2(ref - now);
                // the scores' product came after the output's, which is therefore done
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
              const bool past = fabsf(ref) >= kLarge && ref > -INFINITY;
              if (!CAP && __any_sync(0xffffffffu, real && past)) {
                less_reference(s_tmem, past, c, ref);
                large = less = true;
                renew = false;
                continue;  // none is above 2^kHeadroom now
              }
            }
            const float shift = ref == -INFINITY || (less && fabsf(ref) >= kLarge) ? 0.f : -ref;
            shift2 = make_float2(shift, shift);
            part[0] = part[1] = make_float2(0.f, 0.f);
            exponentials(s, 0, 32);
            if (renew) break;
            tmem_ld64_end(s2);
            if (CAP && !capped) cap.near<true>(s2, most_x);
            mask(s2, pos0 + 64);
            const float so_far = (part[0].x + part[0].y) + (part[1].x + part[1].y);
            const bool beyond = CAP && real && most_x >= cap.edge;
            if (!__any_sync(0xffffffffu, beyond || (real && (so_far > kMostSum || most(s2) + shift > kMost))) || less) break;
            if (CAP && !capped) {
              far = __any_sync(0xffffffffu, beyond);  // the item's other units at once
              cap.all(s_tmem, real);
              capped = true;
            }
            renew = true;
          }
          tmem_st32u(s_tmem, packed);
          exponentials(s2, 0, 16);
          hand_over(0);  // the stores have had time
          exponentials(s2, 16, 32);
          tmem_st32u(s_tmem + 32, packed);
          hand_over(1);
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
      if (ok) next_item(number + 1);  // while the last products run
      if (!ok || !__all_sync(0xffffffffu, mbar_wait(bar(kPO + t), items++ & 1, status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // What the CTAs that share the item have of this tile's rows becomes one: first their
      // references and sums, then the outputs, each CTA's share of the columns at that CTA, from warp
      // to warp of the same rows.
      [[maybe_unused]] auto join = [&]() -> bool {
        const int parts = ((t == 0 ? it.total0 : it.total1) + it.share - 1) / it.share;  // CTAs that have some, the first ones
        const uint32_t mail = base + Cfg::kOffStage + warp * Cfg::kStage, mail_stats = mail + Cfg::kSlabs * Cfg::kSlab;
        auto place = [](int of, int at) { return of < at ? of : of - 1; };  // of a CTA among the others of CTA `at`
        auto gate = [&](int place, int what) { return base + Cfg::kOffJoin + 8 * ((warp * (kMaxParts - 1) + place) * kGates + what); };
        auto here = [&](int place, int what, uint32_t phase, int bytes) {
          if (bytes > 0 && lane == 0) mbar_arrive_expect_tx(gate(place, what), bytes);
          return __all_sync(0xffffffffu, mbar_wait_cluster(gate(place, what), phase >> place & 1, status, kWaitLimitNs));
        };
        // the sum's sign says whether infinities and NaN were taken out
        const float told = flags[number % kFlags] == number + 1 ? __uint_as_float(__float_as_uint(sum) | 0x80000000u) : sum;
        for (int q = 0; q < parts; ++q)
          if (q != rank) {
            // the last item's slab has been read there, and before it the last item's sums
            if (!here(place(q, rank), kSlabRead, ~sent, 0)) return false;
            const uint32_t to = mail_stats + place(rank, q) * Cfg::kStats + lane * 8;
            if (EXL3_SMEM(to, 8)) store_there(map_to_rank(to, q), map_to_rank(gate(place(rank, q), kStatsHere), q), ref, told);
          }
        float refs[kMaxParts - 1], sums[kMaxParts - 1], top = ref;
        uint32_t taken = __float_as_uint(told);
#pragma unroll
        for (int k = 0; k < kMaxParts - 1; ++k) {
          refs[k] = -INFINITY;
          sums[k] = 0.f;
          if (k + (k >= rank) < parts) {
            if (!here(k, kStatsHere, stats_got, Cfg::kStats)) return false;
            stats_got ^= 1u << k;
            uint32_t w;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=f"(refs[k]), "=r"(w) : "r"(mail_stats + k * Cfg::kStats + lane * 8) : "memory");
            sums[k] = __uint_as_float(w & 0x7fffffffu);
            taken |= w;
            top = fmaxf(top, refs[k]);
          }
        }
        float mine = ref == -INFINITY ? 0.f : ex2(ref - top), total = mine * sum;
#pragma unroll
        for (int k = 0; k < kMaxParts - 1; ++k) {
          refs[k] = refs[k] == -INFINITY ? 0.f : ex2(refs[k] - top);
          total = fmaf(refs[k], sums[k], total);
        }
        const float f = total == 0.f ? 0.f : 1.0f / total;
        mine *= f;
        uint32_t read = taken;  // bits of all that other CTAs sent
#pragma unroll
        for (int k = 0; k < kMaxParts - 1; ++k) {
          refs[k] *= f;
          read |= __float_as_uint(refs[k]);
        }
        const int head = it.h * p.group + head_in;
        const int64_t off = (int64_t)(it.row0 + pos) * p.a.ldo + (int64_t)head * D;
        const bool fits = real && EXL3_SPAN(off, D, (int64_t)(p.a.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D);
        if (rank == 0 && fits && p.a.lse) p.a.lse[(int64_t)(it.row0 + pos) * p.a.n_heads + head] = log_sum(top + kHeadroom, total * 0x1p-8f);
        const int wide = parts == 2 ? 2 * Cfg::kSlabs / 3 : Cfg::kSlabs / 3;  // slabs that go to a CTA at a time: one place for each other
#pragma unroll 1
        for (int first = 0; first < D; first += 8 * wide * parts) {
          for (int i = 1; i < parts; ++i) {
            const int q = rank + i < parts ? rank + i : rank + i - parts, at = place(q, rank), k = first + 8 * wide * q;
            if (k >= D) continue;
            if (!here(at, kSlabRead, ~sent, 0)) return false;
            sent ^= 1u << at;
            const uint32_t bar_there = map_to_rank(gate(place(rank, q), kSlabHere), q);
            for (int c = 0; c < wide; ++c) {
              float o[8];
              tmem_ld8(o_tmem + k + 8 * c, o);
              const uint32_t to = mail + (place(rank, q) * wide + c) * Cfg::kSlab + lane * 32;
              if (EXL3_SMEM(to, 32)) {
                const uint32_t there = map_to_rank(to, q);
                store_there(there, bar_there, o[0], o[1], o[2], o[3]);
                store_there(there + 16, bar_there, o[4], o[5], o[6], o[7]);
              }
            }
          }
          if (first + 8 * wide * rank >= D) continue;
#pragma unroll
          for (int i = 0; i < kMaxParts - 1; ++i) {
            if (i + (i >= rank) >= parts) continue;
            if (!here(i, kSlabHere, got, wide * Cfg::kSlab)) return false;
            got ^= 1u << i;
          }
          for (int c = 0; c < wide; ++c) {
            const int k = first + 8 * (wide * rank + c);
            float o[8];
            tmem_ld8(o_tmem + k, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= mine;
#pragma unroll
            for (int i = 0; i < kMaxParts - 1; ++i) {
              if (i + (i >= rank) >= parts) continue;
              float x[8];
              const uint32_t from = mail + (i * wide + c) * Cfg::kSlab + lane * 32;
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(from) : "memory");
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "r"(from + 16) : "memory");
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o[e] = fmaf(refs[i], x[e], o[e]);
                read |= __float_as_uint(x[e]);
              }
            }
            if (fits && taken >> 31) {  // as below
#pragma unroll 1
              for (int at = it.first_masked * kTokens; at < limit; ++at) {
                const int64_t from = (int64_t)(it.row0 + at) * p.a.ldv + (int64_t)it.h * D + k;
                if (!EXL3_SPAN(from, 8, (int64_t)(p.a.rows - 1) * p.a.ldv + (int64_t)p.a.n_kv_heads * D)) continue;
                const __half *v = static_cast<const __half *>(p.a.v) + from;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float x = __half2float(v[e]);
                  if (!isfinite(x)) o[e] += x;
                }
              }
            }
            if (fits) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __half2 h2 = __floats2half2_rn(o[2 * x], o[2 * x + 1]);
                w[x] = *reinterpret_cast<const uint32_t *>(&h2);
              }
              *reinterpret_cast<uint4 *>(static_cast<__half *>(p.a.out) + off + k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          // One arrival for the warp. A release would wait for the stores to memory too (8192 tokens of one head:
          // 39.6 us for 37.3); what orders the reads before the next slab is that the arrival's address
          // depends on all of them.
          const uint32_t seen = __reduce_or_sync(0xffffffffu, read) & p.nothing;
          if (lane < kMaxParts - 1 && lane + (lane >= rank) < parts) {
            const int q = lane + (lane >= rank);
            asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(gate(place(rank, q), kSlabRead), q) + seen) : "memory");
          }
        }
        return true;
      };
      if constexpr (SPLIT) {
        if (live && !join()) {
          ok = false;
          break;
        }
      } else if (live) {
        const float f = sum == 0.f ? 0.f : 1.0f / sum;
        const int head = it.h * p.group + head_in;
        const int64_t off = (int64_t)(it.row0 + pos) * p.a.ldo + (int64_t)head * D;
        const bool fits = real && EXL3_SPAN(off, D, (int64_t)(p.a.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D);
        const bool back = fits && flags[number % kFlags] == number + 1;
        // Through shared memory, so that a store's lanes have 64 bytes of each of 8 rows, not 16 of
        // each of 32 (which take the SM's store path 32 cycles each).
        const uint32_t stage = base + Cfg::kOffStage + warp * 2048;
        const uint32_t rows_fit = __ballot_sync(0xffffffffu, fits);
        int64_t to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(0xffffffffu, off, 8 * i + (lane >> 2)) + 8 * (lane & 3);
#pragma unroll 1
        for (int k = 0; k < D; k += 64) {
          float o[64];
          __syncwarp();
          tmem_ld64(o_tmem + k, o);
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] *= f;
          if (back) {  // infinities and NaN that this row sees, of the units where they were taken out
#pragma unroll 1
            for (int at = it.first_masked * kTokens; at < limit; ++at) {
              const int64_t from = (int64_t)(it.row0 + at) * p.a.ldv + (int64_t)it.h * D + k;
              if (!EXL3_SPAN(from, 64, (int64_t)(p.a.rows - 1) * p.a.ldv + (int64_t)p.a.n_kv_heads * D)) continue;
              const __half *v = static_cast<const __half *>(p.a.v) + from;
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const float x = __half2float(v[e]);
                if (!isfinite(x)) o[e] += x;
              }
            }
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __half2 h2 = __floats2half2_rn(o[32 * part + 8 * e + 2 * x], o[32 * part + 8 * e + 2 * x + 1]);
                w[x] = *reinterpret_cast<const uint32_t *>(&h2);
              }
              sts16(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2);
              uint4 w;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                           : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)));
              if (rows_fit >> r & 1) *reinterpret_cast<uint4 *>(static_cast<__half *>(p.a.out) + to[i] + k + 32 * part) = w;
            }
          }
        }
        // a logarithm near 8 would be 2^-21 off: with the reference back at the maximum first
        if (fits && p.a.lse) p.a.lse[(int64_t)(it.row0 + pos) * p.a.n_heads + head] = log_sum(ref + kHeadroom, sum * 0x1p-8f);
      }
      tc_fence_before();  // the output has been read: before the next item's first products
    }
  }
  tc_fence_before();
  if constexpr (SPLIT) {  // nothing comes from another CTA any more
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// clusters: of 2 and of 4 CTAs that run at once.
template <int D>
cudaError_t prompt_attention(const PromptAttention &a, int num_sms, const int (&clusters)[2], cudaStream_t st) {
  PromptParams p;
  p.a = a;
  p.group = a.n_heads / a.n_kv_heads;
  p.tile_tokens = kTile / p.group;
  p.nothing = 0;
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
  // items at most
  auto items = [&](int n_seqs) { return (ceil_div(a.rows, 2 * p.tile_tokens) + n_seqs) * a.n_kv_heads; };
  p.ranks = prompt_ranks(a.n_seqs, a.rows, a.causal, items(a.n_seqs), num_sms, clusters);
  if (p.ranks > 1) {
    const int64_t most = items(a.n_seqs), at_once = clusters[p.ranks == 4];
    return launch_overlapped(a.softcap > 0.f ? prompt_attention_kernel<D, true, true> : prompt_attention_kernel<D, false, true>,
                             dim3((unsigned)(p.ranks * (most < at_once ? most : at_once))), kPromptThreads, PromptCfg<D, true>::kSmem, st, p.ranks,
                             tq, tk, tv, p);
  }
  for (int s0 = 0; s0 < a.n_seqs; s0 += kPromptSeqs) {
    p.a.q_start = a.q_start + s0;
    p.a.n_seqs = a.n_seqs - s0 < kPromptSeqs ? a.n_seqs - s0 : kPromptSeqs;
    const int64_t most = items(p.a.n_seqs);
    const cudaError_t e =
        launch_overlapped(a.softcap > 0.f ? prompt_attention_kernel<D, true, false> : prompt_attention_kernel<D, false, false>,
                          dim3((unsigned)(most < num_sms ? most : num_sms)), kPromptThreads, PromptCfg<D, false>::kSmem, st, 1, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t init_kernels(int (&clusters)[2]) {
  cudaError_t e = cudaSuccess;
  for (const void *f : {(const void *)prompt_attention_kernel<D, false, false>, (const void *)prompt_attention_kernel<D, true, false>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<D, false>::kSmem);
  for (const void *f : {(const void *)prompt_attention_kernel<D, false, true>, (const void *)prompt_attention_kernel<D, true, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptCfg<D, true>::kSmem);
  for (int four = 0; four < 2 && e == cudaSuccess; ++four) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = four ? 4 : 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(attr.val.clusterDim.x);
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = PromptCfg<D, true>::kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters[four], prompt_attention_kernel<D, false, true>, &cfg);
  }
  return e;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptAttention &a, int num_sms, const int (&clusters)[2][2], cudaStream_t st) {
  return a.head_dim == 64 ? prompt_attention<64>(a, num_sms, clusters[0], st) : prompt_attention<128>(a, num_sms, clusters[1], st);
}

cudaError_t init_prompt_attention_kernels(int *status, int (&clusters)[2][2]) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  if (e == cudaSuccess) e = init_kernels<64>(clusters[0]);
  if (e == cudaSuccess) e = init_kernels<128>(clusters[1]);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_prompt_attention(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
