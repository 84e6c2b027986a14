// Attention over the 8-bit key/value cache, and the accumulated attention weight
// of its tokens. Formulas in include/exl3.h.
//
// Stream kernel, for few rows (row of the sequence x head of the group). A segment is
// a (sequence, key/value head, tile of up to 16 rows). All work is cut into units of
// 32 cached tokens; the units of all segments lie one behind the other, and each
// warp of a persistent grid takes one equal, contiguous range of them, whatever the
// sequences' lengths are (they are read on the device). A warp keeps its own ring
// of TMA copies in flight and its own running maximum, sum and output, so warps do
// not wait for one another. Where ranges end inside a segment, the partial results
// are joined in the order of the ranges: those of a CTA's warps through shared
// memory when the CTA is done, those of several CTAs through the workspace by a
// second kernel.
//
// The bound is the cache stream: D + D bytes a token and head. The tensor core's
// narrow side takes the rows (S^T = K Q^T and O^T = V^T P^T, m16n8k16): 8 rows
// of a group cost half the products and registers that 16 would, and the
// transposed probabilities come from one movmatrix each. Codes become fp16
// exactly. The dimension is permuted so that a lane's 16 bytes of a key serve
// four k-steps and its 16 bytes of a value four rows of the output, without a
// shuffle.
//
// Measured, 40 heads on 8, D = 128: two sequences of 98K to 131K tokens 87 us (471
// MB, 5.4 TB/s: DRAM is 74 % busy, the slowest SM 10 % over the average); 16 sequences
// of 61 to 8192 tokens 36 us (136 MB, 3.8 TB/s: launch, plan and page numbers before
// the first units and the two joins after the last weigh more); one of 777 tokens 12
// us, all latency.
#include <cuda.h>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"
#include "exl3_tcgen05.cuh"

namespace exl3 {

namespace {

constexpr int kUnit = 32;         // tokens
constexpr int kMaxSeqs = 1024;    // sequences of one launch
// What a warp spends on entering a segment (queries, page numbers and scales of
// another head), in units: counted as that many units of no tokens in front of
// each segment, so that ranges of many short sequences are not longer than the
// others. 16 sequences of 61 to 8192 tokens: the slowest CTA 82K cycles of 59K on
// average without it.
constexpr int kEntry = 3;

// NT x 8 rows. 8 rows leave room for 12 warps an SM (168 registers a
// thread), 16 rows for 8; the kernel is bound by the latency of dependent
// instructions until there are about 12.
template <int D, int NT, bool WEIGH>
struct StreamCfg {
  static constexpr int kWarps = NT == 1 ? 12 : 8, kThreads = 32 * kWarps;
  static constexpr int kHalf = kUnit * D;                     // bytes of a unit's keys (or values)
  static constexpr int kStage = WEIGH ? kHalf : 2 * kHalf;
  static constexpr int kStages = 192 * 1024 / kWarps / kStage;  // 192 KB of copies in flight per SM
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kOffPlan = kRing;
  static constexpr int kOffBar = kOffPlan + (kMaxSeqs + 32) * 8 + (kMaxSeqs + 8) * 8;
  static constexpr int kSmem = 1024 + kOffBar + kWarps * kStages * 8;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct StreamParams {
  KvAttention a;
  int group;      // query heads of a key/value head
  // Workspace: partial results of the CTAs (slot 0: a segment that began before
  // the CTA's range, slot 1: one that began in it and goes on after it), and the
  // plan for the join.
  float *part_o;      // CTAs x 2 x rows x D
  float *part_ml;     // CTAs x 2 x rows x 2 (maximum in log2 units, sum)
  float *first;       // warps x rows x (D + 2): see Parts
  int64_t *plan;      // prefix of build_plan
  int warps;          // of the stream grid
  int64_t part_rows;  // 2 * CTAs * rows
};

__device__ __forceinline__ int units_of(int len) { return (len + kUnit - 1) / kUnit; }

// The sequences of a launch in shared memory.
struct Plan {
  int64_t *prefix;  // kMaxSeqs + 1: units (with those of entering) of all sequences before each; then scratch
  int2 *seq;        // kMaxSeqs + 1: first row and length of each sequence (length -1: not to be served)
  __device__ __forceinline__ KvSeq at(int s) const {
    const int2 a = seq[s];
    return KvSeq{a.x, a.y < 0 ? 0 : seq[s + 1].x - a.x, a.y < 0 ? 0 : a.y};
  }
};

__device__ __forceinline__ int64_t segment_units(int len) { return len > 0 ? units_of(len) + kEntry : 0; }

// Tiles of `tile` rows that a sequence's rows make.
template <bool TILED>
__device__ __forceinline__ int row_tiles(int rows, int group, int tile) {
  return TILED ? (rows * group + tile - 1) / tile : 1;
}

// Every thread of the CTA takes part; ends with a barrier.
template <bool TILED>
__device__ __forceinline__ void build_plan(const KvView &kv, int group, int tile, const Plan &plan) {
  int64_t *warp_sum = plan.prefix + kMaxSeqs + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  int64_t carry = 0;
  if (threadIdx.x == 0) plan.prefix[0] = 0;
  for (int c = 0; c < kv.n_seqs; c += blockDim.x) {
    const int s = c + (int)threadIdx.x;
    int64_t n = 0;
    if (s < kv.n_seqs) {
      const KvSeq q = kv_sequence(kv, s);
      if (q.rows > 0) n = segment_units(q.len) * kv.n_kv_heads * row_tiles<TILED>(q.rows, group, tile);
      plan.seq[s] = make_int2(kv.q_start[s], q.rows > 0 ? q.len : -1);
      if (s + 1 == kv.n_seqs) plan.seq[s + 1] = make_int2(kv.q_start[s + 1], -1);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += o;
    }
    if (lane == 31) warp_sum[warp] = n;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < nwarps; ++w) {
      const int64_t x = warp_sum[w];
      if (w < warp) n += x;
      total += x;
    }
    if (s < kv.n_seqs) plan.prefix[s + 1] = carry + n;
    carry += total;
    __syncthreads();
  }
  __syncthreads();
}

// A place in the unit order; u < 0: entering the segment.
struct Cursor {
  KvSeq q;
  int s, h, rt, u;    // sequence, key/value head, row tile, unit of the segment
  int units, tiles;   // of this sequence's segments
};
template <bool TILED>
__device__ __forceinline__ void enter_sequence(const Plan &plan, int group, int tile, Cursor &c) {
  c.q = plan.at(c.s);
  c.units = units_of(c.q.len);
  c.tiles = row_tiles<TILED>(c.q.rows, group, tile);
}
template <bool TILED>
__device__ __forceinline__ Cursor locate(const KvView &kv, int group, int tile, const Plan &plan, int64_t z) {
  Cursor c;
  int lo = 0, hi = kv.n_seqs - 1;  // the s with prefix[s] <= z < prefix[s + 1]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (plan.prefix[mid + 1] > z) hi = mid;
    else lo = mid + 1;
  }
  c.s = lo;
  enter_sequence<TILED>(plan, group, tile, c);
  const int64_t rem = z - plan.prefix[lo];
  const int seg = rem < ((int64_t)1 << 31) ? (int)((uint32_t)rem / (uint32_t)(c.units + kEntry)) : (int)(rem / (c.units + kEntry));
  c.u = (int)(rem - (int64_t)seg * (c.units + kEntry)) - kEntry;
  c.h = TILED ? seg / c.tiles : seg;
  c.rt = TILED ? seg - c.h * c.tiles : 0;
  return c;
}
// The next place; z moves with it.
template <bool TILED>
__device__ __forceinline__ void advance(const KvView &kv, int group, int tile, const Plan &plan, Cursor &c, int64_t &z) {
  ++z;
  if (++c.u < c.units) return;
  c.u = -kEntry;
  if (TILED) {
    if (++c.rt < c.tiles) return;
    c.rt = 0;
  }
  if (++c.h < kv.n_kv_heads) return;
  c.h = 0;
  do ++c.s;
  while (c.s < kv.n_seqs && plan.prefix[c.s + 1] == plan.prefix[c.s]);
  if (c.s < kv.n_seqs) enter_sequence<TILED>(plan, group, tile, c);
}
// Past the places of entering.
__device__ __forceinline__ void skip_entry(Cursor &c, int64_t &z) {
  if (c.u < 0) {
    z -= c.u;
    c.u = 0;
  }
}

// Page numbers and scales of 32 consecutive blocks of one (sequence, head), one
// block a lane.
struct Blocks {
  int s = -1, h = -1, base = 0;
  int page = -1;
  float ks = 0.f, vs = 0.f;
  __device__ __forceinline__ bool holds(const Cursor &c) const {
    const int b = c.u >> 1;
    return c.s == s && c.h == h && b >= base && b < base + 32;
  }
  template <bool WEIGH>
  __device__ __forceinline__ void load(const KvView &kv, const Cursor &c, int lane) {
    s = c.s;
    h = c.h;
    base = c.u >> 1;
    page = -1;
    ks = 0.f;
    vs = 0.f;
    const int b = base + lane;
    if (b * 2 < c.units) page = kv_page(kv, s, b);
    if (page >= 0) {
      const int64_t slab = (int64_t)page * kv.n_kv_heads + h;
      ks = kv.k_scale[slab];
      if (!WEIGH) vs = kv.v_scale[slab];
    }
  }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t lo_codes(uint32_t w) { return e4m3x2_to_half2((uint16_t)(w & 0xFFFFu)); }
__device__ __forceinline__ uint32_t hi_codes(uint32_t w) { return e4m3x2_to_half2((uint16_t)(w >> 16)); }

// Address of 16-byte piece c of token row r in a copied tile (128-byte swizzle
// for 128-byte rows, 64-byte swizzle for 64-byte rows).
template <int D>
__device__ __forceinline__ uint32_t piece(uint32_t base, int r, int c) {
  return D == 128 ? base + r * 128 + ((c ^ (r & 7)) << 4) : base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
template <int W>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t *w) {
  if (!EXL3_SMEM(addr, 4 * W)) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    return;
  }
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// The B operand of S^T: this lane's D / 4 elements of row j (from lane / 4).
template <int D>
__device__ __forceinline__ void load_query(const StreamParams &p, const Cursor &c, int j, int lane, uint32_t (&qf)[D / 8]) {
  const int t = lane & 3;
  const int i = j / p.group;
#pragma unroll
  for (int k = 0; k < D / 8; ++k) qf[k] = 0;
  if (i >= c.q.rows) return;
  const int64_t off = (int64_t)(c.q.row0 + i) * p.a.ldq + (int64_t)(c.h * p.group + j - i * p.group) * D + t * (D / 4);
  const __half *q = static_cast<const __half *>(p.a.q) + off;
#pragma unroll
  for (int k = 0; k < D / 32; ++k)
    if (EXL3_SPAN(off + 8 * k, 8, (int64_t)(p.a.kv.rows - 1) * p.a.ldq + (int64_t)p.a.n_heads * D)) {
      const uint4 v = reinterpret_cast<const uint4 *>(q)[k];
      qf[4 * k] = v.x;
      qf[4 * k + 1] = v.y;
      qf[4 * k + 2] = v.z;
      qf[4 * k + 3] = v.w;
    }
}

// Tokens that row j of a segment sees: 0 for rows past the last.
__device__ __forceinline__ int row_limit(const StreamParams &p, const Cursor &c, int j) {
  const int i = j / p.group;
  if (i >= c.q.rows) return 0;
  return p.a.causal ? c.q.len - c.q.rows + i + 1 : c.q.len;
}

// The keys of a unit: word j of w[mi][r] holds the A operands of k-step j for
// token 16 mi + 8 r + lane / 4.
template <int D>
__device__ __forceinline__ void load_keys(uint32_t base, int lane, uint32_t (&w)[2][2][D / 16]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) lds<4>(piece<D>(base, 16 * mi + 8 * r + g, (D / 64) * t + x), &w[mi][r][4 * x]);
}

// S^T of a unit for NT x 8 rows; the chains of the two 16-token halves and
// of even and odd k-steps are independent.
template <int D, int NT>
__device__ __forceinline__ void score_products(const uint32_t (&w)[2][2][D / 16], const uint32_t (&qf)[NT][D / 8],
                                               float (&s)[NT][2][4]) {
  float odd[NT][2][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][mi][k] = odd[n][mi][k] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      const uint32_t a0 = lo_codes(w[mi][0][j]), a1 = lo_codes(w[mi][1][j]);
      const uint32_t a2 = hi_codes(w[mi][0][j]), a3 = hi_codes(w[mi][1][j]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_16816(j & 1 ? odd[n][mi] : s[n][mi], a0, a1, a2, a3, qf[n][2 * j], qf[n][2 * j + 1]);
    }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][mi][k] += odd[n][mi][k];
}

// Scores of two products in log2 units. c: key scale * softmax scale * log2 e.
template <bool CAP>
__device__ __forceinline__ float2 score(float acc0, float acc1, float c, const SoftCap &cap) {
  const float2 s = mul2(make_float2(acc0, acc1), make_float2(c, c));
  if constexpr (CAP) return cap(s);
  return s;
}

// A warp's ring of copies: issues the keys (and values) of units in order.
template <int D, int NT, bool WEIGH>
struct Ring {
  using Cfg = StreamCfg<D, NT, WEIGH>;
  uint32_t base, bars;
  int put = 0, get = 0;
  uint32_t get_phase = 0;
  int in_flight = 0;

  __device__ __forceinline__ void issue(const CUtensorMap *tk, const CUtensorMap *tv, const KvView &kv, const Cursor &c,
                                        int page, int lane) {
    if (lane == 0) {
      const uint32_t bar = bars + 8 * put, dst = base + put * Cfg::kStage;
      const int64_t row = ((int64_t)max(page, 0) * kv.n_kv_heads + c.h) * kKvBlock + (c.u & 1) * kUnit;
      // a page that the table does not name: nothing is copied, the consumer skips the unit
      const bool ok = page >= 0 && EXL3_SPAN(row, kUnit, kv.n_pages * kv.n_kv_heads * kKvBlock) &&
                      EXL3_SMEM(dst, Cfg::kStage) && EXL3_SMEM(bar, 8);
      mbar_arrive_expect_tx(bar, ok ? Cfg::kStage : 0);
      if (ok) {
        tma_load_2d(dst, tk, bar, 0, (int)row);
        if (!WEIGH) tma_load_2d(dst + Cfg::kHalf, tv, bar, 0, (int)row);
      }
    }
    if (++put == Cfg::kStages) put = 0;
    ++in_flight;
  }
  __device__ __forceinline__ uint32_t stage() const { return base + get * Cfg::kStage; }
  __device__ __forceinline__ bool wait(int *status) {
    return __all_sync(0xffffffffu, mbar_wait(bars + 8 * get, get_phase, status));
  }
  __device__ __forceinline__ void next() {
    if (++get == Cfg::kStages) {
      get = 0;
      get_phase ^= 1u;
    }
    --in_flight;
  }
  // After a wait that ran out: the copies still in flight land before the CTA leaves.
  __device__ __forceinline__ void drain() {
    while (in_flight > 0) {
      mbar_wait_short(bars + 8 * get, get_phase);
      next();
    }
  }
};

// The probabilities' scale in fp16: a row's many small ones keep their bits (one of
// 2^-28 of the largest still has all 11; fp16 ends 2^-39 below it).
constexpr float kHeadroom = 0x1p14f;

template <int D, int NT>
struct RowState {
  float o[NT][D / 16][4];  // O^T in units of 2^e_v / kHeadroom: d by lane / 4, rows 2 t, 2 t + 1
  float m[NT][2], l[NT][2];
  int ev;                  // exponent of the value scale that o is in units of
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    ev = 0;
  }
};

// One unit: scores, running maximum and sum, O^T += V^T P^T.
template <int D, int NT, bool CAP>
__device__ __forceinline__ void attend_unit(const StreamParams &p, uint32_t stage, int pos0, int len, float ks, float vs,
                                            const uint32_t (&qf)[NT][D / 8], const int (&limit)[NT][2], int min_limit,
                                            const SoftCap &cap, int lane, RowState<D, NT> &st) {
  const int g = lane >> 2, t = lane & 3;
  float s[NT][2][4];
  {
    uint32_t w[2][2][D / 16];
    load_keys<D>(stage, lane, w);
    score_products<D, NT>(w, qf, s);
  }
  const float c = ks * p.a.scale * kLog2e;
  const bool masked = pos0 + kUnit > min_limit;  // some row does not see the whole unit
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float2 x = score<CAP>(s[n][mi][k], s[n][mi][k + 1], c, cap);
        const int pos = pos0 + 16 * mi + g + 4 * k;
        s[n][mi][k] = masked && pos >= limit[n][0] ? -INFINITY : x.x;
        s[n][mi][k + 1] = masked && pos >= limit[n][1] ? -INFINITY : x.y;
      }
  const int ev = pow2_exponent(vs);
  const float unit = pow2i(max(min(st.ev - ev, 127), -126));  // exact: O in the new unit
  uint32_t b[NT][2][2];
  float alpha[NT][2];
  bool still = ev == st.ev;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      float top = fmaxf(fmaxf(s[n][0][col], s[n][0][2 + col]), fmaxf(s[n][1][col], s[n][1][2 + col]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float now = fmaxf(st.m[n][col], top);
      const float ref = now == -INFINITY ? 0.f : now;
      const float keep = ex2(st.m[n][col] - ref);
      still = still && (keep == 1.0f || st.m[n][col] == -INFINITY);
      float sum = 0.f;
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float e = ex2(s[n][mi][2 * r + col] - ref);
          s[n][mi][2 * r + col] = e;
          sum += e;
        }
      st.m[n][col] = now;
      st.l[n][col] = st.l[n][col] * keep + sum;
      alpha[n][col] = keep * unit;
    }
    // fp16 probabilities times kHeadroom: relative error 2^-12 on average, the size of the result's own rounding
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 scaled = mul2(make_float2(s[n][mi][2 * r], s[n][mi][2 * r + 1]), make_float2(kHeadroom, kHeadroom));
        const __half2 h = __floats2half2_rn(scaled.x, scaled.y);
        b[n][mi][r] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&h));
      }
  }
  if (!__all_sync(0xffffffffu, still)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[n][i][k] *= alpha[n][k & 1];
    st.ev = ev;
  }
  const bool tail = pos0 + kUnit > len;
#pragma unroll
  for (int mi = 0; mi < 2; ++mi) {
    constexpr int W = D / 32;  // words of a lane's piece of a token
    uint32_t v[4][W];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * mi + 2 * t + (r & 1) + 8 * (r >> 1);
      if constexpr (D == 128) lds<4>(piece<D>(stage + kUnit * D, tok, g), v[r]);
      else lds<2>(piece<D>(stage + kUnit * D, tok, g >> 1) + (g & 1) * 8, v[r]);
      if (tail && pos0 + tok >= len) {  // whatever lies past the length (a NaN times 0 is a NaN)
#pragma unroll
        for (int w = 0; w < W; ++w) v[r][w] = 0;
      }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t x = __byte_perm(v[0][w], v[1][w], 0x5140), y = __byte_perm(v[2][w], v[3][w], 0x5140);
      const uint32_t z = __byte_perm(v[0][w], v[1][w], 0x7362), u = __byte_perm(v[2][w], v[3][w], 0x7362);
      const uint32_t a0 = lo_codes(x), a1 = hi_codes(x), a2 = lo_codes(y), a3 = hi_codes(y);
      const uint32_t c0 = lo_codes(z), c1 = hi_codes(z), c2 = lo_codes(u), c3 = hi_codes(u);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816(st.o[n][2 * w], a0, a1, a2, a3, b[n][mi][0], b[n][mi][1]);
        mma_16816(st.o[n][2 * w + 1], c0, c1, c2, c3, b[n][mi][0], b[n][mi][1]);
      }
    }
  }
}

// Writes a finished row's D / 8 consecutive outputs of this lane.
template <int D>
__device__ __forceinline__ void store_out(const KvAttention &a, int64_t row, int head, int d0, const float (&v)[D / 8]) {
  const int64_t off = row * a.ldo + (int64_t)head * D + d0;
  if (!EXL3_SPAN(off, D / 8, (int64_t)(a.kv.rows - 1) * a.ldo + (int64_t)a.n_heads * D)) return;
  __half *out = static_cast<__half *>(a.out) + off;
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint4 *>(out)[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Parts of segments that a CTA's warps do not cover alone, two a warp: 2 w, the
// end of a segment that began before the warp's range (in the workspace), and
// 2 w + 1, its last segment (in shared memory, the ring's).
struct Part {
  int s, h, rt;  // the segment; s < 0: no part
  int begins, ends;
};
template <int D, int NT>
struct Parts {
  using Cfg = StreamCfg<D, NT, false>;
  static constexpr int kWarps = Cfg::kWarps;
  static constexpr int kRows = 8 * NT;
  static constexpr int kFloats = kRows * (D + 2);  // output, then (maximum, sum) of each row
  static constexpr int kHeads = kWarps * kFloats * 4;
  static_assert(kHeads + 2 * kWarps * (int)sizeof(Part) <= Cfg::kRing, "parts fit the ring");
  uint8_t *smem;
  float *first;  // workspace: CTAs x warps x kFloats
  __device__ __forceinline__ float *o(int i) const {
    return i & 1 ? reinterpret_cast<float *>(smem) + (i >> 1) * kFloats
                 : first + ((int64_t)blockIdx.x * kWarps + (i >> 1)) * kFloats;
  }
  __device__ __forceinline__ float2 *ml(int i) const { return reinterpret_cast<float2 *>(o(i) + kRows * D); }
  __device__ __forceinline__ Part *head(int i) const { return reinterpret_cast<Part *>(smem + kHeads) + i; }
};

// The sum of each row over the lanes that share it.
template <int D, int NT>
__device__ __forceinline__ void close_rows(RowState<D, NT> &st) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      float l = st.l[n][col];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      st.l[n][col] = l;
    }
}

// The result of a segment that one warp worked on alone.
template <int D, int NT>
__device__ __forceinline__ void write_rows(const StreamParams &p, const Cursor &c, int lane, const RowState<D, NT> &st) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      const float l = st.l[n][col], f = l == 0.f ? 0.f : pow2i(st.ev) / kHeadroom / l;
      const int j = c.rt * 8 * NT + 8 * n + 2 * t + col, i = j / p.group;
      if (i >= c.q.rows) continue;
      float v[D / 8];
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        v[2 * k] = st.o[n][k][col] * f;
        v[2 * k + 1] = st.o[n][k][2 + col] * f;
      }
      const int head = c.h * p.group + j - i * p.group;
      store_out<D>(p.a, c.q.row0 + i, head, g * (D / 8), v);
      if (p.a.lse && g == 0) p.a.lse[(int64_t)(c.q.row0 + i) * p.a.n_heads + head] = log_sum(st.m[n][col], l);
    }
}

template <int D, int NT>
__device__ __forceinline__ void keep_part(float *part_o, float2 *part_ml, int lane, const RowState<D, NT> &st) {
  const int g = lane >> 2, t = lane & 3;
  const float unit = pow2i(st.ev) / kHeadroom;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      const int r = 8 * n + 2 * t + col;
      float4 *o = reinterpret_cast<float4 *>(part_o + r * D + g * (D / 8));
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        o[k] = make_float4(st.o[n][2 * k][col] * unit, st.o[n][2 * k][2 + col] * unit, st.o[n][2 * k + 1][col] * unit,
                           st.o[n][2 * k + 1][2 + col] * unit);
      if (g == 0) part_ml[r] = make_float2(st.m[n][col], st.l[n][col]);
    }
}

// Joins the CTA's parts, in order. Every thread has four columns of some rows.
template <int D, int NT>
__device__ __forceinline__ void join_cta(const StreamParams &p, const Parts<D, NT> &parts) {
  using P = Parts<D, NT>;
  constexpr int kWarps = P::kWarps;
  constexpr int kPerRow = D / 4, kStep = P::Cfg::kThreads / kPerRow;  // threads of a row, rows at a time
  const int d0 = threadIdx.x % kPerRow * 4, lane = threadIdx.x & 31;
  static_assert(2 * kWarps <= 32, "a bit for each part");
  const uint32_t valid = __ballot_sync(0xffffffffu, lane < 2 * kWarps && parts.head(lane < 2 * kWarps ? lane : 0)->s >= 0);
  for (int r = threadIdx.x / kPerRow; r < P::kRows; r += kStep) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool begins = false;
    for (uint32_t left = valid; left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const Part part = *parts.head(i);
      const float2 ml = parts.ml(i)[r];
      const float4 x = *reinterpret_cast<const float4 *>(parts.o(i) + r * D + d0);
      const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
      const float a = ex2(m - ref), b = ex2(ml.x - ref);
      m = top;
      l = l * a + ml.y * b;
      o = make_float4(o.x * a + x.x * b, o.y * a + x.y * b, o.z * a + x.z * b, o.w * a + x.w * b);
      begins = begins || part.begins;
      // the segment's last part in this CTA: it ends, or no other part follows
      const bool last = part.ends || (left & (left - 1)) == 0;
      if (!last) continue;
      const KvSeq q = kv_sequence(p.a.kv, part.s);
      const int j = part.rt * P::kRows + r, row = j / p.group;
      if (row < q.rows) {
        if (begins && part.ends) {
          const int head = part.h * p.group + j - row * p.group;
          const int64_t off = (int64_t)(q.row0 + row) * p.a.ldo + (int64_t)head * D + d0;
          const float f = l == 0.f ? 0.f : 1.0f / l;
          const __half2 lo = __floats2half2_rn(o.x * f, o.y * f), hi = __floats2half2_rn(o.z * f, o.w * f);
          if (EXL3_SPAN(off, 4, (int64_t)(p.a.kv.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D))
            *reinterpret_cast<uint2 *>(static_cast<__half *>(p.a.out) + off) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
          if (p.a.lse && d0 == 0) p.a.lse[(int64_t)(q.row0 + row) * p.a.n_heads + head] = log_sum(m, l);
        } else {
          const int64_t at = (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * P::kRows + r;
          if (EXL3_SPAN(at, 1, p.part_rows)) {
            *reinterpret_cast<float4 *>(p.part_o + at * D + d0) = o;
            if (d0 == 0) reinterpret_cast<float2 *>(p.part_ml)[at] = make_float2(m, l);
          }
        }
      }
      m = -INFINITY;
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      begins = false;
    }
  }
}

template <int D, int NT, bool CAP, bool TILED>
__global__ void __launch_bounds__(StreamCfg<D, NT, false>::kThreads, 1)
    kv8_stream_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const StreamParams p) {
  using Cfg = StreamCfg<D, NT, false>;
  constexpr int kWarps = Cfg::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const KvView &kv = p.a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Plan plan{reinterpret_cast<int64_t *>(smem + Cfg::kOffPlan), reinterpret_cast<int2 *>(smem + Cfg::kOffPlan + (kMaxSeqs + 32) * 8)};
  Ring<D, NT, false> ring;
  ring.base = smem_u32(smem) + warp * Cfg::kStages * Cfg::kStage;
  ring.bars = smem_u32(smem + Cfg::kOffBar) + warp * Cfg::kStages * 8;
  if (lane == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) mbar_init(ring.bars + 8 * i, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&tk);
    prefetch_tensor_map(&tv);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int tile = 8 * NT;
  build_plan<TILED>(kv, p.group, tile, plan);
  const int64_t T = plan.prefix[kv.n_seqs], W = min((int64_t)p.warps, T);
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= kv.n_seqs; i += Cfg::kThreads) p.plan[i] = plan.prefix[i];
  if ((int64_t)blockIdx.x * kWarps >= W) return;
  const Parts<D, NT> parts{smem, p.first};
  Part first{-1}, last{-1};  // this warp's parts of segments that it does not cover
  RowState<D, NT> st;
  if (w < W) {
    int64_t z = range_start(w, W, T);
    const int64_t z1 = range_start(w + 1, W, T);
    Cursor c = locate<TILED>(kv, p.group, tile, plan, z);
    skip_entry(c, z);
    int64_t zp = z;
    Cursor cp = c;
    Blocks ahead, now;
    const SoftCap cap(p.a.softcap, kLog2e);
    uint32_t qf[NT][D / 8];
    int limit[NT][2], min_limit = 0;  // tokens that this lane's rows see, and the first row
    bool fresh = true, began = false;
    while (z < z1) {
      if (fresh) {  // first: on their way while the page numbers are
        fresh = false;
        began = c.u == 0;
        const int j0 = TILED ? c.rt * tile : 0;
        st.clear();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          load_query<D>(p, c, j0 + 8 * n + (lane >> 2), lane, qf[n]);
          limit[n][0] = row_limit(p, c, j0 + 8 * n + 2 * (lane & 3));
          limit[n][1] = row_limit(p, c, j0 + 8 * n + 2 * (lane & 3) + 1);
        }
        min_limit = row_limit(p, c, j0);  // rows come in order: the first sees the least
      }
      while (zp < z1 && ring.in_flight < Cfg::kStages) {
        if (!ahead.holds(cp)) ahead.load<false>(kv, cp, lane);
        ring.issue(&tk, &tv, kv, cp, __shfl_sync(0xffffffffu, ahead.page, (cp.u >> 1) - ahead.base), lane);
        advance<TILED>(kv, p.group, tile, plan, cp, zp);
        skip_entry(cp, zp);
      }
      if (!now.holds(c)) {
        if (ahead.holds(c)) now = ahead;
        else now.load<false>(kv, c, lane);
      }
      if (!ring.wait(kv.status)) {
        ring.drain();  // the call's outputs are undefined: the error word says so
        break;
      }
      const int at = (c.u >> 1) - now.base;
      const int page = __shfl_sync(0xffffffffu, now.page, at);
      const float ks = __shfl_sync(0xffffffffu, now.ks, at), vs = __shfl_sync(0xffffffffu, now.vs, at);
      if (page >= 0)
        attend_unit<D, NT, CAP>(p, ring.stage(), c.u * kUnit, c.q.len, ks, vs, qf, limit, min_limit, cap, lane, st);
      __syncwarp();  // every lane is done with the stage before it is filled again
      ring.next();
      const bool end = c.u + 1 == c.units;
      const bool done = z + 1 == z1 || (end && z + 1 + kEntry >= z1);  // no unit of the range is left
      if (end || done) {
        close_rows<D, NT>(st);
        if (end && began) {
          write_rows<D, NT>(p, c, lane, st);
        } else if (done) {
          last = Part{c.s, c.h, c.rt, began, end};
          break;  // kept in registers
        } else {
          // the end of a segment that began before this range: the first part of
          // a range only, and the ring is in use, so it goes to the workspace
          first = Part{c.s, c.h, c.rt, false, true};
          keep_part<D, NT>(parts.o(2 * warp), parts.ml(2 * warp), lane, st);
        }
        fresh = true;
      }
      advance<TILED>(kv, p.group, tile, plan, c, z);
      skip_entry(c, z);
    }
  }
  __syncthreads();  // no warp uses its ring any more
  if (lane == 0) {
    *parts.head(2 * warp) = first;
    *parts.head(2 * warp + 1) = last;
  }
  if (last.s >= 0) keep_part<D, NT>(parts.o(2 * warp + 1), parts.ml(2 * warp + 1), lane, st);
  __syncthreads();
  join_cta<D, NT>(p, parts);
}

// Joins the partials of the segments that several CTAs worked on, in the order of
// the CTAs, and writes the rows of segments without tokens. One CTA of G x D threads
// per (row of a group, sequence, key/value head).
template <int D, int NT, bool TILED, int G>
__global__ void __launch_bounds__(D * G) kv8_join_kernel(const StreamParams p) {
  const KvView &kv = p.a.kv;
  constexpr int kRows = 8 * NT, kWarps = StreamCfg<D, NT, false>::kWarps;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.y, h = blockIdx.z, j = blockIdx.x, i = j / p.group;
  const int d = threadIdx.x % D, g = threadIdx.x / D;
  const int64_t z0 = p.plan[s], units_s = p.plan[s + 1] - z0, T = p.plan[kv.n_seqs], W = min((int64_t)p.warps, T);
  const KvSeq q = kv_sequence(kv, s);
  if (i >= q.rows) return;
  const int head = h * p.group + j - i * p.group;
  float m = -INFINITY, l = 0.f, o = 0.f;
  if (units_s > 0) {
    const int units = units_of(q.len);
    const int tiles = row_tiles<TILED>(q.rows, p.group, kRows);
    const int64_t z = z0 + ((int64_t)h * tiles + (TILED ? j / kRows : 0)) * (units + kEntry) + kEntry;
    const int64_t c0 = range_owner(z, W, T) / kWarps, c1 = range_owner(z + units - 1, W, T) / kWarps;
    if (c0 == c1) return;  // the CTA wrote the result
    const int64_t share = (c1 - c0 + G) / G, first = c0 + g * share, last = min(c1, first + share - 1);
#pragma unroll 4
    for (int64_t c = first; c <= last; ++c) {
      const int64_t at = (2 * c + (c == c0 ? 1 : 0)) * kRows + (TILED ? j % kRows : j);
      if (!EXL3_SPAN(at, 1, p.part_rows)) continue;
      const float2 ml = reinterpret_cast<const float2 *>(p.part_ml)[at];
      const float x = p.part_o[at * D + d];
      const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
      const float a = ex2(m - ref), b = ex2(ml.x - ref);
      l = l * a + ml.y * b;
      o = o * a + x * b;
      m = top;
    }
  }
  if constexpr (G > 1) {  // the groups' results, in their order
    __shared__ float so[G][D], sm[G], sl[G];
    so[g][d] = o;
    if (d == 0) {
      sm[g] = m;
      sl[g] = l;
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 1; k < G; ++k) {
      const float top = fmaxf(m, sm[k]), ref = top == -INFINITY ? 0.f : top;
      const float a = ex2(m - ref), b = ex2(sm[k] - ref);
      l = l * a + sl[k] * b;
      o = o * a + so[k][d] * b;
      m = top;
    }
  }
  const int64_t row = q.row0 + i, off = row * p.a.ldo + (int64_t)head * D + d;
  if (EXL3_SPAN(off, 1, (int64_t)(kv.rows - 1) * p.a.ldo + (int64_t)p.a.n_heads * D))
    static_cast<__half *>(p.a.out)[off] = __float2half_rn(l == 0.f ? 0.f : o / l);
  if (p.a.lse && threadIdx.x == 0) p.a.lse[row * p.a.n_heads + head] = log_sum(m, l);
}

// Accumulated weight: the same stream over the keys alone; a unit's weights are
// the sums over all rows of the sequence, formed by the warp that owns the unit.
// 16 sequences of 61 to 8192 tokens, 40 heads on 8, D = 128: 20 us (72 MB, 3.6 TB/s;
// bound as the attention is, and the shorter the stream the larger the share of its
// beginning and end).
template <int D, bool CAP>
__global__ void __launch_bounds__(StreamCfg<D, 1, true>::kThreads, 1)
    kv8_weigh_kernel(const __grid_constant__ CUtensorMap tk, const StreamParams p) {
  using Cfg = StreamCfg<D, 1, true>;
  constexpr int kWarps = Cfg::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const KvView &kv = p.a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Plan plan{reinterpret_cast<int64_t *>(smem + Cfg::kOffPlan), reinterpret_cast<int2 *>(smem + Cfg::kOffPlan + (kMaxSeqs + 32) * 8)};
  Ring<D, 1, true> ring;
  ring.base = smem_u32(smem) + warp * Cfg::kStages * Cfg::kStage;
  ring.bars = smem_u32(smem + Cfg::kOffBar) + warp * Cfg::kStages * 8;
  if (lane == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) mbar_init(ring.bars + 8 * i, 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) prefetch_tensor_map(&tk);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  build_plan<false>(kv, p.group, 0, plan);
  const int64_t T = plan.prefix[kv.n_seqs], W = min((int64_t)p.warps, T);
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  if (w >= W) return;
  int64_t z = range_start(w, W, T);
  const int64_t z1 = range_start(w + 1, W, T);
  Cursor c = locate<false>(kv, p.group, 0, plan, z);
  skip_entry(c, z);
  int64_t zp = z;
  Cursor cp = c;
  Blocks ahead, now;
  const SoftCap cap(p.a.softcap, kLog2e);
  uint32_t qf[1][D / 8];
  int limit[2];
  float lse[2];  // in log2 units
  int held_s = -1, held_h = -1, held_j = -1;
  // The queries, limits and lse of the 8 rows from j0 on, unless they are held.
  auto hold = [&](int j0) {
    if (held_s == c.s && held_h == c.h && held_j == j0) return;
    held_s = c.s;
    held_h = c.h;
    held_j = j0;
    load_query<D>(p, c, j0 + g, lane, qf[0]);
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      const int j = j0 + 2 * t + col, i = j / p.group;
      limit[col] = row_limit(p, c, j);
      lse[col] = limit[col] > 0 ? p.a.lse[(int64_t)(c.q.row0 + i) * p.a.n_heads + c.h * p.group + j - i * p.group] : 0.f;
      if (lse[col] == -INFINITY) limit[col] = 0;
      lse[col] *= kLog2e;
    }
  };
  // The first row that sees a token of the cursor's unit.
  auto first_row = [&]() { return p.a.causal ? max(0, c.u * kUnit - (c.q.len - c.q.rows)) * p.group : 0; };

  while (z < z1) {
    if (held_s != c.s || held_h != c.h) hold(first_row() & ~7);  // on their way while the page numbers are
    while (zp < z1 && ring.in_flight < Cfg::kStages) {
      if (!ahead.holds(cp)) ahead.load<true>(kv, cp, lane);
      ring.issue(&tk, nullptr, kv, cp, __shfl_sync(0xffffffffu, ahead.page, (cp.u >> 1) - ahead.base), lane);
      advance<false>(kv, p.group, 0, plan, cp, zp);
      skip_entry(cp, zp);
    }
    if (!now.holds(c)) {
      if (ahead.holds(c)) now = ahead;
      else now.load<true>(kv, c, lane);
    }
    if (!ring.wait(kv.status)) {
      ring.drain();
      return;
    }
    const int at = (c.u >> 1) - now.base;
    const int page = __shfl_sync(0xffffffffu, now.page, at);
    const float ks = __shfl_sync(0xffffffffu, now.ks, at) * p.a.scale * kLog2e;
    if (page >= 0) {
      uint32_t words[2][2][D / 16];
      load_keys<D>(ring.stage(), lane, words);
      const int pos0 = c.u * kUnit, J = c.q.rows * p.group;
      const int first = first_row();
      float sum[2][2] = {};
      for (int j0 = first & ~7; j0 < J; j0 += 8) {
        hold(j0);
        float s[1][2][4];
        score_products<D, 1>(words, qf, s);
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float2 x = score<CAP>(s[0][mi][k], s[0][mi][k + 1], ks, cap);
            const int pos = pos0 + 16 * mi + g + 4 * k;
            if (pos < limit[0]) sum[mi][k >> 1] += ex2(x.x - lse[0]);
            if (pos < limit[1]) sum[mi][k >> 1] += ex2(x.y - lse[1]);
          }
      }
      const int64_t slab = (int64_t)page * kv.n_kv_heads + c.h;
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = sum[mi][r];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          const int tok = 16 * mi + g + 8 * r;
          const int64_t off = slab * kKvBlock + (c.u & 1) * kUnit + tok;
          if (t == 0 && pos0 + tok < c.q.len && EXL3_SPAN(off, 1, kv.n_pages * kv.n_kv_heads * kKvBlock))
            atomicAdd(&kv.weight[off], x);  // alone but for sequences that share the block; no wait for the old value
        }
    }
    __syncwarp();
    ring.next();
    advance<false>(kv, p.group, 0, plan, c, z);
    skip_entry(c, z);
  }
}

// Rows of a (sequence, head) up to which the stream kernels take a call; more go to
// the tensor-core kernels of exl3_kv8_chunk.cu and exl3_kv8_weigh_chunk.cu, whose time
// hardly depends on the rows below 128. Attention, one tile of 16 rows after another,
// 5 heads a group: 16 sequences of up to 8192 tokens 69 / 85 / 109 / 123 us at 20 / 45 /
// 50 / 65 rows (there 103), one of 60000 tokens 60 / 81 / 99 / 121 (there 95), one of
// 777 tokens 15.5 (there 16.3). Weights, the rows 8 at a time over a unit's
// keys in registers: 34 / 63 / 102 / 148 us at 20 / 50 / 100 / 160 rows for the 16 (there
// 127 to 131), 31 / 53 / 91 / 135 for the one (there 108 to 121).
constexpr int64_t kStreamRows = 48, kWeighRows = 112;

// Up to 8 rows of a (sequence, head): half the registers and products of 16 (5 rows
// over 16 sequences 35.6 us, 41.8 in the form of 16; one of 777 tokens 12.1 and 13.6).
bool narrow(int64_t rows) { return rows <= 8; }

template <int D>
bool cache_map(CUtensorMap *m, const KvView &kv, const uint8_t *codes) {
  const uint64_t rows = (uint64_t)kv.n_pages * kv.n_kv_heads * kKvBlock;
  return encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, D, rows, D, D, kUnit,
                              D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, int NT, bool TILED>
cudaError_t run_stream(const CUtensorMap &tk, const CUtensorMap &tv, const StreamParams &params, cudaStream_t st) {
  using Cfg = StreamCfg<D, NT, false>;
  StreamParams p = params;
  const int grid = p.a.num_sms, kThreads = Cfg::kThreads;
  p.warps = grid * Cfg::kWarps;
  const size_t smem = Cfg::kSmem;
  const cudaError_t e =
      p.a.softcap > 0.f ? launch_overlapped(kv8_stream_kernel<D, NT, true, TILED>, grid, kThreads, smem, st, 1, tk, tv, p)
                        : launch_overlapped(kv8_stream_kernel<D, NT, false, TILED>, grid, kThreads, smem, st, 1, tk, tv, p);
  if (e != cudaSuccess) return e;
  const dim3 join((unsigned)(p.a.kv.max_rows * (int64_t)p.group), p.a.kv.n_seqs, p.a.kv.n_kv_heads);
  // A long sequence's segments are spread over all CTAs: with few heads, groups of
  // threads share a row's many partials. One token over 72000, 1 head, D = 64: 17.7 us
  // with 8 groups, 39.6 with one; 16 tokens over 500 to 4000, 2 heads: 14.7 and 16.7.
  // With 8 heads a row has 19 at most, and larger CTAs would only cost.
  constexpr int G = 512 / D;
  if (p.a.kv.n_kv_heads * 24 < p.a.num_sms)
    return launch_overlapped(kv8_join_kernel<D, NT, TILED, G>, join, D * G, 0, st, 1, p);
  return launch_overlapped(kv8_join_kernel<D, NT, TILED, 1>, join, D, 0, st, 1, p);
}

// Floats of the workspace's parts, in the order of StreamParams; the plan first.
struct StreamWorkspace {
  int64_t part_rows, o, ml, first, total;
};
StreamWorkspace stream_workspace(int64_t rows, int D, int num_sms) {
  StreamWorkspace w;
  const int64_t kept = narrow(rows) ? 8 : 16;
  w.part_rows = num_sms * 2 * kept;
  w.o = 2 * (kMaxSeqs + 8);  // the plan's int64
  w.ml = w.o + w.part_rows * D;
  w.first = w.ml + w.part_rows * 2;
  w.total = w.first + (int64_t)num_sms * (narrow(rows) ? StreamCfg<128, 1, false>::kWarps : StreamCfg<128, 2, false>::kWarps) * kept * (D + 2);
  return w;
}

template <int D>
cudaError_t attention(const KvAttention &a, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!cache_map<D>(&tk, a.kv, a.kv.k) || !cache_map<D>(&tv, a.kv, a.kv.v)) return cudaErrorInvalidValue;
  StreamParams p;
  p.a = a;
  p.group = a.n_heads / a.kv.n_kv_heads;
  const int64_t rows = (int64_t)a.kv.max_rows * p.group;
  const StreamWorkspace w = stream_workspace(rows, D, a.num_sms);
  float *ws = static_cast<float *>(a.workspace);
  p.part_rows = w.part_rows;
  p.plan = reinterpret_cast<int64_t *>(ws);
  p.part_o = ws + w.o;
  p.part_ml = ws + w.ml;
  p.first = ws + w.first;
  for (int s0 = 0; s0 < a.kv.n_seqs; s0 += kMaxSeqs) {
    p.a.kv = kv_slice(a.kv, s0, a.kv.n_seqs - s0 < kMaxSeqs ? a.kv.n_seqs - s0 : kMaxSeqs);
    const cudaError_t e = narrow(rows) ? run_stream<D, 1, false>(tk, tv, p, st)
                          : rows <= 16 ? run_stream<D, 2, false>(tk, tv, p, st)
                                       : run_stream<D, 2, true>(tk, tv, p, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t weigh(const KvAttention &a, cudaStream_t st) {
  CUtensorMap tk;
  if (!cache_map<D>(&tk, a.kv, a.kv.k)) return cudaErrorInvalidValue;
  StreamParams p{};
  p.a = a;
  p.group = a.n_heads / a.kv.n_kv_heads;
  using Cfg = StreamCfg<D, 1, true>;
  constexpr int kThreads = Cfg::kThreads;
  p.warps = a.num_sms * Cfg::kWarps;
  const size_t smem = Cfg::kSmem;
  for (int s0 = 0; s0 < a.kv.n_seqs; s0 += kMaxSeqs) {
    p.a.kv = kv_slice(a.kv, s0, a.kv.n_seqs - s0 < kMaxSeqs ? a.kv.n_seqs - s0 : kMaxSeqs);
    const cudaError_t e = a.softcap > 0.f ? launch_overlapped(kv8_weigh_kernel<D, true>, a.num_sms, kThreads, smem, st, 1, tk, p)
                                          : launch_overlapped(kv8_weigh_kernel<D, false>, a.num_sms, kThreads, smem, st, 1, tk, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t init_dim() {
  cudaError_t e = cudaSuccess;
  for (const void *f : {(const void *)kv8_stream_kernel<D, 1, false, false>, (const void *)kv8_stream_kernel<D, 1, true, false>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamCfg<D, 1, false>::kSmem);
  for (const void *f : {(const void *)kv8_stream_kernel<D, 2, false, false>, (const void *)kv8_stream_kernel<D, 2, true, false>,
                        (const void *)kv8_stream_kernel<D, 2, false, true>, (const void *)kv8_stream_kernel<D, 2, true, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamCfg<D, 2, false>::kSmem);
  for (const void *f : {(const void *)kv8_weigh_kernel<D, false>, (const void *)kv8_weigh_kernel<D, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamCfg<D, 1, true>::kSmem);
  // the join takes the stream kernel's split of shared memory and L1: no SM waits to change it
  for (const void *f : {(const void *)kv8_join_kernel<D, 1, false, 1>, (const void *)kv8_join_kernel<D, 2, false, 1>,
                        (const void *)kv8_join_kernel<D, 2, true, 1>, (const void *)kv8_join_kernel<D, 1, false, 512 / D>,
                        (const void *)kv8_join_kernel<D, 2, false, 512 / D>, (const void *)kv8_join_kernel<D, 2, true, 512 / D>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  return e;
}

}  // namespace

size_t kv8_attention_workspace_bytes(const exl3_kv8_cache &c, const exl3_kv8_batch &b, int n_heads, int num_sms) {
  if (b.rows == 0 || b.n_seqs == 0 || b.max_rows == 0) return 16;
  const int64_t rows = (int64_t)b.max_rows * (n_heads / c.n_kv_heads);
  if (rows > kStreamRows) return kv8_chunk_workspace_bytes(c.head_dim, num_sms);
  return (size_t)stream_workspace(rows, c.head_dim, num_sms).total * sizeof(float);
}

cudaError_t launch_kv8_attention(const KvAttention &a, cudaStream_t st) {
  if (a.kv.rows == 0 || a.kv.n_seqs == 0 || a.kv.max_rows == 0) return cudaSuccess;
  if ((int64_t)a.kv.max_rows * (a.n_heads / a.kv.n_kv_heads) > kStreamRows) return launch_kv8_chunk_attention(a, st);
  return a.kv.head_dim == 64 ? attention<64>(a, st) : attention<128>(a, st);
}

cudaError_t launch_kv8_weigh(const KvAttention &a, cudaStream_t st) {
  if (a.kv.rows == 0 || a.kv.n_seqs == 0 || a.kv.max_rows == 0) return cudaSuccess;
  if ((int64_t)a.kv.max_rows * (a.n_heads / a.kv.n_kv_heads) > kWeighRows) return launch_kv8_weigh_chunk(a, st);
  return a.kv.head_dim == 64 ? weigh<64>(a, st) : weigh<128>(a, st);
}

cudaError_t init_kv8_attention_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  if (e == cudaSuccess) e = init_dim<64>();
  return e == cudaSuccess ? init_dim<128>() : e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_kv8_attention(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
