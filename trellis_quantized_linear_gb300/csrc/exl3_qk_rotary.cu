// Norm and rotation of query and key heads. Formulas in include/exl3.h.
//
// A thread has 16 elements of a head, in two pieces of 8 that hold both partners of its
// 8 pairs, and the angles of those pairs in registers for all heads of the row that it works
// on. Bound by the bytes, or by launch and the way position - angles - store.
//
// Measured (in a graph, 48 heads of 128, normed): 16 rows 2.0 us, 6827 rows 27.8 us (6.0 TB/s;
// loads after the position 33.8). 9 heads, a row at a time 12.7 us, several 8.0; 3 heads
// 10.2 and 3.9.
#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

constexpr int kRotaryThreads = 128, kFlatThreads = 256;

struct Piece {
  float v[8];
  __device__ __forceinline__ explicit Piece(uint4 w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ void store(__half *p) const {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      x[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(x[0], x[1], x[2], x[3]);
  }
};

// D / 16 lanes a head; blockIdx.y takes its share of the heads, `each` of them. A thread's
// heads are loaded kAhead at a time, before the position is there. FLAT: a CTA has `tall` rows
// at once, a head for each place.
template <int D, bool INTERLEAVED, bool NORM, bool FLAT>
__global__ void __launch_bounds__(FLAT ? kFlatThreads : kRotaryThreads) qk_rotary_kernel(const QkRotary p, int each, int tall) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kLanes = D / 16, kAtOnce = (FLAT ? kFlatThreads : kRotaryThreads) / kLanes, kAhead = FLAT ? 1 : 3;
  const int l = threadIdx.x % kLanes, place = threadIdx.x / kLanes;
  const int heads = p.q_heads + p.k_heads, h0 = blockIdx.y * each, h1 = min(h0 + each, heads);
  const int below = FLAT ? place / heads : 0, slot = place - below * heads;
  const bool turns = 16 * l < p.rot_dim;
  // first elements of the two pieces
  const int a0 = INTERLEAVED || !turns ? 16 * l : 8 * l;
  const int b0 = INTERLEAVED || !turns ? 16 * l + 8 : p.rot_dim / 2 + 8 * l;
  [[maybe_unused]] const int64_t size_x = (int64_t)(p.rows - 1) * p.ldx + (int64_t)heads * D;
  [[maybe_unused]] const int64_t size_o = (int64_t)(p.rows - 1) * p.ldo + (int64_t)heads * D;
  const int rows_at_once = FLAT ? tall : 1;
  for (int64_t first_row = (int64_t)blockIdx.x * rows_at_once; first_row < p.rows; first_row += (int64_t)gridDim.x * rows_at_once) {
    const int64_t row = first_row + below;
    const bool mine = !FLAT || (below < tall && row < p.rows);
    const int pos = mine ? p.position[row] : -1;
    float cs[8], sn[8];
    bool known = false, turned = true;
    for (int first = h0; first < h1; first += kAhead * kAtOnce) {
      uint4 ra[kAhead], rb[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int h = first + i * kAtOnce + slot;
        const int64_t from = row * p.ldx + (int64_t)h * D;
        ra[i] = rb[i] = make_uint4(0, 0, 0, 0);
        if (mine && h < h1 && EXL3_SPAN(from, D, size_x)) {
          ra[i] = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(p.x) + from + a0);
          rb[i] = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(p.x) + from + b0);
        }
      }
      if (!known) {
        known = true;
        if (pos >= p.n_positions && slot == 0 && l == 0) report_index(p.status);
        turned = pos >= 0 && pos < p.n_positions;
        if (!FLAT && !turned) break;  // the same in the whole CTA
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
        if (turned && turns) {
          const int64_t at = (int64_t)pos * p.rot_dim + 8 * l;
          if (EXL3_SPAN(at, p.rot_dim / 2 + 8, (int64_t)p.n_positions * p.rot_dim)) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const float4 c = *reinterpret_cast<const float4 *>(p.cos_sin + at + e);
              const float4 s = *reinterpret_cast<const float4 *>(p.cos_sin + at + p.rot_dim / 2 + e);
              cs[e] = c.x, cs[e + 1] = c.y, cs[e + 2] = c.z, cs[e + 3] = c.w;
              sn[e] = s.x, sn[e + 1] = s.y, sn[e + 2] = s.z, sn[e + 3] = s.w;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {  // all lanes of a warp go round as often as each other: the norm's shuffles
        const int h = first + i * kAtOnce + slot;
        const int64_t to = row * p.ldo + (int64_t)h * D;
        const bool there = turned && h < h1 && EXL3_SPAN(to, D, size_o);
        Piece a(ra[i]), b(rb[i]);
        if constexpr (NORM) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(a.v[e], a.v[e], fmaf(b.v[e], b.v[e], sum));
#pragma unroll
          for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const float r = rsqrtf(sum / (float)D + p.eps);
          if (there) {
            const __half *w = static_cast<const __half *>(h < p.q_heads ? p.q_weight : p.k_weight);
            const Piece wa(*reinterpret_cast<const uint4 *>(w + a0)), wb(*reinterpret_cast<const uint4 *>(w + b0));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              a.v[e] *= r * (wa.v[e] + p.weight_offset);
              b.v[e] *= r * (wb.v[e] + p.weight_offset);
            }
          }
        }
        if (!there) continue;
        Piece oa, ob;
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            oa.v[2 * e] = a.v[2 * e] * cs[e] - a.v[2 * e + 1] * sn[e];
            oa.v[2 * e + 1] = a.v[2 * e + 1] * cs[e] + a.v[2 * e] * sn[e];
            ob.v[2 * e] = b.v[2 * e] * cs[4 + e] - b.v[2 * e + 1] * sn[4 + e];
            ob.v[2 * e + 1] = b.v[2 * e + 1] * cs[4 + e] + b.v[2 * e] * sn[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            oa.v[e] = a.v[e] * cs[e] - b.v[e] * sn[e];
            ob.v[e] = b.v[e] * cs[e] + a.v[e] * sn[e];
          }
        }
        // not rotated: as they are, also infinities and NaN, which 0 times would spread
        (turns ? oa : a).store(static_cast<__half *>(p.out) + to + a0);
        (turns ? ob : b).store(static_cast<__half *>(p.out) + to + b0);
      }
    }
  }
}

template <int D, bool INTERLEAVED>
cudaError_t rotary(const QkRotary &p, int num_sms, cudaStream_t st) {
  const int heads = p.q_heads + p.k_heads;
  const bool norm = p.q_weight || p.k_weight;
  // Up to 2048 columns of heads leave most of a CTA without work, or a few rows of it: several rows at once, whose threads
  // read the angles for one head each (6827 rows of 16 heads of 128 or fewer: 3 to 11 us, 10 to 14 by rows; 20 heads: 19 and 16).
  if (heads * D <= 2048) {
    const int tall = kFlatThreads * 16 / D / heads;
    const int64_t ctas = ceil_div(p.rows, tall), most = (int64_t)num_sms * (2048 / kFlatThreads);
    return launch_overlapped(norm ? qk_rotary_kernel<D, INTERLEAVED, true, true> : qk_rotary_kernel<D, INTERLEAVED, false, true>,
                             dim3((unsigned)(ctas < most ? ctas : most)), kFlatThreads, 0, st, 1, p, heads, tall);
  }
  // Few rows: the heads of a row are shared by CTAs, as far as those are resident at once (48 heads of 128: 1 row 1.9 us, by
  // one CTA 2.2; 304 rows 2.9 and 3.8; 700 rows, shared as if there were fewer, 5.1, not 4.3).
  constexpr int kAtOnce = kRotaryThreads * 16 / D;
  const int64_t most = (int64_t)num_sms * (2048 / kRotaryThreads), top = ceil_div(heads, kAtOnce), full = most / 2 / p.rows;
  const int64_t shares = full < 1 ? 1 : full < top ? full : top;
  const int each = (int)(ceil_div(ceil_div(heads, shares), kAtOnce) * kAtOnce);
  const dim3 grid((unsigned)(p.rows < most ? p.rows : most), (unsigned)ceil_div(heads, each));
  return launch_overlapped(norm ? qk_rotary_kernel<D, INTERLEAVED, true, false> : qk_rotary_kernel<D, INTERLEAVED, false, false>, grid,
                           kRotaryThreads, 0, st, 1, p, each, 1);
}

}  // namespace

cudaError_t launch_qk_rotary(const QkRotary &p, int num_sms, cudaStream_t st) {
  if (p.interleaved) return p.head_dim == 64 ? rotary<64, true>(p, num_sms, st) : rotary<128, true>(p, num_sms, st);
  return p.head_dim == 64 ? rotary<64, false>(p, num_sms, st) : rotary<128, false>(p, num_sms, st);
}

cudaError_t init_qk_rotary_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  cudaFuncAttributes attr;
  for (const void *f : {(const void *)qk_rotary_kernel<64, false, false, false>, (const void *)qk_rotary_kernel<64, false, true, false>,
                        (const void *)qk_rotary_kernel<64, true, false, false>, (const void *)qk_rotary_kernel<64, true, true, false>,
                        (const void *)qk_rotary_kernel<128, false, false, false>, (const void *)qk_rotary_kernel<128, false, true, false>,
                        (const void *)qk_rotary_kernel<128, true, false, false>, (const void *)qk_rotary_kernel<128, true, true, false>,
                        (const void *)qk_rotary_kernel<64, false, false, true>, (const void *)qk_rotary_kernel<64, false, true, true>,
                        (const void *)qk_rotary_kernel<64, true, false, true>, (const void *)qk_rotary_kernel<64, true, true, true>,
                        (const void *)qk_rotary_kernel<128, false, false, true>, (const void *)qk_rotary_kernel<128, false, true, true>,
                        (const void *)qk_rotary_kernel<128, true, false, true>, (const void *)qk_rotary_kernel<128, true, true, true>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, f);
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_qk_rotary(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
