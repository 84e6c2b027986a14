// Root-mean-square norm with the residual's addition, fp16 or 8-bit output. Formulas in
// include/exl3.h.
//
// A row is read once and stays in registers until its outputs are stored: 8 elements a
// thread and piece, the sum of squares by shuffles and, where a row has more than a warp, one
// exchange through shared memory. Bound by the bytes, or by launch and one row's latency.
// Many rows of more than 2048 columns come by bulk copies into a ring of shared memory, the
// next rows while one is worked on: loads into registers have a row at a time in flight for
// each resident CTA.
//
// Measured (in a graph, over three sets of buffers, the sum in the residual's place; here and at the rules between
// the forms, which stand at by_size with both sides): one row of 5120 fp16 2.0 us; 8192 rows 57 us (5.9 TB/s); 777 rows
// fp32 with E4M3 codes 11.0 us (4.7 TB/s: 107 MB of buffers, of which the L2 holds a part; 12.1 us, 4.3 TB/s, with the sum apart,
// 155 MB; 2.6 rows for each CTA of the ring, 3 for some); 2400 rows of 17408 58 us (5.8 TB/s, from registers 94).
#include <math.h>

#include <type_traits>

#include "exl3_internal.h"
#include "exl3_kv8.cuh"

namespace exl3 {

namespace {

constexpr float kCodeMax = 448.0f, kLeastScale = 0x1p-40f;
constexpr int kWarpRowThreads = 256;
constexpr int kRingThreads = 640, kMaxStages = 8;  // two CTAs an SM with two pieces a thread (more of fewer threads), one with four
constexpr int kRingBytes = 220 * 1024, kRingOther = 2 * 1024;  // of an SM's shared memory; what a CTA has besides its stages

struct Eight {
  float v[8];
  __device__ __forceinline__ void load(const __half *p) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void load(const float *p) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  // From shared memory: every other four lanes read the second half first, so that 8 lanes have all 32 banks.
  __device__ __forceinline__ void load_shared(const __half *p) { load(p); }
  __device__ __forceinline__ void load_shared(const float *p) {
    const bool second = threadIdx.x & 4;
    const float4 x = reinterpret_cast<const float4 *>(p)[second], y = reinterpret_cast<const float4 *>(p)[!second];
    const float4 a = second ? y : x, b = second ? x : y;
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ void store(__half *p) const {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      x[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Sum (or maximum) over the row's threads: `lanes` of a warp, or the whole CTA.
template <bool CTA_ROW, bool MAX>
__device__ __forceinline__ float over_row(float x, int lanes, float *scratch) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  if constexpr (!CTA_ROW) {
    for (int d = lanes >> 1; d > 0; d >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  } else {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, d));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) scratch[warp] = x;
    __syncthreads();
    x = lane < warps ? scratch[lane] : 0.f;  // 0: of sums of squares and of magnitudes
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  }
}

// A thread's pieces of the weight, as fp16 (ones where there is none, without the offset).
template <int V>
struct Weights {
  uint4 w[V];
  float offset;
  __device__ __forceinline__ void load(const exl3_norm &p, int per_row, int at) {
    offset = p.weight ? p.weight_offset : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      w[i] = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);
      if (p.weight && c < (int)(p.cols >> 3) && EXL3_SPAN(c * 8, 8, p.cols)) w[i] = static_cast<const uint4 *>(p.weight)[c];
    }
  }
  __device__ __forceinline__ void times(int i, Eight &h) const {
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[e]));
      h.v[2 * e] *= f.x + offset;
      h.v[2 * e + 1] *= f.y + offset;
    }
  }
};

// From a row's sums h to its outputs. Threads without a row take part with zeros.
template <typename Rt, int V, bool CTA_ROW>
__device__ __forceinline__ void finish_row(const exl3_norm &p, int64_t row, Eight (&h)[V], const Weights<V> &w, int per_row, int at,
                                           int lanes, float (&scratch)[3][32], int turn) {
  const int pieces = (int)(p.cols >> 3);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(h[i].v[e], h[i].v[e], s);
    sum += s;
  }
  if (p.residual_out) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      if (row < p.rows && c < pieces && EXL3_SPAN(row * p.ldro + c * 8, 8, (p.rows - 1) * p.ldro + p.cols))
        h[i].store(static_cast<Rt *>(p.residual_out) + row * p.ldro + c * 8);
    }
  }
  sum = over_row<CTA_ROW, false>(sum, lanes, scratch[turn]);
  const float r = rsqrtf(sum / (float)p.cols + p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) w.times(i, h[i]);
  if (p.codes) {
    // the row's factor cancels in y / (max |y| / 448): codes are of h * w times 448 / max |h * w|
    float most[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      most[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(h[i].v[e]);
        most[i] = fmaxf(most[i], a <= 3.402823466e38f ? a : 0.f);
      }
    }
    const int cols = (int)p.cols, group = p.group;
    const bool whole = group == cols;
    if (whole) {
      float m = most[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, most[i]);
      m = over_row<CTA_ROW, true>(m, lanes, scratch[2]);
      if constexpr (CTA_ROW) __syncthreads();  // its buffer is used by every row
#pragma unroll
      for (int i = 0; i < V; ++i) most[i] = m;
    } else {
      for (int d = group >> 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) most[i] = fmaxf(most[i], __shfl_xor_sync(0xffffffffu, most[i], d));
    }
    const int shift = 31 - __clz(group), groups = whole ? 1 : cols >> shift;  // a power of two, if not the whole row
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      if (row >= p.rows || c >= pieces) continue;
      const float raw = most[i] * r / kCodeMax;
      const bool least = !(raw >= kLeastScale);
      const float f = least ? r / kLeastScale : kCodeMax / most[i];
      const int64_t to = row * groups + (whole ? 0 : c * 8 >> shift);
      if ((whole ? c : c * 8 & (group - 1)) == 0 && EXL3_SPAN(to, 1, p.rows * groups)) p.scales[to] = least ? kLeastScale : raw;
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = to_e4m3x2(h[i].v[2 * e] * f, h[i].v[2 * e + 1] * f);
      if (EXL3_SPAN(row * p.ldc + c * 8, 8, (p.rows - 1) * p.ldc + p.cols))
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.ldc + c * 8) =
            make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
  }
  if (p.y) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      if (row >= p.rows || c >= pieces) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i].v[e] *= r;
      if (EXL3_SPAN(row * p.ldy + c * 8, 8, (p.rows - 1) * p.ldy + p.cols))
        h[i].store(static_cast<__half *>(p.y) + row * p.ldy + c * 8);
    }
  }
}

// X, R: types of x and of the residual (void: none). V: pieces of 8 elements a thread.
// A row is `lanes` lanes' of a warp, or the CTA's.
template <typename X, typename R, int V, bool CTA_ROW>
__global__ void __launch_bounds__(CTA_ROW ? 1024 : kWarpRowThreads) rms_norm_kernel(const exl3_norm p, int lanes) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float scratch[3][32];
  constexpr bool kResidual = !std::is_void<R>::value;
  using Rt = typename std::conditional<kResidual, R, float>::type;
  const int per_row = CTA_ROW ? (int)blockDim.x : lanes, at = threadIdx.x % per_row;
  const int rows_at_once = CTA_ROW ? 1 : (int)blockDim.x / lanes;
  const int pieces = (int)(p.cols >> 3);
  Weights<V> w;
  w.load(p, per_row, at);
  int turn = 0;  // sums alternate between two buffers, so that one barrier a row is enough
  // every lane of a warp stays to the end: rows past the last are nobody's, but their lanes take part in the shuffles
  for (int64_t first = (int64_t)blockIdx.x * rows_at_once; first < p.rows; first += (int64_t)gridDim.x * rows_at_once, turn ^= 1) {
    const int64_t row = first + (CTA_ROW ? 0 : threadIdx.x / per_row);
    Eight h[V], r[kResidual ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      const bool there = row < p.rows && c < pieces;
      if (there && EXL3_SPAN(row * p.ldx + c * 8, 8, (p.rows - 1) * p.ldx + p.cols)) h[i].load(static_cast<const X *>(p.x) + row * p.ldx + c * 8);
      else h[i].zero();
      if constexpr (kResidual) {
        if (there && EXL3_SPAN(row * p.ldr + c * 8, 8, (p.rows - 1) * p.ldr + p.cols)) r[i].load(static_cast<const Rt *>(p.residual) + row * p.ldr + c * 8);
        else r[i].zero();
      }
    }
    if constexpr (kResidual) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i].v[e] += r[i].v[e];
    }
    finish_row<Rt, V, CTA_ROW>(p, row, h, w, per_row, at, lanes, scratch, turn);
  }
}

// The same for many rows: x and the residual come by bulk copies, `stages` rows of the CTA at a
// time. A stage is given back when every thread has its pieces in registers, which the row's
// barrier (that of the sum of squares) says; so the next copy into it is issued after it.
template <typename X, typename R, int V>
__global__ void __launch_bounds__(kRingThreads, V <= 2 ? 2 : 1) rms_norm_ring_kernel(const exl3_norm p, int stages, int stage_bytes, int *status) {
  extern __shared__ __align__(128) uint8_t smem[];  // stages of x, then residual
  __shared__ float scratch[3][32];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  constexpr bool kResidual = !std::is_void<R>::value;
  using Rt = typename std::conditional<kResidual, R, float>::type;
  const int at = threadIdx.x, per_row = blockDim.x, pieces = (int)(p.cols >> 3);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(full + i), 1);
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  const uint32_t x_bytes = (uint32_t)(p.cols * sizeof(X)), r_bytes = kResidual ? (uint32_t)(p.cols * sizeof(Rt)) : 0;
  auto fetch = [&](int64_t row, int st) {  // one thread
    const uint32_t dst = smem_u32(smem) + st * stage_bytes, bar = smem_u32(full + st);
    mbar_arrive_expect_tx(bar, x_bytes + r_bytes);
    if (EXL3_SPAN(row * p.ldx, p.cols, (p.rows - 1) * p.ldx + p.cols) && EXL3_SMEM(dst, x_bytes + r_bytes))
      bulk_g2s(dst, static_cast<const X *>(p.x) + row * p.ldx, x_bytes, bar);
    if constexpr (kResidual)
      if (EXL3_SPAN(row * p.ldr, p.cols, (p.rows - 1) * p.ldr + p.cols))
        bulk_g2s(dst + x_bytes, static_cast<const Rt *>(p.residual) + row * p.ldr, r_bytes, bar);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + (int64_t)i * gridDim.x < p.rows) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
  Weights<V> w;
  w.load(p, per_row, at);
  int st = 0, turn = 0;
  uint32_t phase = 0;
  bool ok = true;  // after a wait that ran out, a thread only keeps step with the others
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    ok = ok && mbar_wait(smem_u32(full + st), phase, status);
    Eight h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * per_row + at;
      if (c < pieces) {
        h[i].load_shared(reinterpret_cast<const X *>(smem + st * stage_bytes) + c * 8);
        if constexpr (kResidual) {
          Eight r;
          r.load_shared(reinterpret_cast<const Rt *>(smem + st * stage_bytes + x_bytes) + c * 8);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i].v[e] += r.v[e];
        }
      } else {
        h[i].zero();
      }
    }
    finish_row<Rt, V, true>(p, row, h, w, per_row, at, 32, scratch, turn);
    // past the row's barrier: all have read the stage
    if (threadIdx.x == 0 && ok && row + (int64_t)stages * gridDim.x < p.rows) fetch(row + (int64_t)stages * gridDim.x, st);
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
  // nothing is on its way into this CTA's memory when it ends (only after a wait that ran out)
  if (threadIdx.x == 0 && !ok)
    for (int i = 0; i < stages; ++i) mbar_wait_short(smem_u32(full + i), i < st ? phase ^ 1 : phase);
}

template <typename X, typename R, int V, bool CTA_ROW>
cudaError_t launch(const exl3_norm &p, int threads, int lanes, int num_sms, cudaStream_t st) {
  const int64_t ctas = CTA_ROW ? p.rows : ceil_div(p.rows, threads / lanes);
  // Rows of one piece a thread have a CTA each: 8192 rows of 2048 fp16 take 21.7 us, 22.5 from CTAs that stay; the widest
  // ones stay, with their weight (1000 rows of 32768 fp16: 62.3 us, 66.3 with a CTA each).
  const int64_t most = CTA_ROW && V == 1 ? INT32_MAX : (int64_t)num_sms * (2048 / threads);
  return launch_overlapped(rms_norm_kernel<X, R, V, CTA_ROW>, dim3((unsigned)(ctas < most ? ctas : most)), threads, 0, st, 1, p, lanes);
}

template <typename X, typename R>
constexpr int element_bytes() {
  if constexpr (std::is_void<R>::value) return sizeof(X);
  else return sizeof(X) + sizeof(R);
}

template <typename X, typename R>
cudaError_t by_size(const exl3_norm &p, int num_sms, int *status, cudaStream_t st) {
  const int pieces = (int)(p.cols / 8);
  // A row of at most 1024 columns is a warp's, or a part's; where rows are few, one of more than 256 is a CTA's: 304 rows of
  // 1024 take 1.8 us, 2.3 by warps; 608 rows 2.0 and 2.3 (with codes 2.6 and 3.7), 1216 rows 2.7 and 2.4, 2400 rows 4.0 and
  // 3.1, 8192 rows 11.8 and 13.4 (of 512: 8.6 and 5.1).
  if (pieces <= 32 || (pieces <= 128 && p.rows > 4 * num_sms)) {
    int lanes = 16;
    while (lanes < 32 && lanes < pieces) lanes *= 2;
    if (pieces <= 32) return launch<X, R, 1, false>(p, kWarpRowThreads, lanes, num_sms, st);
    return pieces <= 64 ? launch<X, R, 2, false>(p, kWarpRowThreads, lanes, num_sms, st)
                        : launch<X, R, 4, false>(p, kWarpRowThreads, lanes, num_sms, st);
  }
  auto threads = [&](int v) { return (int)(ceil_div(ceil_div(pieces, v), 32) * 32); };
  // The ring, with as many CTAs as have two stages each: from three rows an SM on (fp16: 500 rows of 5120 3.9 us, 4.4 from
  // registers; 400 rows 4.0 and 3.5; 2400 rows 17.6 and 18.2, without a residual 10.7 and 14.8, fp32 with codes 27.5 and 30.4) and above
  // 2048 columns (2400 rows of 2560: 8.1 and 9.3; 8192 of 2048: 23.4 and 21.7). What is read and written in equal parts by many rows
  // would be a little better off in registers (8192 rows of 5120, fp16 57.0 and 55.3, fp32 95 and 86; without a residual 32 and 44).
  // Rows too wide for one piece a thread: from one an SM on (160 rows of 17408: 5.9 us and 9.1; 2400: 58 and 94), as far as the
  // threads reach: 2400 rows of 20480 columns 66 us, of 20488, from registers, 106.
  if (pieces > 256 && p.rows > (threads(1) > 1024 ? 1 : 3) * num_sms && threads(4) <= kRingThreads) {
    const bool two = threads(2) <= kRingThreads;
    const int t = threads(two ? 2 : 4), stage = (int)p.cols * element_bytes<X, R>();
    auto stages_of = [&](int ctas) { return ((kRingBytes + kRingOther) / ctas - kRingOther) / stage; };
    int ctas = two ? 2 * kRingThreads / t : 1;
    while (ctas > 1 && stages_of(ctas) < 2) --ctas;
    const int stages = stages_of(ctas) < kMaxStages ? stages_of(ctas) : kMaxStages;
    if (stages >= 2)
      return launch_overlapped(two ? rms_norm_ring_kernel<X, R, 2> : rms_norm_ring_kernel<X, R, 4>, ctas * num_sms, t, (size_t)stages * stage, st, 1,
                               p, stages, stage, status);
  }
  if (threads(1) <= 1024) return launch<X, R, 1, true>(p, threads(1), 32, num_sms, st);
  return launch<X, R, 4, true>(p, threads(4), 32, num_sms, st);
}

template <typename X>
cudaError_t by_residual(const exl3_norm &p, int num_sms, int *status, cudaStream_t st) {
  if (!p.residual) return by_size<X, void>(p, num_sms, status, st);
  return p.residual_dtype == EXL3_F32 ? by_size<X, float>(p, num_sms, status, st) : by_size<X, __half>(p, num_sms, status, st);
}

template <typename X, typename R>
cudaError_t load_kernels() {
  cudaFuncAttributes attr;
  cudaError_t e = cudaSuccess;
  for (const void *f : {(const void *)rms_norm_kernel<X, R, 1, false>, (const void *)rms_norm_kernel<X, R, 2, false>,
                        (const void *)rms_norm_kernel<X, R, 4, false>, (const void *)rms_norm_kernel<X, R, 1, true>,
                        (const void *)rms_norm_kernel<X, R, 4, true>})
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, f);
  for (const void *f : {(const void *)rms_norm_ring_kernel<X, R, 2>, (const void *)rms_norm_ring_kernel<X, R, 4>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  return e;
}

}  // namespace

cudaError_t launch_rms_norm(const exl3_norm &p, int num_sms, int *status, cudaStream_t st) {
  return p.x_dtype == EXL3_F32 ? by_residual<float>(p, num_sms, status, st) : by_residual<__half>(p, num_sms, status, st);
}

cudaError_t init_rms_norm_kernels(int *status) {
  cudaError_t e = EXL3_BIND_BOUNDS_WORD(status);
  if (e == cudaSuccess) e = load_kernels<__half, void>();
  if (e == cudaSuccess) e = load_kernels<__half, __half>();
  if (e == cudaSuccess) e = load_kernels<__half, float>();
  if (e == cudaSuccess) e = load_kernels<float, void>();
  if (e == cudaSuccess) e = load_kernels<float, __half>();
  if (e == cudaSuccess) e = load_kernels<float, float>();
  return e;
}

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_rms_norm(cudaStream_t st) { return launch_bounds_probe(st); }
#endif

}  // namespace exl3
