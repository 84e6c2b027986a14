// Device helpers of the 8-bit key/value cache (layout in include/exl3.h).
#pragma once

#include <stdint.h>

#include <utility>

#include "exl3_common.cuh"
#include "exl3_serve.h"
#include "exl3_tcgen05.cuh"

namespace exl3 {

constexpr int kKvBlock = EXL3_KV8_BLOCK;
constexpr int kMinExp = -32, kMaxExp = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void report_index(int *status) {
  atomicCAS(status, 0, (int)EXL3_ERR_DEVICE_INDEX);
}

// What the device buffers say of one sequence, checked against what the call
// declared: lengths and row ranges outside it are reported, and the sequence
// is then empty.
struct KvSeq {
  int row0, rows, len;
};
__device__ __forceinline__ int kv_length(const KvView &kv, int s) {
  const int len = kv.kv_len[s];
  if (len < 0 || len > kv.max_pages * (int64_t)kKvBlock) {
    report_index(kv.status);
    return 0;
  }
  return len;
}
__device__ __forceinline__ KvSeq kv_sequence(const KvView &kv, int s) {
  KvSeq q{kv.q_start[s], 0, kv_length(kv, s)};
  q.rows = kv.q_start[s + 1] - q.row0;
  if (q.row0 < 0 || q.rows < 0 || q.rows > kv.max_rows || q.row0 + (int64_t)q.rows > kv.rows) {
    report_index(kv.status);
    q = KvSeq{0, 0, 0};
  }
  return q;
}

// Page of block b of sequence s, or -1 (reported) when the table's entry names
// no page. b < max_pages.
__device__ __forceinline__ int kv_page(const KvView &kv, int s, int b) {
  const int p = kv.page_table[(int64_t)s * kv.max_pages + b];
  if (p < 0 || p >= kv.n_pages) {
    report_index(kv.status);
    return -1;
  }
  return p;
}

// 2^e for -126 <= e <= 127, and the exponent of a power of two.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int pow2_exponent(float s) { return ((__float_as_int(s) >> 23) & 255) - 127; }

// Smallest e in kMinExp .. kMaxExp with a <= 448 * 2^e, for an fp16 value a >= 0.
// With a = m 2^x, m in [1/2, 1), and 448 = 7/8 * 2^9: x - 9, one more when m > 7/8.
__device__ __forceinline__ int block_exponent(float a) {
  const int b = __float_as_int(a);
  const int e = (b >> 23) - 126 - 9 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// Two fp32 values to two E4M3 codes (a in the low byte): nearest even,
// saturating, NaN to NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two E4M3 codes to two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// Eight codes times 2^d, rounded to nearest even.
__device__ __forceinline__ uint2 rescale_codes(uint2 c, float factor) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = e4m3x2_to_half2((uint16_t)(w[i] & 0xFFFF)), hi = e4m3x2_to_half2((uint16_t)(w[i] >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    o[i] = to_e4m3x2(a.x * factor, a.y * factor) | (to_e4m3x2(b.x * factor, b.y * factor) << 16);
  }
  return make_uint2(o[0], o[1]);
}

// Byte offset of 16-byte piece c (of 8) of 128-byte row r in a swizzled operand half.
__device__ __forceinline__ uint32_t swizzled(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if (EXL3_SMEM(addr, 16))
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes to 16 fp16 values, exact.
__device__ __forceinline__ void codes_to_half(uint4 w, uint32_t (&o)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = e4m3x2_to_half2((uint16_t)(x[i] & 0xFFFFu));
    o[2 * i + 1] = e4m3x2_to_half2((uint16_t)(x[i] >> 16));
  }
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tcgen05.mma cuts its fp32 accumulator off towards zero at each of a score's D / 16
// steps. Of scores whose partial sums grow evenly, as those of heavy tokens do, that takes
// 1.05 * 2^-23 on average at D = 128 and 0.46 * 2^-23 at D = 64 (measured over 20000 scores
// each; of random vectors 0.47 and 0.2; mma.sync 0.43 and 0.17). So at D = 128 both kernels
// that form scores with it, attention and weights, raise them by 2^-23 of themselves, a step
// of fp32 and no more than one more rounding might do: weights of 10240 rows then are 4e-7 to
// 8e-7 from the formula (elementary fp32 operations as much), 2e-6 without.
template <int D>
struct Raised {
  static constexpr float kOne = D == 128 ? 1.0f + 0x1p-23f : 1.0f;
  static constexpr float kLog2e = (float)(1.4426950408889634 * (D == 128 ? 1.0 + 0x1p-23 : 1.0));
};

// log of a sum l of exponentials around m (log2 units).
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2; }

// First unit of worker w of W over T units, and the worker that owns unit z
// (a 32-bit division where the numbers allow it: a 64-bit one takes about as long
// as a load from memory).
__device__ __forceinline__ int64_t range_start(int64_t w, int64_t W, int64_t T) {
  return W * T < ((int64_t)1 << 31) ? (int64_t)((uint32_t)(w * T) / (uint32_t)W) : w * T / W;
}
__device__ __forceinline__ int64_t range_owner(int64_t z, int64_t W, int64_t T) {
  return W * T < ((int64_t)1 << 31) ? (int64_t)(((uint32_t)((z + 1) * W) - 1) / (uint32_t)T) : ((z + 1) * W - 1) / T;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A cap in the unit of the scores (`unit` of it: 1, or log2 e), and its inverse. A cap
// whose double leaves fp32 is lowered: no score comes near it.
struct SoftCap {
  float cap, inv;
  __device__ __forceinline__ SoftCap(float softcap, float unit)
      : cap(fminf(softcap * unit, 1.5e38f)), inv(1.0f / (softcap * unit)) {}
  // cap * tanh(x), x = s / cap, of two scores, to 2^-19 of each. |x| < 1/5: s (1 - x^2 / 3
  // + 2 x^4 / 15 - 17 x^6 / 315), tanh's power series, whose next term is 2^-24 there, and
  // which does not depend on the cap where that is far above the scores. Else through
  // 1 - 2 / (exp(2 x) + 1), an absolute error near cap * 2^-22, which a direct tanh
  // approximation (relative error 2^-11 of a score near the cap) would not give. exp
  // overflows to inf: tanh is then 1. 2048 rows of 40 heads over 8192 tokens, cap 30:
  // weights 409 us, 394 by the exponential alone; attention 617, and 22 less.
  __device__ __forceinline__ float2 operator()(float2 s) const {
    auto both = [](float v) { return make_float2(v, v); };
    const float2 x = mul2(s, both(inv)), y = mul2(x, x), e = mul2(x, both(2.0f * kLog2e));
    float2 series = fma2(y, both(-17.0f / 315.0f), both(2.0f / 15.0f));
    series = fma2(y, series, both(-1.0f / 3.0f));
    series = fma2(mul2(s, y), series, s);
    const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.0f));
    const float2 far = fma2(both(-2.0f * cap), make_float2(rcp(d.x), rcp(d.y)), both(cap));
    return make_float2(y.x < 0.04f ? series.x : far.x, y.y < 0.04f ? series.y : far.y);
  }
};

// A launch that may start while the kernel before it in the stream is ending.
// The kernels wait (griddepcontrol.wait) before they touch memory, and read it
// through ordinary loads: a read-only load could move above the wait.
// cluster: CTAs of a cluster along x.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                              Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace exl3
