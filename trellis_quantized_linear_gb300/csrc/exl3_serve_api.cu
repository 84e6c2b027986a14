// C ABI of the serving operators: argument validation. Declarations and
// argument contracts are in include/exl3.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/exl3.h"
#include "exl3_common.cuh"
#include "exl3_internal.h"
#include "exl3_serve.h"

namespace exl3 {

namespace {

bool aligned(const void *p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
exl3_status from_cuda(cudaError_t e) { return e == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA; }

bool cache_shape_ok(const exl3_kv8_cache &c) {
  return (c.head_dim == 64 || c.head_dim == 128) && c.n_kv_heads >= 1 && c.n_kv_heads <= 1024 && c.n_pages >= 1 &&
         c.n_pages <= INT32_MAX && c.n_pages * c.n_kv_heads * EXL3_KV8_BLOCK <= INT32_MAX;
}
bool batch_shape_ok(const exl3_kv8_batch &b) {
  return b.n_seqs >= 0 && b.n_seqs <= 65535 && b.max_pages >= 0 && b.max_pages <= INT32_MAX / EXL3_KV8_BLOCK &&
         b.rows >= 0 && b.max_rows >= 0 && b.max_rows <= b.rows;
}

// Nothing to do: a call without rows or sequences is over after its shape checks, and may
// come with the null pointers that empty tensors have.
bool no_rows(const exl3_kv8_batch &b) { return b.rows == 0 || b.n_seqs == 0 || b.max_rows == 0; }

// Shape checks come first (they need no pointers), then alignment, then the
// device, as in every entry point of the library.
exl3_status validate_kv(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, bool rows, const DeviceInfo **dev,
                        KvView *kv) {
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(cache->k_scale, 4) || !aligned(cache->v_scale, 4) ||
      (cache->weight && !aligned(cache->weight, 16)) || !aligned(batch->page_table, 4) || !aligned(batch->kv_len, 4) ||
      (rows && !aligned(batch->q_start, 4)))
    return EXL3_ERR_ALIGNMENT;
  *dev = initialized_device();
  if (!*dev) return EXL3_ERR_NOT_INITIALIZED;
  *kv = KvView{static_cast<uint8_t *>(cache->k), static_cast<uint8_t *>(cache->v), cache->k_scale, cache->v_scale,
               cache->weight, batch->page_table, batch->kv_len, batch->q_start, cache->n_pages, cache->n_kv_heads,
               cache->head_dim, batch->n_seqs, batch->max_pages, batch->rows, batch->max_rows, (*dev)->status};
  return EXL3_OK;
}

bool attention_shape_ok(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, int32_t n_heads) {
  return cache && batch && cache_shape_ok(*cache) && batch_shape_ok(*batch) && n_heads >= 1 && n_heads <= 65535 &&
         n_heads % cache->n_kv_heads == 0 && (int64_t)batch->rows * n_heads <= INT32_MAX;
}

// 0 is off; below 1e-30 the scores' quotient by it would leave fp32.
bool softcap_ok(float c) { return c == 0.f || (isfinite(c) && c >= 1e-30f); }

bool ld_ok(int64_t ld, int64_t width) { return ld >= width && ld % 8 == 0 && ld <= INT32_MAX; }

}  // namespace

}  // namespace exl3

using namespace exl3;

extern "C" {

exl3_status exl3_kv8_append(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *k, int64_t ldk,
                            const void *v, int64_t ldv, void *stream) {
  if (!cache || !batch || !cache_shape_ok(*cache) || !batch_shape_ok(*batch)) return EXL3_ERR_INVALID_ARG;
  const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
  if (!ld_ok(ldk, width) || !ld_ok(ldv, width)) return EXL3_ERR_INVALID_ARG;
  if (no_rows(*batch)) return EXL3_OK;
  if (!aligned(k, 16) || !aligned(v, 16)) return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev;
  KvView kv;
  const exl3_status s = validate_kv(cache, batch, true, &dev, &kv);
  if (s != EXL3_OK) return s;
  return from_cuda(launch_kv8_append(kv, k, ldk, v, ldv, static_cast<cudaStream_t>(stream)));
}

size_t exl3_kv8_attention_workspace_bytes(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, int32_t n_heads) {
  if (!attention_shape_ok(cache, batch, n_heads)) return 0;
  int d = -1, sms = 0;
  if (const DeviceInfo *dev = initialized_device()) sms = dev->num_sms;
  else if (cudaGetDevice(&d) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d) != cudaSuccess)
    return 0;
  return kv8_attention_workspace_bytes(*cache, *batch, n_heads, sms);
}

exl3_status exl3_kv8_attention(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *q, int64_t ldq,
                               int32_t n_heads, float scale, float softcap, int causal, void *out, int64_t ldo,
                               float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  if (!attention_shape_ok(cache, batch, n_heads)) return EXL3_ERR_INVALID_ARG;
  const int64_t width = (int64_t)n_heads * cache->head_dim;
  if (!ld_ok(ldq, width) || !ld_ok(ldo, width) || !isfinite(scale) || !softcap_ok(softcap))
    return EXL3_ERR_INVALID_ARG;
  if (no_rows(*batch)) return EXL3_OK;
  if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) || !aligned(workspace, 16))
    return EXL3_ERR_ALIGNMENT;
  KvAttention p{};
  const DeviceInfo *dev;
  const exl3_status s = validate_kv(cache, batch, true, &dev, &p.kv);
  if (s != EXL3_OK) return s;
  if (kv8_attention_workspace_bytes(*cache, *batch, n_heads, dev->num_sms) > workspace_bytes)
    return EXL3_ERR_WORKSPACE_TOO_SMALL;
  p.q = q;
  p.ldq = ldq;
  p.n_heads = n_heads;
  p.scale = scale;
  p.softcap = softcap;
  p.causal = causal != 0;
  p.out = out;
  p.ldo = ldo;
  p.lse = lse;
  p.workspace = workspace;
  p.num_sms = dev->num_sms;
  return from_cuda(launch_kv8_attention(p, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_kv8_weigh(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const void *q, int64_t ldq,
                           int32_t n_heads, float scale, float softcap, int causal, const float *lse, void *stream) {
  if (!attention_shape_ok(cache, batch, n_heads)) return EXL3_ERR_INVALID_ARG;
  if (!ld_ok(ldq, (int64_t)n_heads * cache->head_dim) || !isfinite(scale) || !softcap_ok(softcap))
    return EXL3_ERR_INVALID_ARG;
  if (no_rows(*batch)) return EXL3_OK;
  if (!cache->weight || !aligned(q, 16) || !aligned(lse, 4)) return EXL3_ERR_ALIGNMENT;
  KvAttention p{};
  const DeviceInfo *dev;
  const exl3_status s = validate_kv(cache, batch, true, &dev, &p.kv);
  if (s != EXL3_OK) return s;
  p.q = q;
  p.ldq = ldq;
  p.n_heads = n_heads;
  p.scale = scale;
  p.softcap = softcap;
  p.causal = causal != 0;
  p.lse = const_cast<float *>(lse);
  p.num_sms = dev->num_sms;
  return from_cuda(launch_kv8_weigh(p, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_kv8_evict(const exl3_kv8_cache *cache, const exl3_kv8_batch *batch, const int32_t *dst_pages,
                           int32_t budget, int32_t recent, int32_t *kept, int32_t *new_len, void *stream) {
  if (!cache || !batch || !cache_shape_ok(*cache) || batch->n_seqs < 0 || batch->n_seqs > 65535 || batch->max_pages < 0 ||
      batch->max_pages > INT32_MAX / EXL3_KV8_BLOCK || budget < 1 || budget > (1 << 30) || recent < 0 || recent > budget)
    return EXL3_ERR_INVALID_ARG;
  if (batch->n_seqs == 0) return EXL3_OK;
  if (!cache->weight || !aligned(dst_pages, 4) || !aligned(kept, 4) || !aligned(new_len, 4)) return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev;
  KvView kv;
  const exl3_status s = validate_kv(cache, batch, false, &dev, &kv);
  if (s != EXL3_OK) return s;
  return from_cuda(launch_kv8_evict(kv, dst_pages, budget, recent, kept, new_len, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_logits_adjust(const float *logits, int64_t ldl, int64_t M, int64_t n, const exl3_logits_rules *rules,
                               float *out, int64_t ldo, int32_t *argmax, void *stream) {
  if (!rules || M < 0 || M > 65535 || n < 1 || n > (1 << 19) || ldl < n || ldl % 4 || ldo < n || ldo % 4 ||
      rules->history_size < 0 || rules->history_size > (1 << 29) || rules->bias_size < 0 || rules->bias_size > (1 << 29))
    return EXL3_ERR_INVALID_ARG;
  // rows of one buffer at two distances would run into one another
  if (logits == out && ldl != ldo && M > 1) return EXL3_ERR_INVALID_ARG;
  const exl3_logits_rules &r = *rules;
  // parts of a rule go together
  if ((r.history == nullptr) != (r.history_start == nullptr) || (r.generated_from && !r.history) ||
      (r.bias_id == nullptr) != (r.bias_value == nullptr) || (r.bias_id == nullptr) != (r.bias_start == nullptr))
    return EXL3_ERR_INVALID_ARG;
  if (M == 0) return EXL3_OK;
  if (!aligned(logits, 16) || !aligned(out, 16) || !aligned(argmax, 4)) return EXL3_ERR_ALIGNMENT;
  for (const void *p : {(const void *)r.history, (const void *)r.history_start, (const void *)r.generated_from,
                        (const void *)r.repetition, (const void *)r.presence, (const void *)r.frequency,
                        (const void *)r.bias_id, (const void *)r.bias_value, (const void *)r.bias_start,
                        (const void *)r.allowed})
    if (p && !aligned(p, 4)) return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev = initialized_device();
  if (!dev) return EXL3_ERR_NOT_INITIALIZED;
  return from_cuda(launch_logits_adjust(logits, ldl, M, n, r, out, ldo, argmax, dev->status, dev->num_sms,
                                        static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_selftest_bounds_serving(int *units_reported, int *units_total, void *stream) {
  if (!units_reported || !units_total) return EXL3_ERR_INVALID_ARG;
  *units_reported = 0;
  *units_total = 0;
  if (!initialized_device()) return EXL3_ERR_NOT_INITIALIZED;
#if EXL3_DEBUG_BOUNDS
  const exl3_status pending = exl3_get_device_status(stream);
  if (pending != EXL3_OK) return pending;
  cudaError_t (*const probes[])(cudaStream_t) = {bounds_probe_kv8_cache, bounds_probe_kv8_attention, bounds_probe_kv8_chunk,
                                                 bounds_probe_kv8_weigh_chunk,
                                                 bounds_probe_logits_adjust};
  for (auto *probe : probes) {
    ++*units_total;
    if (probe(static_cast<cudaStream_t>(stream)) != cudaSuccess) return EXL3_ERR_CUDA;
    const exl3_status s = exl3_get_device_status(stream);
    if (s == EXL3_ERR_OUT_OF_BOUNDS) ++*units_reported;
    else if (s != EXL3_OK) return s;
  }
#else
  (void)stream;
#endif
  return EXL3_OK;
}

}  // extern "C"
