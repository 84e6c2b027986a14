// C ABI of the step operators (block tables, norm, rotation, prompt attention):
// argument validation. Declarations and argument contracts are in include/exl3.h.
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
bool ld_ok(int64_t ld, int64_t width) { return ld >= width && ld % 8 == 0 && ld <= INT32_MAX; }
bool dtype_ok(int32_t t) { return t == EXL3_F16 || t == EXL3_F32; }
// Two matrices that start at one address are one buffer: same type, same rows.
bool one_buffer_ok(const void *a, int32_t ta, int64_t lda, const void *b, int32_t tb, int64_t ldb) {
  return a != b || a == nullptr || (ta == tb && lda == ldb);
}

}  // namespace

}  // namespace exl3

using namespace exl3;

extern "C" {

exl3_status exl3_kv8_plan(const exl3_kv8_batch *batch, const int32_t *tokens, const int32_t *cached, int32_t *free_pages,
                          int32_t free_capacity, const int32_t *free_count, int32_t *free_left, int64_t n_pages,
                          int32_t *position, int32_t *slot, int32_t *served, void *stream) {
  constexpr int32_t kMost = (1 << 30) - 1;
  if (!batch || batch->n_seqs < 0 || batch->n_seqs > 65535 || batch->max_pages < 0 ||
      batch->max_pages > INT32_MAX / EXL3_KV8_BLOCK || batch->rows < 0 || batch->rows > kMost || batch->max_rows < 0 ||
      free_capacity < 0 || free_capacity > kMost || n_pages < 1 || n_pages > INT32_MAX / EXL3_KV8_BLOCK)
    return EXL3_ERR_INVALID_ARG;
  // empty arrays may come with null pointers
  if (!aligned(free_count, 4) || !aligned(free_left, 4) || !aligned(served, 4) || !aligned(batch->q_start, 4) ||
      (free_capacity > 0 && !aligned(free_pages, 4)) || (batch->rows > 0 && (!aligned(position, 4) || !aligned(slot, 4))) ||
      (batch->n_seqs > 0 && (!aligned(tokens, 4) || !aligned(cached, 4) || !aligned(batch->kv_len, 4) ||
                             (batch->max_pages > 0 && !aligned(batch->page_table, 4)))))
    return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev = initialized_device();
  if (!dev) return EXL3_ERR_NOT_INITIALIZED;
  KvPlan p;
  p.tokens = tokens;
  p.cached = cached;
  p.free_count = free_count;
  p.page_table = const_cast<int32_t *>(batch->page_table);
  p.kv_len = const_cast<int32_t *>(batch->kv_len);
  p.q_start = const_cast<int32_t *>(batch->q_start);
  p.free_pages = free_pages;
  p.free_left = free_left;
  p.position = position;
  p.slot = slot;
  p.served = served;
  p.n_seqs = batch->n_seqs;
  p.max_pages = batch->max_pages;
  p.rows = batch->rows;
  p.max_rows = batch->max_rows;
  p.free_capacity = free_capacity;
  p.n_pages = (int)n_pages;
  p.status = dev->status;
  return from_cuda(launch_kv8_plan(p, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_rms_norm(const exl3_norm *norm, void *stream) {
  if (!norm) return EXL3_ERR_INVALID_ARG;
  const exl3_norm &n = *norm;
  if (n.rows < 0 || n.rows > INT32_MAX || n.cols < 8 || n.cols > 32768 || n.cols % 8 || !dtype_ok(n.x_dtype) || !ld_ok(n.ldx, n.cols) ||
      !isfinite(n.eps) || n.eps < 0.f || !isfinite(n.weight_offset) || (n.codes == nullptr) != (n.scales == nullptr) ||
      (n.residual_out && !n.residual))
    return EXL3_ERR_INVALID_ARG;
  if (n.residual && (!dtype_ok(n.residual_dtype) || !ld_ok(n.ldr, n.cols) || (n.residual_out && !ld_ok(n.ldro, n.cols))))
    return EXL3_ERR_INVALID_ARG;
  if (n.y && !ld_ok(n.ldy, n.cols)) return EXL3_ERR_INVALID_ARG;
  if (n.codes && (!ld_ok(n.ldc, n.cols) ||
                  !(n.group == n.cols || ((n.group == 32 || n.group == 64 || n.group == 128) && n.cols % n.group == 0))))
    return EXL3_ERR_INVALID_ARG;
  if (!one_buffer_ok(n.x, n.x_dtype, n.ldx, n.residual_out, n.residual_dtype, n.ldro) ||
      !one_buffer_ok(n.residual, n.residual_dtype, n.ldr, n.residual_out, n.residual_dtype, n.ldro) ||
      !one_buffer_ok(n.x, n.x_dtype, n.ldx, n.y, EXL3_F16, n.ldy) ||
      !one_buffer_ok(n.residual, n.residual_dtype, n.ldr, n.y, EXL3_F16, n.ldy) ||
      (n.y && n.y == n.residual_out) || (n.codes && (n.codes == n.x || n.codes == n.residual || n.codes == n.y || n.codes == n.residual_out)))
    return EXL3_ERR_INVALID_ARG;
  if (n.rows == 0) return EXL3_OK;  // with the null pointers that empty tensors have
  if (!n.residual_out && !n.y && !n.codes) return EXL3_ERR_INVALID_ARG;
  if (!aligned(n.x, 16) || (n.residual && !aligned(n.residual, 16)) || (n.residual_out && !aligned(n.residual_out, 16)) ||
      (n.weight && !aligned(n.weight, 16)) || (n.y && !aligned(n.y, 16)) || (n.codes && !aligned(n.codes, 16)) ||
      (n.scales && !aligned(n.scales, 4)))
    return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev = initialized_device();
  if (!dev) return EXL3_ERR_NOT_INITIALIZED;
  return from_cuda(launch_rms_norm(n, dev->num_sms, dev->status, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_qk_rotary(const void *x, int64_t ldx, void *out, int64_t ldo, int64_t rows, int32_t q_heads,
                           int32_t k_heads, int32_t head_dim, const int32_t *position, const float *cos_sin,
                           int64_t n_positions, int32_t rot_dim, int interleaved, const void *q_weight,
                           const void *k_weight, float eps, float weight_offset, void *stream) {
  if (rows < 0 || rows > INT32_MAX || q_heads < 0 || k_heads < 0 || (int64_t)q_heads + k_heads < 1 ||
      (int64_t)q_heads + k_heads > 65535 || (head_dim != 64 && head_dim != 128) || n_positions < 1 || n_positions > INT32_MAX ||
      rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 || !isfinite(eps) || eps < 0.f || !isfinite(weight_offset))
    return EXL3_ERR_INVALID_ARG;
  const int64_t width = ((int64_t)q_heads + k_heads) * head_dim;
  if (!ld_ok(ldx, width) || !ld_ok(ldo, width) || (x == out && x != nullptr && ldx != ldo)) return EXL3_ERR_INVALID_ARG;
  // both weights, or none; one that no head has may be missing
  if ((q_weight || k_weight) && ((!q_weight && q_heads > 0) || (!k_weight && k_heads > 0))) return EXL3_ERR_INVALID_ARG;
  if (rows == 0) return EXL3_OK;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(position, 4) || !aligned(cos_sin, 16) || (q_weight && !aligned(q_weight, 16)) ||
      (k_weight && !aligned(k_weight, 16)))
    return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev = initialized_device();
  if (!dev) return EXL3_ERR_NOT_INITIALIZED;
  QkRotary p;
  p.x = x;
  p.out = out;
  p.ldx = ldx;
  p.ldo = ldo;
  p.rows = (int)rows;
  p.q_heads = q_heads;
  p.k_heads = k_heads;
  p.head_dim = head_dim;
  p.position = position;
  p.cos_sin = cos_sin;
  p.n_positions = (int)n_positions;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.weight_offset = weight_offset;
  p.status = dev->status;
  return from_cuda(launch_qk_rotary(p, dev->num_sms, static_cast<cudaStream_t>(stream)));
}

exl3_status exl3_prompt_attention(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                  int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, const int32_t *q_start,
                                  int32_t n_seqs, int64_t rows, float scale, float softcap, int causal, void *out,
                                  int64_t ldo, float *lse, void *stream) {
  if ((head_dim != 64 && head_dim != 128) || n_heads < 1 || n_heads > 65535 || n_kv_heads < 1 || n_heads % n_kv_heads ||
      n_heads / n_kv_heads > 128 || n_seqs < 0 || n_seqs > 65535 || rows < 0 || rows > INT32_MAX || rows * n_heads > INT32_MAX ||
      !isfinite(scale) || !(softcap == 0.f || (isfinite(softcap) && softcap >= 1e-30f)))
    return EXL3_ERR_INVALID_ARG;
  const int64_t width = (int64_t)n_heads * head_dim, kv_width = (int64_t)n_kv_heads * head_dim;
  if (!ld_ok(ldq, width) || !ld_ok(ldk, kv_width) || !ld_ok(ldv, kv_width) || !ld_ok(ldo, width)) return EXL3_ERR_INVALID_ARG;
  if (rows == 0 || n_seqs == 0) return EXL3_OK;
  if (out && (out == q || out == k || out == v)) return EXL3_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(q_start, 4) || (lse && !aligned(lse, 4)))
    return EXL3_ERR_ALIGNMENT;
  const DeviceInfo *dev = initialized_device();
  if (!dev) return EXL3_ERR_NOT_INITIALIZED;
  PromptAttention p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.n_heads = n_heads;
  p.n_kv_heads = n_kv_heads;
  p.head_dim = head_dim;
  p.q_start = q_start;
  p.n_seqs = n_seqs;
  p.rows = (int)rows;
  p.scale = scale;
  p.softcap = softcap;
  p.causal = causal != 0;
  p.out = out;
  p.ldo = ldo;
  p.lse = lse;
  p.status = dev->status;
  return from_cuda(launch_prompt_attention(p, dev->num_sms, dev->prompt_clusters, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
