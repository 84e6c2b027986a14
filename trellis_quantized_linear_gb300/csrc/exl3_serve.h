// Host-side interfaces of the serving operators (8-bit paged key/value cache,
// logits adjustment).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/exl3.h"

namespace exl3 {

// One call's cache and sequences, as the kernels take them.
struct KvView {
  uint8_t *k, *v;
  float *k_scale, *v_scale, *weight;
  const int32_t *page_table, *kv_len, *q_start;
  int64_t n_pages;
  int n_kv_heads, head_dim;
  int n_seqs, max_pages, rows, max_rows;
  int *status;  // device error word
};

struct KvAttention {
  KvView kv;
  const void *q;
  int64_t ldq;
  int n_heads;
  float scale, softcap;
  int causal;
  void *out;
  int64_t ldo;
  float *lse;
  void *workspace;
  int num_sms;
};

// The sequences [s0, s0 + n) of a call.
inline KvView kv_slice(const KvView &kv, int s0, int n) {
  KvView v = kv;
  v.page_table += (int64_t)s0 * kv.max_pages;
  v.kv_len += s0;
  v.q_start += s0;
  v.n_seqs = n;
  return v;
}

cudaError_t init_kv8_cache_kernels(int *status);
cudaError_t init_kv8_attention_kernels(int *status);
cudaError_t init_kv8_chunk_kernels(int *status);
cudaError_t init_kv8_weigh_chunk_kernels(int *status);
cudaError_t init_logits_adjust_kernels(int *status);

cudaError_t launch_kv8_append(const KvView &kv, const void *k, int64_t ldk, const void *v, int64_t ldv, cudaStream_t st);
cudaError_t launch_kv8_evict(const KvView &kv, const int32_t *dst_pages, int budget, int recent, int32_t *kept,
                             int32_t *new_len, cudaStream_t st);
size_t kv8_attention_workspace_bytes(const exl3_kv8_cache &cache, const exl3_kv8_batch &batch, int n_heads, int num_sms);
cudaError_t launch_kv8_attention(const KvAttention &p, cudaStream_t st);
// More rows than the stream kernel takes (exl3_kv8_chunk.cu).
size_t kv8_chunk_workspace_bytes(int head_dim, int num_sms);
cudaError_t launch_kv8_chunk_attention(const KvAttention &p, cudaStream_t st);
// lse of the call that p describes; adds to p.kv.weight.
cudaError_t launch_kv8_weigh(const KvAttention &p, cudaStream_t st);
// The same for many rows (exl3_kv8_weigh_chunk.cu).
cudaError_t launch_kv8_weigh_chunk(const KvAttention &p, cudaStream_t st);
cudaError_t launch_logits_adjust(const float *logits, int64_t ldl, int64_t M, int64_t n, const exl3_logits_rules &r,
                                 float *out, int64_t ldo, int32_t *argmax, int *status, int num_sms, cudaStream_t st);

// What a step does around its projections (exl3_step_api.cu).
struct PromptAttention {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  int n_heads, n_kv_heads, head_dim;
  const int32_t *q_start;
  int n_seqs, rows;
  float scale, softcap;
  int causal;
  void *out;
  int64_t ldo;
  float *lse;
  int *status;
};
struct KvPlan {
  const int32_t *tokens, *cached, *free_count;
  int32_t *page_table, *kv_len, *q_start, *free_pages, *free_left, *position, *slot, *served;
  int n_seqs, max_pages, rows, max_rows, free_capacity, n_pages;
  int *status;
};
struct QkRotary {
  const void *x;
  void *out;
  int64_t ldx, ldo;
  int rows, q_heads, k_heads, head_dim;
  const int32_t *position;
  const float *cos_sin;
  int n_positions, rot_dim, interleaved;
  const void *q_weight, *k_weight;
  float eps, weight_offset;
  int *status;
};
cudaError_t init_prompt_attention_kernels(int *status, int (&clusters)[2][2]);
cudaError_t init_kv8_plan_kernels(int *status);
cudaError_t init_rms_norm_kernels(int *status);
cudaError_t init_qk_rotary_kernels(int *status);
cudaError_t launch_prompt_attention(const PromptAttention &p, int num_sms, const int (&clusters)[2][2], cudaStream_t st);
cudaError_t launch_kv8_plan(const KvPlan &p, cudaStream_t st);
cudaError_t launch_rms_norm(const exl3_norm &p, int num_sms, int *status, cudaStream_t st);
cudaError_t launch_qk_rotary(const QkRotary &p, int num_sms, cudaStream_t st);

#if EXL3_DEBUG_BOUNDS
cudaError_t bounds_probe_prompt_attention(cudaStream_t st);
cudaError_t bounds_probe_kv8_plan(cudaStream_t st);
cudaError_t bounds_probe_rms_norm(cudaStream_t st);
cudaError_t bounds_probe_qk_rotary(cudaStream_t st);
cudaError_t bounds_probe_kv8_cache(cudaStream_t st);
cudaError_t bounds_probe_kv8_attention(cudaStream_t st);
cudaError_t bounds_probe_kv8_chunk(cudaStream_t st);
cudaError_t bounds_probe_kv8_weigh_chunk(cudaStream_t st);
cudaError_t bounds_probe_logits_adjust(cudaStream_t st);
#endif

}  // namespace exl3
