// pkv_kernels.h -- internal launchers behind the C ABI (host side).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

// Rows of num_kv_heads x head_dim bf16 (head_dim a multiple of 8), page size 16.
int launch_append(const void* k_new, const void* v_new, const int32_t* slot_mapping, int32_t n_tokens, void* k_pages,
                  void* v_pages, int32_t num_pages, int32_t num_kv_heads, int32_t head_dim, int* status, int num_sms,
                  cudaStream_t stream);

// Decode (decode.cu, decode_kernel.cuh): page size 16, head_dim 64 or 128, num_q_heads / num_kv_heads
// from 1 to 8. Workspace = [status header | counters | records], laid out in decode_kernel.cuh.
bool decode_supported(int num_q_heads, int num_kv_heads, int head_dim, int page_size);
size_t decode_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim, int32_t batch, int num_sms);
// k_new / v_new (nullable): fused append of each request's new token at position seq_lens[b] - 1.
// rope (nullable, needs k_new): cos/sin table [rope_max_pos][head_dim]; the new key row and the
// query rows are rotated at that position. flags: 0 or PKV_DECODE_EARLY_PREFETCH.
int launch_decode(const void* q, const void* k_new, const void* v_new, const void* k_pages, const void* v_pages,
                  const int32_t* block_table, const int32_t* seq_lens, const float* rope, int32_t rope_max_pos,
                  void* out, float scale, int num_q_heads, int num_kv_heads, int head_dim, int32_t batch,
                  int32_t max_pages, int32_t num_pages, void* workspace, int num_sms, cudaStream_t stream,
                  uint32_t flags);
// The 8-bit cache (decode_fp8_d64.cu, decode_fp8_d128.cu): the same geometries and workspace.
struct DecodeFp8 {
  const void* q;
  const void* k_new;  // fused step: the new rows, written at seq_lens - 1; nullptr: attention alone
  const void* v_new;
  const void* k_pages;
  const void* v_pages;
  const void* kv_scales;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* rope;  // fused step: optional table, and norm weights
  int32_t rope_max_pos;
  const void* q_weight;
  const void* k_weight;
  float eps;
  void* out;
  float scale;
};
int launch_decode_fp8(const DecodeFp8& f, int num_q_heads, int num_kv_heads, int head_dim, int32_t batch,
                      int32_t max_pages, int32_t num_pages, void* workspace, int num_sms, cudaStream_t stream,
                      uint32_t flags);
int decode_max_batch();

// Append with the rotary embedding and per-head norm (append_rope.cu): head_dim 64 or 128, page size 16.
struct AppendRopeArgs {
  const __nv_bfloat16* q;  // [n_tokens][hq][D], token stride q_stride elements; hq = 0: no query rows
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  long long q_stride, k_stride, v_stride;
  const int32_t* positions;     // with cos_sin
  const int32_t* slot_mapping;  // negative: the token's k and v are not written
  const float* cos_sin;         // [rope_max_pos][D], or nullptr: no rotation
  const __nv_bfloat16* q_weight;  // [D], or nullptr: no norm
  const __nv_bfloat16* k_weight;
  __nv_bfloat16* q_out;  // [n_tokens][hq][D]
  void* k_pages;         // bf16, or e4m3 where scales is given
  void* v_pages;
  uint8_t* scales;
  int* status;
  float eps;
  int n_tokens, hq, hkv, rope_max_pos, num_pages;
};
int launch_append_rope(const AppendRopeArgs& a, int head_dim, int num_sms, cudaStream_t stream);

// Pages of the 8-bit cache as bf16 pages (expand_fp8.cu): head_dim 64 or 128, page size 16.
struct ExpandArgs {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const uint8_t* scales;
  const int32_t* block_table;  // [num_seqs][max_pages]
  const int32_t* seq_lens;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  const int32_t* out_block_table;
  int* status;
  int num_seqs, max_pages, hkv, num_pages, out_pages;
};
int launch_expand_fp8(const ExpandArgs& a, int head_dim, int num_sms, cudaStream_t stream);

// Rotary-embedding table (rope.cu): fp32 [max_pos][head_dim], row p = cos(p w_i) for i < head_dim / 2,
// then sin(p w_i), w_i = theta^(-2 i / head_dim), angles in double rounded to float once.
int launch_rope_table(float* table, int32_t max_pos, int32_t head_dim, double theta, cudaStream_t stream);

// Chunked prefill (prefill.cu): page size 16, head_dim 64 or 128, 1 to 8 query heads per KV head.
bool prefill_supported(int num_q_heads, int num_kv_heads, int head_dim, int page_size);
size_t prefill_workspace_bytes(int num_q_heads, int num_kv_heads, int32_t num_seqs, int32_t max_q_len, int num_sms);
int prefill_max_seqs();
// The decode half of a mixed step (16/8/128 only): decode requests attended in the prefill launch.
struct MixedDecode {
  const void* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  int32_t batch;
  int32_t max_pages;
};
// Workspace of the mixed step: the prefill workspace, then the decode chunks' counters and records.
size_t mixed_workspace_bytes(int32_t num_seqs, int32_t max_q_len, int32_t dec_batch, int32_t dec_max_pages,
                             int num_sms);
// dec: nullptr for prefill alone; otherwise the launch also attends the decode requests (the mixed step).
int launch_prefill(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                   const int32_t* prefix_lens, const int32_t* cu_q_lens, int32_t num_seqs, int32_t total_q,
                   void* out, float scale, int num_q_heads, int num_kv_heads, int head_dim, int32_t max_pages,
                   int32_t max_q_len, int32_t num_pages, void* workspace, cudaStream_t stream,
                   const MixedDecode* dec = nullptr);

int launch_wait_timeout_selftest(void* workspace, long long limit_cycles, cudaStream_t stream);

}  // namespace pkv
