// Parameters of the attention kernels over rows of new tokens: whole prompts
// (16-bit K and V rows) and chunks over the packed cache.
#pragma once
#include "kvq_internal.h"

namespace kvq {

// A strided tensor of rows [tokens][heads][head_dim] (strides in elements).
struct Rows {
  const void* data;
  long long st, sh;
};

struct RowAttnParams {
  Rows q, k, v;  // k and v: prompts only
  // packed cache: chunks only
  const uint8_t *k_codes, *v_codes;
  const uint16_t *k_scale, *k_zero, *v_scale, *v_zero;
  const int32_t* seq_lens;
  const int32_t* page_table;
  const int32_t* cu;  // [batch + 1] row offsets of the sequences
  void* out;          // [total][num_q_heads][head_dim]
  float* lse;         // [total][num_q_heads] or null
  uint32_t* dev_status;
  int batch, total, num_q_heads, num_kv_heads, gq;  // gq: query heads per KV head
  int head_dim, group, bits, k_scheme, v_scheme, max_blocks, num_pages;
  int causal, fp16;
  float scale_log2;  // sm_scale * log2(e)
  uint32_t flags;
};

// Rows of sequence b in the packed row tensors: [first, first + n); a bad
// entry (negative, decreasing, past `total`) gives an empty sequence.
struct SeqRows {
  int first, n;
  bool bad;
};
__device__ __forceinline__ SeqRows seq_rows(const int32_t* cu, int b, int total) {
  const int a = cu[b], e = cu[b + 1];
  const bool bad = a < 0 || e < a || e > total;
  return {bad ? 0 : a, bad ? 0 : e - a, bad};
}


cudaError_t launch_prompt_attn(const RowAttnParams& p, cudaStream_t stream);

// Rotation of the first `dim` channels of a row by its position: angles
// [positions][dim], cosines and then sines.
struct Turn {
  const float* angles;
  int dim, interleaved;
  float one;  // 1, at run time (append_rotary.cuh)
};
struct AppendParams {
  Rows x[2];  // K, V rows
  int dtype;
  const int32_t* cu;
  const int32_t* seq_lens;
  const int32_t* page_table;
  const float* window[2];
  float* window_out[2];
  uint8_t* codes[2];
  uint16_t* scale[2];
  uint16_t* zero[2];
  uint32_t* dev_status;
  int scheme[2];
  int bits, head_dim, group, num_kv_heads, num_pages, max_blocks, batch, total;
  long long most;  // tokens a sequence may have
  Turn turn;       // append_rotary: K's
};
cudaError_t launch_append_chunk(const AppendParams& p, cudaStream_t stream);

// Rows turned by their positions and written as rows of the same type
// (append_rotary.cu): queries, and keys where an attention over rows follows.
struct TurnRowsParams {
  Rows x[2];     // q, k
  void* out[2];  // [total][heads][head_dim]
  int heads[2];  // 0: none
  int dtype, head_dim, batch, total;
  const int32_t* cu;
  const int32_t* seq_lens;
  long long most;
  Turn turn;
};
cudaError_t launch_append_rotary(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream);

}  // namespace kvq
