// C-ABI entry points for rows of new tokens: attention over whole prompts,
// appending a chunk to the packed cache, attention of a chunk over the cache.
// Argument checks and launches only; nothing here allocates memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "chunk_attn.h"

namespace kvq {
namespace {

constexpr int kMaxGroup = 16;  // query heads per KV head

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A row tensor of elements of `size` bytes: 16-byte aligned base and strides.
bool rows_ok(const kvq_rows* r, int size) {
  if (r == nullptr || r->data == nullptr || !aligned16(r->data)) return false;
  const long long unit = 16 / size, most = 1LL << 38;  // a 40-bit byte stride
  return r->stride_token > 0 && r->stride_head > 0 && r->stride_token % unit == 0 && r->stride_head % unit == 0 &&
         r->stride_token < most / size && r->stride_head < most / size;
}
Rows rows_of(const kvq_rows* r) { return {r->data, r->stride_token, r->stride_head}; }

kvq_status check_heads(int head_dim, int num_q_heads, int num_kv_heads, int batch, int total, int dtype) {
  if (num_kv_heads < 1 || num_q_heads < 1 || batch < 1 || batch > 65535 || total < 0) return KVQ_ERR_INVALID_ARG;
  if (dtype != KVQ_BF16 && dtype != KVQ_FP16) return dtype == KVQ_FP32 ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kMaxGroup || num_kv_heads > 65535)
    return KVQ_ERR_UNSUPPORTED;
  if ((long long)total * num_q_heads > (1LL << 30)) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq_status check_chunk(const kvq_chunk_desc* d) {
  if (d == nullptr) return KVQ_ERR_INVALID_ARG;
  kvq_status s = check_cache(&d->cache);
  if (s != KVQ_OK) return s;
  s = check_heads(d->cache.head_dim, d->num_q_heads, d->cache.num_kv_heads, d->batch, d->total_tokens, d->dtype);
  if (s != KVQ_OK) return s;
  if (d->max_blocks < 1 || (d->causal != 0 && d->causal != 1)) return KVQ_ERR_INVALID_ARG;
  if (d->max_blocks > (1 << 23)) return KVQ_ERR_UNSUPPORTED;  // positions are 32-bit
  if (!std::isfinite(d->sm_scale) || (d->flags & ~KVQ_FLAG_TEST_STALL) != 0) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

float scale_log2(float sm_scale, int head_dim) {
  return (sm_scale > 0.0f ? sm_scale : 1.0f / std::sqrt((float)head_dim)) * 1.4426950408889634f;
}

// The arguments of an append call, checked, as the kernels take them.
kvq_status append_params(const kvq_cache_desc* cache, int32_t dtype, const kvq_rows* k, const kvq_rows* v, int32_t batch,
                         int32_t total_tokens, const int32_t* cu_seqlens, const int32_t* seq_lens,
                         const int32_t* page_table, int32_t max_blocks, const float* k_window, const float* v_window,
                         float* k_window_out, float* v_window_out, uint8_t* k_codes, uint16_t* k_scale,
                         uint16_t* k_zero, uint8_t* v_codes, uint16_t* v_scale, uint16_t* v_zero, uint32_t* dev_status,
                         AppendParams* params) {
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (dtype != KVQ_BF16 && dtype != KVQ_FP16 && dtype != KVQ_FP32) return KVQ_ERR_INVALID_ARG;
  if (batch < 1 || batch > 65535 || total_tokens < 0 || max_blocks < 1 || max_blocks > (1 << 23) ||
      cache->num_kv_heads > 65535)
    return KVQ_ERR_INVALID_ARG;
  if (page_table == nullptr && (long long)batch * max_blocks > cache->num_pages) return KVQ_ERR_INVALID_ARG;
  const int size = dtype == KVQ_FP32 ? 4 : 2;
  if (total_tokens > 0 && (!rows_ok(k, size) || !rows_ok(v, size))) return KVQ_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr || seq_lens == nullptr) return KVQ_ERR_INVALID_ARG;
  const void* ints[] = {cu_seqlens, seq_lens, page_table};
  for (const void* ptr : ints)
    if (!aligned4(ptr)) return KVQ_ERR_INVALID_ARG;
  const void* arrays[] = {k_codes, k_scale, k_zero, v_codes, v_scale, v_zero};
  for (const void* ptr : arrays)
    if (ptr == nullptr || !aligned16(ptr)) return KVQ_ERR_INVALID_ARG;
  const float* window[2] = {k_window, v_window};
  float* window_out[2] = {k_window_out, v_window_out};
  for (int i = 0; i < 2; ++i) {
    if ((window[i] == nullptr) != (window_out[i] == nullptr)) return KVQ_ERR_INVALID_ARG;
    if (window[i] == nullptr && (i ? cache->v_scheme : cache->k_scheme) == KVQ_CHANNELWISE) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(window[i]) || !aligned16(window_out[i])) return KVQ_ERR_INVALID_ARG;
  }
  AppendParams& p = *params;
  p = AppendParams{};
  if (total_tokens > 0) { p.x[0] = rows_of(k); p.x[1] = rows_of(v); }
  p.dtype = dtype;
  p.cu = cu_seqlens; p.seq_lens = seq_lens; p.page_table = page_table;
  for (int i = 0; i < 2; ++i) { p.window[i] = window[i]; p.window_out[i] = window_out[i]; }
  p.codes[0] = k_codes; p.scale[0] = k_scale; p.zero[0] = k_zero;
  p.codes[1] = v_codes; p.scale[1] = v_scale; p.zero[1] = v_zero;
  p.dev_status = dev_status; p.scheme[0] = cache->k_scheme; p.scheme[1] = cache->v_scheme;
  p.bits = cache->bits; p.head_dim = cache->head_dim; p.group = group_of(cache);
  p.num_kv_heads = cache->num_kv_heads; p.num_pages = cache->num_pages; p.max_blocks = max_blocks;
  p.batch = batch; p.total = total_tokens;
  p.most = (long long)max_blocks * kBlockTokens;
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

KVQ_API kvq_status kvq_prompt_attn(const kvq_prompt_desc* d, const kvq_rows* q, const kvq_rows* k, const kvq_rows* v,
                                   const int32_t* cu_seqlens, void* out, float* lse, uint32_t* dev_status,
                                   void* stream) {
  if (d == nullptr) return KVQ_ERR_INVALID_ARG;
  kvq_status s = check_heads(d->head_dim, d->num_q_heads, d->num_kv_heads, d->batch, d->total_tokens, d->dtype);
  if (s != KVQ_OK) return s;
  if ((d->causal != 0 && d->causal != 1) || !std::isfinite(d->sm_scale) || (d->flags & ~KVQ_FLAG_TEST_STALL) != 0)
    return KVQ_ERR_INVALID_ARG;
  if (d->total_tokens == 0) return check_device(nullptr);  // no rows: nothing to read or write
  if (!rows_ok(q, 2) || !rows_ok(k, 2) || !rows_ok(v, 2) || cu_seqlens == nullptr || !aligned4(cu_seqlens) ||
      out == nullptr || !aligned16(out) || !aligned4(lse))
    return KVQ_ERR_INVALID_ARG;
  s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  RowAttnParams p{};
  p.q = rows_of(q); p.k = rows_of(k); p.v = rows_of(v);
  p.cu = cu_seqlens; p.out = out; p.lse = lse; p.dev_status = dev_status;
  p.batch = d->batch; p.total = d->total_tokens; p.num_q_heads = d->num_q_heads; p.num_kv_heads = d->num_kv_heads;
  p.gq = d->num_q_heads / d->num_kv_heads;
  p.head_dim = d->head_dim; p.causal = d->causal; p.fp16 = d->dtype == KVQ_FP16;
  p.scale_log2 = scale_log2(d->sm_scale, d->head_dim); p.flags = d->flags;
  return launch_prompt_attn(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_append_chunk(const kvq_cache_desc* cache, int32_t dtype, const kvq_rows* k, const kvq_rows* v,
                                    int32_t batch, int32_t total_tokens, const int32_t* cu_seqlens,
                                    const int32_t* seq_lens, const int32_t* page_table, int32_t max_blocks,
                                    const float* k_window, const float* v_window, float* k_window_out,
                                    float* v_window_out, uint8_t* k_codes, uint16_t* k_scale, uint16_t* k_zero,
                                    uint8_t* v_codes, uint16_t* v_scale, uint16_t* v_zero, uint32_t* dev_status,
                                    void* stream) {
  AppendParams p;
  kvq_status s = append_params(cache, dtype, k, v, batch, total_tokens, cu_seqlens, seq_lens, page_table, max_blocks,
                               k_window, v_window, k_window_out, v_window_out, k_codes, k_scale, k_zero, v_codes,
                               v_scale, v_zero, dev_status, &p);
  if (s == KVQ_OK) s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  return launch_append_chunk(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_append_rotary(const kvq_cache_desc* cache, int32_t dtype, const kvq_rotary* rotary,
                                     const kvq_rows* q, int32_t num_q_heads, const kvq_rows* k, const kvq_rows* v,
                                     int32_t batch, int32_t total_tokens, const int32_t* cu_seqlens,
                                     const int32_t* seq_lens, const int32_t* page_table, int32_t max_blocks,
                                     const float* k_window, const float* v_window, float* k_window_out,
                                     float* v_window_out, uint8_t* k_codes, uint16_t* k_scale, uint16_t* k_zero,
                                     uint8_t* v_codes, uint16_t* v_scale, uint16_t* v_zero, void* q_out, void* k_out,
                                     uint32_t* dev_status, void* stream) {
  AppendParams p;
  kvq_status s = append_params(cache, dtype, k, v, batch, total_tokens, cu_seqlens, seq_lens, page_table, max_blocks,
                               k_window, v_window, k_window_out, v_window_out, k_codes, k_scale, k_zero, v_codes,
                               v_scale, v_zero, dev_status, &p);
  if (s != KVQ_OK) return s;
  if (rotary == nullptr || rotary->angles == nullptr || !aligned16(rotary->angles) || rotary->positions < 1 ||
      (rotary->interleaved != 0 && rotary->interleaved != 1))
    return KVQ_ERR_INVALID_ARG;
  if (rotary->dim < 16 || rotary->dim % 16 != 0 || rotary->dim > cache->head_dim) return KVQ_ERR_UNSUPPORTED;
  const bool queries = q != nullptr && total_tokens > 0;
  if ((q != nullptr) != (q_out != nullptr) && total_tokens > 0) return KVQ_ERR_INVALID_ARG;
  if (queries && (!rows_ok(q, dtype == KVQ_FP32 ? 4 : 2) || num_q_heads < 1 || num_q_heads > 65535)) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(k_out)) return KVQ_ERR_INVALID_ARG;
  s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  p.turn = Turn{rotary->angles, rotary->dim, rotary->interleaved, 1.0f};
  if (rotary->positions < p.most) p.most = rotary->positions;
  TurnRowsParams t{};
  if (queries) { t.x[0] = rows_of(q); t.out[0] = q_out; t.heads[0] = num_q_heads; }
  if (k_out != nullptr) { t.x[1] = p.x[0]; t.out[1] = k_out; t.heads[1] = p.num_kv_heads; }
  t.dtype = dtype; t.head_dim = p.head_dim; t.batch = batch; t.total = total_tokens;
  t.cu = cu_seqlens; t.seq_lens = seq_lens; t.most = p.most; t.turn = p.turn;
  return launch_append_rotary(p, t, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_chunk_workspace_size(const kvq_chunk_desc* d, size_t* bytes) {
  kvq_status s = check_chunk(d);
  if (s != KVQ_OK) return s;
  if (bytes == nullptr) return KVQ_ERR_INVALID_ARG;
  *bytes = chunk_plan(d->cache.head_dim, group_of(&d->cache), d->cache.bits, d->batch, d->total_tokens, d->num_q_heads, d->cache.num_kv_heads).total;
  return KVQ_OK;
}

KVQ_API kvq_status kvq_chunk_attn(const kvq_chunk_desc* d, const kvq_rows* q, const uint8_t* k_codes,
                                  const uint16_t* k_scale, const uint16_t* k_zero, const uint8_t* v_codes,
                                  const uint16_t* v_scale, const uint16_t* v_zero, const int32_t* cu_seqlens,
                                  const int32_t* seq_lens, const int32_t* page_table, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  kvq_status s = check_chunk(d);
  if (s != KVQ_OK) return s;
  if (d->total_tokens == 0) return check_device(nullptr);  // no rows: nothing to read or write
  const void* arrays[] = {k_codes, k_scale, k_zero, v_codes, v_scale, v_zero, out};
  for (const void* ptr : arrays)
    if (ptr == nullptr || !aligned16(ptr)) return KVQ_ERR_INVALID_ARG;
  if (!rows_ok(q, 2) || cu_seqlens == nullptr || seq_lens == nullptr) return KVQ_ERR_INVALID_ARG;
  const void* words[] = {cu_seqlens, seq_lens, page_table, lse};
  for (const void* ptr : words)
    if (!aligned4(ptr)) return KVQ_ERR_INVALID_ARG;
  if (page_table == nullptr && (long long)d->batch * d->max_blocks > d->cache.num_pages) return KVQ_ERR_INVALID_ARG;
  const ChunkPlan plan =
      chunk_plan(d->cache.head_dim, group_of(&d->cache), d->cache.bits, d->batch, d->total_tokens, d->num_q_heads, d->cache.num_kv_heads);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < plan.total)
    return KVQ_ERR_WORKSPACE;
  s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  RowAttnParams p{};
  p.q = rows_of(q);
  p.k_codes = k_codes; p.k_scale = k_scale; p.k_zero = k_zero;
  p.v_codes = v_codes; p.v_scale = v_scale; p.v_zero = v_zero;
  p.seq_lens = seq_lens; p.page_table = page_table; p.cu = cu_seqlens; p.out = out; p.lse = lse;
  p.dev_status = dev_status; p.batch = d->batch; p.total = d->total_tokens; p.num_q_heads = d->num_q_heads;
  p.num_kv_heads = d->cache.num_kv_heads; p.gq = d->num_q_heads / d->cache.num_kv_heads;
  p.head_dim = d->cache.head_dim; p.group = group_of(&d->cache); p.bits = d->cache.bits;
  p.k_scheme = d->cache.k_scheme; p.v_scheme = d->cache.v_scheme; p.max_blocks = d->max_blocks;
  p.num_pages = d->cache.num_pages; p.causal = d->causal; p.fp16 = d->dtype == KVQ_FP16;
  p.scale_log2 = scale_log2(d->sm_scale, p.head_dim); p.flags = d->flags;
  return launch_chunk_attn(p, plan, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
