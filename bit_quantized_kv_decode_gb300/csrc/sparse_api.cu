// C-ABI entry points of decode steps over part of a cache: the selection of
// blocks and decode attention over lists of them.  Argument checks and launches
// only; nothing here allocates memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sparse_decode.h"

namespace kvq {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What both calls have in common.
kvq_status check_step(const kvq_cache_desc* cache, int batch, int num_q_heads, int max_blocks, int list_len) {
  kvq_status s = check_cache(cache);
  if (s != KVQ_OK) return s;
  if (batch < 1 || batch > 65535 || num_q_heads < 1 || max_blocks < 1 || list_len < 1) return KVQ_ERR_INVALID_ARG;
  if (num_q_heads % cache->num_kv_heads != 0) return KVQ_ERR_UNSUPPORTED;
  const int g = num_q_heads / cache->num_kv_heads;
  if (g != 1 && g != 2 && g != 4 && g != 8) return KVQ_ERR_UNSUPPORTED;
  if (max_blocks > (1 << 23)) return KVQ_ERR_UNSUPPORTED;  // positions are 32-bit
  if ((long long)batch * cache->num_kv_heads * list_len > (1LL << 30)) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq_status check_sparse(const kvq_sparse_desc* d) {
  if (d == nullptr) return KVQ_ERR_INVALID_ARG;
  kvq_status s = check_step(&d->cache, d->batch, d->num_q_heads, d->max_blocks, d->list_len);
  if (s != KVQ_OK) return s;
  if (!std::isfinite(d->sm_scale) || (d->flags & ~(KVQ_FLAG_TEST_STALL | KVQ_FLAG_TEST_STALL_MMA)) != 0)
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

KVQ_API kvq_status kvq_select_blocks(const kvq_select_desc* d, const uint16_t* q, const uint16_t* k_scale,
                                     const uint16_t* k_zero, const int32_t* seq_lens, const int32_t* page_table,
                                     int32_t* blocks, int32_t* counts, uint32_t* dev_status, void* stream) {
  if (d == nullptr) return KVQ_ERR_INVALID_ARG;
  kvq_status s = check_step(&d->cache, d->batch, d->num_q_heads, d->max_blocks, d->budget);
  if (s != KVQ_OK) return s;
  if (d->cache.k_scheme != KVQ_CHANNELWISE || d->max_blocks > kSelectMaxBlocks) return KVQ_ERR_UNSUPPORTED;
  if (d->first < 0 || d->last < 0 || d->first > d->budget || d->last > d->budget - d->first) return KVQ_ERR_INVALID_ARG;
  const void* arrays[] = {q, k_scale, k_zero};
  for (const void* ptr : arrays)
    if (ptr == nullptr || !aligned16(ptr)) return KVQ_ERR_INVALID_ARG;
  const void* words[] = {seq_lens, blocks, counts};
  for (const void* ptr : words)
    if (ptr == nullptr || !aligned4(ptr)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(page_table)) return KVQ_ERR_INVALID_ARG;
  if (page_table == nullptr && (long long)d->batch * d->max_blocks > d->cache.num_pages) return KVQ_ERR_INVALID_ARG;
  s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  SelectParams p{};
  p.q = q; p.k_scale = k_scale; p.k_zero = k_zero; p.seq_lens = seq_lens; p.page_table = page_table;
  p.blocks = blocks; p.counts = counts; p.dev_status = dev_status;
  p.batch = d->batch; p.num_q_heads = d->num_q_heads; p.num_kv_heads = d->cache.num_kv_heads;
  p.gq = d->num_q_heads / d->cache.num_kv_heads; p.max_blocks = d->max_blocks; p.num_pages = d->cache.num_pages;
  p.bits = d->cache.bits; p.head_dim = d->cache.head_dim; p.group = group_of(&d->cache);
  p.budget = d->budget; p.first = d->first; p.last = d->last;
  return launch_select(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_sparse_workspace_size(const kvq_sparse_desc* d, size_t* bytes) {
  kvq_status s = check_sparse(d);
  if (s != KVQ_OK) return s;
  if (bytes == nullptr) return KVQ_ERR_INVALID_ARG;
  *bytes = sparse_plan(d).total;
  return KVQ_OK;
}

KVQ_API kvq_status kvq_sparse_decode_attn(const kvq_sparse_desc* d, const uint16_t* q, const uint8_t* k_codes,
                                          const uint16_t* k_scale, const uint16_t* k_zero, const uint8_t* v_codes,
                                          const uint16_t* v_scale, const uint16_t* v_zero, const int32_t* seq_lens,
                                          const int32_t* page_table, const int32_t* blocks, const int32_t* counts,
                                          uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                          uint32_t* dev_status, void* stream) {
  kvq_status s = check_sparse(d);
  if (s != KVQ_OK) return s;
  const void* arrays[] = {q, k_codes, k_scale, k_zero, v_codes, v_scale, v_zero, out};
  for (const void* ptr : arrays)
    if (ptr == nullptr || !aligned16(ptr)) return KVQ_ERR_INVALID_ARG;
  const void* words[] = {seq_lens, blocks, counts};
  for (const void* ptr : words)
    if (ptr == nullptr || !aligned4(ptr)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(lse)) return KVQ_ERR_INVALID_ARG;
  if (page_table == nullptr && (long long)d->batch * d->max_blocks > d->cache.num_pages) return KVQ_ERR_INVALID_ARG;
  const SparsePlan plan = sparse_plan(d);
  if (plan.total > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
                         workspace_bytes < plan.total))
    return KVQ_ERR_WORKSPACE;
  s = check_device(nullptr);
  if (s != KVQ_OK) return s;
  ListParams p{};
  p.q = q; p.k_codes = k_codes; p.k_scale = k_scale; p.k_zero = k_zero;
  p.v_codes = v_codes; p.v_scale = v_scale; p.v_zero = v_zero;
  p.seq_lens = seq_lens; p.page_table = page_table; p.dev_status = dev_status;
  if (plan.total > 0) {
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.part_lse = reinterpret_cast<float*>(ws + plan.part_lse);
    p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
  }
  p.batch = d->batch; p.num_kv_heads = d->cache.num_kv_heads; p.num_q_heads = d->num_q_heads;
  p.max_blocks = d->max_blocks; p.num_pages = d->cache.num_pages; p.gq = plan.gq;
  p.units_per_seq = d->cache.num_kv_heads;
  p.sm_scale_log2 = (d->sm_scale > 0.0f ? d->sm_scale : 1.0f / std::sqrt((float)d->cache.head_dim)) * 1.4426950408889634f;
  p.flags = d->flags;
  p.wait_limit_ns = d->flags != 0 ? 50ull * 1000 * 1000 : 2ull * 1000 * 1000 * 1000;
  p.nibble_mul = 1u << 28;
  p.minus_one = 0xffffffffu;
  p.blocks = blocks; p.counts = counts; p.out = out; p.lse = lse;
  p.list_len = d->list_len; p.splits = plan.splits; p.head_dim = d->cache.head_dim;
  return launch_sparse_decode(d->cache, plan, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
