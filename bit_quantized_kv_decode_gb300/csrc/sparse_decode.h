// Attention over lists of blocks and the selection of such lists: parameters,
// the split of the lists, launch entries.
#pragma once
#include "decode_general.h"

namespace kvq {

// How the lists of a call are cut, from its sizes alone (host only).
struct SparsePlan {
  GenLaunch launch;
  int nh, gq;       // query heads a unit holds (4 or 8), and has
  int units;        // sequences x KV heads
  int splits;       // ranges of a unit's list, at most
  size_t part_lse, part_o, total;  // workspace offsets and size
};
SparsePlan sparse_plan(const kvq_sparse_desc* d);

// The kernels of a call over lists of blocks (p's part pointers set).
cudaError_t launch_sparse_decode(const kvq_cache_desc& cache, const SparsePlan& plan, const ListParams& p,
                                 cudaStream_t stream);

struct SelectParams {
  const uint16_t* q;  // bf16 [B][Hq][D]
  const uint16_t* k_scale;
  const uint16_t* k_zero;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int32_t* blocks;  // [B][Hkv][budget]
  int32_t* counts;  // [B][Hkv]
  uint32_t* dev_status;
  int batch, num_q_heads, num_kv_heads, gq, max_blocks, num_pages;
  int bits, head_dim, group;
  int budget, first, last;
};
constexpr int kSelectMaxBlocks = 16384;  // blocks of a sequence that a selection takes (their scores are in shared memory)
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream);

}  // namespace kvq
