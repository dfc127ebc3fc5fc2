// Decode attention over lists of blocks: how the lists are cut, the dispatch of
// the kernel instances (decode_general_kernel with LISTED), and the log-sum-exp
// merge of the ranges.
#include "decode_general.cuh"
#include "sparse_decode.h"

namespace kvq {

namespace {

constexpr int kSms = 152;          // of a GB300
constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024;

// What a CTA takes besides its blocks, in blocks.
constexpr int kFixedBlocks = 3;

// Ranges per list: the count with the least time when every list is full --
// waves of resident CTAs times what one of them takes -- and of equals the
// fewest, as each range adds a part to the merge.
int sparse_splits(long long units, int list_len, long long resident) {
  long long best = -1;
  int splits = 1;
  for (int s = 1; s <= list_len; ++s) {
    const long long waves = (units * s + resident - 1) / resident;
    const long long cost = waves * ((list_len + s - 1) / s + kFixedBlocks);
    if (best < 0 || cost < best) {
      best = cost;
      splits = s;
    }
    if (units * s > 8 * resident) break;
  }
  return splits;
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// One CTA per (sequence, query head): groups of D / 4 threads take every
// kParts-th part of the row, a float4 of channels each.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) listed_merge_kernel(const ListParams p) {
  gen::grid_dep_wait();  // the decode kernel's parts
  __shared__ float top[kMergeThreads / 32], sum[kMergeThreads / 32];
  __shared__ __align__(16) float4 acc[kMergeThreads];
  const int D4 = p.head_dim / 4, groups = kMergeThreads / D4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, b = row / p.num_q_heads, head = row % p.num_q_heads;
  const int u = b * p.units_per_seq + head / p.gq, k = head % p.gq;
  const int nr = min(p.splits, listed_unit(p, u).n);
  const size_t slot0 = (size_t)u * p.splits;
  auto lse_of = [&](int s) { return p.part_lse[(slot0 + s) * p.gq + k]; };
  float m = -INFINITY;
  for (int s = tid; s < nr; s += kMergeThreads) m = fmaxf(m, lse_of(s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) top[warp] = m;
  __syncthreads();
  m = top[0];
#pragma unroll
  for (int w = 1; w < kMergeThreads / 32; ++w) m = fmaxf(m, top[w]);
  const bool none = m == -INFINITY;  // no entry, or bad ones alone
  float t = 0.f;
  for (int s = tid; s < nr && !none; s += kMergeThreads) t += expf(lse_of(s) - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) sum[warp] = t;
  const int g = tid / D4, d = tid % D4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!none) {
#pragma unroll 4
    for (int s = g; s < nr; s += groups) {
      const float w = expf(lse_of(s) - m);
      const float4 v = reinterpret_cast<const float4*>(p.part_o + ((slot0 + s) * p.gq + k) * p.head_dim)[d];
      a.x = fmaf(w, v.x, a.x);
      a.y = fmaf(w, v.y, a.y);
      a.z = fmaf(w, v.z, a.z);
      a.w = fmaf(w, v.w, a.w);
    }
  }
  acc[tid] = a;
  __syncthreads();
  t = sum[0];
#pragma unroll
  for (int w = 1; w < kMergeThreads / 32; ++w) t += sum[w];
  if (g == 0) {
    for (int i = 1; i < groups; ++i) {
      const float4 v = acc[i * D4 + d];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float inv = none ? 0.f : 1.f / t;
    const ushort4 o = make_ushort4(gen::bf16_bits(a.x * inv), gen::bf16_bits(a.y * inv), gen::bf16_bits(a.z * inv),
                                   gen::bf16_bits(a.w * inv));
    reinterpret_cast<ushort4*>(p.out + (size_t)row * p.head_dim)[d] = o;
  }
  if (tid == 0 && p.lse != nullptr) p.lse[row] = none ? -INFINITY : m + logf(t);
}

}  // namespace

SparsePlan sparse_plan(const kvq_sparse_desc* d) {
  const kvq_cache_desc& c = d->cache;
  SparsePlan plan;
  plan.gq = d->num_q_heads / c.num_kv_heads;
  plan.nh = plan.gq > 4 ? 8 : 4;
  plan.units = d->batch * c.num_kv_heads;
  plan.launch = general_launch_shape(c.bits, c.k_scheme, c.v_scheme, c.head_dim, group_of(&c), false, plan.nh,
                                     kSmemPerSm, kSmemReserved);
  plan.splits = sparse_splits(plan.units, d->list_len, (long long)plan.launch.ctas_per_sm * kSms);
  plan.part_lse = plan.part_o = plan.total = 0;
  if (plan.splits > 1) {
    const size_t rows = (size_t)plan.units * plan.splits * plan.gq;
    plan.part_o = round_up(rows * sizeof(float));
    plan.total = plan.part_o + round_up(rows * c.head_dim * sizeof(float));
  }
  return plan;
}

cudaError_t launch_listed_d64(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                              const GenLaunch& shape, cudaStream_t s);
cudaError_t launch_listed_d64_h8(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                                 const GenLaunch& shape, cudaStream_t s);
cudaError_t launch_listed_d128(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                               const GenLaunch& shape, cudaStream_t s);
cudaError_t launch_listed_d128_h8(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                                  const GenLaunch& shape, cudaStream_t s);
cudaError_t launch_listed_d256(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                               const GenLaunch& shape, cudaStream_t s);
cudaError_t launch_listed_d256_h8(int bits, bool kcw, bool vcw, int group, const ListParams& p, int grid,
                                  const GenLaunch& shape, cudaStream_t s);

cudaError_t launch_sparse_decode(const kvq_cache_desc& cache, const SparsePlan& plan, const ListParams& p,
                                 cudaStream_t stream) {
  const bool kcw = cache.k_scheme == KVQ_CHANNELWISE, vcw = cache.v_scheme == KVQ_CHANNELWISE, wide = plan.nh > 4;
  const auto launch = cache.head_dim == 64    ? (wide ? launch_listed_d64_h8 : launch_listed_d64)
                      : cache.head_dim == 128 ? (wide ? launch_listed_d128_h8 : launch_listed_d128)
                                              : (wide ? launch_listed_d256_h8 : launch_listed_d256);
  cudaError_t e = launch(cache.bits, kcw, vcw, group_of(&cache), p, plan.units * plan.splits, plan.launch, stream);
  if (e != cudaSuccess || plan.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.num_q_heads));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, listed_merge_kernel, p);
}

}  // namespace kvq
