// Decode attention over lists of blocks: how the lists are cut, the dispatch of
// the kernel instances (decode_general_kernel with LISTED), and the log-sum-exp
// merge of the ranges.
#include "decode_general.cuh"
#include "sparse_decode.h"

namespace kvq {

namespace {

constexpr int kSms = 152;          // of a GB300
constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024;

// Ranges per list, by what a call takes when every list is full, in tenths of a
// microsecond (head dim 128): a block takes 12 in a CTA by itself, and 5 of an
// SM's time however many CTAs share it; a CTA 8 of it besides; half a range is
// idle at the end; several ranges need a merge.  Measured (us): 8 lists of 256
// blocks, 16 / 32 / 64 / 128 ranges 32.0 / 22.8 / 21.1 / 23.3; 512 lists of up to
// 64, 1 / 2 / 4 / 8 ranges 165 / 127 / 109 / 107; 1,024 of 32, 1 / 2 / 4 ranges 136
// / 132 / 138.
int sparse_splits(long long units, int list_len) {
  long long best = -1;
  int splits = 1;
  int blocks = list_len;  // of a range
  for (int s = 1;; s = (list_len - 1) / (blocks - 1) + 1) {  // (the next s with fewer: those between add only CTAs)
    if (units * (s - 1) > 32 * kSms) break;  // (so units * s <= 64 * kSms = 9,728, which callers may rely on)
    blocks = (list_len + s - 1) / s;
    const long long ctas = units * s;
    const long long alone = 12LL * blocks, shared = ctas * (5LL * blocks + 8) / kSms;
    const long long cost = (alone > shared ? alone : shared) + alone / 2 + (s > 1 ? 30 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      splits = s;
    }
    if (blocks == 1) break;
  }
  return splits;
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// WARPS warps per (sequence, query head): each takes every WARPS-th part, a lane
// D / 32 channels of it.  Every warp works out the weights by itself, so that
// nothing but the sums is exchanged.
constexpr int kMergeThreads = 256;

template <int D, int WARPS>
__global__ void __launch_bounds__(kMergeThreads) listed_merge_kernel(const ListParams p) {
  constexpr int kRows = kMergeThreads / 32 / WARPS, V = D / 32;
  __shared__ float acc[WARPS > 1 ? WARPS : 1][WARPS > 1 ? D : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kRows + warp / WARPS, w0 = warp % WARPS;
  gen::grid_dep_wait();  // the decode kernel's parts
  if (row >= p.batch * p.num_q_heads) return;  // (WARPS > 1: never)
  const int b = row / p.num_q_heads, head = row % p.num_q_heads;
  const int u = b * p.units_per_seq + head / p.gq, k = head % p.gq;
  const int nr = min(p.splits, listed_unit(p, u).n);
  const float* lses = p.part_lse + (size_t)u * p.splits * p.gq + k;
  const float* parts = p.part_o + ((size_t)u * p.splits * p.gq + k) * D + lane * V;
  float m = -INFINITY;
  bool some = false;
  for (int s = lane; s < nr; s += 32) {
    const float x = lses[(size_t)s * p.gq];
    m = fmaxf(m, x);
    some |= x != -INFINITY;  // (the maximum passes over what is not a number: m alone would not tell)
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool none = !__any_sync(0xffffffffu, some);  // no entry, or bad ones alone
  float t = 0.f;
  for (int s = lane; s < nr; s += 32) t += none ? 0.f : expf(lses[(size_t)s * p.gq] - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const float inv = none ? 0.f : 1.f / t;
  float a[V];
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = 0.f;
  if (!none) {
#pragma unroll 4
    for (int s = w0; s < nr; s += WARPS) {
      const float w = expf(lses[(size_t)s * p.gq] - m) * inv;
      const float2* src = reinterpret_cast<const float2*>(parts + (size_t)s * p.gq * D);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 v = src[i];
        a[2 * i] = fmaf(w, v.x, a[2 * i]);
        a[2 * i + 1] = fmaf(w, v.y, a[2 * i + 1]);
      }
    }
  }
  if (w0 == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = none ? -INFINITY : m + logf(t);
  if (WARPS > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[WARPS > 1 ? w0 : 0][lane * V + i] = a[i];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < D) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) o += acc[WARPS > 1 ? w : 0][c];
      p.out[(size_t)row * D + c] = gen::bf16_bits(o);
    }
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (size_t)row * D + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dst[i] = gen::bf16_bits(a[2 * i]) | (uint32_t)gen::bf16_bits(a[2 * i + 1]) << 16;
  }
}

template <int D>
cudaError_t launch_merge_of(const ListParams& p, cudaStream_t stream) {
  const int rows = p.batch * p.num_q_heads;
  const bool many = p.splits > 8;  // parts of a row
  constexpr int kRows = kMergeThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(many ? rows : (rows + kRows - 1) / kRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, listed_merge_kernel<D, kRows>, p)
              : cudaLaunchKernelEx(&cfg, listed_merge_kernel<D, 1>, p);
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
  plan.splits = sparse_splits(plan.units, d->list_len);
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
  if (cache.head_dim == 64) return launch_merge_of<64>(p, stream);
  return cache.head_dim == 128 ? launch_merge_of<128>(p, stream) : launch_merge_of<256>(p, stream);
}

}  // namespace kvq
