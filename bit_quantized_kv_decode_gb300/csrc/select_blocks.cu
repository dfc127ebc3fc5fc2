// Selection of the blocks of a sequence that a query may look at.
//
// K is channel-wise: channel c of token group g holds values in [z_gc, z_gc + m
// s_gc], m = 2^bits - 1.  A block's score is the largest sum over the query
// heads of a KV head that a token's scores can have,
//   max_g sum_h max_{k in box g} q_h . k = max_g sum_c (Q_c z_gc + m P_c s_gc),
//   Q = sum_h q_h,  P = sum_h max(q_h, 0),
// so one pass over K's scales and offsets (512 of a block's 17,408 bytes at
// 4 bits, D = G = 128) scores all heads of the group.
//
// A cluster of 1 to 8 CTAs per (sequence, KV head) scores the blocks -- 8
// channels a lane, 16-byte loads -- and leaves the scores in the first CTA's
// shared memory, which selects: a bisection over the scores' bit patterns.
//
// The list is the one that scores without rounding give (ties to the lowest
// index), whatever the order of the sums: an fp32 score is off by at most E =
// 2^-19 A, A the largest sum of magnitudes (7 additions of the heads, 16 + 5 of
// the channels, one for the factor m: 29 roundings of 2^-24), so a cut between
// scores more than 2 E apart is certain.  Else the blocks within 2 E of the cut
// are scored again in fp64 (about one list in a hundred; two blocks as a rule).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "sparse_decode.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kBound = 1.f / (1 << 19);  // E / A

// Numbers as unsigned integers of the same order; what is not a number comes
// with minus infinity.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x != x ? -INFINITY : x + 0.f);  // (-0 is 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const double y = x != x ? -INFINITY : x + 0.0;
  const uint64_t b = (uint64_t)__double_as_longlong(y);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

struct Shared {
  float bound;  // the cluster's largest sum of magnitudes
  int warp_count[2][kWarps];
  uint32_t warp_lo[kWarps], warp_hi[kWarps];
  uint32_t taken[kSelectMaxBlocks / 32];  // scored blocks of the list
};

// Sum of v over the CTA, in every thread; `turn` counts the calls.
__device__ __forceinline__ int cta_sum(Shared& sh, int v, int& turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  int* buf = sh.warp_count[turn++ & 1];
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += buf[w];
  return t;
}

// The largest t with at least k of the n keys >= t, or a t with exactly k keys
// >= t (and then *exact).  0 < k <= n.
template <typename Key>
__device__ __forceinline__ Key cut(Shared& sh, const Key* keys, int n, int k, Key lo, Key hi, int& turn, bool* exact) {
  *exact = false;
  while (lo < hi) {  // count(>= lo) >= k; the answer is in [lo, hi]
    const Key mid = lo + (hi - lo) / 2 + 1;
    int c = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) c += keys[i] >= mid;
    c = cta_sum(sh, c, turn);
    if (c == k) {
      *exact = true;
      return mid;
    }
    if (c > k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Smallest and largest of the keys that `pass` lets through, in every thread.
template <class Pass>
__device__ __forceinline__ void extremes(Shared& sh, const uint32_t* keys, int n, Pass pass, uint32_t& lo, uint32_t& hi) {
  uint32_t a = 0xffffffffu, b = 0u;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t k = keys[i];
    if (pass(k)) {
      a = min(a, k);
      b = max(b, k);
    }
  }
  a = __reduce_min_sync(0xffffffffu, a);
  b = __reduce_max_sync(0xffffffffu, b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.warp_lo[threadIdx.x >> 5] = a;
    sh.warp_hi[threadIdx.x >> 5] = b;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    a = min(a, sh.warp_lo[w]);
    b = max(b, sh.warp_hi[w]);
  }
  lo = a;
  hi = b;
}

__device__ __forceinline__ int page_of(const SelectParams& p, int b, int j) {
  return p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
}

// Score of block j in fp64, by a warp (minus infinity for a bad page).
template <int D>
__device__ __forceinline__ double exact_score(const SelectParams& p, int b, int h, int j, int len) {
  const int lane = threadIdx.x & 31, page = page_of(p, b, j);
  if (page < 0 || page >= p.num_pages) return -INFINITY;
  const size_t at = ((size_t)page * p.num_kv_heads + h) * (kBlockTokens / p.group * D);
  const uint16_t* q = p.q + ((size_t)b * p.num_q_heads + (size_t)h * p.gq) * D;
  const double most = (1 << p.bits) - 1;
  const int groups = (min(kBlockTokens, len - j * kBlockTokens) + p.group - 1) / p.group;
  double best = -INFINITY;
  for (int g = 0; g < groups; ++g) {
    double s = 0.0;
    for (int c = lane; c < D; c += 32) {
      double all = 0.0, up = 0.0;
      for (int k = 0; k < p.gq; ++k) {
        const double v = bf16_value(q[k * D + c]);
        all += v;
        up += v > 0.0 ? v : v == v ? 0.0 : v;
      }
      s += all * (double)__half2float(__ushort_as_half(p.k_zero[at + g * D + c])) +
           most * (up * (double)__half2float(__ushort_as_half(p.k_scale[at + g * D + c])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    best = s != s ? best : s > best ? s : best;
  }
  return best;
}

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Shared sh;
  uint32_t* keys = reinterpret_cast<uint32_t*>(dynamic);  // of the scored blocks, in order (first CTA)
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = blockIdx.x / ranks, b = u / p.num_kv_heads, h = u % p.num_kv_heads;
  int len = p.seq_lens[b];
  if (len < 0 || len > p.max_blocks * kBlockTokens) {
    if (tid == 0 && rank == 0) report(p.dev_status, KVQ_DEV_BAD_SEQ_LEN);
    len = 0;
  }
  const int n = (len + kBlockTokens - 1) / kBlockTokens;
  int32_t* list = p.blocks + (size_t)u * p.budget;
  if (rank == 0 && tid == 0) p.counts[u] = min(n, p.budget);
  if (n <= p.budget) {  // every block
    if (rank == 0)
      for (int i = tid; i < p.budget; i += kThreads) list[i] = i < n ? i : -1;
    return;
  }
  const int m = n - p.first - p.last, want = p.budget - p.first - p.last;  // blocks to score, and to take of them

  if (want > 0) {
    // ---- the scores
    if (tid == 0) sh.bound = 0.f;
    cluster.sync();
    uint32_t* out = cluster.map_shared_rank(keys, 0);
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a block, blocks of a warp at a time
    const int sub = lane / kLanes, c0 = lane % kLanes * 8;
    float qs[8], ps[8], ws[8];  // sums over the heads of q, of its positive part times m, and of its magnitude
#pragma unroll
    for (int i = 0; i < 8; ++i) qs[i] = ps[i] = ws[i] = 0.f;
    const uint16_t* q = p.q + ((size_t)b * p.num_q_heads + (size_t)h * p.gq) * D + c0;
    for (int k = 0; k < p.gq; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + k * D);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = i & 1 ? __uint_as_float(w[i / 2] & 0xffff0000u) : bf16_value(w[i / 2] & 0xffffu);
        qs[i] += x;
        ps[i] += x != x ? x : fmaxf(x, 0.f);
        ws[i] += fabsf(x);
      }
    }
    const float most = (float)((1 << p.bits) - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) ps[i] *= most;
    const int groups = kBlockTokens / p.group, nsz = groups * D;
    const int each = (m + ranks * kWarps - 1) / (ranks * kWarps);  // blocks of a warp
    const int from = min(m, (rank * kWarps + warp) * each), to = min(m, from + each);
    uint32_t magnitude = 0u;  // bits: NaN is the largest
    for (int i0 = from; i0 < to; i0 += 32) {
      int page = -1;  // of block i0 + lane
      if (i0 + lane < to) {
        page = page_of(p, b, p.first + i0 + lane);
        if (page < 0 || page >= p.num_pages) {
          report(p.dev_status, KVQ_DEV_BAD_PAGE);
          page = -1;
        }
      }
      const int here = min(32, to - i0);
      for (int i = 0; i < here; i += kRows) {
        const int mine = __shfl_sync(0xffffffffu, page, min(i + sub, 31));
        const int j = p.first + i0 + i + sub;
        const bool live = i + sub < here && mine >= 0;
        const size_t at = ((size_t)(live ? mine : 0) * p.num_kv_heads + h) * nsz + c0;
        const int used = live ? (min(kBlockTokens, len - j * kBlockTokens) + p.group - 1) / p.group : 0;
        float best = -INFINITY;
        for (int g = 0; g < groups; ++g) {
          float s = 0.f, a = 0.f;
          if (g < used) {
            const uint4 zv = __ldg(reinterpret_cast<const uint4*>(p.k_zero + at + g * D));
            const uint4 sv = __ldg(reinterpret_cast<const uint4*>(p.k_scale + at + g * D));
            const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w}, sw[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&zw[k]));
              const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&sw[k]));
              s = fmaf(z.x, qs[2 * k], s);
              s = fmaf(w.x, ps[2 * k], s);
              s = fmaf(z.y, qs[2 * k + 1], s);
              s = fmaf(w.y, ps[2 * k + 1], s);
              a = fmaf(fabsf(z.x), ws[2 * k], a);
              a = fmaf(fabsf(w.x), ps[2 * k], a);
              a = fmaf(fabsf(z.y), ws[2 * k + 1], a);
              a = fmaf(fabsf(w.y), ps[2 * k + 1], a);
            }
          }
          magnitude = max(magnitude, __float_as_uint(a) & 0x7fffffffu);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (g < used) best = best == best ? (s <= best ? best : s) : best;
        }
        if (i + sub < here && lane % kLanes == 0) out[i0 + i + sub] = ordered(best);
      }
    }
    // the lanes' largest partial sums, added up, are at least the largest sum
    float total = __uint_as_float(magnitude);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(total) & 0x7fffffffu);
    if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(cluster.map_shared_rank(&sh.bound, 0)), bits);
    cluster.sync();
  }
  if (rank != 0) return;

  // ---- the selection
  int turn = 0;
  for (int i = tid; i < (m + 31) / 32; i += kThreads) sh.taken[i] = 0u;
  __syncthreads();
  if (want > 0) {
    const float bound = 2.f * (kBound * sh.bound);
    uint32_t lo, hi;
    extremes(sh, keys, m, [](uint32_t) { return true; }, lo, hi);
    bool exact;
    const uint32_t t = cut(sh, keys, m, want, lo, hi, turn, &exact);
    bool sure = exact;
    float at = value_of(t);  // the last score taken
    if (exact) {
      uint32_t low, high, unused;
      extremes(sh, keys, m, [t](uint32_t k) { return k >= t; }, low, unused);
      extremes(sh, keys, m, [t](uint32_t k) { return k < t; }, unused, high);
      at = value_of(low);
      sure = at - value_of(high) > bound;
    }
    if (sure) {
      for (int i0 = warp * 32; i0 < m; i0 += kThreads) {
        const uint32_t w = __ballot_sync(0xffffffffu, i0 + lane < m && keys[i0 + lane] >= t);
        if (lane == 0) sh.taken[i0 / 32] = w;
      }
      __syncthreads();
    } else {
      // Blocks certain to be in, and the candidates: those that may be on
      // either side of the cut.  (Comparisons that NaN or infinite bounds make
      // void leave every block a candidate.)
      __syncthreads();  // (the last reduction is read)
      const float above = at + bound, below = at - bound;
      uint64_t* exact_keys = reinterpret_cast<uint64_t*>(dynamic + (((size_t)p.max_blocks * 4 + 15) & ~(size_t)15));
      int* candidates = reinterpret_cast<int*>(keys);  // over the scores, behind their reading
      int in = 0, found = 0;
      for (int i0 = 0; i0 < m; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t key = i < m ? keys[i] : 0u;
        const float s = value_of(key);
        const bool sure_in = i < m && s > above, candidate = i < m && !sure_in && !(s < below);
        const uint32_t w = __ballot_sync(0xffffffffu, sure_in), cw = __ballot_sync(0xffffffffu, candidate);
        if (lane == 0) {
          if (i0 + warp * 32 < m) sh.taken[i0 / 32 + warp] = w;
          sh.warp_lo[warp] = __popc(cw);
        }
        in += cta_sum(sh, sure_in, turn);  // (its barrier: the scores of this round are read)
        int pos = found;
        for (int k = 0; k < kWarps; ++k) {
          if (k < warp) pos += (int)sh.warp_lo[k];
          found += (int)sh.warp_lo[k];
        }
        if (candidate) {
          const int slot = pos + __popc(cw & ((1u << lane) - 1u));
          candidates[slot] = i;
          exact_keys[slot] = key;
        }
        __syncthreads();
      }
      const int rest = want - in;  // candidates to take
      if (bound != 0.f) {          // (0: nothing but zeros was added up)
        for (int i = warp; i < found; i += kWarps) {
          const double s = exact_score<D>(p, b, h, p.first + candidates[i], len);
          if (lane == 0) exact_keys[i] = ordered(s);
        }
        __syncthreads();
      }
      bool separate;
      const uint64_t t64 = cut<uint64_t>(sh, exact_keys, found, rest, 0ull, ~0ull, turn, &separate);
      int over = 0;  // keys above the cut: all of them; at it: the first ones
      for (int i = tid; i < found; i += kThreads) over += exact_keys[i] > t64;
      over = cta_sum(sh, over, turn);
      int equal = separate ? found : rest - over;  // equal ones still to take
      for (int i0 = 0; i0 < found; i0 += kThreads) {
        const int i = i0 + tid;
        const bool same = i < found && exact_keys[i] == t64;
        const uint32_t w = __ballot_sync(0xffffffffu, same);
        if (lane == 0) sh.warp_lo[warp] = __popc(w);
        const int all = cta_sum(sh, same, turn);
        int before = __popc(w & ((1u << lane) - 1u));
        for (int k = 0; k < warp; ++k) before += (int)sh.warp_lo[k];
        if (i < found && (exact_keys[i] > t64 || (same && before < equal)))
          atomicOr(&sh.taken[candidates[i] / 32], 1u << (candidates[i] & 31));
        equal = max(0, equal - all);
        __syncthreads();
      }
    }
  }

  // ---- the list, in order: the first blocks, those taken, the last ones
  for (int i = tid; i < p.first; i += kThreads) list[i] = i;
  for (int i = tid; i < p.last; i += kThreads) list[p.budget - p.last + i] = n - p.last + i;
  int done = p.first;
  for (int i0 = 0; i0 < m && want > 0; i0 += kThreads * 32) {  // a word of 32 blocks per thread
    const int i = i0 / 32 + tid;
    uint32_t w = i < (m + 31) / 32 ? sh.taken[i] : 0u;
    const int mine = __popc(w);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sh.warp_lo[warp] = (uint32_t)incl;
    __syncthreads();
    int pos = done + incl - mine;
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) pos += (int)sh.warp_lo[k];
      done += (int)sh.warp_lo[k];
    }
    for (; w != 0u; w &= w - 1u) list[pos++] = p.first + i * 32 + __ffs((int)w) - 1;
  }
}

template <int D>
cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
  // scores, and exact scores of as many candidates as there can be
  const size_t smem = (((size_t)p.max_blocks * 4 + 15) & ~(size_t)15) + (size_t)p.max_blocks * 8;
  cudaError_t e = cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // CTAs per list: up to 8 while the lists alone do not give every SM two, and
  // each has 32 blocks a warp or more to score
  const long long units = (long long)p.batch * p.num_kv_heads;
  int ranks = 1;
  while (ranks < 8 && units * ranks < 304 && p.max_blocks > ranks * 64) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<D>, p);
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  if (p.head_dim == 64) return launch<64>(p, stream);
  if (p.head_dim == 128) return launch<128>(p, stream);
  return launch<256>(p, stream);
}

}  // namespace kvq
