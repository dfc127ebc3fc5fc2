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
// A cluster of up to 8 CTAs per (sequence, KV head) scores the blocks -- 8
// channels a lane, 16-byte copies kept under way in shared memory -- and leaves the
// scores in the first CTA's shared memory, which selects: a bisection over the
// scores' bit patterns, of up to 1,024 blocks by one warp without a barrier (20
// steps of some 60 cycles).  Measured: 1,024 lists of 256 blocks, 134 MB: 32.4 us,
// 4.1 TB/s, the chain of copies, sums and selection of a list; 8 lists of 8,192
// blocks: 24 us, of which the selection by one CTA is about half.
//
// The list is the one that scores without rounding give (ties to the lowest
// index), whatever the order of the sums: an fp32 score is off by at most E =
// 2^-19 A, A the sum over the channels of the largest magnitudes that any block
// has there (7 additions of the heads, one for the factor m, 9 of a lane's
// channels, 5 of the lanes: 22 roundings of 2^-24), and by 2^-140 where numbers
// are too small for that (512 products, 2^-150 each; q is a multiple of 2^-133, its
// sums are exact).  So a cut between scores more than 2 E apart is certain.  Else
// the blocks within 2 E of the cut are scored again in fp64 (about one list in a
// hundred; two blocks as a rule).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "attn_core.cuh"
#include "sparse_decode.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kMaxWarps = 16;
constexpr float kBound = 1.f / (1 << 19);  // E / A
constexpr float kTiny = 0x1p-139f;         // 2 E of the smallest numbers

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

// Copy steps of a warp under way.
constexpr int kAhead = 6;
// Dynamic shared memory: a key per block, a bit per block, then the copies.
__host__ __device__ constexpr int keys_room(int max_blocks) { return (max_blocks + 3) / 4 * 4; }
__host__ __device__ constexpr size_t copies_at(int max_blocks) {
  return ((size_t)keys_room(max_blocks) + (max_blocks + 127) / 128 * 4) * 4;
}

// The larger of each half of two fp16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t max_nan_2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Eight neighbouring bf16 values in shared memory.
__device__ __forceinline__ void eight(const uint4* at, float (&x)[8]) {
  const uint4 v = *at;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = i & 1 ? __uint_as_float(w[i / 2] & 0xffff0000u) : bf16_value(w[i / 2] & 0xffffu);
}

// The cluster's barrier, in halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

struct Shared {
  uint4 q[8 * 256 / 8];  // the query heads
  float bound;  // the cluster's largest sum of magnitudes
  uint32_t low, high;  // the cluster's smallest and largest key
  int in, found, few[32];
  int warp_count[2][kMaxWarps];
  uint32_t warp_lo[kMaxWarps], warp_hi[kMaxWarps];
};

// Sum of v over the CTA, in every thread; `turn` counts the calls.
template <int NT>
__device__ __forceinline__ int cta_sum(Shared& sh, int v, int& turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  int* buf = sh.warp_count[turn++ & 1];
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < NT / 32 ? buf[lane] : 0);
}

// The largest t with at least k of the n keys >= t, or a t with exactly k keys
// >= t (and then *exact).  0 < k <= n; lo: at most the smallest key, hi: at least
// the largest.
template <int NT, typename Key>
__device__ __forceinline__ Key cut(Shared& sh, const Key* keys, int n, int k, Key lo, Key hi, int& turn, bool* exact) {
  // the first keys of a thread stay in its registers
  constexpr int kHeld = sizeof(Key) == 4 ? 16 : 4;
  Key mine[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int at = i * NT + threadIdx.x;
    mine[i] = at < n ? keys[at] : 0;  // (the cut is above 0)
  }
  *exact = false;
  while (lo < hi) {  // count(>= lo) >= k; the answer is in [lo, hi]
    const Key mid = lo + (hi - lo) / 2 + 1;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) c += mine[i] >= mid;
    for (int i = kHeld * NT + threadIdx.x; i < n; i += NT) c += keys[i] >= mid;
    c = cta_sum<NT>(sh, c, turn);
    if (c == k) {
      *exact = true;
      return mid;
    }
    if (c > k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The smallest of the keys >= t and the largest of the others, in every thread
// (all ones, and 0, where there is none).
template <int NT>
__device__ __forceinline__ void beside(Shared& sh, const uint32_t* keys, int n, uint32_t t, uint32_t& low, uint32_t& high) {
  uint32_t a = 0xffffffffu, b = 0u;
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint32_t k = keys[i];
    if (k >= t) a = min(a, k);
    else b = max(b, k);
  }
  a = __reduce_min_sync(0xffffffffu, a);
  b = __reduce_max_sync(0xffffffffu, b);
  const int lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) {
    sh.warp_lo[threadIdx.x >> 5] = a;
    sh.warp_hi[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  low = __reduce_min_sync(0xffffffffu, lane < NT / 32 ? sh.warp_lo[lane] : 0xffffffffu);
  high = __reduce_max_sync(0xffffffffu, lane < NT / 32 ? sh.warp_hi[lane] : 0u);
}

// The same cut by one warp, with the keys in its registers: no barriers.
template <int kEach>  // keys of a lane
__device__ __forceinline__ void warp_cut(const uint32_t* keys, int n, int k, uint32_t lo, uint32_t hi, uint32_t& t,
                                         bool& exact, uint32_t& low, uint32_t& high) {
  const int lane = threadIdx.x & 31;
  uint32_t mine[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) mine[i] = 32 * i + lane < n ? keys[32 * i + lane] : 0u;  // (0: below every key)
  exact = false;
  while (lo < hi && !exact) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) c += mine[i] >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    exact = c == k;
    if (c >= k) lo = mid;
    else hi = mid - 1;
  }
  t = lo;
  uint32_t a = 0xffffffffu, b = 0u;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (mine[i] >= t) a = min(a, mine[i]);
    else b = max(b, mine[i]);
  }
  low = __reduce_min_sync(0xffffffffu, a);
  high = __reduce_max_sync(0xffffffffu, b);
}

__device__ __forceinline__ int page_of(const SelectParams& p, int b, int j) {
  return p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
}

// Scores in fp64, a block at a time by a warp.
template <int D, int NG>
struct Exact {
  double all[D / 32], up[D / 32];  // Q and m P of channels lane, lane + 32, ...
  const SelectParams& p;
  const int b, h, len;
  __device__ __forceinline__ Exact(const SelectParams& params, int b_, int h_, int len_) : p(params), b(b_), h(h_), len(len_) {
    const uint16_t* q = p.q + ((size_t)b * p.num_q_heads + (size_t)h * p.gq) * D + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      all[i] = up[i] = 0.0;
      for (int k = 0; k < p.gq; ++k) {
        const float v = bf16_value(q[k * D + 32 * i]);
        all[i] += (double)v;
        up[i] += (double)fmaxf(v, 0.f);
      }
      up[i] *= (double)((1 << p.bits) - 1);
    }
  }
  __device__ __forceinline__ double score(int j) const {  // minus infinity for a bad page
    const int lane = threadIdx.x & 31, page = page_of(p, b, j);
    if (page < 0 || page >= p.num_pages) return -INFINITY;
    const size_t at = ((size_t)page * p.num_kv_heads + h) * (NG * D) + lane;
    double best = -INFINITY;
    for (int g = 0; g < NG; ++g) {
      if (j * kBlockTokens + g * (kBlockTokens / NG) >= len) break;
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int c = g * D + 32 * i;
        s = fma(all[i], (double)__half2float(__ushort_as_half(p.k_zero[at + c])), s);
        s = fma(up[i], (double)__half2float(__ushort_as_half(p.k_scale[at + c])), s);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      best = s > best ? s : best;  // (NaN: minus infinity)
    }
    return best;
  }
};

template <int D, int NG, int NT>  // NG: token groups of a block; NT: threads
__global__ void __launch_bounds__(NT, 1024 / NT) select_kernel(const SelectParams p) {
  constexpr int kThreads = NT, kWarps = NT / 32;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ Shared sh;
  uint32_t* keys = reinterpret_cast<uint32_t*>(dynamic);  // of the scored blocks, in order (first CTA)
  uint32_t* taken = keys + keys_room(p.max_blocks);       // those of them that the list has
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
    if (tid == 0) {
      sh.bound = 0.f;
      sh.low = 0xffffffffu;
      sh.high = 0u;
      sh.in = sh.found = 0;
    }
    if (ranks > 1) {  // (now, while there is nothing that it would wait for: with the copies under way it takes longer)
      __syncthreads();
      cluster_arrive();
    }
    // A warp takes kRows blocks at a time, 8 channels a lane; its lanes copy what
    // they will read to places of their own in shared memory, kAhead steps ahead:
    // more bytes under way than registers would hold.
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int sub = lane / kLanes, c0 = lane % kLanes * 8;
    const long long stride = (long long)p.num_kv_heads * (NG * D), base = (long long)h * (NG * D) + c0;
    const int each = (m + ranks * kWarps - 1) / (ranks * kWarps);  // blocks of a warp
    const int from = min(m, (rank * kWarps + warp) * each), to = min(m, from + each);
    uint4* ring = reinterpret_cast<uint4*>(dynamic + copies_at(p.max_blocks)) + warp * (kAhead * 64) + lane;
    int page0 = 0, page1 = 0, steps = 0;  // of blocks lane and 32 + lane of the 64 under way
    uint32_t good0 = 0u, good1 = 0u;
    int here_last = 0;  // last of them
    auto fetch = [&](int st, int slot) {  // (a group of copies at each call, empty ones at the end)
      if (st < steps) {
        const int at = min(st / NG * kRows + sub, here_last);  // lanes past the last block take it again
        const int a = __shfl_sync(0xffffffffu, page0, at & 31), c = __shfl_sync(0xffffffffu, page1, at & 31);
        const long long src = (long long)(at < 32 ? a : c) * stride + base + st % NG * D;
        copy16(ring + slot * 64, p.k_zero + src);
        copy16(ring + slot * 64 + 32, p.k_scale + src);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto begin = [&](int i0) {  // pages of the next 64 blocks, first copies; a bad page is read as page 0, and not used
      here_last = min(64, to - i0) - 1;  // (-1: none)
      steps = (here_last + kRows) / kRows * NG;
      page0 = lane <= here_last ? page_of(p, b, p.first + i0 + lane) : 0;
      page1 = lane + 32 <= here_last ? page_of(p, b, p.first + i0 + 32 + lane) : 0;
      const bool bad0 = page0 < 0 || page0 >= p.num_pages, bad1 = page1 < 0 || page1 >= p.num_pages;
      if (bad0 || bad1) report(p.dev_status, KVQ_DEV_BAD_PAGE);
      page0 = bad0 ? 0 : page0;
      page1 = bad1 ? 0 : page1;
      good0 = ~__ballot_sync(0xffffffffu, bad0);
      good1 = ~__ballot_sync(0xffffffffu, bad1);
#pragma unroll 1
      for (int st = 0; st < kAhead; ++st) fetch(st, st);
    };
    // (the queries first: behind the others' copies they would wait)
    const uint16_t* query = p.q + ((size_t)b * p.num_q_heads + (size_t)h * p.gq) * D;
    for (int i = tid; i < p.gq * (D / 8); i += kThreads) copy16(sh.q + i, query + 8 * i);
    asm volatile("cp.async.commit_group;" ::: "memory");
    begin(from);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    __syncthreads();

    // sums over the heads of q and of its positive part times m, in pairs
    const uint4* q = sh.q + lane % kLanes;
    uint64_t qs[4], ps[4];
    {
      float all[8], up[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) all[i] = up[i] = 0.f;
#pragma unroll 4
      for (int k = 0; k < p.gq; ++k) {
        float x[8];
        eight(q + k * kLanes, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          all[i] += x[i];
          up[i] += fmaxf(x[i], 0.f);  // (a NaN shows in the other sum)
        }
      }
      const float most = (float)((1 << p.bits) - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qs[i] = rows::pair(all[2 * i], all[2 * i + 1]);
        ps[i] = rows::pair(up[2 * i] * most, up[2 * i + 1] * most);
      }
    }
    uint32_t zmax[4] = {0u, 0u, 0u, 0u}, smax[4] = {0u, 0u, 0u, 0u};  // largest magnitudes of the channels, fp16 pairs
    if (ranks > 1) cluster_wait();  // every CTA of the list is there, and the first one's numbers
    uint32_t* out = cluster.map_shared_rank(keys, 0);
    uint32_t low = 0xffffffffu, high = 0u;
    for (int i0 = from; i0 < to; i0 += 64) {
      if (i0 > from) begin(i0);
      // four steps at a time, their sums reduced together
      int slot = 0;
      for (int st = 0; st < steps; st += 4) {
        float sum[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
          const uint4 zv = ring[slot * 64], sv = ring[slot * 64 + 32];
          const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w}, sw[4] = {sv.x, sv.y, sv.z, sv.w};
          uint64_t s2 = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&zw[k]));
            const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&sw[k]));
            s2 = rows::fma2(rows::pair(z.x, z.y), qs[k], s2);
            s2 = rows::fma2(rows::pair(w.x, w.y), ps[k], s2);
            if (st + r < steps) {  // (what is behind the last step is not a copy of these)
              zmax[k] = max_nan_2(zmax[k], zw[k] & 0x7fff7fffu);
              smax[k] = max_nan_2(smax[k], sw[k]);
            }
          }
          fetch(st + r + kAhead, slot);  // into the pieces just read, which no other lane reads
          slot = slot + 1 < kAhead ? slot + 1 : 0;
          float odd;
          rows::unpair(s2, sum[r], odd);
          sum[r] += odd;
        }
        // over the block's lanes: lane l of them is left with step l / (kLanes / 4)
#pragma unroll
        for (int n = 4, o = kLanes / 2; n > 1; n >>= 1, o >>= 1) {
          const bool upper = (lane & o) != 0;
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? sum[i] : sum[i + n / 2], o);
            sum[i] = (upper ? sum[i + n / 2] : sum[i]) + got;
          }
        }
#pragma unroll
        for (int o = kLanes / 8; o > 0; o >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        const int mine = st + lane % kLanes / (kLanes / 4), at = mine / NG * kRows + sub, g = mine % NG;
        float best = sum[0];
        if (NG > 1) {  // the largest of a block's groups (those behind the last token have none)
          if (g > 0 && (p.first + i0 + at) * kBlockTokens + g * (kBlockTokens / NG) >= len) best = -INFINITY;
#pragma unroll
          for (int o = kLanes / 4; o < kLanes / 4 * NG; o <<= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, best, o);
            best = best != best ? best : other <= best ? best : other;
          }
        }
        const bool good = ((at < 32 ? good0 : good1) >> (at & 31) & 1u) != 0u;
        const uint32_t key = ordered(good ? best : -INFINITY);
        if (at <= here_last) {
          low = min(low, key);
          high = max(high, key);
          if (g == 0 && lane % (kLanes / 4) == 0) out[i0 + at] = key;
        }
      }
    }
    // the largest magnitude of each channel, whatever its block: at least the largest sum
    float total = 0.f, ws[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ws[i] = 0.f;
    for (int k = 0; k < p.gq; ++k) {
      float x[8];
      eight(q + k * kLanes, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) ws[i] += fabsf(x[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&zmax[k]));
      const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&smax[k]));
      float p0, p1;
      rows::unpair(ps[k], p0, p1);
      total = __fmaf_ru(z.x, ws[2 * k], total);  // (rounded up: 0 only if there is nothing to add up)
      total = __fmaf_ru(z.y, ws[2 * k + 1], total);
      total = __fmaf_ru(w.x, p0, total);
      total = __fmaf_ru(w.y, p1, total);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(total) & 0x7fffffffu);
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
      Shared* first = cluster.map_shared_rank(&sh, 0);
      atomicMax(reinterpret_cast<unsigned int*>(&first->bound), bits);
      atomicMin(&first->low, low);
      atomicMax(&first->high, high);
    }
    if (ranks > 1) {
      cluster_arrive();
      if (rank != 0) return;  // (nothing of this CTA's is read by others)
      cluster_wait();
    } else {
      __syncthreads();
    }
  }
  if (rank != 0) return;

  // ---- the selection
  int turn = 0;
  for (int i = tid; i < (m + 31) / 32; i += kThreads) taken[i] = 0u;
  __syncthreads();
  if (want > 0) {
    const float bound = sh.bound == 0.f ? 0.f : 2.f * (kBound * sh.bound) + kTiny;
    uint32_t t;       // keys from here on are taken, if `exact`
    bool exact;
    uint32_t low, high;  // then: the smallest key taken, the largest left
    if (m <= 1024) {
      if (warp == 0) {
        if (m <= 256) warp_cut<8>(keys, m, want, sh.low, sh.high, t, exact, low, high);
        else warp_cut<32>(keys, m, want, sh.low, sh.high, t, exact, low, high);
        if (lane == 0) {
          sh.warp_lo[0] = t;
          sh.warp_lo[1] = exact;
          sh.warp_hi[0] = low;
          sh.warp_hi[1] = high;
        }
      }
      __syncthreads();
      t = sh.warp_lo[0];
      exact = sh.warp_lo[1] != 0u;
      low = sh.warp_hi[0];
      high = sh.warp_hi[1];
    } else {
      t = cut<kThreads>(sh, keys, m, want, sh.low, sh.high, turn, &exact);
      beside<kThreads>(sh, keys, m, t, low, high);
    }
    const float at = value_of(exact ? low : t);  // the last score taken
    const bool sure = exact && at - value_of(high) > bound;
    if (sure) {
      for (int i0 = warp * 32; i0 < m; i0 += kThreads) {
        const uint32_t w = __ballot_sync(0xffffffffu, i0 + lane < m && keys[i0 + lane] >= t);
        if (lane == 0) taken[i0 / 32] = w;
      }
      __syncthreads();
    } else {
      // Blocks certain to be in, and the candidates: those that may be on
      // either side of the cut.  (Comparisons that NaN or infinite bounds make
      // void leave every block a candidate.)
      const float above = at + bound, below = at - bound;
      uint64_t* exact_keys = reinterpret_cast<uint64_t*>(dynamic + copies_at(p.max_blocks));
      for (int i0 = warp * 32; i0 < m; i0 += kThreads) {
        const int i = i0 + lane;
        const uint32_t key = i < m ? keys[i] : 0u;
        const float s = value_of(key);
        const bool sure_in = i < m && s > above, candidate = i < m && !sure_in && !(s < below);
        const uint32_t w = __ballot_sync(0xffffffffu, sure_in), cw = __ballot_sync(0xffffffffu, candidate);
        int slot = 0;
        if (lane == 0) {
          taken[i0 / 32] = w;
          if (w != 0u) atomicAdd(&sh.in, __popc(w));
          if (cw != 0u) slot = atomicAdd(&sh.found, __popc(cw));
        }
        slot = __shfl_sync(0xffffffffu, slot, 0) + __popc(cw & ((1u << lane) - 1u));
        if (candidate && slot < 32) {
          sh.few[slot] = i;
          exact_keys[slot] = key;
        }
      }
      __syncthreads();
      const int in = sh.in, found = sh.found;
      int* candidates = sh.few;
      if (found > 32) {  // many: over the scores, in order
        candidates = reinterpret_cast<int*>(keys);
        int done = 0;
        for (int i0 = 0; i0 < m; i0 += kThreads) {
          const int i = i0 + tid;
          const uint32_t key = i < m ? keys[i] : 0u;
          const float s = value_of(key);
          const bool candidate = i < m && !(s > above) && !(s < below);
          const uint32_t cw = __ballot_sync(0xffffffffu, candidate);
          if (lane == 0) sh.warp_lo[warp] = __popc(cw);
          __syncthreads();  // the scores of this round are read
          int pos = done;
          for (int k = 0; k < kWarps; ++k) {
            if (k < warp) pos += (int)sh.warp_lo[k];
            done += (int)sh.warp_lo[k];
          }
          if (candidate) {
            const int slot = pos + __popc(cw & ((1u << lane) - 1u));
            candidates[slot] = i;
            exact_keys[slot] = key;
          }
          __syncthreads();
        }
      }
      const int rest = want - in;  // candidates to take
      if (bound != 0.f) {          // (0: nothing but zeros was added up)
        if (warp < found) {
          const Exact<D, NG> in_full(p, b, h, len);
          for (int i = warp; i < found; i += kWarps) {
            const double s = in_full.score(p.first + candidates[i]);
            if (lane == 0) exact_keys[i] = ordered(s);
          }
        }
        __syncthreads();
      }
      if (found <= 32) {  // as a rule: ranked by one warp
        if (warp == 0) {
          const uint64_t mine = lane < found ? exact_keys[lane] : 0ull;
          const int block = lane < found ? sh.few[lane] : 0;
          int over = 0;
          for (int i = 0; i < found; ++i) {
            const uint64_t other = __shfl_sync(0xffffffffu, mine, i);
            const int other_block = __shfl_sync(0xffffffffu, block, i);
            over += other > mine || (other == mine && other_block < block);
          }
          if (lane < found && over < rest) atomicOr(&taken[block / 32], 1u << (block & 31));
        }
        __syncthreads();
      } else {
        bool separate;
        const uint64_t t64 = cut<kThreads, uint64_t>(sh, exact_keys, found, rest, 0ull, ~0ull, turn, &separate);
        int over = 0;  // keys above the cut: all of them; at it: the first ones
        for (int i = tid; i < found; i += kThreads) over += exact_keys[i] > t64;
        over = cta_sum<kThreads>(sh, over, turn);
        int equal = separate ? found : rest - over;  // equal ones still to take
        for (int i0 = 0; i0 < found; i0 += kThreads) {
          const int i = i0 + tid;
          const bool same = i < found && exact_keys[i] == t64;
          const uint32_t w = __ballot_sync(0xffffffffu, same);
          if (lane == 0) sh.warp_lo[warp] = __popc(w);
          const int all = cta_sum<kThreads>(sh, same, turn);
          int before = __popc(w & ((1u << lane) - 1u));
          for (int k = 0; k < warp; ++k) before += (int)sh.warp_lo[k];
          if (i < found && (exact_keys[i] > t64 || (same && before < equal)))
            atomicOr(&taken[candidates[i] / 32], 1u << (candidates[i] & 31));
          equal = max(0, equal - all);
          __syncthreads();
        }
      }
    }
  }

  // ---- the list, in order: the first blocks, those taken, the last ones
  for (int i = tid; i < p.first; i += kThreads) list[i] = i;
  for (int i = tid; i < p.last; i += kThreads) list[p.budget - p.last + i] = n - p.last + i;
  int done = p.first;
  for (int i0 = 0; i0 < m && want > 0; i0 += kThreads * 32) {  // a word of 32 blocks per thread
    const int i = i0 / 32 + tid;
    uint32_t w = i < (m + 31) / 32 ? taken[i] : 0u;
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

template <int D, int NG, int NT>
cudaError_t launch_nt(const SelectParams& p, int ranks, cudaStream_t stream) {
  // scores; the copies under way, and then exact scores of as many candidates as there can be
  const size_t ring = (size_t)NT * kAhead * 32, exact = (size_t)p.max_blocks * 8;
  const size_t smem = copies_at(p.max_blocks) + (ring > exact ? ring : exact);
  const auto kernel = select_kernel<D, NG, NT>;
  if (smem > 40 * 1024) {  // (less, with the static part, is granted without asking; the same limit in every call)
    constexpr int kMost = (int)(copies_at(kSelectMaxBlocks) + (size_t)kSelectMaxBlocks * 8);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.num_kv_heads * ranks));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Warps of a list: one for 64 of its blocks, and more, up to one for 16, as long
// as all lists' warps are resident at once (32 to an SM): 512 lists of up to 1,024
// blocks, 64 / 32 / 16 blocks a warp: 30 / 34 / 50 us; 1,024 of 256: 35 / 39 / 44;
// 256 of 256: 17.2 / 16.6 / 16.9.  (1,024 lists of 256 are one wave then, in which
// lists copy together and then select together, and memory idles at both ends.)
// CTAs of 4 warps, of 16 where a cluster of 8 such has not enough.
template <int D, int NG>
cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
  const long long units = (long long)p.batch * p.num_kv_heads, resident = 152 * 32 / units;
  const long long most = (p.max_blocks + 15) / 16, least = (p.max_blocks + 63) / 64;
  const long long warps = most < resident ? most : least > resident ? least : resident;
  const int per = warps > 32 ? 16 : 4;
  int ranks = 1;
  while (ranks < 8 && ranks * per < warps && units * ranks < (1 << 28)) ranks *= 2;
  return per == 16 ? launch_nt<D, NG, 512>(p, ranks, stream) : launch_nt<D, NG, 128>(p, ranks, stream);
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const int groups = kBlockTokens / p.group;
  if (p.head_dim == 64) return groups == 2 ? launch<64, 2>(p, stream) : launch<64, 4>(p, stream);
  if (p.head_dim == 128)
    return groups == 1 ? launch<128, 1>(p, stream) : groups == 2 ? launch<128, 2>(p, stream) : launch<128, 4>(p, stream);
  return groups == 1 ? launch<256, 1>(p, stream) : groups == 2 ? launch<256, 2>(p, stream) : launch<256, 4>(p, stream);
}

}  // namespace kvq
