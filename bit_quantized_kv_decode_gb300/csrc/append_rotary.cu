// Append with the position rotation on the way, and rows turned on their own.
//
// The first R channels of a row at position p are pairs (x1, x2) -- channel i
// with i + R / 2, or neighbours -- that become
//   (fl(fl(x1 c) - fl(x2 s)), fl(fl(x2 c) + fl(x1 s))),  c, s = cos, sin of the pair's angle at p,
// in fp32.  K goes into the cache from there, without a rounding to the rows'
// type between; turned queries (and keys, where attention over rows follows)
// are rounded to it once.
#include <cuda_bf16.h>

#include "append_core.cuh"

namespace kvq {
namespace {

template <typename T, int BITS, int W>
cudaError_t launch_w(const AppendParams& p, cudaStream_t stream) {
  const unsigned heads = (unsigned)p.num_kv_heads, planes = (unsigned)(2 * (p.head_dim / W));
  const long long two = p.batch < p.total / 2 ? p.batch : p.total / 2;
  const long long blocks = p.batch + two + (p.total - 2 * two) / kBlockTokens;  // (as for append_chunk's edges)
  append_edges_kernel<T, BITS, W, kEvery, true><<<dim3((unsigned)blocks, heads, planes), 32 * kEdgeWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  if (p.bits == 4) return p.head_dim < 128 ? launch_w<T, 4, 64>(p, stream) : launch_w<T, 4, 128>(p, stream);
  return p.head_dim < 128 ? launch_w<T, 2, 64>(p, stream) : launch_w<T, 2, 128>(p, stream);
}

// ------------------------------------------------------------- rows alone

// Eight neighbouring channels of a row, in fp32.
template <typename T>
struct Eight {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, long long at) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = wide<T>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void put(const float (&x)[8]) {
    constexpr bool kHalf = sizeof(T) == sizeof(__half);
    v = make_uint4(rows::round2<kHalf>(x[0], x[1]), rows::round2<kHalf>(x[2], x[3]), rows::round2<kHalf>(x[4], x[5]),
                   rows::round2<kHalf>(x[6], x[7]));
  }
  __device__ __forceinline__ void store(void* p, long long at) const {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = v;
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, long long at) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = __ldg(src);
    b = __ldg(src + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void put(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void store(void* p, long long at) const {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    dst[0] = a;
    dst[1] = b;
  }
};

// The sequence that row t belongs to (cu[b] <= t < cu[b + 1]) by a warp, 32
// entries at a time; -1 where there is none.  Behind an entry that goes back a
// row may be missed, never taken for another sequence's.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;  // the last entry <= t, if any, is one of lo ... lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, i < n && cu[lo + min(i, n - 1)] <= t);
    if (le == 0u) return -1;
    const int k = 31 - __clz((int)le);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// One warp per token and piece of the heads: a lane has two pieces of 8
// channels of a head -- the two halves of 8 pairs -- and their angles for all
// heads it comes to.
constexpr int kTurnThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kTurnThreads) turn_rows_kernel(const TurnRowsParams p, int heads_each) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kTurnThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.total) return;
  const int b = sequence_of(p.cu, p.batch, t);
  if (b < 0) return;
  const SeqRows s = seq_rows(p.cu, b, p.total);
  const int len = p.seq_lens[b];
  if (s.bad || len < 0 || (long long)len + s.n > p.most) return;
  const int pos = len + t - s.first;
  const int D = p.head_dim, R = p.turn.dim, half = R / 2;
  const int lanes = D / 16, sub = lane / lanes, i = lane % lanes;  // lanes of a head, head of this pass, pairs 8 i ...
  const bool turns = i * 16 < R;
  const bool apart = turns && !p.turn.interleaved;
  const int c0 = apart ? 8 * i : 16 * i, c1 = apart ? half + 8 * i : 16 * i + 8;
  float c[8], sn[8];
  if (turns) {
    const float* at = p.turn.angles + (size_t)pos * R + 8 * i;
    Eight<float> v;
    v.load(at, 0);
    v.get(c);
    v.load(at, half);
    v.get(sn);
  }
  const int h0 = blockIdx.y * heads_each, all = p.heads[0] + p.heads[1];
  for (int hh = h0 + sub; hh < min(all, h0 + heads_each); hh += 32 / lanes) {
    const int which = hh >= p.heads[0], h = which ? hh - p.heads[0] : hh;
    const Rows& x = p.x[which];
    const long long from = (long long)t * x.st + (long long)h * x.sh, to = ((long long)t * p.heads[which] + h) * D;
    Eight<T> u, v;
    u.load(x.data, from + c0);
    v.load(x.data, from + c1);
    if (turns) {
      float a[8], d[8];
      u.get(a);
      v.get(d);
      if (apart) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x1 = a[k], x2 = d[k];
          a[k] = __fsub_rn(__fmul_rn(x1, c[k]), __fmul_rn(x2, sn[k]));
          d[k] = __fadd_rn(__fmul_rn(x2, c[k]), __fmul_rn(x1, sn[k]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x1 = a[2 * k], x2 = a[2 * k + 1];
          a[2 * k] = __fsub_rn(__fmul_rn(x1, c[k]), __fmul_rn(x2, sn[k]));
          a[2 * k + 1] = __fadd_rn(__fmul_rn(x2, c[k]), __fmul_rn(x1, sn[k]));
          x1 = d[2 * k], x2 = d[2 * k + 1];
          d[2 * k] = __fsub_rn(__fmul_rn(x1, c[k + 4]), __fmul_rn(x2, sn[k + 4]));
          d[2 * k + 1] = __fadd_rn(__fmul_rn(x2, c[k + 4]), __fmul_rn(x1, sn[k + 4]));
        }
      }
      u.put(a);
      v.put(d);
    }
    u.store(p.out[which], to + c0);
    v.store(p.out[which], to + c1);
  }
}

template <typename T>
cudaError_t launch_turn(const TurnRowsParams& p, cudaStream_t stream) {
  const int all = p.heads[0] + p.heads[1], pass = 512 / p.head_dim;  // heads of a warp at a time
  const int each = pass * 4;
  turn_rows_kernel<T><<<dim3((unsigned)((p.total + kTurnThreads / 32 - 1) / (kTurnThreads / 32)), (unsigned)((all + each - 1) / each)),
                        kTurnThreads, 0, stream>>>(p, each);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rotary(const AppendParams& p, cudaStream_t stream) {
  if (p.dtype == KVQ_FP32) return launch<float>(p, stream);
  if (p.dtype == KVQ_FP16) return launch<__half>(p, stream);
  return launch<Bf16Tag>(p, stream);
}

cudaError_t launch_turn_rows(const TurnRowsParams& p, cudaStream_t stream) {
  if (p.total == 0 || p.heads[0] + p.heads[1] == 0) return cudaSuccess;
  if (p.dtype == KVQ_FP32) return launch_turn<float>(p, stream);
  if (p.dtype == KVQ_FP16) return launch_turn<__half>(p, stream);
  return launch_turn<Bf16Tag>(p, stream);
}

}  // namespace kvq
