// Append with the position rotation (append_rotary.cuh): rows turned on their own,
// and the dispatch.
#include <cuda_bf16.h>

#include "append_rotary.cuh"

namespace kvq {
namespace {

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

// One warp per token and piece of q's (or k's) heads: a lane has two pieces of 8
// channels of a head -- the two halves of 8 pairs -- and their angles for the
// kPasses heads it comes to, whose loads go out together.  What bounds it is
// memory: 32,768 tokens x 40 heads of 128 in bf16, 671 MB: 98 us, 6.8 TB/s.
constexpr int kTurnThreads = 128, kPasses = 4;

template <typename T>
__device__ __forceinline__ void turn_rows(const TurnRowsParams& p, int q_pieces) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kTurnThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.total) return;
  const int D = p.head_dim, R = p.turn.dim, half = R / 2;
  const int lanes = D / 16, sub = lane / lanes, i = lane % lanes, each = 32 / lanes;  // lanes of a head, heads at a time
  const bool turns = i * 16 < R, near = !turns || p.turn.interleaved;
  const int c0 = near ? 16 * i : 8 * i, c1 = near ? 16 * i + 8 : half + 8 * i;
  const bool key = blockIdx.y >= q_pieces;
  const int heads = key ? p.heads[1] : p.heads[0], h0 = (blockIdx.y - (key ? q_pieces : 0)) * each * kPasses + sub;
  const Rows x = key ? p.x[1] : p.x[0];
  Eight<T> u[kPasses], v[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int h = h0 + k * each;
    if (h < heads) {
      const long long from = (long long)t * x.st + (long long)h * x.sh;
      u[k].load(x.data, from + c0);
      v[k].load(x.data, from + c1);
    }
  }
  const int b = sequence_of(p.cu, p.batch, t);
  if (b < 0) return;
  const SeqRows s = seq_rows(p.cu, b, p.total);
  const int len = p.seq_lens[b];
  if (s.bad || len < 0 || (long long)len + s.n > p.most) return;
  const int pos = len + t - s.first;
  uint64_t c[4], sn[4];  // of the pairs two by two
  if (turns) {
    const float* at = p.turn.angles + (size_t)pos * R + 8 * i;
    const ulonglong2 *cp = reinterpret_cast<const ulonglong2*>(at), *sp = reinterpret_cast<const ulonglong2*>(at + half);
    const ulonglong2 ca = __ldg(cp), cb = __ldg(cp + 1), sa = __ldg(sp), sb = __ldg(sp + 1);
    c[0] = ca.x; c[1] = ca.y; c[2] = cb.x; c[3] = cb.y;
    sn[0] = sa.x; sn[1] = sa.y; sn[2] = sb.x; sn[3] = sb.y;
  }
  const uint64_t minus = rows::pair(-p.turn.one, -p.turn.one), plus = rows::pair(p.turn.one, p.turn.one);
  void* out = key ? p.out[1] : p.out[0];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int h = h0 + k * each;
    if (h >= heads) break;
    if (turns) {
      float a[8], d[8];
      u[k].get(a);
      v[k].get(d);
      if (near) {  // even and odd channels apart, and together again
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* y = e < 2 ? a + 4 * e : d + 4 * (e - 2);  // two pairs
          const uint64_t x1 = rows::pair(y[0], y[2]), x2 = rows::pair(y[1], y[3]);
          rows::unpair(rows::fma2(rows::mul2(x2, sn[e]), minus, rows::mul2(x1, c[e])), y[0], y[2]);
          rows::unpair(rows::fma2(rows::mul2(x1, sn[e]), plus, rows::mul2(x2, c[e])), y[1], y[3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t x1 = rows::pair(a[2 * e], a[2 * e + 1]), x2 = rows::pair(d[2 * e], d[2 * e + 1]);
          rows::unpair(rows::fma2(rows::mul2(x2, sn[e]), minus, rows::mul2(x1, c[e])), a[2 * e], a[2 * e + 1]);
          rows::unpair(rows::fma2(rows::mul2(x1, sn[e]), plus, rows::mul2(x2, c[e])), d[2 * e], d[2 * e + 1]);
        }
      }
      u[k].put(a);
      v[k].put(d);
    }
    const long long to = ((long long)t * heads + h) * D;
    u[k].store(out, to + c0);
    v[k].store(out, to + c1);
  }
}

template <typename T>
__global__ void __launch_bounds__(kTurnThreads) turn_rows_kernel(const TurnRowsParams p, int q_pieces) {
  let_next_start();
  turn_rows<T>(p, q_pieces);
  end_after_last();
}

template <typename T>
cudaError_t launch_turn(const TurnRowsParams& p, Chain& chain) {
  const int each = 512 / p.head_dim * kPasses;  // heads of a warp
  const int q_pieces = (p.heads[0] + each - 1) / each, k_pieces = (p.heads[1] + each - 1) / each;
  return chain.launch(dim3((unsigned)((p.total + kTurnThreads / 32 - 1) / (kTurnThreads / 32)), (unsigned)(q_pieces + k_pieces)),
                      kTurnThreads, 0, turn_rows_kernel<T>, p, q_pieces);
}

}  // namespace

bool rows_to_turn(const TurnRowsParams& rows) { return rows.total > 0 && rows.heads[0] + rows.heads[1] > 0; }

cudaError_t launch_turn_rows(const TurnRowsParams& rows, Chain& chain) {
  if (rows.dtype == KVQ_FP32) return launch_turn<float>(rows, chain);
  if (rows.dtype == KVQ_FP16) return launch_turn<__half>(rows, chain);
  return launch_turn<Bf16Tag>(rows, chain);
}

cudaError_t launch_append_rotary(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  return p.bits == 4 ? launch_append_rotary_i4(p, rows, stream) : launch_append_rotary_i2(p, rows, stream);
}

}  // namespace kvq
