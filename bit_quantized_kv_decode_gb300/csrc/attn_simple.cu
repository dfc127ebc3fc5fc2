// Attention over rows of new tokens, the plain way: one CTA per 32 rows
// (token, head of the KV group) of one sequence and KV head, K and V staged
// 32 tokens at a time as fp32 in shared memory, an online softmax per row.
// Four threads share a row; each forms 8 of a tile's 32 scores and owns a
// quarter of the output channels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_rows.h"

namespace kvq {
namespace {

constexpr int kRows = 32, kTile = 32, kThreads = 128;

__device__ __forceinline__ float load16(const void* p, long long i, int fp16) {
  return fp16 ? __half2float(static_cast<const __half*>(p)[i])
              : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Value (t, c) of page `page`, KV head h, as fp16 (the operand precision).
__device__ float cache_value(const RowAttnParams& p, int which, int page, int h, int t, int c) {
  const int D = p.head_dim, G = p.group, bits = p.bits;
  const size_t blk = (size_t)page * p.num_kv_heads + h;
  const uint8_t* codes = (which ? p.v_codes : p.k_codes) + blk * (size_t)(kBlockTokens * D * bits / 8);
  const int row = which ? c : t, col = which ? t : c, nrows = which ? D : kBlockTokens;
  const int byte = col * bits / 8;
  const uint32_t code = (codes[((byte / 16) * nrows + row) * 16 + byte % 16] >> (col * bits % 8)) & ((1u << bits) - 1);
  const int scheme = which ? p.v_scheme : p.k_scheme;
  const size_t e = blk * (kBlockTokens * D / G) + (scheme == KVQ_TOKENWISE ? t * (D / G) + c / G : (t / G) * D + c);
  float s = __half2float(__ushort_as_half((which ? p.v_scale : p.k_scale)[e]));
  float z = __half2float(__ushort_as_half((which ? p.v_zero : p.k_zero)[e]));
  const float qmax = (float)((1 << bits) - 1);
  if (!(fmaf(s, qmax, z) <= 65504.f) || !(z >= -65504.f)) {  // past the fp16 range, or not finite
    report(p.dev_status, KVQ_DEV_NONFINITE);
    if (!isfinite(s) || !isfinite(z)) s = z = 0.f;
    else s = __half2float(__float2half_rd((65504.f - z) / qmax));
  }
  return __half2float(__float2half_rn(fmaf(s, (float)code, z)));
}

template <int D>
__global__ void __launch_bounds__(kThreads) simple_kernel(const RowAttnParams p, bool cached) {
  extern __shared__ float sm[];
  float* qs = sm;                         // [32][D + 1]
  float* ks = qs + kRows * (D + 1);       // [32][D + 1]
  float* vs = ks + kTile * (D + 1);       // [32][D]
  float* ps = vs + kTile * D;             // [32][33]
  const int tid = threadIdx.x, h = blockIdx.y;
  // this CTA's sequence and first row
  int b = 0, r0 = blockIdx.x;
  SeqRows s{};
  for (; b < p.batch; ++b) {
    s = seq_rows(p.cu, b, p.total);
    if (s.bad && r0 == 0 && h == 0 && tid == 0) report(p.dev_status, KVQ_DEV_BAD_SEQ_LEN);
    const int tiles = (s.n * p.gq + kRows - 1) / kRows;
    if (r0 < tiles) break;
    r0 -= tiles;
  }
  if (b == p.batch) return;
  r0 *= kRows;
  int len = cached ? p.seq_lens[b] : s.n;
  if (cached && (len < 0 || len > p.max_blocks * kBlockTokens)) {
    if (r0 == 0 && h == 0 && tid == 0) report(p.dev_status, KVQ_DEV_BAD_SEQ_LEN);
    len = 0;
  }
  const int before = len - s.n;  // position of the chunk's first token
  const int rows = min(kRows, s.n * p.gq - r0);
  for (int i = tid; i < rows * D; i += kThreads) {
    const int r = i / D, c = i % D, t = (r0 + r) / p.gq, g = (r0 + r) % p.gq;
    qs[r * (D + 1) + c] = load16(p.q.data, (s.first + t) * p.q.st + (h * p.gq + g) * p.q.sh + c, p.fp16);
  }
  const int r = tid / 4, part = tid % 4;
  const int my = r < rows ? (p.causal ? before + (r0 + r) / p.gq : len - 1) : -1;   // last position seen
  const int top = p.causal ? min(len - 1, before + (r0 + rows - 1) / p.gq) : len - 1;  // ... by any row
  float m = -INFINITY, l = 0.f, acc[D / 4];
#pragma unroll
  for (int c = 0; c < D / 4; ++c) acc[c] = 0.f;
  for (int t0 = 0; t0 <= top; t0 += kTile) {
    __syncthreads();
    for (int i = tid; i < kTile * D; i += kThreads) {
      const int t = i / D, c = i % D;
      float k = 0.f, v = 0.f;
      if (t0 + t < len) {
        if (cached) {
          const int j = (t0 + t) / kBlockTokens;
          const int page = p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
          if (page < 0 || page >= p.num_pages) {
            if (h == 0 && c == 0) report(p.dev_status, KVQ_DEV_BAD_PAGE);
          } else {
            k = cache_value(p, 0, page, h, (t0 + t) % kBlockTokens, c);
            v = cache_value(p, 1, page, h, (t0 + t) % kBlockTokens, c);
          }
        } else {
          k = load16(p.k.data, (s.first + t0 + t) * p.k.st + h * p.k.sh + c, p.fp16);
          v = load16(p.v.data, (s.first + t0 + t) * p.v.st + h * p.v.sh + c, p.fp16);
        }
      }
      ks[t * (D + 1) + c] = k;
      vs[t * D + c] = v;
    }
    __syncthreads();
    float sc[8], mt = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = part + 4 * i;
      float d = 0.f;
      for (int c = 0; c < D; ++c) d = fmaf(qs[r * (D + 1) + c], ks[t * (D + 1) + c], d);
      sc[i] = t0 + t <= my ? d * p.scale_log2 : -INFINITY;
      mt = fmaxf(mt, sc[i]);
    }
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
    const float mn = fmaxf(m, mt);
    const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
    float lt = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = mn == -INFINITY ? 0.f : exp2f(sc[i] - mn);
      lt += e;
      ps[r * 33 + part + 4 * i] = p.fp16 || cached ? __half2float(__float2half_rn(e * 128.f)) / 128.f
                                                   : __bfloat162float(__float2bfloat16_rn(e));
    }
    lt += __shfl_xor_sync(0xffffffffu, lt, 1);
    lt += __shfl_xor_sync(0xffffffffu, lt, 2);
    l = l * a + lt;
    m = mn;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < D / 4; ++c) acc[c] *= a;
    for (int t = 0; t < kTile; ++t) {
      const float e = ps[r * 33 + t];
      if (e == 0.f) continue;
#pragma unroll
      for (int c = 0; c < D / 4; ++c) acc[c] = fmaf(e, vs[t * D + part + 4 * c], acc[c]);
    }
  }
  if (r >= rows) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const long long row = (long long)(s.first + (r0 + r) / p.gq) * p.num_q_heads + h * p.gq + (r0 + r) % p.gq;
#pragma unroll
  for (int c = 0; c < D / 4; ++c) {
    const float o = acc[c] * inv;
    if (p.fp16) static_cast<__half*>(p.out)[row * D + part + 4 * c] = __float2half_rn(o);
    else static_cast<__nv_bfloat16*>(p.out)[row * D + part + 4 * c] = __float2bfloat16_rn(o);
  }
  if (p.lse != nullptr && part == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
cudaError_t launch(const RowAttnParams& p, bool cached, cudaStream_t stream) {
  constexpr int smem = (kRows * (D + 1) + kTile * (D + 1) + kTile * D + kRows * 33) * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(simple_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long long)p.total * p.gq / kRows + p.batch), p.num_kv_heads);
  simple_kernel<D><<<grid, kThreads, smem, stream>>>(p, cached);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_row_attn_simple(const RowAttnParams& p, bool cached, cudaStream_t stream) {
  if (p.head_dim == 64) return launch<64>(p, cached, stream);
  if (p.head_dim == 128) return launch<128>(p, cached, stream);
  return launch<256>(p, cached, stream);
}

}  // namespace kvq
