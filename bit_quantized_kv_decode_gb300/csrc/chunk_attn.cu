// Chunk attention: launch shape, workspace and the merge of cut tiles.
#include "chunk_attn.cuh"

namespace kvq {
namespace chunk {
namespace {

constexpr int kGrid = 152;  // one CTA per SM; they do not wait on one another, so fewer SMs only take longer
constexpr int kSmem = 227 * 1024;
constexpr int kMergeThreads = 256, kMergeRows = 32, kMergeLanes = kMergeThreads / kMergeRows;  // lanes of a row

// Joins the parts of the tile that the border between CTAs blockIdx.x and
// blockIdx.x + 1 is the first to cut, rows blockIdx.y * 32 on:
// lse = log2 sum 2^lse_i, out = sum 2^(lse_i - lse) o_i.  Eight lanes to a row,
// so that a CTA's rows are all read at once: what it takes is latency.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Params P, int nt, int grid) {
  __shared__ long long scan[kMergeThreads / 32], range[3];
  __shared__ Place at;
  __shared__ int list[kGrid], parts;
  const RowAttnParams& p = P.r;
  const int cta = blockIdx.x + 1, tid = threadIdx.x;
  const int tok_tile = kTile / p.gq, tok_cta = tok_tile * nt;
  find_place<kMergeThreads>(p, tok_cta, cta, grid, scan, &at, range, false);
  // every CTA waits, those that have nothing to join too: what follows in the
  // stream waits for this grid, which must not be done before that one is
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long total = range[2];
  if (range[0] >= total || at.x == 0) return;  // past the last step (`at` is unset), or between two tiles
  const long long tile0 = at.tile0, before = total * (cta - 1) / grid;
  if (before > tile0) return;  // an earlier border cut this tile
  uint32_t bad = 0;
  const Seq s = load_seq(p, at.b, &bad);
  const int work = work_steps(key_tiles(s, at.t, tok_cta, p.causal));
  if (at.x >= work) return;  // the border lies behind the tile's work
  const long long end = tile0 + work;
  const int slot0 = 2 * (cta - 1) + (before == tile0 ? 0 : 1);
  // The parts: CTA cta - 1's, then one of every CTA that begins before the end
  // and has steps (all have, where there are as many steps as CTAs).
  if (tid == 0) {
    int n = 0;
    for (int c = cta; c < grid && total * c / grid < end; ++c)
      if (total >= grid || total * (c + 1) / grid > total * c / grid) list[n++] = 2 * c;
    parts = n;
  }
  __syncthreads();
  const size_t pitch = (size_t)nt * kTile;
  const int prow = blockIdx.y * kMergeRows + tid / kMergeLanes, r = prow & (kTile - 1), sub = tid % kMergeLanes;
  const int tile_tok = at.t * tok_cta + (prow / kTile) * tok_tile, tok = tile_tok + r / p.gq;
  const bool mine = r < tok_tile * p.gq && tok < s.n;
  auto part = [&](int k) { return (size_t)(k == 0 ? slot0 : list[k - 1]) * pitch + prow; };
  float m = -INFINITY;
  if (mine)
    for (int k = sub; k <= parts; k += kMergeLanes) m = fmaxf(m, P.part_lse[part(k)]);
#pragma unroll
  for (int o = kMergeLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!mine) return;
  constexpr int kPer = D / 4 / kMergeLanes;  // of four channels, kMergeLanes apart
  float4 acc[kPer];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k <= parts; ++k) {
    const size_t at_part = part(k);
    const float l = P.part_lse[at_part];
    const float w = l == -INFINITY ? 0.f : exp2f(l - m);  // 0: nothing seen in this part (NaN stays, m passes it over)
    sum += w;
    const float4* o = reinterpret_cast<const float4*>(P.part_o + at_part * D) + sub;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float4 v = o[e * kMergeLanes];
      acc[e].x = fmaf(w, v.x, acc[e].x);
      acc[e].y = fmaf(w, v.y, acc[e].y);
      acc[e].z = fmaf(w, v.z, acc[e].z);
      acc[e].w = fmaf(w, v.w, acc[e].w);
    }
  }
  const float inv = sum > 0.f || isnan(sum) ? 1.f / sum : 0.f;
  const long long row = (long long)(s.first + tok) * p.num_q_heads + at.h * p.gq + r % p.gq;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D) + sub;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float4 v = make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
    dst[e * kMergeLanes] = p.fp16 ? make_uint2(rows::round2<true>(v.x, v.y), rows::round2<true>(v.z, v.w))
                                  : make_uint2(rows::round2<false>(v.x, v.y), rows::round2<false>(v.z, v.w));
  }
  if (sub == 0 && p.lse != nullptr)
    p.lse[row] = sum > 0.f || isnan(sum) ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace
}  // namespace chunk

namespace chunk {
namespace {

struct Memory {
  int table_bytes, unit_bytes, units;
  size_t total;
};
// What an instance's shared memory is divided into: units = 0 where the
// ring of packed blocks would not hold one for each team.
Memory memory_of(int head_dim, int group, int bits, int nt) {
  Memory m;
  const int nsz = kBlockTokens * head_dim / group, teams = teams_of(head_dim);
  m.table_bytes = 4 * nsz;
  m.unit_bytes = kBlockTokens * head_dim * bits / 8 + 4 * nsz;
  const int fixed = fixed_bytes(head_dim, nt) + teams * 2 * m.table_bytes;
  m.units = (kSmem - fixed) / m.unit_bytes;
  if (m.units > kMaxUnits) m.units = kMaxUnits;
  m.units -= m.units % teams;  // a unit's place in the ring belongs to one dequantising team
  m.total = (size_t)fixed + (size_t)m.units * m.unit_bytes;
  return m;
}

}  // namespace
}  // namespace chunk

ChunkPlan chunk_plan(int head_dim, int group, int bits, int batch, int total, int num_q_heads, int num_kv_heads) {
  ChunkPlan c;
  // two row tiles where the sequences have more rows than one on average
  // (head dim 256: one, its accumulators fill tensor memory; nor where shared
  // memory is too small for two, as with 4-bit codes in groups of 32 at 128)
  const long long rows = (long long)total * (num_q_heads / num_kv_heads);
  const int most = head_dim <= 128 && chunk::memory_of(head_dim, group, bits, 2).units > 0 ? 2 : 1;
  c.nt = rows > (long long)batch * chunk::kTile ? most : 1;
  c.grid = chunk::kGrid;
  // the workspace of the larger shape for both: fewer sequences may take two row
  // tiles where more take one, and a buffer made for the larger call serves both
  const size_t slots = (size_t)2 * c.grid * most * chunk::kTile;
  c.part_lse = slots * head_dim * sizeof(float);
  c.total = c.part_lse + slots * sizeof(float);
  return c;
}

cudaError_t launch_chunk_attn(const RowAttnParams& p, const ChunkPlan& plan, void* workspace, cudaStream_t stream) {
  using namespace chunk;
  Params P{};
  P.r = p;
  P.part_o = static_cast<float*>(workspace);
  P.part_lse = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + plan.part_lse);
  P.gshift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
  const Memory m = memory_of(p.head_dim, p.group, p.bits, plan.nt);
  P.table_bytes = m.table_bytes;
  P.unit_bytes = m.unit_bytes;
  P.units = m.units;
  if (m.units < 1) return cudaErrorInvalidValue;
  cudaError_t e = p.bits == 2 ? launch_i2(p.head_dim, plan.nt, P, plan.grid, m.total, stream)
                              : launch_i4(p.head_dim, plan.nt, P, plan.grid, m.total, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(plan.grid - 1), (unsigned)(plan.nt * kTile / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.head_dim == 64) return cudaLaunchKernelEx(&cfg, merge_kernel<64>, P, plan.nt, plan.grid);
  if (p.head_dim == 128) return cudaLaunchKernelEx(&cfg, merge_kernel<128>, P, plan.nt, plan.grid);
  return cudaLaunchKernelEx(&cfg, merge_kernel<256>, P, plan.nt, plan.grid);
}

}  // namespace kvq
