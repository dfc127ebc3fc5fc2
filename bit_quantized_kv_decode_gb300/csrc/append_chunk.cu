// Quantise and append a chunk of new tokens to the packed K and V caches.
//
// One CTA per (block touched, KV head, 64- or 128-channel slab, K or V);
// sequence b touches blocks seq_lens[b] / 128 to (seq_lens[b] + n - 1) / 128.
// The tile (128 tokens x 64 or 128 channels) is read once into registers: a
// thread has 4 neighbouring channels of 4 to 16 consecutive tokens, so rows are
// read as 8-byte (fp32: 16-byte) pieces of full lines, a channel-wise group is
// reduced in registers and across warps, a token-wise one across the lanes that
// share the token, and V's codes, packed along tokens, come out of one thread's
// registers as whole words.  The packed block is put together in shared memory
// and written in 16-byte pieces.
//
// Two kernels.  append_blocks_kernel takes the blocks that consist of new
// 16-bit tokens alone: the tile stays in its 16-bit form (half the registers,
// so more loads in flight), ranges are formed on 16-bit pairs.
// append_edges_kernel takes the rest in fp32 -- the first and last block of a
// chunk, with the window's rows and the tokens that stay, and every block of
// fp32 rows.  They write disjoint places; the second starts once the last CTA of
// the first has, so that the two overlap in the first one's last wave.
//
// The work is one pass over the rows, and memory would bound it below about ten
// instructions a value; it takes 16 with everything, so whole blocks are bound
// by instructions and barriers (65,536 tokens x 8 heads of 128, bf16 to 4 bits,
// K channel-wise, V token-wise: 86 us, 4.0 TB/s, 66% of the issue slots; as fp32
// rows, all of them edges: 212 us, 2.9 TB/s), edges by the latency of one block
// (128 sequences of a token, windows re-quantised: 39 us, 3.6 TB/s).  Slower
// when tried: 16 warps to a whole block (140 -> 164 us); K and V of a block in
// one CTA, V's loads under K's stores, gained 2%.
//
// The code of a value is clamp(rint(fl(fl(x - z) / s))) in IEEE fp32.  With
// d = fl(x - z) and r = fl(1 / s) once per group, the quotient is corrected once
// after Markstein ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): q = fl(d r), q' = fma(fma(-q, s, d), r, q) is
// fl(d / s), since s, an fp16 number, has no all-ones fp32 significand (checked
// for every s and the 13 fp32 numbers nearest to each half of a code); adding
// 1.5 x 2^23 then rounds it to the nearest even integer.  No clamp is needed:
// q' >= 0, because z was rounded down, and at most 2^b - 1 up to rounding,
// because s was rounded up.  (Deciding by d r alone and dividing where it lies
// near a half was slower: coarse 16-bit values meet exact halves 0.07% of the
// time, in three warps of four.)
#include "append_core.cuh"

namespace kvq {
namespace {

template <typename T, int BITS, int W>
__global__ void __launch_bounds__(32 * kBlockWarps, kBlockCtas) append_blocks_kernel(const AppendParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the edges' kernel runs beside this one
  append_block<T, BITS, W>(p, blockIdx.z & 1, blockIdx.z >> 1);
}

template <typename T, int BITS, int W, Part PART>
__global__ void __launch_bounds__(32 * kEdgeWarps, sizeof(Raw<T>) == 8 ? 2 : 1) append_edges_kernel(const AppendParams p) {
  append_edge<T, BITS, W, PART, false>(p);
  // overlaps append_blocks_kernel: what follows in the stream waits for
  // this grid, which is not done before that one is
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T, int BITS, int W>
cudaError_t launch_w(const AppendParams& p, cudaStream_t stream) {
  constexpr bool kHalf = sizeof(Raw<T>) == 8;
  const unsigned heads = (unsigned)p.num_kv_heads, planes = (unsigned)(2 * (p.head_dim / W));
  const bool whole = kHalf && p.total >= kBlockTokens;  // there may be blocks of new tokens alone
  if constexpr (kHalf) {
    if (whole) {
      append_blocks_kernel<T, BITS, W><<<dim3((unsigned)(p.total / kBlockTokens), heads, planes), 32 * kBlockWarps, 0, stream>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  const long long blocks = edge_blocks(p.batch, p.total, kHalf);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, heads, planes);
  cfg.blockDim = dim3(32 * kEdgeWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = whole ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, append_edges_kernel<T, BITS, W, kHalf ? kEdges : kEvery>, p);
}

template <typename T>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  if (p.bits == 4) return p.head_dim < 128 ? launch_w<T, 4, 64>(p, stream) : launch_w<T, 4, 128>(p, stream);
  return p.head_dim < 128 ? launch_w<T, 2, 64>(p, stream) : launch_w<T, 2, 128>(p, stream);
}

}  // namespace

cudaError_t launch_append_chunk(const AppendParams& p, cudaStream_t stream) {
  if (p.dtype == KVQ_FP32) return launch<float>(p, stream);
  if (p.dtype == KVQ_FP16) return launch<__half>(p, stream);
  return launch<Bf16Tag>(p, stream);
}

}  // namespace kvq
