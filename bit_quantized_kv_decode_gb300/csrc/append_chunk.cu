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
// K channel-wise, V token-wise: 90 us, 3.8 TB/s, 67% of the issue slots; as fp32
// rows, all of them edges: 242 us, 2.5 TB/s), edges by the latency of one block
// (128 sequences of a token, windows re-quantised: 51 us, 2.7 TB/s).  Slower
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
#include <cuda_fp16.h>

#include "attn_core.cuh"

namespace kvq {
namespace {

// Warps of a block.  Edges: twice as many, each with half the tokens (8 of a
// thread): their loads and stores depend on one another, so what counts is how
// many warps wait at a time (256 sequences of a token: 67 -> 54 us).
constexpr int kBlockWarps = 8, kEdgeWarps = 16;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Group {
  float s, z;  // s NaN: the group is refused (not finite, or past the fp16 range) and left zero
  uint16_t s_bits, z_bits;
};
// Scale and offset of a group with minimum mn and maximum mx (NaN where a
// value is NaN; mn > mx: no value at all).
__device__ __forceinline__ Group group_of_range(float mn, float mx, float qmax) {
  Group g{0.f, 0.f, 0, 0};
  if (mn > mx) return g;
  const __half zh = __float2half_rd(mn);
  const float z = __half2float(zh), width = __fsub_rn(mx, z);
  const __half sh = width != 0.f ? __float2half_ru(__fdiv_rn(width, qmax)) : __float2half_rn(0.f);
  if (!(fabsf(mn) < INFINITY) || !(fabsf(mx) < INFINITY) || __hisinf(zh) || __hisinf(sh)) {
    g.s = NAN;
    return g;
  }
  return Group{__half2float(sh), z, __half_as_ushort(sh), __half_as_ushort(zh)};
}
// What the codes of a group are made with: its scale's reciprocal, 0 where
// every code is 0.
__device__ __forceinline__ float reciprocal(float s) { return s > 0.f ? __frcp_rn(s) : 0.f; }

constexpr float kMagic = 12582912.f;  // 1.5 x 2^23: adding it leaves rint in the low bits
constexpr uint32_t kMagicBits = 0x4b400000u;

// The codes of two values plus kMagicBits (r = 0: zero): the fp32 pipe takes
// pairs, each half rounded as by itself.  zn, sn: -z, -s.
__device__ __forceinline__ void code_pair(float x0, float x1, uint64_t sn, uint64_t zn, uint64_t r, uint32_t& y0,
                                          uint32_t& y1) {
  const uint64_t d = rows::add2(rows::pair(x0, x1), zn), q = rows::mul2(d, r);
  float a, b;
  rows::unpair(rows::add2(rows::fma2(rows::fma2(q, sn, d), r, q), rows::pair(kMagic, kMagic)), a, b);
  y0 = __float_as_uint(a);
  y1 = __float_as_uint(b);
}

// Reductions over the lanes of a group of LG lanes for N values a lane at
// once, halving the values held at each exchange: afterwards lane l of the
// group holds value v[0], number l >> log2(LG / N) (LG >= N), or the N / LG
// values from l * N / LG on.
template <int N, bool MAX>
__device__ __forceinline__ void reduce_group(float (&v)[N], int lg) {
  int o = lg >> 1;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    if (o > 0) {
      const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float keep = upper ? v[i + n / 2] : v[i];
        const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + n / 2], o);
        v[i] = MAX ? max_nan(keep, got) : min_nan(keep, got);
      }
      o >>= 1;
    }
  }
  for (; o > 0; o >>= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
    v[0] = MAX ? max_nan(v[0], got) : min_nan(v[0], got);
  }
}

// Four neighbouring values at `at` (elements).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 v;
  __device__ __forceinline__ void load(const void* p, long long at) {
    v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
  }
  __device__ __forceinline__ float4 get() const { return v; }
};
struct Raw16 {
  uint2 v;
  __device__ __forceinline__ void load(const void* p, long long at) {
    v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at));
  }
};
struct Bf16Tag {};
template <>
struct Raw<Bf16Tag> : Raw16 {
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
  }
};
template <>
struct Raw<__half> : Raw16 {
  __device__ __forceinline__ float4 get() const {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

// Tokens of sequence b's chunk and of its cache; a bad entry has no blocks.
struct Chunk {
  SeqRows rows;
  int len;
  bool bad;
};
__device__ __forceinline__ Chunk load_chunk(const AppendParams& p, int b) {
  Chunk c;
  c.rows = seq_rows(p.cu, b, p.total);
  c.len = p.seq_lens[b];
  c.bad = c.rows.bad || c.len < 0 || (long long)c.len + c.rows.n > (long long)p.max_blocks * kBlockTokens;
  return c;
}
// Blocks of a sequence that a kernel takes, in order.  Whole: those of new
// tokens alone.  Edges: the others (one for an empty chunk: its window).
__device__ __forceinline__ int whole_blocks(const Chunk& c) {
  return c.bad ? 0 : max(0, (c.len + c.rows.n) / kBlockTokens - (c.len + kBlockTokens - 1) / kBlockTokens);
}
__device__ __forceinline__ int touched_blocks(const Chunk& c) {
  return c.bad ? 0 : c.rows.n == 0 ? 1 : (c.len + c.rows.n - 1) / kBlockTokens - c.len / kBlockTokens + 1;
}
enum Part { kWhole, kEdges, kEvery };
template <Part PART>
__device__ __forceinline__ int part_blocks(const Chunk& c) {
  return PART == kWhole ? whole_blocks(c) : PART == kEdges ? touched_blocks(c) - whole_blocks(c) : touched_blocks(c);
}

// The i-th block of a sequence that the kernel takes, counted from the
// sequence's first touched one.
template <Part PART>
__device__ __forceinline__ int block_of(const Chunk& c, int i) {
  const int lead = c.len % kBlockTokens != 0 ? 1 : 0;  // an edge before the whole ones?
  return PART == kWhole ? lead + i : PART == kEdges && i >= lead ? i + whole_blocks(c) : i;
}

// The sequence and block of a CTA, by one warp: found[0] = sequence (-1:
// none), found[1] = block.  With SKIP blocks of every sequence left out, the
// rank-th of the rest.
template <Part PART, int SKIP>
__device__ __forceinline__ void find_block(const AppendParams& p, int rank, int* found) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) found[0] = -1;
  __syncwarp();
  constexpr int kAt = 4;  // sequences of a lane at a time: their loads overlap
  for (int b0 = 0; b0 < p.batch && rank >= 0; b0 += 32 * kAt) {
    Chunk c[kAt];
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      const int b = b0 + 32 * k + lane;
      c[k] = Chunk{{0, 0, false}, 0, true};
      if (b < p.batch) c[k] = load_chunk(p, b);
    }
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      if (b0 + 32 * k >= p.batch) break;
      const int blocks = max(0, part_blocks<PART>(c[k]) - SKIP);
      int incl = blocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int i = rank - (incl - blocks);
      if (i >= 0 && i < blocks) {
        found[0] = b0 + 32 * k + lane;
        found[1] = block_of<PART>(c[k], i + SKIP);
      }
      rank -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

// Channel-wise groups of a tile, by the whole block: the warps' ranges in
// `ranges` ([low, high][warp][channel]) become scales and offsets ([s,
// z][token group][channel]); their 16-bit forms go to s_out, z_out.
template <int BITS, int W, int NW>
__device__ __forceinline__ void channel_groups(float (*ranges)[NW][W], int groups, int gw, uint16_t* s_out,
                                               uint16_t* z_out, uint32_t* dev_status) {
  constexpr int kThreads = 32 * NW, kEach = 512 / kThreads;  // groups * W <= 512
  const int tid = threadIdx.x;
  Group mine[kEach];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = tid + k * kThreads;
    if (e < groups * W) {
      const int g = e / W, c = e % W;
      float a = INFINITY, z = -INFINITY;
      for (int w = g * gw; w < (g + 1) * gw; ++w) {
        a = min_nan(a, ranges[0][w][c]);
        z = max_nan(z, ranges[1][w][c]);
      }
      mine[k] = group_of_range(a, z, (float)((1 << BITS) - 1));
      if (isnan(mine[k].s)) report(dev_status, KVQ_DEV_NONFINITE);
      s_out[e] = mine[k].s_bits;
      z_out[e] = mine[k].z_bits;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = tid + k * kThreads;
    if (e < groups * W) {
      ranges[0][e / W][e % W] = mine[k].s;
      ranges[1][e / W][e % W] = mine[k].z;
    }
  }
  __syncthreads();
}

template <typename T, int BITS, int W, Part PART>  // W: channels of the slab
__device__ __forceinline__ void append_edge(const AppendParams& p) {
  constexpr int kWarps = kEdgeWarps, kThreads = 32 * kWarps, kWarpTok = kBlockTokens / kWarps;  // tokens of a warp
  constexpr int kLanes = W / 4;                 // lanes that share a token
  constexpr int kTok = kWarpTok * kLanes / 32;  // tokens of a thread (8 or 4)
  constexpr int kPer = 128 / BITS;              // codes of a 16-byte piece
  constexpr int kPieces = W * BITS;             // 16-byte pieces of the slab's block: 128 W BITS / 128
  constexpr float kMax = (float)((1 << BITS) - 1);
  // packed block: K [chunk][128 tokens], V [chunk][W channels], a piece of padding per chunk against bank conflicts
  __shared__ __align__(16) unsigned char packed[(kPieces + W * BITS / 64 + 8) * 16];
  // channel-wise: ranges per warp, then s / z (as [group][W]); token-wise: s, z of every (token, group)
  __shared__ __align__(16) float ranges[2][kWarps][W];
  float(*lo_s)[W] = ranges[0], (*hi_s)[W] = ranges[1];
  __shared__ __align__(16) uint16_t s_out[128 * 4], z_out[128 * 4];
  __shared__ int found[2];
  const int D = p.head_dim;
  const int h = blockIdx.y, which = blockIdx.z & 1, slab = blockIdx.z >> 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = h == 0 && blockIdx.z == 0;
  // the first `batch` CTAs take the first block of a sequence each (every thread
  // looks for itself), the others what more there is
  int b = blockIdx.x, nth = 0;
  if (blockIdx.x >= p.batch) {
    if (warp == 0) find_block<PART, 1>(p, blockIdx.x - p.batch, found);
    __syncthreads();
    b = found[0];
    nth = found[1];
    if (b < 0) return;
  }
  const Chunk chunk = load_chunk(p, b);
  if (blockIdx.x < p.batch) {
    if (chunk.bad && lead && tid == 0) report(p.dev_status, KVQ_DEV_BAD_SEQ_LEN);
    if (part_blocks<PART>(chunk) <= 0) return;
    nth = block_of<PART>(chunk, 0);
  }
  const SeqRows s = chunk.rows;
  const int len = chunk.len, end = len + s.n;
  const int j = len / kBlockTokens + nth, t0 = j * kBlockTokens;
  const int nv = min(kBlockTokens, end - t0);  // rows of this block
  const int from = min(max(len - t0, 0), nv);  // ... that were there before
  // (asked for now, needed at the end; an empty chunk may be at the end of its table)
  const int page = s.n == 0 ? -1 : p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
  const bool tokenwise = p.scheme[which] == KVQ_TOKENWISE;
  const size_t win_at = ((size_t)b * p.num_kv_heads + h) * kBlockTokens * D + slab * W;
  const float* win = p.window[which] ? p.window[which] + win_at : nullptr;
  const int sub = lane / kLanes, ch = (lane % kLanes) * 4;  // this thread's channels ch ... ch + 3
  const int tok = warp * kWarpTok + sub * kTok;                   // ... and tokens tok ... tok + kTok - 1
  const Rows& rows = p.x[which];
  const long long at0 = (long long)h * rows.sh + slab * W + ch;

  // ---- the rows, in fp32
  float x[kTok][4];
  {
    Raw<T> raw[kTok];
    if (from == 0 && nv == kBlockTokens) {  // a whole block of new tokens, as most are
#pragma unroll
      for (int i = 0; i < kTok; ++i)
        raw[i].load(rows.data, (long long)(s.first + t0 + tok + i - len) * rows.st + at0);
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const float4 v = raw[i].get();
        x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
      }
    } else {
      // all loads before the first use.  Earlier tokens: for a group along the
      // tokens, or to be copied to another window.
      const bool old = win != nullptr && (!tokenwise || p.window_out[which] != p.window[which]);
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int t = tok + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (old && t < from) v = *reinterpret_cast<const float4*>(win + (size_t)t * D + ch);
        x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int t = tok + i;
        if (t >= from && t < nv) raw[i].load(rows.data, (long long)(s.first + t0 + t - len) * rows.st + at0);
      }
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int t = tok + i;
        if (t >= from && t < nv) {
          const float4 v = raw[i].get();
          x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
        }
      }
    }
  }

  // ---- the window of the new partial last block.  The sequence's first block
  //      reads the window's rows (above) where it was begun before, and then is
  //      the one that writes the new ones; else its last block does.
  const int last = end / kBlockTokens * kBlockTokens;  // the partial block's first position
  if (win != nullptr && end > last) {
    float* wout = p.window_out[which] + win_at;
    if (last == t0 && (nth == 0 || len % kBlockTokens == 0)) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        const int t = tok + i;
        if (t < nv && (t >= from || wout != win)) {
          *reinterpret_cast<float4*>(wout + (size_t)t * D + ch) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        }
      }
    } else if (nth == 0 && len % kBlockTokens != 0) {
      if (!tokenwise) __syncthreads();  // every thread has its rows of the old window
      for (int e = tid; e < (end - last) * kLanes; e += kThreads) {
        const int t = e / kLanes, c = (e % kLanes) * 4;
        Raw<T> raw;
        raw.load(rows.data, (long long)(s.first + last + t - len) * rows.st + (long long)h * rows.sh + slab * W + c);
        *reinterpret_cast<float4*>(wout + (size_t)t * D + c) = raw.get();
      }
    }
  }
  if (s.n == 0) return;
  if (page < 0 || page >= p.num_pages) {
    if (lead && tid == 0) report(p.dev_status, KVQ_DEV_BAD_PAGE);
    return;
  }
  const int G = p.group, gps = W / G;  // channel groups of a token in this slab (token-wise)
  const int nsz = kBlockTokens * D / G;
  const size_t blk = (size_t)page * p.num_kv_heads + h;

  // Where codes go.  K, one token: the thread's 4 codes are 16 (8) bits of the
  // token's row; kMagicBits is zero there, so the codes are summed in place.
  auto put_k = [&](int t, const uint32_t (&y)[4]) {
    const uint32_t w = y[0] + (y[1] << BITS) + (y[2] << 2 * BITS) + (y[3] << 3 * BITS);
    unsigned char* at = packed + ((ch / kPer) * 129 + t) * 16 + (ch % kPer) * BITS / 8;
    if (BITS == 4) *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
    else *at = (unsigned char)w;
  };
  // V, one channel: kTok codes along the row, up to 32 bits to a word.
  constexpr int kWordTok = 32 / BITS < kTok ? 32 / BITS : kTok, kWords = kTok / kWordTok;
  constexpr uint32_t kWordMagic = [] {
    uint32_t m = 0;
    for (int i = 0; i < kWordTok; ++i) m += kMagicBits << (i * BITS);
    return m;
  }();
  auto put_v = [&](const uint32_t (&acc)[kWords][4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      unsigned char* at = packed + ((tok / kPer) * (W + 1) + ch + c) * 16 + (tok % kPer) * BITS / 8;
      if (kWords == 2) *reinterpret_cast<uint2*>(at) = make_uint2(acc[0][c] - kWordMagic, acc[kWords - 1][c] - kWordMagic);
      else if (kTok * BITS == 32) *reinterpret_cast<uint32_t*>(at) = acc[0][c] - kWordMagic;
      else if (kTok * BITS == 16) *reinterpret_cast<uint16_t*>(at) = (uint16_t)acc[0][c];  // (kMagicBits is zero there)
      else *at = (unsigned char)acc[0][c];
    }
  };
  const bool past = warp * kWarpTok >= nv;  // none of this warp's tokens is there: codes 0
  auto put_none = [&] {
    if (which == 0) {
      const uint32_t none[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < kTok; ++i) put_k(tok + i, none);
    } else {
      uint32_t none[kWords][4];
#pragma unroll
      for (int i = 0; i < kWords * 4; ++i) none[i / 4][i % 4] = kWordMagic;
      put_v(none);
    }
  };
  if (tokenwise && (warp + 1) * kWarpTok <= from) {
    // tokens that stay, all of this warp's: nothing of theirs is written
  } else if (tokenwise && past) {
    for (int e = warp * kWarpTok * gps + lane; e < (warp + 1) * kWarpTok * gps; e += 32) s_out[e] = z_out[e] = 0;
    put_none();
  } else if (tokenwise) {
    // ranges of the thread's tokens over its 4 channels, then over the group's lanes
    const int lg = G / 4, gl = lane & (lg - 1);  // lanes of a group, place in it
    float mn[kTok], mx[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      mn[i] = min_nan(min_nan(x[i][0], x[i][1]), min_nan(x[i][2], x[i][3]));
      mx[i] = max_nan(max_nan(x[i][0], x[i][1]), max_nan(x[i][2], x[i][3]));
    }
    reduce_group<kTok, false>(mn, lg);
    reduce_group<kTok, true>(mx, lg);
    float4* sz = reinterpret_cast<float4*>(ranges);  // [token][group] s, z, 1 / s: at most 128 x W / 32 of them
    static_assert(sizeof(ranges) >= 128 * (W / 32) * sizeof(float4), "table");
    const int each = kTok / lg > 1 ? kTok / lg : 1, share = lg / kTok > 1 ? lg / kTok : 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k < each && gl % share == 0) {
        const int t = tok + (each > 1 ? gl * each + k : gl / share);
        const bool live = t >= from && t < nv;
        const Group g = live ? group_of_range(mn[k], mx[k], kMax) : Group{0.f, 0.f, 0, 0};
        if (isnan(g.s)) report(p.dev_status, KVQ_DEV_NONFINITE);
        const int e = t * gps + ch / G;
        sz[e] = make_float4(g.s, g.z, reciprocal(g.s), 0.f);
        s_out[e] = g.s_bits;
        z_out[e] = g.z_bits;
      }
    }
    __syncwarp();  // a group's lanes are one warp's
    uint32_t acc[kWords][4] = {};
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      float4 g = sz[(tok + i) * gps + ch / G];
      if (isnan(g.x)) {
        g.x = 0.f;
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
      }
      uint32_t y[4];
      const uint64_t sn = rows::pair(-g.x, -g.x), zn = rows::pair(-g.y, -g.y), r = rows::pair(g.z, g.z);
      code_pair(x[i][0], x[i][1], sn, zn, r, y[0], y[1]);
      code_pair(x[i][2], x[i][3], sn, zn, r, y[2], y[3]);
      if (which == 0) {
        put_k(tok + i, y);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i / kWordTok][c] += y[c] << (i % kWordTok * BITS);
      }
    }
    if (which == 1) put_v(acc);
  } else {
    // ranges of the thread's tokens per channel, then across the warps (and
    // half-warps) of the group's tokens
    float mn[4], mx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mn[c] = INFINITY;
      mx[c] = -INFINITY;
    }
    if (tok + kTok <= nv) {
#pragma unroll
      for (int i = 0; i < kTok; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mn[c] = min_nan(mn[c], x[i][c]);
          mx[c] = max_nan(mx[c], x[i][c]);
        }
    } else if (!past) {
#pragma unroll
      for (int i = 0; i < kTok; ++i)
        if (tok + i < nv) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mn[c] = min_nan(mn[c], x[i][c]);
            mx[c] = max_nan(mx[c], x[i][c]);
          }
        }
    }
    if (kLanes < 32) {  // both halves of the warp hold the same channels
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mn[c] = min_nan(mn[c], __shfl_xor_sync(0xffffffffu, mn[c], 16));
        mx[c] = max_nan(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 16));
      }
    }
    *reinterpret_cast<float4*>(&lo_s[warp][ch]) = make_float4(mn[0], mn[1], mn[2], mn[3]);
    *reinterpret_cast<float4*>(&hi_s[warp][ch]) = make_float4(mx[0], mx[1], mx[2], mx[3]);
    const int gw = G / kWarpTok, groups = kBlockTokens / G;  // warps of a token group, token groups
    channel_groups<BITS, W, kWarps>(ranges, groups, gw, s_out, z_out, p.dev_status);
    if (past) {
      put_none();
    } else {
      const int g = warp * kWarpTok / G;
      const float4 s4 = *reinterpret_cast<const float4*>(&lo_s[g][ch]);
      const float4 z4 = *reinterpret_cast<const float4*>(&hi_s[g][ch]);
      float sc[4] = {s4.x, s4.y, s4.z, s4.w}, rc[4];
      const float zc[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (isnan(sc[c])) {
          sc[c] = 0.f;
#pragma unroll
          for (int i = 0; i < kTok; ++i) x[i][c] = 0.f;
        }
        rc[c] = reciprocal(sc[c]);
      }
      uint64_t sn[2], zn[2], r2[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sn[c] = rows::pair(-sc[2 * c], -sc[2 * c + 1]);
        zn[c] = rows::pair(-zc[2 * c], -zc[2 * c + 1]);
        r2[c] = rows::pair(rc[2 * c], rc[2 * c + 1]);
      }
      if (nv < kBlockTokens) {  // tokens past the end have code 0
#pragma unroll
        for (int i = 0; i < kTok; ++i)
          if (tok + i >= nv) {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[i][c] = zc[c];
          }
      }
      uint32_t acc[kWords][4] = {};
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        uint32_t y[4];
#pragma unroll
        for (int c = 0; c < 4; c += 2) code_pair(x[i][c], x[i][c + 1], sn[c / 2], zn[c / 2], r2[c / 2], y[c], y[c + 1]);
        if (which == 0) {
          put_k(tok + i, y);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i / kWordTok][c] += y[c] << (i % kWordTok * BITS);
        }
      }
      if (which == 1) put_v(acc);
    }
  }
  __syncthreads();

  // ---- out: the slab's pieces of the block (K: chunks of every token, V: rows of every chunk)
  const int keep = tokenwise ? from : 0;  // earlier tokens keep their codes, s and z
  uint8_t* dst = p.codes[which] + blk * (size_t)(kBlockTokens * D * BITS / 8);
  if (which == 0) {
    for (int e = tid; e < kPieces; e += kThreads) {
      const int chunk = e >> 7, t = e & 127;
      if (t >= keep)
        *reinterpret_cast<uint4*>(dst + ((size_t)(slab * (W / kPer) + chunk) * kBlockTokens + t) * 16) =
            *reinterpret_cast<const uint4*>(packed + (chunk * 129 + t) * 16);
    }
  } else {
    for (int e = tid; e < kPieces; e += kThreads) {
      const int chunk = e / W, r = e % W, t = chunk * kPer;
      if (t + kPer <= keep) continue;
      uint4 v = *reinterpret_cast<const uint4*>(packed + (chunk * (W + 1) + r) * 16);
      uint4* at = reinterpret_cast<uint4*>(dst + ((size_t)chunk * D + slab * W + r) * 16);
      if (t < keep) {
        const uint4 was = *at;
        const uint32_t old[4] = {was.x, was.y, was.z, was.w};
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = min(max((keep - t) * BITS - 32 * k, 0), 32);  // bits to keep
          const uint32_t mask = n == 32 ? 0xffffffffu : (1u << n) - 1u;
          w[k] = (w[k] & ~mask) | (old[k] & mask);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *at = v;
    }
  }
  uint16_t* so = p.scale[which] + blk * nsz;
  uint16_t* zo = p.zero[which] + blk * nsz;
  if (tokenwise) {  // entry token * (D / G) + group
    for (int e = tid + keep * gps; e < kBlockTokens * gps; e += kThreads) {
      const int t = e / gps, at = t * (D / G) + slab * gps + e - t * gps;
      so[at] = s_out[e];
      zo[at] = z_out[e];
    }
  } else {  // entry token group * D + channel
    for (int e = tid; e < kBlockTokens / G * W; e += kThreads) {
      const int at = e / W * D + slab * W + e % W;
      so[at] = s_out[e];
      zo[at] = z_out[e];
    }
  }
}

template <typename T, int BITS, int W, Part PART>
__global__ void __launch_bounds__(32 * kEdgeWarps, sizeof(Raw<T>) == 8 ? 2 : 1) append_edges_kernel(const AppendParams p) {
  append_edge<T, BITS, W, PART>(p);
  // overlaps append_blocks_kernel: what follows in the stream waits for
  // this grid, which is not done before that one is
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------- whole blocks

// 16-bit pairs: the smaller (larger) of each half, NaN if either is.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (sizeof(T) == sizeof(__half)) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (sizeof(T) == sizeof(__half)) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ float2 wide(uint32_t v) {
  if (sizeof(T) == sizeof(__half)) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// reduce_group's exchange for 16-bit pairs, the smaller of each half kept.
template <typename T, int N>
__device__ __forceinline__ void reduce_group2(uint32_t (&v)[N], int lg) {
  int o = lg >> 1;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    if (o > 0) {
      const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const uint32_t keep = upper ? v[i + n / 2] : v[i];
        v[i] = min2<T>(keep, __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + n / 2], o));
      }
      o >>= 1;
    }
  }
  for (; o > 0; o >>= 1) v[0] = min2<T>(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
}

// (four CTAs to an SM: 64 registers, two of them spilled at 4 bits, and still
// 8% faster than three with 80, as their loads and barriers overlap better)
template <typename T, int BITS, int W>
__global__ void __launch_bounds__(32 * kBlockWarps, 4) append_blocks_kernel(const AppendParams p) {
  constexpr int kWarps = kBlockWarps, kThreads = 32 * kWarps, kWarpTok = kBlockTokens / kWarps;  // tokens of a warp
  constexpr int kLanes = W / 4, kTok = kWarpTok * kLanes / 32, kPer = 128 / BITS;
  constexpr int kPieces = W * BITS;
  constexpr float kMax = (float)((1 << BITS) - 1);
  // packed block: K [chunk][128 tokens], a piece of padding per chunk; V
  // [chunk][channel mod 4][channel / 4], two pieces of padding per plane: lanes,
  // which have every fourth channel, then meet no bank twice, nor do the
  // pieces as they are read
  constexpr int kPlane = W / 4 + 2;
  __shared__ __align__(16) unsigned char packed[BITS * 4 * kPlane * 16];
  static_assert(BITS * 4 * kPlane >= kPieces + W / kPer, "K's padding fits too");
  __shared__ __align__(16) float ranges[2][kWarps][W];
  __shared__ __align__(16) uint16_t s_out[128 * 4], z_out[128 * 4];
  __shared__ int found[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the edges' kernel runs beside this one
  const int D = p.head_dim;
  const int h = blockIdx.y, which = blockIdx.z & 1, slab = blockIdx.z >> 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) find_block<kWhole, 0>(p, blockIdx.x, found);
  __syncthreads();
  const int b = found[0];
  if (b < 0) return;
  const int len = p.seq_lens[b], j = len / kBlockTokens + found[1];
  const int page = p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
  const int ch = (lane % kLanes) * 4, tok = warp * kWarpTok + (lane / kLanes) * kTok;
  uint2 x[kTok];
  {
    const long long row = (long long)p.cu[b] + j * kBlockTokens - len + tok;
    const uint16_t* src = static_cast<const uint16_t*>(p.x[which].data) + row * p.x[which].st +
                          (long long)h * p.x[which].sh + slab * W + ch;
    const long long st = p.x[which].st;
#pragma unroll
    for (int i = 0; i < kTok; ++i, src += st) x[i] = __ldcs(reinterpret_cast<const uint2*>(src));
  }
  if (page < 0 || page >= p.num_pages) {
    if (h == 0 && blockIdx.z == 0 && tid == 0) report(p.dev_status, KVQ_DEV_BAD_PAGE);
    return;
  }
  const int G = p.group, gps = W / G, nsz = kBlockTokens * D / G;
  const size_t blk = (size_t)page * p.num_kv_heads + h;
  const bool tokenwise = p.scheme[which] == KVQ_TOKENWISE;

  unsigned char* k_at = packed + ((ch / kPer) * 129 + tok) * 16 + (ch % kPer) * BITS / 8;
  auto put_k = [&](int i, const uint32_t (&y)[4]) {
    const uint32_t w = y[0] + (y[1] << BITS) + (y[2] << 2 * BITS) + (y[3] << 3 * BITS);
    if (BITS == 4) *reinterpret_cast<uint16_t*>(k_at + i * 16) = (uint16_t)w;
    else k_at[i * 16] = (unsigned char)w;
  };
  constexpr int kWordTok = 32 / BITS < kTok ? 32 / BITS : kTok, kWords = kTok / kWordTok;
  constexpr uint32_t kWordMagic = [] {
    uint32_t m = 0;
    for (int i = 0; i < kWordTok; ++i) m += kMagicBits << (i * BITS);
    return m;
  }();
  auto put_v = [&](const uint32_t (&acc)[kWords][4]) {
    unsigned char* at = packed + ((tok / kPer) * 4 * kPlane + ch / 4) * 16 + (tok % kPer) * BITS / 8;
#pragma unroll
    for (int c = 0; c < 4; ++c, at += kPlane * 16) {
      if (kWords == 2) *reinterpret_cast<uint2*>(at) = make_uint2(acc[0][c] - kWordMagic, acc[kWords - 1][c] - kWordMagic);
      else if (kTok * BITS == 32) *reinterpret_cast<uint32_t*>(at) = acc[0][c] - kWordMagic;
      else *reinterpret_cast<uint16_t*>(at) = (uint16_t)acc[0][c];  // (kMagicBits is zero there)
    }
  };
  uint32_t acc[kWords][4] = {};
  // the codes of token i of this thread; values of a refused group (s NaN) are taken as z = 0
  auto emit = [&](int i, const uint64_t (&sn)[2], const uint64_t (&zn)[2], const uint64_t (&r)[2]) {
    uint32_t y[4];
    const float2 a = wide<T>(x[i].x), c = wide<T>(x[i].y);
    code_pair(a.x, a.y, sn[0], zn[0], r[0], y[0], y[1]);
    code_pair(c.x, c.y, sn[1], zn[1], r[1], y[2], y[3]);
    if (which == 0) {
      put_k(i, y);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i / kWordTok][k] += y[k] << (i % kWordTok * BITS);
    }
  };

  if (tokenwise) {
    const int lg = G / 4, gl = lane & (lg - 1);
    uint32_t v[kTok];  // the token's smallest value over this thread's channels, and its largest negated
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const uint32_t lo = min2<T>(x[i].x, x[i].y), hi = max2<T>(x[i].x, x[i].y) ^ 0x80008000u;
      v[i] = min2<T>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    }
    reduce_group2<T, kTok>(v, lg);
    float4* sz = reinterpret_cast<float4*>(ranges);  // [token][group] -s, -z, 1 / s
    static_assert(sizeof(ranges) >= 128 * (W / 32) * sizeof(float4), "table");
    const int each = kTok / lg > 1 ? kTok / lg : 1, share = lg / kTok > 1 ? lg / kTok : 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k < each && gl % share == 0) {
        const float2 range = wide<T>(v[k]);
        const Group g = group_of_range(range.x, -range.y, kMax);
        const int e = (tok + (each > 1 ? gl * each + k : gl / share)) * gps + ch / G;
        if (isnan(g.s)) report(p.dev_status, KVQ_DEV_NONFINITE);
        sz[e] = make_float4(-g.s, -g.z, reciprocal(g.s), 0.f);
        s_out[e] = g.s_bits;
        z_out[e] = g.z_bits;
      }
    }
    __syncwarp();  // a group's lanes are one warp's
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      float4 g = sz[(tok + i) * gps + ch / G];
      if (isnan(g.x)) {
        g.x = 0.f;
        x[i] = make_uint2(0u, 0u);
      }
      const uint64_t sn = rows::pair(g.x, g.x), zn = rows::pair(g.y, g.y), r = rows::pair(g.z, g.z);
      emit(i, {sn, sn}, {zn, zn}, {r, r});
    }
  } else {
    uint2 lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < kTok; ++i) {
      lo = make_uint2(min2<T>(lo.x, x[i].x), min2<T>(lo.y, x[i].y));
      hi = make_uint2(max2<T>(hi.x, x[i].x), max2<T>(hi.y, x[i].y));
    }
    if (kLanes < 32) {  // both halves of the warp hold the same channels
      lo = make_uint2(min2<T>(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, 16)),
                      min2<T>(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, 16)));
      hi = make_uint2(max2<T>(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, 16)),
                      max2<T>(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, 16)));
    }
    float2 a = wide<T>(lo.x), c = wide<T>(lo.y);
    *reinterpret_cast<float4*>(&ranges[0][warp][ch]) = make_float4(a.x, a.y, c.x, c.y);
    a = wide<T>(hi.x);
    c = wide<T>(hi.y);
    *reinterpret_cast<float4*>(&ranges[1][warp][ch]) = make_float4(a.x, a.y, c.x, c.y);
    channel_groups<BITS, W, kWarps>(ranges, kBlockTokens / G, G / kWarpTok, s_out, z_out, p.dev_status);
    const int g = warp * kWarpTok / G;
    const float4 s4 = *reinterpret_cast<const float4*>(&ranges[0][g][ch]);
    const float4 z4 = *reinterpret_cast<const float4*>(&ranges[1][g][ch]);
    float sc[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
    float rc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (isnan(sc[k])) {
        sc[k] = 0.f;
        keep[k / 2] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
      }
      rc[k] = reciprocal(sc[k]);
    }
    if ((keep[0] & keep[1]) != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) x[i] = make_uint2(x[i].x & keep[0], x[i].y & keep[1]);
    }
    const uint64_t sn[2] = {rows::pair(-sc[0], -sc[1]), rows::pair(-sc[2], -sc[3])};
    const uint64_t zn[2] = {rows::pair(-z4.x, -z4.y), rows::pair(-z4.z, -z4.w)};
    const uint64_t r[2] = {rows::pair(rc[0], rc[1]), rows::pair(rc[2], rc[3])};
#pragma unroll
    for (int i = 0; i < kTok; ++i) emit(i, sn, zn, r);
  }
  if (which == 1) put_v(acc);
  __syncthreads();

  uint8_t* dst = p.codes[which] + blk * (size_t)(kBlockTokens * D * BITS / 8);
  if (which == 0) {
    dst += (size_t)slab * (W / kPer) * kBlockTokens * 16;
#pragma unroll
    for (int e = tid; e < kPieces; e += kThreads)
      *reinterpret_cast<uint4*>(dst + e * 16) = *reinterpret_cast<const uint4*>(packed + (e + (e >> 7)) * 16);
  } else {
#pragma unroll
    for (int e = tid; e < kPieces; e += kThreads) {
      const int chunk = e / W, r = e % W;
      *reinterpret_cast<uint4*>(dst + ((size_t)chunk * D + slab * W + r) * 16) =
          *reinterpret_cast<const uint4*>(packed + (chunk * 4 * kPlane + (r & 3) * kPlane + (r >> 2)) * 16);
    }
  }
  uint16_t* so = p.scale[which] + blk * nsz;
  uint16_t* zo = p.zero[which] + blk * nsz;
  const int wide_gps = tokenwise ? gps : W, pitch = tokenwise ? D / G : D;  // entries of a row here, and in the cache
  const int entries = kBlockTokens * W / G, shift = 31 - __clz(wide_gps);
  for (int e = tid; e < entries; e += kThreads) {
    const int at = (e >> shift) * pitch + slab * wide_gps + (e & (wide_gps - 1));
    so[at] = s_out[e];
    zo[at] = z_out[e];
  }
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
  // one edge per sequence, two where a chunk of two tokens or more can cross
  // into the next block; every block: one more for each 128 tokens past that
  const long long two = p.batch < p.total / 2 ? p.batch : p.total / 2;
  const long long blocks = p.batch + two + (kHalf ? 0 : (p.total - 2 * two) / kBlockTokens);
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
