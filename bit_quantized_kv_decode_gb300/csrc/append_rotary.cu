// Append with the position rotation on the way, and rows turned on their own.
//
// The first R channels of a row at position p are pairs (x1, x2) -- channel i
// with i + R / 2, or neighbours -- that become
//   (fl(fl(x1 c) - fl(x2 s)), fl(fl(x2 c) + fl(x1 s))),  c, s = cos, sin of the pair's angle at p,
// in fp32, on pairs of values: product, product times sign plus product, where the
// sign is a number that the compiler does not know (Turn::one), so that it does
// not make an addition and then one fused operation of it.  K goes into the cache
// from there, without a rounding to the rows'
// type between; turned queries (and keys, where attention over rows follows)
// are rounded to it once.
#include <cuda_bf16.h>

#include "append_core.cuh"

namespace kvq {
namespace {

// The kernels of a call write disjoint places and read what none of them writes;
// each may start once the last CTA of the one before has, and ends no earlier
// than that one, so that what follows in the stream follows all of them.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void end_after_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// V's blocks of new 16-bit tokens alone.
template <typename T, int BITS, int W>
__global__ void __launch_bounds__(32 * kBlockWarps, kBlockCtas) rotary_v_kernel(const AppendParams p) {
  let_next_start();
  append_block<T, BITS, W>(p, 1, blockIdx.z);
  end_after_last();
}

// K's: CTAs of 16 warps, two to an SM, that take a block through `each` columns
// of 128 channels (a head; two heads of 64; half a head of 256) with the block's
// angles in shared memory.  A thread has 4 channels of 8 tokens.  A value's partner
// is another lane's, but for heads of 256 (CROSS), where it may be of the other
// column and is loaded, as are the angles, which would not fit twice.
constexpr int kColumn = 128;

template <typename T, int BITS, bool CROSS>
__global__ void __launch_bounds__(32 * kEdgeWarps, 2) rotary_k_kernel(const AppendParams p, int each) {
  constexpr int kWarps = kEdgeWarps, kThreads = 32 * kWarps, kTok = kBlockTokens / kWarps;
  constexpr int kPer = 128 / BITS, kPieces = kColumn * BITS;  // codes of a 16-byte piece, pieces of a column
  constexpr float kMax = (float)((1 << BITS) - 1);
  __shared__ __align__(16) unsigned char packed[kColumn / kPer * 129 * 16];  // [chunk][128 tokens], a piece of padding
  __shared__ __align__(16) float ranges[2][kWarps][kColumn];  // channel-wise: ranges, then s and z; token-wise: of every group
  __shared__ __align__(16) uint16_t s_out[128 * 4], z_out[128 * 4];
  __shared__ int found[2];
  let_next_start();
  const int D = p.head_dim, H = p.num_kv_heads, G = p.group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tok = warp * kTok, ch = lane * 4;
  if (warp == 0) find_block<kWhole, 0>(p, blockIdx.x, found);
  __syncthreads();
  const int b = found[0];
  const int len = b < 0 ? 0 : p.seq_lens[b], j = len / kBlockTokens + (b < 0 ? 0 : found[1]);
  const int page = b < 0 ? 0 : p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
  const bool good = page >= 0 && page < p.num_pages;
  if (!good && blockIdx.y == 0 && tid == 0) report(p.dev_status, KVQ_DEV_BAD_PAGE);
  const int columns = (H * D + kColumn - 1) / kColumn, q0 = blockIdx.y * each;
  const int q1 = b < 0 || !good ? q0 : min(columns, q0 + each);
  // head and channel of column q's channel c
  auto head_of = [&](int q, int c) { return D == 64 ? 2 * q + (c >> 6) : D == 256 ? q >> 1 : q; };
  auto channel_of = [&](int q, int c) { return D == 64 ? c & 63 : D == 256 ? (q & 1) * kColumn + c : c; };
  const int half = p.turn.dim >> 1, nsz = kBlockTokens * D / G;
  const bool near = p.turn.interleaved != 0, tokenwise = p.scheme[0] == KVQ_TOKENWISE;
  const long long row0 = b < 0 ? 0 : ((long long)p.cu[b] + j * kBlockTokens - len + tok) * p.x[0].st;
  const float* angles = p.turn.angles + (size_t)(j * kBlockTokens) * p.turn.dim;  // of the block's tokens
  unsigned char* k_at = packed + ((ch / kPer) * 129 + tok) * 16 + (ch % kPer) * BITS / 8;

  Raw<T> raw[kTok];
  auto load = [&](int q) {
    const int h = min(head_of(q, ch), H - 1);  // (of a last, single head of 64: once more, and not kept)
    long long at = row0 + (long long)h * p.x[0].sh + channel_of(q, ch);
#pragma unroll
    for (int i = 0; i < kTok; ++i, at += p.x[0].st) raw[i].load(p.x[0].data, at);
  };
  extern __shared__ __align__(16) float near_angles[];  // not CROSS: the same, in shared memory
  if (!CROSS && q0 < q1) {
    for (int e = tid; e < kBlockTokens / 4 * p.turn.dim; e += kThreads) copy16(near_angles + 4 * e, angles + 4 * e);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
  }
  const float* my_angles = (CROSS ? angles : near_angles) + tok * p.turn.dim;
  auto angle4 = [](const float* at) { return CROSS ? __ldg(reinterpret_cast<const float4*>(at)) : *reinterpret_cast<const float4*>(at); };
  auto angle2 = [](const float* at) { return CROSS ? __ldg(reinterpret_cast<const float2*>(at)) : *reinterpret_cast<const float2*>(at); };
  for (int q = q0; q < q1; ++q) {
    load(q);
    if (q + 1 < q1 && tid < 2 * kBlockTokens) {  // (the next column's rows are on their way to L2 meanwhile: two lines a row)
      const int c = (tid & 1) * 64, h = min(head_of(q + 1, c), H - 1);
      const long long at = row0 + (long long)((tid >> 1) - tok) * p.x[0].st + (long long)h * p.x[0].sh + channel_of(q + 1, c);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint16_t*>(p.x[0].data) + at));
    }
    const int hc = channel_of(q, ch);
    float x[kTok][4];
    // ---- turned, in fp32
    const bool on = hc < p.turn.dim, upper = hc >= half;
    if (near) {
      const float* at = my_angles + (on ? hc >> 1 : 0);
#pragma unroll
      for (int i = 0; i < kTok; ++i, at += p.turn.dim) {
        const float4 v = raw[i].get();
        const float2 c = angle2(at), s = angle2(at + half);
        const uint64_t sign = rows::pair(-p.turn.one, p.turn.one);
        float4 y;
        rows::unpair(rows::fma2(rows::mul2(rows::pair(v.y, v.x), rows::pair(s.x, s.x)), sign,
                                rows::mul2(rows::pair(v.x, v.y), rows::pair(c.x, c.x))), y.x, y.y);
        rows::unpair(rows::fma2(rows::mul2(rows::pair(v.w, v.z), rows::pair(s.y, s.y)), sign,
                                rows::mul2(rows::pair(v.z, v.w), rows::pair(c.y, c.y))), y.z, y.w);
        x[i][0] = on ? y.x : v.x; x[i][1] = on ? y.y : v.y; x[i][2] = on ? y.z : v.z; x[i][3] = on ? y.w : v.w;
      }
    } else {
      const float* at = my_angles + (on ? upper ? hc - half : hc : 0);
      const int away = on ? upper ? -half : half : 0;  // the partner, in channels
      const float one = upper ? p.turn.one : -p.turn.one;
      const uint64_t sign = rows::pair(one, one);
      long long other = row0 + (long long)min(head_of(q, ch), H - 1) * p.x[0].sh + hc + away;
#pragma unroll
      for (int i = 0; i < kTok; ++i, at += p.turn.dim, other += p.x[0].st) {
        const float4 c = angle4(at), s = angle4(at + half);
        Raw<T> partner;
        if (CROSS) {
          partner.load(p.x[0].data, other);
        } else {
          partner.v.x = __shfl_sync(0xffffffffu, raw[i].v.x, lane + away / 4);
          partner.v.y = __shfl_sync(0xffffffffu, raw[i].v.y, lane + away / 4);
        }
        const float4 v = raw[i].get(), w = partner.get();
        float4 y;
        rows::unpair(rows::fma2(rows::mul2(rows::pair(w.x, w.y), rows::pair(s.x, s.y)), sign,
                                rows::mul2(rows::pair(v.x, v.y), rows::pair(c.x, c.y))), y.x, y.y);
        rows::unpair(rows::fma2(rows::mul2(rows::pair(w.z, w.w), rows::pair(s.z, s.w)), sign,
                                rows::mul2(rows::pair(v.z, v.w), rows::pair(c.z, c.w))), y.z, y.w);
        x[i][0] = on ? y.x : v.x; x[i][1] = on ? y.y : v.y; x[i][2] = on ? y.z : v.z; x[i][3] = on ? y.w : v.w;
      }
    }
    // ---- groups and codes
    auto put = [&](int i, const uint64_t (&sn)[2], const uint64_t (&zn)[2], const uint64_t (&r)[2]) {
      uint32_t y[4];
      code_pair(x[i][0], x[i][1], sn[0], zn[0], r[0], y[0], y[1]);
      code_pair(x[i][2], x[i][3], sn[1], zn[1], r[1], y[2], y[3]);
      const uint32_t w = y[0] + (y[1] << BITS) + (y[2] << 2 * BITS) + (y[3] << 3 * BITS);
      if (BITS == 4) *reinterpret_cast<uint16_t*>(k_at + i * 16) = (uint16_t)w;
      else k_at[i * 16] = (unsigned char)w;
    };
    const int gps = kColumn / G;  // channel groups of a token, in the column
    if (tokenwise) {
      const int lg = G / 4, gl = lane & (lg - 1);  // lanes of a group, place in it
      float mn[kTok], mx[kTok];
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        mn[i] = min_nan(min_nan(x[i][0], x[i][1]), min_nan(x[i][2], x[i][3]));
        mx[i] = max_nan(max_nan(x[i][0], x[i][1]), max_nan(x[i][2], x[i][3]));
      }
      reduce_group<kTok, false>(mn, lg);
      reduce_group<kTok, true>(mx, lg);
      float4* sz = reinterpret_cast<float4*>(ranges);  // [token][group] -s, -z, 1 / s
      static_assert(sizeof(ranges) >= 128 * (kColumn / 32) * sizeof(float4), "table");
      const int share = lg / kTok;  // (lg >= kTok: a lane has one value at most)
      if (gl % share == 0) {
        const Group g = group_of_range(mn[0], mx[0], kMax);
        const int e = (tok + gl / share) * gps + ch / G;
        if (isnan(g.s)) report(p.dev_status, KVQ_DEV_NONFINITE);
        sz[e] = make_float4(-g.s, -g.z, reciprocal(g.s), 0.f);
        s_out[e] = g.s_bits;
        z_out[e] = g.z_bits;
      }
      __syncwarp();  // a group's lanes are one warp's
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        float4 g = sz[(tok + i) * gps + ch / G];
        if (isnan(g.x)) {
          g.x = 0.f;
          x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
        }
        const uint64_t sn = rows::pair(g.x, g.x), zn = rows::pair(g.y, g.y), r = rows::pair(g.z, g.z);
        put(i, {sn, sn}, {zn, zn}, {r, r});
      }
    } else {
      float mn[4], mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mn[c] = mx[c] = x[0][c];
#pragma unroll
        for (int i = 1; i < kTok; ++i) {
          mn[c] = min_nan(mn[c], x[i][c]);
          mx[c] = max_nan(mx[c], x[i][c]);
        }
      }
      *reinterpret_cast<float4*>(&ranges[0][warp][ch]) = make_float4(mn[0], mn[1], mn[2], mn[3]);
      *reinterpret_cast<float4*>(&ranges[1][warp][ch]) = make_float4(mx[0], mx[1], mx[2], mx[3]);
      channel_groups<BITS, kColumn, kWarps>(ranges, kBlockTokens / G, G / kTok, s_out, z_out, p.dev_status);
      const int g = tok / G;
      const float4 s4 = *reinterpret_cast<const float4*>(&ranges[0][g][ch]);
      const float4 z4 = *reinterpret_cast<const float4*>(&ranges[1][g][ch]);
      float sc[4] = {s4.x, s4.y, s4.z, s4.w}, rc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (isnan(sc[c])) {
          sc[c] = 0.f;
#pragma unroll
          for (int i = 0; i < kTok; ++i) x[i][c] = 0.f;
        }
        rc[c] = reciprocal(sc[c]);
      }
      const uint64_t sn[2] = {rows::pair(-sc[0], -sc[1]), rows::pair(-sc[2], -sc[3])};
      const uint64_t zn[2] = {rows::pair(-z4.x, -z4.y), rows::pair(-z4.z, -z4.w)};
      const uint64_t r[2] = {rows::pair(rc[0], rc[1]), rows::pair(rc[2], rc[3])};
#pragma unroll
      for (int i = 0; i < kTok; ++i) put(i, sn, zn, r);
    }
    __syncthreads();

    // ---- out
    for (int e = tid; e < kPieces; e += kThreads) {
      const int chunk = e >> 7, t = e & 127, h = head_of(q, chunk * kPer), c = channel_of(q, chunk * kPer);
      if (h < H)
        *reinterpret_cast<uint4*>(p.codes[0] + ((size_t)page * H + h) * (size_t)(kBlockTokens * D * BITS / 8) +
                                  ((size_t)(c / kPer) * kBlockTokens + t) * 16) =
            *reinterpret_cast<const uint4*>(packed + (chunk * 129 + t) * 16);
    }
    for (int e = tid; e < kBlockTokens * kColumn / G; e += kThreads) {
      const int first = tokenwise ? e % gps * G : e % kColumn;  // the entry's (first) channel in the column
      const int h = head_of(q, first), c = channel_of(q, first);
      const size_t at = ((size_t)page * H + h) * nsz + (tokenwise ? e / gps * (D / G) + c / G : e / kColumn * D + c);
      if (h < H) {
        p.scale[0][at] = s_out[e];
        p.zero[0][at] = z_out[e];
      }
    }
    __syncthreads();  // (the shared arrays are free again)
  }
  end_after_last();
}

// The rest of both.
template <typename T, int BITS, int W, Part PART>
__global__ void __launch_bounds__(32 * kEdgeWarps, sizeof(Raw<T>) == 8 ? 2 : 1) rotary_edges_kernel(const AppendParams p) {
  append_edge<T, BITS, W, PART, true>(p);
  end_after_last();
}

struct Chain {
  cudaStream_t stream;
  bool first = true;  // waits for what is in the stream; the others for its last CTA to start
  template <class... Args>
  cudaError_t launch(dim3 grid, int threads, size_t smem, void (*kernel)(Args...), Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = first ? 0 : 1;
    first = false;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
  }
};

template <typename T, int BITS, int W>
cudaError_t launch_w(const AppendParams& p, Chain& chain) {
  constexpr bool kHalf = sizeof(Raw<T>) == 8;
  const unsigned heads = (unsigned)p.num_kv_heads, slabs = (unsigned)(p.head_dim / W);
  if constexpr (kHalf) {
    if (p.total >= kBlockTokens) {  // there may be blocks of new tokens alone
      const unsigned most = (unsigned)(p.total / kBlockTokens);
      const int columns = (p.num_kv_heads * p.head_dim + kColumn - 1) / kColumn;
      cudaError_t e = chain.launch(dim3(most, heads, slabs), 32 * kBlockWarps, 0, rotary_v_kernel<T, BITS, W>, p);
      // two columns or more to a CTA once every SM has six CTAs
      const long long tiles = (long long)most * columns;
      const int each = tiles < 2 * 912 ? 1 : tiles < 4 * 912 ? 2 : 4;
      const dim3 grid(most, (unsigned)((columns + each - 1) / each));
      if (e != cudaSuccess) return e;
      if (p.head_dim == 256) {
        e = chain.launch(grid, 32 * kEdgeWarps, 0, rotary_k_kernel<T, BITS, true>, p, each);
      } else {
        const auto kernel = rotary_k_kernel<T, BITS, false>;
        const size_t smem = (size_t)kBlockTokens * p.turn.dim * sizeof(float);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = chain.launch(grid, 32 * kEdgeWarps, smem, kernel, p, each);
      }
      if (e != cudaSuccess) return e;
    }
  }
  const long long two = p.batch < p.total / 2 ? p.batch : p.total / 2;  // (as for append_chunk's edges)
  const long long blocks = p.batch + two + (kHalf ? 0 : (p.total - 2 * two) / kBlockTokens);
  return chain.launch(dim3((unsigned)blocks, heads, 2 * slabs), 32 * kEdgeWarps, 0, rotary_edges_kernel<T, BITS, W, kHalf ? kEdges : kEvery>, p);
}

template <typename T>
cudaError_t launch(const AppendParams& p, Chain& chain) {
  if (p.bits == 4) return p.head_dim < 128 ? launch_w<T, 4, 64>(p, chain) : launch_w<T, 4, 128>(p, chain);
  return p.head_dim < 128 ? launch_w<T, 2, 64>(p, chain) : launch_w<T, 2, 128>(p, chain);
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

// One warp per token and piece of q's (or k's) heads: a lane has two pieces of 8
// channels of a head -- the two halves of 8 pairs -- and their angles for the
// kPasses heads it comes to, whose loads go out together.  What bounds it is
// memory: 32,768 tokens x 40 heads of 128 in bf16, 671 MB: 107 us, 6.3 TB/s.
constexpr int kTurnThreads = 128, kPasses = 4;

template <typename T>
__global__ void __launch_bounds__(kTurnThreads) turn_rows_kernel(const TurnRowsParams p, int q_pieces) {
  let_next_start();
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
cudaError_t launch_turn(const TurnRowsParams& p, Chain& chain) {
  const int each = 512 / p.head_dim * kPasses;  // heads of a warp
  const int q_pieces = (p.heads[0] + each - 1) / each, k_pieces = (p.heads[1] + each - 1) / each;
  return chain.launch(dim3((unsigned)((p.total + kTurnThreads / 32 - 1) / (kTurnThreads / 32)), (unsigned)(q_pieces + k_pieces)),
                      kTurnThreads, 0, turn_rows_kernel<T>, p, q_pieces);
}

template <typename T>
cudaError_t launch_all(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  Chain chain{stream};
  if (rows.total > 0 && rows.heads[0] + rows.heads[1] > 0) {
    const cudaError_t e = launch_turn<T>(rows, chain);
    if (e != cudaSuccess) return e;
  }
  return launch<T>(p, chain);
}

}  // namespace

cudaError_t launch_append_rotary(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  if (p.dtype == KVQ_FP32) return launch_all<float>(p, rows, stream);
  if (p.dtype == KVQ_FP16) return launch_all<__half>(p, rows, stream);
  return launch_all<Bf16Tag>(p, rows, stream);
}

}  // namespace kvq
