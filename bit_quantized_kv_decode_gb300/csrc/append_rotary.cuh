// Append with the position rotation on the way, and rows turned on their own.
//
// The first R channels of a row at position p are pairs (x1, x2) -- channel i
// with i + R / 2, or neighbours -- that become
//   (fl(fl(x1 c) - fl(x2 s)), fl(fl(x2 c) + fl(x1 s))),  c, s = cos, sin of the pair's angle at p,
// in fp32, on pairs of values: product, product times sign plus product, where the
// sign is a number that the compiler does not know (Turn::one) and so cannot fuse
// into one operation with the product before it.  K goes into the cache from
// there, without a rounding to the rows' type between; turned queries (and keys,
// where attention over rows follows) are rounded to it once.
//
// A call is one chain of kernels -- whole blocks of K, rows, whole blocks of V,
// edges -- that write disjoint places and overlap.  It is one pass over the rows:
// 32,768 tokens of 32 query and 8 KV heads of 128, bf16 to 4 bits, turned K given
// back: 153 us, 5.1 TB/s, most of it the rows' kernel at memory's rate; a token of
// each of 128 sequences: 41 us, 3.4 TB/s, set by the number of instructions that a
// warp of a begun block goes through.
#pragma once
#include "append_core.cuh"

namespace kvq {

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

// Adds the kernel of the rows alone, where there are any, to a call's chain.
bool rows_to_turn(const TurnRowsParams& rows);
cudaError_t launch_turn_rows(const TurnRowsParams& rows, Chain& chain);
cudaError_t launch_append_rotary_i2(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream);
cudaError_t launch_append_rotary_i4(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream);

namespace {

// The kernels of a call write disjoint places and read what none of them writes;
// each may start once the last CTA of the one before has, and ends no earlier
// than that one, so that what follows in the stream follows all of them.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void end_after_last() {  // one CTA waits for all of them, so that the others make room
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// V's blocks of new 16-bit tokens alone.
template <typename T, int BITS, int W>
__global__ void __launch_bounds__(32 * kBlockWarps, kBlockCtas) rotary_v_kernel(const AppendParams p) {
  let_next_start();
  append_block<T, BITS, W>(p, 1, blockIdx.z);
  end_after_last();
}

// K's: CTAs of 16 warps that go from item to item -- a block's next `each` columns
// of 128 channels (a head; two heads of 64; half a head of 256) -- with the block's
// angles in shared memory.  A thread has 4 channels of 8 tokens.  A value's partner
// is another lane's, but for heads of 256 (CROSS), where it may be of the other
// column and is loaded, as are the angles, which would not fit twice.
//
// A column is loads, barriers and arithmetic in turn, so this kernel is bound by
// neither memory nor instructions (32,768 tokens x 8 heads of 128: 15% and 30%).  It
// is launched first, with one CTA to an SM where there are rows to turn: 62 us by
// itself, 1.4 times what two take, but the rows' kernel then runs beside it (the
// call: 168 -> 157 us).
constexpr int kColumn = 128, kSms = 152;

template <typename T, int BITS, bool CROSS>
__global__ void __launch_bounds__(32 * kEdgeWarps, 2) rotary_k_kernel(const AppendParams p, int each) {
  constexpr int kWarps = kEdgeWarps, kThreads = 32 * kWarps, kTok = kBlockTokens / kWarps;
  constexpr int kPer = 128 / BITS, kPieces = kColumn * BITS;  // codes of a 16-byte piece, pieces of a column
  constexpr float kMax = (float)((1 << BITS) - 1);
  __shared__ __align__(16) unsigned char packed[kColumn / kPer * 129 * 16];  // [chunk][128 tokens], a piece of padding
  // channel-wise: ranges per warp, and groups; token-wise: s, z of every group
  __shared__ __align__(16) float ranges[2][kWarps][kColumn], groups_of[3][4][kColumn];
  __shared__ __align__(16) uint16_t s_out[128 * 4], z_out[128 * 4];
  __shared__ int found[2];
  let_next_start();
  const int D = p.head_dim, H = p.num_kv_heads, G = p.group, lgG = 31 - __clz(G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tok = warp * kTok, ch = lane * 4;
  const int columns = (H * D + kColumn - 1) / kColumn, pieces = (columns + each - 1) / each;
  for (int item = blockIdx.x; item < p.total / kBlockTokens * pieces; item += gridDim.x) {
    if (warp == 0) find_block<kWhole, 0>(p, item / pieces, found);
    __syncthreads();
    const int b = found[0];
    if (b < 0) break;  // (nor are there any further ones)
    const int len = p.seq_lens[b], j = len / kBlockTokens + found[1];
    const int page = p.page_table ? p.page_table[(size_t)b * p.max_blocks + j] : b * p.max_blocks + j;
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && item % pieces == 0 && tid == 0) report(p.dev_status, KVQ_DEV_BAD_PAGE);
    const int q0 = item % pieces * each, q1 = good ? min(columns, q0 + each) : q0;
    // head and channel of column q's channel c
    auto head_of = [&](int q, int c) { return D == 64 ? 2 * q + (c >> 6) : D == 256 ? q >> 1 : q; };
    auto channel_of = [&](int q, int c) { return D == 64 ? c & 63 : D == 256 ? (q & 1) * kColumn + c : c; };
    const int half = p.turn.dim >> 1, nsz = kBlockTokens * D >> lgG;
    const bool near = p.turn.interleaved != 0, tokenwise = p.scheme[0] == KVQ_TOKENWISE;
    const long long row0 = ((long long)p.cu[b] + j * kBlockTokens - len + tok) * p.x[0].st;
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
    auto angle4 = [](const float* at) {
      return CROSS ? __ldg(reinterpret_cast<const float4*>(at)) : *reinterpret_cast<const float4*>(at);
    };
    auto angle2 = [](const float* at) {
      return CROSS ? __ldg(reinterpret_cast<const float2*>(at)) : *reinterpret_cast<const float2*>(at);
    };
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
      const int gps = kColumn >> lgG;  // channel groups of a token, in the column
      if (tokenwise) {
        const int lg = G >> 2, gl = lane & (lg - 1);  // lanes of a group, place in it
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
        const int lg_share = lgG - 2 - 3;  // lg / kTok lanes to a value (lg >= kTok: a lane has one at most)
        static_assert(kTok == 8, "values of a group");
        if ((gl & ((1 << lg_share) - 1)) == 0) {
          const Group g = group_of_range(mn[0], mx[0], kMax);
          const int e = (tok + (gl >> lg_share)) * gps + (ch >> lgG);
          if (isnan(g.s)) report(p.dev_status, KVQ_DEV_NONFINITE);
          sz[e] = make_float4(-g.s, -g.z, reciprocal(g.s), 0.f);
          s_out[e] = g.s_bits;
          z_out[e] = g.z_bits;
        }
        __syncwarp();  // a group's lanes are one warp's
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
          float4 g = sz[(tok + i) * gps + (ch >> lgG)];
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
        channel_groups<BITS, kColumn, kWarps>(ranges, groups_of, kBlockTokens >> lgG, G / kTok, s_out, z_out, p.dev_status);
        const int g = tok >> lgG;
        const float4 s4 = *reinterpret_cast<const float4*>(&groups_of[0][g][ch]);
        const float4 z4 = *reinterpret_cast<const float4*>(&groups_of[1][g][ch]);
        const float4 r4 = *reinterpret_cast<const float4*>(&groups_of[2][g][ch]);
        float sc[4] = {s4.x, s4.y, s4.z, s4.w};
        if (isnan(s4.x + s4.y + s4.z + s4.w)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (isnan(sc[c])) {
              sc[c] = 0.f;
#pragma unroll
              for (int i = 0; i < kTok; ++i) x[i][c] = 0.f;
            }
        }
        const uint64_t sn[2] = {rows::pair(-sc[0], -sc[1]), rows::pair(-sc[2], -sc[3])};
        const uint64_t zn[2] = {rows::pair(-z4.x, -z4.y), rows::pair(-z4.z, -z4.w)};
        const uint64_t r[2] = {rows::pair(r4.x, r4.y), rows::pair(r4.z, r4.w)};
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
      const int lg_gps = 7 - lgG;  // of kColumn channels
      for (int e = tid; e < kBlockTokens * kColumn >> lgG; e += kThreads) {
        const int first = tokenwise ? (e & (gps - 1)) << lgG : e % kColumn;  // the entry's (first) channel in the column
        const int h = head_of(q, first), c = channel_of(q, first);
        const size_t at = ((size_t)page * H + h) * nsz + (tokenwise ? (e >> lg_gps) * (D >> lgG) + (c >> lgG) : e / kColumn * D + c);
        if (h < H) {
          p.scale[0][at] = s_out[e];
          p.zero[0][at] = z_out[e];
        }
      }
      __syncthreads();  // (the shared arrays are free again)
    }
    __syncthreads();
  }
  end_after_last();
}

// The rest of both.
template <typename T, int BITS, int W, Part PART>
__global__ void __launch_bounds__(32 * kEdgeWarps, sizeof(Raw<T>) == 8 ? 2 : 1) rotary_edges_kernel(const AppendParams p) {
  append_edge<T, BITS, W, PART, true>(p);
  end_after_last();
}

// Whole blocks of K, rows, whole blocks of V, edges.
template <typename T, int BITS, int W>
cudaError_t launch_w(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  constexpr bool kHalf = sizeof(Raw<T>) == 8;
  const unsigned heads = (unsigned)p.num_kv_heads, slabs = (unsigned)(p.head_dim / W);
  // Kernels for blocks of new tokens alone, where there are likely to be some (a
  // step of one token each is 5 us faster without); else the edges' takes those too.
  const bool whole = kHalf && p.total >= kBlockTokens && (p.total >= 2048 || p.total >= 64LL * p.batch);
  const bool turn = rows_to_turn(rows);
  Chain chain{stream};
  cudaError_t e = cudaSuccess;
  if constexpr (kHalf) {
    if (whole) {
      const long long columns = (p.num_kv_heads * p.head_dim + kColumn - 1) / kColumn;
      const long long tiles = p.total / kBlockTokens * columns;
      const int each = tiles < 2 * 912 ? 1 : 2;  // (two once every SM has six items)
      const long long items = p.total / kBlockTokens * ((columns + each - 1) / each), most = turn ? kSms : 2 * kSms;
      const dim3 grid((unsigned)(items < most ? items : most));
      if (p.head_dim == 256) {
        e = chain.launch(grid, 32 * kEdgeWarps, 0, rotary_k_kernel<T, BITS, true>, p, each);
      } else {
        const auto kernel = rotary_k_kernel<T, BITS, false>;
        const size_t smem = (size_t)kBlockTokens * p.turn.dim * sizeof(float);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockTokens * kColumn * (int)sizeof(float));
        if (e == cudaSuccess) e = chain.launch(grid, 32 * kEdgeWarps, smem, kernel, p, each);
      }
      if (e != cudaSuccess) return e;
    }
  }
  if (turn) e = launch_turn_rows(rows, chain);
  if (e != cudaSuccess) return e;
  if constexpr (kHalf) {
    const dim3 grid((unsigned)(p.total / kBlockTokens), heads, slabs);
    if (whole) e = chain.launch(grid, 32 * kBlockWarps, 0, rotary_v_kernel<T, BITS, W>, p);
    if (e != cudaSuccess) return e;
  }
  const long long blocks = edge_blocks(p.batch, p.total, whole);
  const dim3 grid((unsigned)blocks, heads, 2 * slabs);
  if constexpr (kHalf) {
    if (whole) return chain.launch(grid, 32 * kEdgeWarps, 0, rotary_edges_kernel<T, BITS, W, kEdges>, p);
  }
  return chain.launch(grid, 32 * kEdgeWarps, 0, rotary_edges_kernel<T, BITS, W, kEvery>, p);
}

template <typename T, int BITS>
cudaError_t launch_t(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  return p.head_dim < 128 ? launch_w<T, BITS, 64>(p, rows, stream) : launch_w<T, BITS, 128>(p, rows, stream);
}
template <int BITS>
cudaError_t launch_bits(const AppendParams& p, const TurnRowsParams& rows, cudaStream_t stream) {
  if (p.dtype == KVQ_FP32) return launch_t<float, BITS>(p, rows, stream);
  if (p.dtype == KVQ_FP16) return launch_t<__half, BITS>(p, rows, stream);
  return launch_t<Bf16Tag, BITS>(p, rows, stream);
}

}  // namespace
}  // namespace kvq
