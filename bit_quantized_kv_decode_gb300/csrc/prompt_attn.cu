// Attention over whole prompts on tcgen05: out = softmax(scale Q K^T) V per
// packed sequence, K and V 16-bit rows read where they lie.
//
// A CTA has NT tiles of 128 rows of one sequence and KV head (tokens x the
// heads of the group) and walks the key tiles of 128 tokens from its
// last visible one down, so that the tiles that need masks come first.
// Warps 0-3 (and 4-7) own one tile each: a thread per row takes the row's 128
// scores from tensor memory, keeps the running maximum and sum, and puts the
// probabilities back as the A operand of the second product.  Warp 8 copies Q,
// K and V by TMA into a ring of slots; warp 9 issues the MMAs:
//   S_i = Q_i K^T (both from shared memory), O_i += P_i V (P from tensor memory).
// Only a few MMAs queue up in the tensor core, so whatever the issuing thread
// does in between that takes longer leaves it idle.  Warp 10 therefore does its
// waiting for copies: it arrives at the probabilities' barriers too, once the
// tile's V (and, two row tiles, the next K, which is copied with it) is there,
// and the issuing thread waits for that barrier alone.
// With two tiles (head dims 64 and 128) the tensor cores work on one tile's
// products while the other's softmax runs; with one (head dim 256: two
// accumulators would not fit tensor memory) the scores are double-buffered
// along the keys instead and S of tile j + 2 follows PV of tile j.
//
// What bounds it: with long prompts the tensor cores and the hand-overs between
// them and the softmax (16,384 tokens, 32 heads of 128, bf16, causal: 1.65 ms,
// 1.34 PFLOP/s, 69% of a large library product's rate; a step of two tiles
// takes 1.9 us of which 1.1 us are MMAs).  With short ones it is what a CTA
// takes besides its steps, about 6 us (its tile found, first copies, the
// diagonal's V, the last product, output): 24 prompts of 12,289 tokens in all
// take 172 us where their products would take 52.  Slower when tried: a second issuing warp (1.66 -> 1.99 ms), the
// probabilities handed over in halves (1.66 -> 1.81 ms).
//
// Tensor memory (512 columns): S_0, S_1 (128 each; P_i over S_i), O_0, O_1.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_core.cuh"

namespace kvq {
namespace rows {
namespace {

// 3-D tensor map of a row tensor (channels, heads, tokens), 128-byte swizzle,
// boxes of 64 channels x `box_heads` x `box_tokens`.
cudaError_t encode_rows_map(void* map, const Rows& r, int head_dim, int heads, int total, int box_heads, int box_tokens,
                            bool fp16) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)total};
  const cuuint64_t strides[2] = {(cuuint64_t)r.sh * 2, (cuuint64_t)r.st * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult e = encode(static_cast<CUtensorMap*>(map),
                            fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                            const_cast<void*>(r.data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
struct Shape {
  static constexpr int kNT = D > 128 ? 1 : 2;      // row tiles
  static constexpr int kAhead = D > 128 ? 2 : 1;   // score tiles issued ahead of their PV, per row tile
  static constexpr int kChunks = D / 64;           // 64-channel chunks of a row (16 KB per 128 rows)
  static constexpr int kSlotCh = D > 128 ? 2 : kChunks;  // chunks of a ring slot
  static constexpr int kParts = kChunks / kSlotCh;       // slots of a K or V tile
  static constexpr int kSlotBytes = kSlotCh * 16384;
  static constexpr int kQBytes = kNT * kChunks * 16384;
  // Two row tiles: K of the first key tile in slot 0, then pairs (V of tile j,
  // K of tile j + 1), copied and given up together.  One: single slots.
  static constexpr int kPairs = D == 64 ? 3 : 2;
  static constexpr int kSlots = kNT == 2 ? 1 + 2 * kPairs : 5;
  static constexpr int kThreads = 384;  // three warpgroups: softmax, softmax, copies and products
  static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + 512 + 4 * D;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Aux {  // after the ring
  uint64_t full[8], empty[8], first, q, fixed[2], s[2], p[2], sums, done;
  uint32_t tmem;
  int fail, any_bad;
  int seq_first, seq_n, tile;  // this CTA's sequence (rows [first, first + n)) and tile; tile < 0: none
};
static_assert(sizeof(Aux) <= 512, "Aux");

// The first tokens, counted from the first key tile that is not seen whole
// (two such tiles at most), at which a channel of V holds a NaN, +inf, -inf:
// ten bits each, kNone where there is none.
constexpr uint32_t kNone = 0x3ff;
constexpr uint32_t kNoneAll = kNone | kNone << 10 | kNone << 20;

// Reports entries of cu_seqlens that are out of range or go back, wherever they
// stand: find_tile reads no further than the CTA's own sequence.  Run by one warp
// of the first CTA beside find_tile.  (Among the roles, by a warp that has none,
// the code in their midst cost 2% on long prompts and 1% on packed ones.)
__device__ void check_starts(const RowAttnParams& p) {
  bool bad = false;
#pragma unroll 8
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) bad |= seq_rows(p.cu, b, p.total).bad;
  if (bad) report(p.dev_status, KVQ_DEV_BAD_SEQ_LEN);
}

// Which sequence and tile the rank-th CTA of a KV head has.  Run by one warp.
// Causal tiles cost in proportion to their place in the sequence, so they are
// handed out by falling place over all sequences at once: the rank's place t
// is found by bisection on cum(t) = sum_b max(0, tiles_b - t), the number of
// tiles at places >= t.  (Up to 256 sequences, eight to a lane; beyond that,
// and without a causal mask, in order of the sequences: 65,536 ragged tokens
// took 802 us as 256 prompts and 740 us as 257 others, so the border shows
// less than the lengths do.)
__device__ void find_tile(const RowAttnParams& p, int rank, int per_tile, Aux* aux) {
  const int lane = threadIdx.x & 31;
  int seq = -1, tile = -1;
  if (p.causal && p.batch <= 256) {
    int nt[8], most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int b = lane + 32 * i;
      nt[i] = 0;
      if (32 * i >= p.batch) continue;
      if (b < p.batch) nt[i] = (seq_rows(p.cu, b, p.total).n + per_tile - 1) / per_tile;
      most = max(most, nt[i]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    auto cum = [&](int t) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * i < p.batch) n += max(0, nt[i] - t);
      return __reduce_add_sync(0xffffffffu, n);
    };
    if (rank < cum(0)) {
      int lo = 0, hi = most;  // cum(lo) > rank >= cum(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum(mid) > rank) lo = mid;
        else hi = mid;
      }
      tile = lo;
      int k = rank - cum(lo + 1);  // the k-th sequence with more than `tile` tiles
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (seq >= 0 || 32 * i >= p.batch) continue;
        const uint32_t has = __ballot_sync(0xffffffffu, nt[i] > tile);
        const int before = __popc(has & ((1u << lane) - 1));
        const uint32_t kth = __ballot_sync(0xffffffffu, nt[i] > tile && before == k);
        if (kth != 0) seq = 32 * i + __ffs(kth) - 1;
        else k -= __popc(has);
      }
      if (seq < 0) tile = -1;  // (more tiles than 31 bits, of sequences that share their rows)
    }
  } else {
    for (int b0 = 0; b0 < p.batch && seq < 0; b0 += 32) {
      const int b = b0 + lane;
      SeqRows s{0, 0, false};
      if (b < p.batch) s = seq_rows(p.cu, b, p.total);
      const int n = (s.n + per_tile - 1) / per_tile;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > rank);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        seq = b0 + l;
        tile = rank - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, n, l));
        break;
      }
      rank -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane == 0) {
    aux->tile = tile;
    if (tile >= 0) {
      const SeqRows s = seq_rows(p.cu, seq, p.total);
      aux->seq_first = s.first;
      aux->seq_n = s.n;
    }
  }
}

// A V tile that some rows see only in part: tokens from `valid` on (another
// sequence's rows, or none) become zeros, and values that are not finite are
// zeroed and noted in `bad`, so that a zero probability keeps them out of the
// rows before them; the epilogue adds them to the rows from there on (without a
// causal mask: to all).  token0: the tile's first token as `bad` counts them.
// By THREADS threads, in their own time: this one is number `me`.
template <bool FP16, int THREADS>
__device__ __forceinline__ void mend_values(int me, unsigned char* slot, int chunks, int channel0, int token0, int valid,
                                            uint32_t* bad, int* any_bad) {
  const uint32_t inf = FP16 ? 0x7c00u : 0x7f80u;
  uint32_t acc = 0;
  const int n = chunks * kTile * 8;
#pragma unroll 4
  for (int i = me; i < n; i += THREADS) {  // 16 bytes each; rows of 8
    const int t = (i >> 3) & (kTile - 1);
    uint4* at = reinterpret_cast<uint4*>(slot) + i;
    if (t >= valid) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 v = *at;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // an all-ones exponent in either half carries into its sign bit
        const uint32_t e = (w[j] & (inf * 0x10001u)) + (FP16 ? 0x04000400u : 0x00800080u);
        acc |= e & 0x80008000u;
      }
    }
  }
  if (!__any_sync(0xffffffffu, acc != 0)) return;
  if ((me & 31) == 0) *any_bad = 1;
#pragma unroll 1
  for (int i = me; i < n; i += THREADS) {
    const int t = (i >> 3) & (kTile - 1), chunk = (i >> 3) / kTile, c16 = (i & 7) ^ (t & 7);
    if (t >= valid) continue;
    uint16_t* at = reinterpret_cast<uint16_t*>(slot) + i * 8;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = at[j];
      if ((w & inf) != inf) continue;
      const int shift = (w & 0x7fffu) != inf ? 0 : (w >> 15) ? 20 : 10;
      uint32_t* word = &bad[channel0 + chunk * 64 + c16 * 8 + j];
      uint32_t was = *word;
      while (((was >> shift) & kNone) > (uint32_t)(token0 + t)) {
        const uint32_t got = atomicCAS(word, was, (was & ~(kNone << shift)) | (uint32_t)(token0 + t) << shift);
        if (got == was) break;
        was = got;
      }
      at[j] = 0;
    }
  }
}

template <int D, bool FP16>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const RowAttnParams p) {
  using Sh = Shape<D>;
  constexpr int NT = Sh::kNT;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* q_s = smem;
  unsigned char* ring = smem + Sh::kQBytes;
  Aux* aux = reinterpret_cast<Aux*>(ring + Sh::kSlots * Sh::kSlotBytes);
  uint32_t* bad = reinterpret_cast<uint32_t*>(reinterpret_cast<unsigned char*>(aux) + 512);  // [D]
  volatile int* fail = &aux->fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.x % p.num_kv_heads, rank = blockIdx.x / p.num_kv_heads;
  const int tok_tile = kTile / p.gq;          // tokens of a row tile
  const int tok_cta = tok_tile * NT;

  if (warp == 0) find_tile(p, rank, tok_cta, aux);
  if (warp == 11 && blockIdx.x == 0) check_starts(p);
  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_map(&map_q);
      tma_prefetch_map(&map_k);
      tma_prefetch_map(&map_v);
      for (int i = 0; i < 8; ++i) {
        mbar_init(&aux->full[i], 1);
        mbar_init(&aux->empty[i], 1);
      }
      mbar_init(&aux->q, 1);
      mbar_init(&aux->first, 1);
      mbar_init(&aux->sums, 1);
      mbar_init(&aux->done, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&aux->fixed[i], 8);
        mbar_init(&aux->s[i], 1);
        mbar_init(&aux->p[i], 5);  // the row tile's warps and the one that waits for copies
      }
      aux->fail = 0;
      aux->any_bad = 0;
      fence_barrier_init();
    }
    __syncwarp();
  }
  if (warp == 9) {
    tmem_alloc(&aux->tmem, 512);
    tmem_relinquish();
  }
  for (int i = tid; i < D; i += Sh::kThreads) bad[i] = kNoneAll;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = aux->tmem;
  const int tile = aux->tile;
  if (tile >= 0) {
    const int first = aux->seq_first, n = aux->seq_n;
    const int tok0 = tile * tok_cta;                        // first token of the CTA, in its sequence
    const int ntok = min(tok_cta, n - tok0);
    const int act = NT == 2 && ntok > tok_tile ? 2 : 1;     // row tiles in use
    const int last = p.causal ? (tok0 + ntok - 1) / kTile : (n - 1) / kTile;  // last visible key tile
    const int tiles = last + 1;
    // the first `mend` tiles of the walk hold tokens that some row must not see
    const int clean = p.causal ? (tok0 + 1) / kTile : n / kTile;  // key tiles below this are seen whole by every row
    const int mend = tiles - min(clean, tiles);
    const int tries = (p.flags & KVQ_FLAG_TEST_STALL) ? kTestTries : kTries;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return bounded_wait(bar, parity, fail, tries); };
    // the same after a failure too: what is in flight must land
    auto drain = [&](uint64_t* bar, uint32_t parity) {
      for (int i = 0; i < tries && !mbar_try_wait_sleep(bar, parity, 20000u); ++i) {}
    };

    // V of the walk's tile j (one of the first two), a share of this thread.
    // Warps 0-7 do it, the softmax's between the probabilities and their
    // arrival: a single warp beside them took longer than that (packed prompts
    // 203 -> 188 us, head dim 256 203 -> 177 us).
    auto mend_tile = [&](int j) -> bool {
      bool ok = true;
      // the tile's first slot, counted from the walk's start.  One row tile: this
      // slot's round before held K of tile j or less, whose scores are there.
      const int at = NT == 2 ? 1 + 2 * j : Sh::kParts * (min(Sh::kAhead, tiles) + j + (j > 0 && tiles > Sh::kAhead));
      for (int part = 0; part < Sh::kParts && ok; ++part) {
        const int sl = NT == 2 ? at : (at + part) % Sh::kSlots;
        ok = __all_sync(0xffffffffu, NT == 2 ? wait(&aux->full[j], 0) : wait(&aux->full[sl], (at + part) / Sh::kSlots & 1));
        if (ok)
          mend_values<FP16, 256>(tid, ring + sl * Sh::kSlotBytes, Sh::kSlotCh, part * Sh::kSlotCh * 64,
                                      (last - j - clean) * kTile, min(kTile, n - (last - j) * kTile), bad, &aux->any_bad);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->fixed[j]);
      return ok;
    };

    // Registers: 384 threads x 168 at launch; the softmax warpgroups take 208
    // each (a row's 128 scores stay in registers), the third keeps 88.
    if (warp >= (NT == 2 ? 8 : 4)) {
      setmaxnreg_dec<88>();
    if (warp == 8) {
      // ------------------------------------------------------------ copies
      int slot = 0, round = 0, issued = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap& map, int j, int part) {  // one slot of key tile j
        if (!ok) return;
        if (round > 0) ok = wait(&aux->empty[slot], (round - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(&aux->full[slot], Sh::kSlotBytes);
#pragma unroll
          for (int c = 0; c < Sh::kSlotCh; ++c)
            tma_load_3d(ring + slot * Sh::kSlotBytes + c * 16384, &map, (part * Sh::kSlotCh + c) * 64, kvh,
                        first + j * kTile, &aux->full[slot]);
        }
        ++issued;
        if (++slot == Sh::kSlots) { slot = 0; ++round; }
      };
      if (lane == 0) {
        const int box = tok_tile * p.gq * 128;
        mbar_arrive_expect_tx(&aux->q, act * Sh::kChunks * box);
        for (int i = 0; i < act; ++i)
          for (int c = 0; c < Sh::kChunks; ++c)
            tma_load_3d(q_s + (i * Sh::kChunks + c) * 16384, &map_q, c * 64, kvh * p.gq, first + tok0 + i * tok_tile,
                        &aux->q);
      }
      const bool stall = (p.flags & KVQ_FLAG_TEST_STALL) && blockIdx.x == 0;  // test hook: V of the first CTA is withheld
      if (NT == 2) {
        auto copy = [&](const CUtensorMap& map, int j, int sl, uint64_t* bar) {
#pragma unroll
          for (int c = 0; c < Sh::kSlotCh; ++c)
            tma_load_3d(ring + sl * Sh::kSlotBytes + c * 16384, &map, c * 64, kvh, first + j * kTile, bar);
        };
        if (lane == 0) {
          mbar_arrive_expect_tx(&aux->first, Sh::kSlotBytes);
          copy(map_k, last, 0, &aux->first);
        }
        for (int j = 0; j < tiles && ok && !stall; ++j) {
          const int m = j % Sh::kPairs;
          if (j >= Sh::kPairs) ok = __all_sync(0xffffffffu, wait(&aux->empty[m], (j / Sh::kPairs - 1) & 1));
          if (!ok) break;
          if (lane == 0) {
            const bool more = j + 1 < tiles;
            mbar_arrive_expect_tx(&aux->full[m], (more ? 2 : 1) * Sh::kSlotBytes);
            copy(map_v, last - j, 1 + 2 * m, &aux->full[m]);
            if (more) copy(map_k, last - j - 1, 2 + 2 * m, &aux->full[m]);
          }
          ++issued;
        }
      } else {
        for (int i = 0; i < Sh::kAhead && i < tiles; ++i)
          for (int part = 0; part < Sh::kParts; ++part) load(map_k, last - i, part);
        for (int i = 0; i < tiles && ok && !stall; ++i) {
          for (int part = 0; part < Sh::kParts; ++part) load(map_v, last - i, part);
          if (i + Sh::kAhead < tiles)
            for (int part = 0; part < Sh::kParts; ++part) load(map_k, last - i - Sh::kAhead, part);
        }
      }
      // copies in flight land before this CTA's shared memory is given up
      constexpr int kRing = NT == 2 ? Sh::kPairs : Sh::kSlots;
      for (int k = issued > kRing ? issued - kRing : 0; k < issued; ++k)
        drain(&aux->full[k % kRing], (k / kRing) & 1);
      if (NT == 2) drain(&aux->first, 0);
      drain(&aux->q, 0);
    } else if (warp == 9) {
      // ------------------------------------------------------------ products
      if (lane == 0) {
        constexpr uint32_t fmt = FP16 ? 0u : 1u;
        constexpr uint32_t idesc_s = make_idesc(fmt, fmt, 0, 0, 128, 128);
        constexpr int kN = D < 128 ? D : 128;
        constexpr uint32_t idesc_o = make_idesc(fmt, fmt, 0, 1, 128, kN);
        const uint32_t q_a = smem_u32(q_s), ring_a = smem_u32(ring);
        bool ok = wait(&aux->q, 0);
        // S of row tile i <- Q_i K^T with K in the slots from `sl`
        auto scores = [&](int i, int buf, int sl) {
#pragma unroll 1
          for (int part = 0; part < Sh::kParts; ++part) {
            issue_scores<Sh::kSlotCh>(tmem + 128 * buf,
                                      make_desc_sw128_lo(q_a + (i * Sh::kChunks + part * Sh::kSlotCh) * 16384, 0),
                                      make_desc_sw128_lo(ring_a + sl * Sh::kSlotBytes, 0), idesc_s, part > 0);
            if (++sl == Sh::kSlots) sl = 0;
          }
        };
        auto values = [&](int i, int buf, int sl, bool add) {
#pragma unroll 1
          for (int part = 0; part < Sh::kParts; ++part) {  // V rows are tokens: 16 of them are 2 KB on
            issue_values(tmem + 256 + i * D + part * 128, tmem + 128 * buf,
                         make_desc_sw128_lo(ring_a + sl * Sh::kSlotBytes, 16384), 128, 512, idesc_o, add);
            if (++sl == Sh::kSlots) sl = 0;
          }
        };
        if (NT == 2) {
          ok = ok && wait(&aux->first, 0);
          int m = 0;  // the pair of tile j
#pragma unroll 1
          for (int j = -1; j < tiles && ok; ++j) {
            const bool more = j + 1 < tiles;
#pragma unroll 1
            for (int i = 0; i < act; ++i) {
              if (j >= 0) {
                if (!(ok = wait(&aux->p[i], j & 1))) break;  // the probabilities, and the pair's copies
                tc_fence_after();
                values(i, i, 1 + 2 * m, j > 0);
              }
              if (more) {
                scores(i, i, j < 0 ? 0 : 2 + 2 * m);
                tc_commit(&aux->s[i]);
              }
            }
            if (j >= 0) {
              tc_commit(&aux->empty[m]);
              if (++m == Sh::kPairs) m = 0;
            }
          }
        } else {
          int slot = 0, round = 0;  // next slot to consume
          auto pass = [&](int& sl) {  // the next tile's slots
            sl = slot;
            for (int part = 0; part < Sh::kParts; ++part)
              if (++slot == Sh::kSlots) { slot = 0; ++round; }
          };
          auto take = [&](int& sl) {  // ... loaded
            const int r0 = round;
            pass(sl);
            for (int part = 0, at = sl, r = r0; part < Sh::kParts && ok; ++part) {
              ok = wait(&aux->full[at], r & 1);
              if (++at == Sh::kSlots) { at = 0; ++r; }
            }
          };
          auto release = [&](int sl) {
            for (int part = 0; part < Sh::kParts; ++part) {
              tc_commit(&aux->empty[sl]);
              if (++sl == Sh::kSlots) sl = 0;
            }
          };
          int ks, vs;
#pragma unroll 1
          for (int j = -Sh::kAhead; j < tiles && ok; ++j) {
            const int buf = j & 1;
            if (j >= 0) {
              pass(vs);
              if (!(ok = wait(&aux->p[buf], j >> 1 & 1))) break;  // the probabilities, and V's copies
              tc_fence_after();
              values(0, buf, vs, j > 0);
              tc_commit(&aux->sums);
              release(vs);
            }
            if (j + Sh::kAhead < tiles) {
              take(ks);
              if (!ok) break;
              scores(0, buf, ks);
              tc_commit(&aux->s[buf]);
              release(ks);
            }
          }
        }
        tc_commit(&aux->done);
        drain(&aux->done, 0);  // nothing in flight when tensor memory is freed
      }
      __syncwarp();
    } else if (warp < 8) {  // (head dim 256: warps 4-7)
      for (int j = 0; j < mend && __all_sync(0xffffffffu, wait(&aux->s[j], 0)) && mend_tile(j); ++j) {}
    } else if (warp == 10 && lane == 0) {
      // ------------------------------------------------------------ copies' arrival, for the products
      bool ok = true;
      int slot = 0, round = 0;  // one row tile: every slot in turn, so that each wait is for the round after the last
      auto next_tile = [&] {
        for (int part = 0; part < Sh::kParts && ok; ++part) {
          ok = wait(&aux->full[slot], round & 1);
          if (++slot == Sh::kSlots) { slot = 0; ++round; }
        }
      };
      if (NT == 1)
        for (int i = 0; i < Sh::kAhead && i < tiles; ++i) next_tile();  // K
#pragma unroll 1
      for (int j = 0; j < tiles && ok; ++j) {
        if (NT == 2) {
          ok = wait(&aux->full[j % Sh::kPairs], j / Sh::kPairs & 1);
        } else {
          if (j > 0 && j - 1 + Sh::kAhead < tiles) next_tile();  // the K tile copied before this V
          next_tile();
        }
        if (ok && j < mend) ok = wait(&aux->fixed[j], 0);
        if (!ok) break;
        // (an arrival counts for the barrier's present phase: the one before must be over)
        if (NT == 2) {
          for (int i = 0; i < act && ok; ++i) {
            if (j > 0) ok = wait(&aux->p[i], (j - 1) & 1);
            mbar_arrive(&aux->p[i]);
          }
        } else {
          if (j > 1) ok = wait(&aux->p[j & 1], (j >> 1 & 1) ^ 1);
          mbar_arrive(&aux->p[j & 1]);
        }
      }
    }
    } else {
      // ------------------------------------------------------------ softmax
      setmaxnreg_inc<208>();
      const int i = NT == 2 ? warp >> 2 : 0;
      const int r = tid & 127;  // row of the tile = lane of tensor memory
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;
      const int rows = min(tok_tile, ntok - i * tok_tile) * p.gq;
      if (i >= act) {
        for (int j = 0; j < mend && mend_tile(j); ++j) {}
      } else {
        const bool mine = r < rows, any = (warp & 3) * 32 < rows;
        const int tok = tok0 + i * tok_tile + r / p.gq;
        const uint32_t t_o = tmem + lanes + 256 + i * D;
        RowState st;
        bool ok = true;
        for (int j = 0; j < tiles && ok; ++j) {
          const int buf = NT == 2 ? i : j & 1;
          ok = __all_sync(0xffffffffu, wait(&aux->s[buf], (NT == 2 ? j : j >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (any) {
            const int k0 = (last - j) * kTile;
            const int seen = !mine ? kTile : (p.causal ? min(n, tok + 1) : n) - k0;
            softmax_tile<D, FP16>(tmem + lanes + 128 * buf, t_o, p.scale_log2, seen, j == 0, st,
                                  [](int x) { return x; },
                                  // two tiles: S of tile j was issued after PV of tile j - 1, and so is done after it
                                  [&] {
                                    if (NT == 1) {
                                      wait(&aux->sums, (j - 1) & 1);
                                      __syncwarp();
                                      tc_fence_after();
                                    }
                                  });
          }
          if (__builtin_expect(j < mend, 0)) ok = mend_tile(j);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&aux->p[buf]);
        }
        ok = ok && __all_sync(0xffffffffu, wait(&aux->done, 0));
        if (ok && any) {
          tc_fence_after();
          const int row = (first + tok) * p.num_q_heads + kvh * p.gq + r % p.gq;  // (at most 2^30 of them)
          const float inv = st.l > 0.f || isnan(st.l) ? 1.f / st.l : 0.f;
          const bool spoiled = aux->any_bad != 0;
          // this row's token as `bad` counts them (-1: the last one before); without a mask every row sees all of them
          const int at = p.causal ? tok - clean * kTile : (int)kNone;
          // The warp's rows go out through Q's place in shared memory (16-byte units
          // at unit ^ (row & 7)), so that neighbouring lanes write neighbouring units:
          // written by its thread alone, a row is D / 8 stores of half sectors (2.7 us
          // of a CTA's time; packed prompts 188 -> 172 us, head dim 256 178 -> 172 us).
          unsigned char* stage = q_s + warp * (32 * D * 2);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_o + 32 * c, o);
            tc_wait_ld();
            float x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(o[k]) * inv;
            if (spoiled) {
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const uint32_t w = bad[32 * c + k];
                if ((w & kNone) != kNone && at >= (int)(w & kNone)) x[k] = NAN;
                if ((w >> 10 & kNone) != kNone && at >= (int)(w >> 10 & kNone)) x[k] += INFINITY;
                if ((w >> 20) != kNone && at >= (int)(w >> 20)) x[k] -= INFINITY;
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(stage + lane * (D * 2) + ((4 * c + k) ^ (lane & 7)) * 16) =
                  make_uint4(round2<FP16>(x[8 * k], x[8 * k + 1]), round2<FP16>(x[8 * k + 2], x[8 * k + 3]),
                             round2<FP16>(x[8 * k + 4], x[8 * k + 5]), round2<FP16>(x[8 * k + 6], x[8 * k + 7]));
          }
          __syncwarp();
          constexpr int kUnits = D / 8, kAtOnce = 32 / kUnits;  // units of a row, rows of a store
          const int rows_w = min(32, rows - (warp & 3) * 32), u = lane % kUnits;
#pragma unroll 4
          for (int i0 = 0; i0 < 32; i0 += kAtOnce) {
            const int rr = i0 + lane / kUnits, to = __shfl_sync(0xffffffffu, row, rr);
            if (rr < rows_w)
              reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (long long)to * D)[u] =
                  *reinterpret_cast<const uint4*>(stage + rr * (D * 2) + (u ^ (rr & 7)) * 16);
          }
          if (mine && p.lse != nullptr) p.lse[row] = row_lse<FP16>(st, p.scale_log2);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (tid == 0 && aux->fail) report(p.dev_status, KVQ_DEV_TIMEOUT);
}

template <int D, bool FP16>
cudaError_t launch(const RowAttnParams& p, cudaStream_t stream) {
  using Sh = Shape<D>;
  CUtensorMap maps[3];
  cudaError_t e = encode_rows_map(&maps[0], p.q, D, p.num_q_heads, p.total, p.gq, kTile / p.gq, FP16);
  if (e == cudaSuccess) e = encode_rows_map(&maps[1], p.k, D, p.num_kv_heads, p.total, 1, kTile, FP16);
  if (e == cudaSuccess) e = encode_rows_map(&maps[2], p.v, D, p.num_kv_heads, p.total, 1, kTile, FP16);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(prompt_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = p.total / (kTile / p.gq * Sh::kNT) + (p.batch < p.total ? p.batch : p.total);
  if (tiles * p.num_kv_heads > 0x7fffffffLL) return cudaErrorInvalidValue;
  prompt_kernel<D, FP16><<<(unsigned)(tiles * p.num_kv_heads), Sh::kThreads, Sh::kSmem, stream>>>(maps[0], maps[1],
                                                                                                 maps[2], p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace rows

cudaError_t launch_prompt_attn(const RowAttnParams& p, cudaStream_t stream) {
  if (p.head_dim == 64) return p.fp16 ? rows::launch<64, true>(p, stream) : rows::launch<64, false>(p, stream);
  if (p.head_dim == 128) return p.fp16 ? rows::launch<128, true>(p, stream) : rows::launch<128, false>(p, stream);
  return p.fp16 ? rows::launch<256, true>(p, stream) : rows::launch<256, false>(p, stream);
}

}  // namespace kvq
