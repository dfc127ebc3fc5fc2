// Attention of chunks of new tokens over the packed cache, on tcgen05.
//
// Work: a row tile is up to NT x 128 (token, head) rows of one sequence and KV
// head, and takes one step per key tile of 128 tokens (a cache block); a few
// more are counted for what it costs besides (tile_cost).  All
// steps of all tiles, in a fixed order, are cut into as many equal ranges as
// there are CTAs; a CTA walks its range tile by tile (a segment each).  A tile
// that a range border cuts leaves partial results (normalised outputs and
// their log-sum-exp) that merge_kernel joins; at most two segments of a CTA are
// partial.  So ragged batches, one long sequence and many short ones balance
// alike, without a host round trip: every CTA works the cut out by itself from
// cu_seqlens and seq_lens.
//
// Few rows (a tile of up to 64, one row tile to a CTA): a row's softmax would be
// the work of one thread while three quarters of the lanes idle, and the
// slowest link of a step.  The rows are laid out two or four times over
// instead, in different quadrants of tensor memory; every copy forms the
// probabilities of its own half or quarter of the key tile and leaves the rest
// zero, with a maximum and a sum of its own, so that its accumulator rows are
// the attention over its share of the tokens.  The copies are joined like the
// parts of a cut tile, at the end of the segment, in shared memory.  The extra
// MMA rows are free.
//
// A step: the block's packed codes, scales and offsets come in by bulk copies
// (warp `copy`); a team of dequantising warps turns them into fp16 operands in
// shared memory (x_hat = s code + z, one rounding); S = Q K^T and O += P V run
// on the tensor cores with fp32 accumulators in tensor memory; a thread per
// row does the softmax in between (attn_core.cuh).  K and V operands are both
// K-major: K rows are tokens, V rows are channels, as the cache packs them, and
// neighbouring codes are split off two at a time (the halves of a 32-bit word),
// which leaves the contraction index in a permuted order within 8 (4-bit) or
// 16 (2-bit) elements; Q's channels and P's tokens are put in the same order.
//
// Roundings: x_hat, q (bf16 rows, 8 bits: none) and the probabilities are fp16,
// 2^-11 each; e4m3 codes with the scales folded into the other operand, as
// decode has them for its 4 to 16 rows, would need three-part splits of 128 rows.
//
// What bounds it: the chain of a step, scores - softmax - probabilities -
// products, more than any unit.  Few rows: 1.2 us a step, of which one thread
// spends 0.75 us issuing 16 MMAs at the tensor cores' pace and the rest waiting
// its turn; without dequantisation it would still be 1.1 us, without softmax
// 1.1 us (64 ragged paged sequences up to 128K, 2 bits, 8 tokens at most:
// 962 us, 1.1 TB/s; four drafted tokens of 8 sequences of 4K: 44 us).  Many rows:
// the tensor cores run half of the time (512 tokens behind 32K cached ones,
// 4 bits, 32 heads of 128: 278 us, 1.0 PFLOP/s).  The roles' code together has
// to stay within the instruction cache: two pieces side by side in the dequantising
// loop took 1.4 times as long, a straight-line softmax 1.2 times.  Slower too:
// a second issuing warp (308 -> 355 us), a warp that waits for operands on the
// issuing one's behalf (304 -> 320 us), a fourth dequantising team (1063 -> 1165).
#pragma once
#include "attn_core.cuh"
#include "chunk_attn.h"

namespace kvq {
namespace chunk {

using rows::kTile;
using rows::RowState;

// ---------------------------------------------------------------- the plan

// Tokens of sequence b's chunk and of its cache; a bad entry empties it.
struct Seq {
  int first, n, len;
};
__device__ __forceinline__ Seq load_seq(const RowAttnParams& p, int b, uint32_t* bad) {
  const SeqRows s = seq_rows(p.cu, b, p.total);
  int len = p.seq_lens[b];
  if (s.bad) *bad |= KVQ_DEV_BAD_SEQ_LEN;
  if (len < 0 || len > p.max_blocks * kBlockTokens) {
    *bad |= KVQ_DEV_BAD_SEQ_LEN;
    len = 0;
  }
  return {s.first, s.n, len};
}
// Key tiles that tile t (tok tokens) of the sequence sees.
__device__ __forceinline__ int key_tiles(const Seq& s, int t, int tok, int causal) {
  const int end = min((t + 1) * tok, s.n);
  const int top = causal ? s.len - s.n + end : s.len;
  return top > 0 ? (top + kTile - 1) / kTile : 0;
}
// Steps of a tile that sees n key tiles: one at least, since a tile that sees
// nothing still has its rows written, and tile_cost more for what a segment
// costs beside its steps (Q, the epilogue, filling the pipeline), so that a CTA
// with many short tiles is not the last.  (32 sequences at head dim 256: 156 us
// without, 132 with 3, 137 with 6; head dim 128, 64 ragged sequences: 1063,
// 1026 with 10; four drafted tokens: 55.6, 52 with 6 or 10, 56 with 16.  Head dim
// 64 has 128's, without a measurement of its own.)
__device__ __forceinline__ int tile_cost(int head_dim) { return head_dim > 128 ? 3 : 8; }
__device__ __forceinline__ int work_steps(int n) { return max(1, n); }
__device__ __forceinline__ int tile_steps(const RowAttnParams& p, const Seq& s, int t, int tok) {
  return work_steps(key_tiles(s, t, tok, p.causal)) + tile_cost(p.head_dim);
}
__device__ __forceinline__ long long seq_steps(const RowAttnParams& p, const Seq& s, int tok) {
  const int nt = (s.n + tok - 1) / tok;
  if (nt == 0) return 0;
  if (!p.causal) return (long long)nt * tile_steps(p, s, 0, tok);
  long long n = 0;
  for (int t = 0; t < nt; ++t) n += tile_steps(p, s, t, tok);
  return n;
}

// A place in the order of all steps: head, sequence, tile, step of the tile.
struct Place {
  int h, b, t, x;
  int pad;
  long long per_head, tile0;  // steps of one head; index of the tile's first step
};

// The place of step `at` (of all per_head * heads), found by the whole block;
// scan: block-wide scratch of blockDim.x / 32 long longs; range: the CTA's
// steps [range[0], range[1]) and range[2] of them in all.
template <int NT>
__device__ __forceinline__ void find_place(const RowAttnParams& p, int tok, int cta, int grid, long long* scan,
                                           Place* out, long long* range, bool report_bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + NT - 1) / NT, b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  uint32_t bad = 0;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_steps(p, load_seq(p, b, &bad), tok);
  if (report_bad && bad) report(p.dev_status, bad);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long base = 0, all = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += scan[w];
    all += scan[w];
  }
  const long long lo = base + incl - mine;  // this thread's sequences: steps [lo, lo + mine) of a head
  const long long total = all * p.num_kv_heads;
  const long long s0 = total * cta / grid, s1 = total * (cta + 1) / grid;
  if (tid == 0) {
    range[0] = s0;
    range[1] = s1;
    range[2] = total;
  }
  if (all > 0 && s0 < total) {
    const int h = (int)(s0 / all);
    long long at = s0 - h * all - lo;
    if (at >= 0 && at < mine) {
      for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(p, b, &bad);
        const long long n = seq_steps(p, s, tok);
        if (at >= n) {
          at -= n;
          continue;
        }
        int t = 0;
        for (;; ++t) {
          const int w = tile_steps(p, s, t, tok);
          if (at < w) break;
          at -= w;
        }
        *out = Place{h, b, t, (int)at, 0, all, s0 - at};
        break;
      }
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------- segments

struct Segment {
  int kvh, first, n, len, tile, b;
  int top, tiles;  // key tiles top, top - 1, ..., top - tiles + 1; tiles < 0: no more segments
  int slot;        // partial results' slot, or -1: the tile is whole
};

struct Aux {
  uint64_t raw_full[kMaxUnits], raw_empty[kMaxUnits];
  uint64_t full[4], empty[4];
  uint64_t seg_full[4], seg_empty[4];
  uint64_t s[2], p[2], q, sums, done, s_free, join;
  uint32_t tmem;
  int fail;
  int raw_bad[kMaxUnits];
  Segment seg[4];
  Place start;
  long long range[3];
};
static_assert(sizeof(Aux) <= kAuxBytes, "Aux");

// ------------------------------------------------------ dequantisation

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) { return (a & m) | o; }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// A word of codes as fp16 integers, two per register: word halves give codes
// (i, i + 4) of 8 four-bit or (i, i + 8) of 16 two-bit codes.  0x6400 | m is
// the fp16 number 1024 + m, so a code in place at bit 2^k is (h - 1024) 2^-k,
// exactly.
template <int BITS>
__device__ __forceinline__ void unpack_word(uint32_t w, __half2* c) {
  const uint32_t w8 = w >> 8;
  if (BITS == 4) {
    const __half2 one = as_h2(0xe400e400u);                                     // -1024
    const __half2 r16 = as_h2(0x2c002c00u), o16 = as_h2(0xd400d400u);           // 1/16, -64
    c[0] = __hadd2(as_h2(and_or(w, 0x000f000fu, 0x64006400u)), one);
    c[1] = __hfma2(as_h2(and_or(w, 0x00f000f0u, 0x64006400u)), r16, o16);
    c[2] = __hadd2(as_h2(and_or(w8, 0x000f000fu, 0x64006400u)), one);
    c[3] = __hfma2(as_h2(and_or(w8, 0x00f000f0u, 0x64006400u)), r16, o16);
  } else {
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const uint32_t v = hi ? w8 : w;
      c[4 * hi] = __hadd2(as_h2(and_or(v, 0x00030003u, 0x64006400u)), as_h2(0xe400e400u));
      c[4 * hi + 1] = __hfma2(as_h2(and_or(v, 0x000c000cu, 0x64006400u)), as_h2(0x34003400u), as_h2(0xdc00dc00u));
      c[4 * hi + 2] = __hfma2(as_h2(and_or(v, 0x00300030u, 0x64006400u)), as_h2(0x2c002c00u), as_h2(0xd400d400u));
      c[4 * hi + 3] = __hfma2(as_h2(and_or(v, 0x00c000c0u, 0x64006400u)), as_h2(0x24002400u), as_h2(0xcc00cc00u));
    }
  }
}
// Operand position of element e within a word's block of codes, and back.
template <int BITS>
__host__ __device__ constexpr int position_of(int e) {
  return BITS == 4 ? (e & ~7) + ((e & 3) << 1) + ((e >> 2) & 1) : (e & ~15) + ((e & 7) << 1) + ((e >> 3) & 1);
}
template <int BITS>
__host__ __device__ constexpr int element_at(int i) {
  return BITS == 4 ? (i & ~7) + ((i & 7) >> 1) + ((i & 1) << 2) : (i & ~15) + ((i & 15) >> 1) + ((i & 1) << 3);
}

// The block's scales and offsets into the table that the dequantising threads
// read: checked (a group whose values would not fit fp16 has its scale
// lowered to fit, one that is not finite is zeroed) and, where they belong to
// columns, in operand order: by_column: [group][column] u16 scales, then
// offsets; else [entry] (scale | offset << 16).
template <int BITS>
__device__ __forceinline__ void prepare_table(int t, const uint16_t* s, const uint16_t* z, int nsz, bool by_column,
                                              bool value, int D, int gshift, bool bad, unsigned char* table,
                                              uint32_t* dev_status) {
  const float most = (float)((1 << BITS) - 1);
  uint16_t* ts = reinterpret_cast<uint16_t*>(table);
  uint16_t* tz = ts + nsz;
  for (int e = t; e < nsz; e += 128) {
    __half sh = __ushort_as_half(s[e]), zh = __ushort_as_half(z[e]);
    const float sf = __half2float(sh), zf = __half2float(zh);
    if (bad) {
      sh = zh = __ushort_as_half(0);
    } else if (!(fmaf(sf, most, zf) <= 65504.f) || !(zf >= -65504.f)) {
      report(dev_status, KVQ_DEV_NONFINITE);
      if (!isfinite(sf) || !isfinite(zf)) sh = zh = __ushort_as_half(0);
      else sh = __float2half_rd((65504.f - zf) / most);
    }
    if (!by_column) {
      reinterpret_cast<uint32_t*>(table)[e] = __half_as_ushort(sh) | (uint32_t)__half_as_ushort(zh) << 16;
    } else {
      int at;
      if (!value) {  // K, channel-wise: entry group * D + channel
        at = (e & ~15) + position_of<BITS>(e & 15);
      } else {       // V, token-wise: entry token * (D / G) + group
        const int gpt = D >> gshift, tok = e >> (31 - __clz(gpt)), g = e & (gpt - 1);
        at = g * kTile + position_of<BITS>(tok);
      }
      ts[at] = __half_as_ushort(sh);
      tz[at] = __half_as_ushort(zh);
    }
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// One slot (part) of a K or V block: codes -> fp16 operand tile of kNR rows
// x kCols columns, 128-byte swizzled, 64 columns to a chunk.  128 threads, a
// 16-byte piece of codes (32 or 64 columns of a row) at a time; every thread
// keeps its row (64 rows: two threads to a row), so that only constants are
// added to its addresses (shared-memory addresses, 32 bits).
template <int BITS, int D, bool VALUE, bool BYCOL>
__device__ __forceinline__ void dequant_part(int t, uint32_t codes, uint32_t table, int nsz, int part, int gshift,
                                             uint32_t slot) {
  constexpr int kRowsAll = VALUE ? D : kTile;                 // rows of the packed block
  constexpr int kNR = VALUE ? (D < 128 ? D : 128) : kTile;    // rows of the part
  constexpr int kCols = VALUE ? kTile : (D < 128 ? D : 128);  // columns of the part
  constexpr int kPer = 128 / BITS;                            // codes of a piece
  constexpr int kChunks = kCols / kPer;
  constexpr int kStep = 128 / kNR;                            // pieces of a row that the threads take at once
  constexpr int kWord = 32 / BITS;                            // codes of a word
  const int row = t & (kNR - 1), chunk0 = t / kNR;
  const int grow = row + (VALUE ? part * 128 : 0);            // row of the block
  const int gchunk0 = chunk0 + (VALUE ? 0 : part * kChunks);  // piece of the row
  uint32_t src = codes + (uint32_t)(gchunk0 * kRowsAll + grow) * 16;
  // 16-byte unit u of the row's 128 bytes of a chunk lies at (u ^ (row & 7)) * 16
  const uint32_t at_row = slot + row * 128, sw = (uint32_t)(row & 7) << 4;
  // by column: scales of the row's group, then offsets nsz entries on; by row:
  // entry (row, column group), a column group every 2^gshift columns
  uint32_t ts = table, step;
  if (BYCOL) {
    ts += (uint32_t)((grow >> gshift) * (VALUE ? kTile : D) + gchunk0 * kPer) * 2;
    step = kStep * kPer * 2;
  } else {
    ts += (uint32_t)(VALUE ? grow : grow * (D >> gshift)) * 4;
    step = 0;
  }
#pragma unroll 1
  for (int i = 0; i < kChunks; i += kStep, src += kStep * kRowsAll * 16, ts += step) {
    const int chunk = i + chunk0;
    const uint4 v = lds128(src);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t dst = at_row + (uint32_t)(chunk * kPer / 64) * (kNR * 128);
    const uint32_t u0 = (uint32_t)(chunk * kPer % 64) / 8 * 16 ^ sw;
    uint32_t sz = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 s4[kWord / 8], z4[kWord / 8];
      if (BYCOL) {
#pragma unroll
        for (int hf = 0; hf < kWord / 8; ++hf) {
          s4[hf] = lds128(ts + (q * kWord + 8 * hf) * 2);
          z4[hf] = lds128(ts + nsz * 2 + (q * kWord + 8 * hf) * 2);
        }
      } else if (q == 0 || (BITS == 2 && q == 2)) {  // a group is at least 32 columns
        const int g = ((gchunk0 + i) * kPer + q * kWord) >> gshift;
        sz = lds32(ts + (VALUE ? g * D : g) * 4);
      }
      __half2 c[kWord / 2];
      unpack_word<BITS>(w[q], c);
      uint32_t x[kWord / 2];
      if (BYCOL) {
#pragma unroll
        for (int hf = 0; hf < kWord / 8; ++hf) {
          x[4 * hf] = as_u32(__hfma2(c[4 * hf], as_h2(s4[hf].x), as_h2(z4[hf].x)));
          x[4 * hf + 1] = as_u32(__hfma2(c[4 * hf + 1], as_h2(s4[hf].y), as_h2(z4[hf].y)));
          x[4 * hf + 2] = as_u32(__hfma2(c[4 * hf + 2], as_h2(s4[hf].z), as_h2(z4[hf].z)));
          x[4 * hf + 3] = as_u32(__hfma2(c[4 * hf + 3], as_h2(s4[hf].w), as_h2(z4[hf].w)));
        }
      } else {
        const __half2 s2 = as_h2(__byte_perm(sz, 0, 0x1010)), z2 = as_h2(__byte_perm(sz, 0, 0x3232));
#pragma unroll
        for (int k = 0; k < kWord / 2; ++k) x[k] = as_u32(__hfma2(c[k], s2, z2));
      }
#pragma unroll
      for (int hf = 0; hf < kWord / 8; ++hf)
        sts128(dst + (u0 ^ (q * (kWord / 8) + hf) * 16), x[4 * hf], x[4 * hf + 1], x[4 * hf + 2], x[4 * hf + 3]);
    }
  }
}

// ------------------------------------------------------------------ Q rows

// 16-byte unit u of row rr of this warp's 32 in a row tile's Q operand.
__device__ __forceinline__ uint4* unit_of(unsigned char* q_s, int rr, int u) {
  const int at = (threadIdx.x & 96) + rr;
  return reinterpret_cast<uint4*>(q_s + u / 8 * 16384 + at * 128 + ((u % 8) ^ (at & 7)) * 16);
}

// This warp's 32 Q rows -> fp16 operand rows, channels in operand order; this
// thread's is at data + off, if `mine`.  A lane has 16 channels of every kR-th
// row, so that lines are read whole.  bf16 rows are scaled by a power of two
// that brings the largest magnitude to [2^13, 2^14): eight significant bits down
// to 2^-30 of it, nothing overflows.  Returns what undoes it in this thread's row.
template <int BITS, int D>
__device__ __forceinline__ float stage_rows(const uint16_t* data, long long off, bool mine, bool fp16, unsigned char* q_s) {
  constexpr int kL = D / 16, kR = 32 / kL, kIts = 32 / kR, kB = 4;  // lanes of a row, rows at once; kB in flight
  const int lane = threadIdx.x & 31, u2 = lane % kL;
  const uint32_t there = __ballot_sync(0xffffffffu, mine);
  int my_ex = 0;
  auto up_of = [](int ex) { return ex > 0 && ex < 255 ? min(13 + 127 - ex, 100) : 0; };
#pragma unroll 1
  for (int b = 0; b < kIts; b += kB) {
    uint4 v[kB][2];
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int rr = (b + k) * kR + lane / kL;
      const uint4* src = reinterpret_cast<const uint4*>(data + __shfl_sync(0xffffffffu, off, rr)) + 2 * u2;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) v[k][hf] = there >> rr & 1 ? src[hf] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int rr = (b + k) * kR + lane / kL;
      const uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
      float mul = 1.f;
      if (!fp16) {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) most = __vmaxu2(most, w[j] & 0x7fff7fffu);
        int ex = (int)(max(most & 0xffffu, most >> 16) >> 7);  // biased exponent
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1) ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, o));
        mul = __uint_as_float((uint32_t)(up_of(ex) + 127) << 23);
        const int got = __shfl_sync(0xffffffffu, ex, lane % kR * kL);
        if (lane / kR == b + k) my_ex = got;  // this thread's own row
      }
      float f[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (fp16) {
          const float2 h = __half22float2(as_h2(w[j]));
          f[2 * j] = h.x;
          f[2 * j + 1] = h.y;
        } else {
          f[2 * j] = __uint_as_float(w[j] << 16) * mul;
          f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * mul;
        }
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = rows::round2<true>(f[element_at<BITS>(8 * hf + 2 * j)], f[element_at<BITS>(8 * hf + 2 * j + 1)]);
        *unit_of(q_s, rr, 2 * u2 + hf) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  return __uint_as_float((uint32_t)(127 - up_of(my_ex)) << 23);
}

// ------------------------------------------------------------- the kernel

template <int BITS, int D, int NT>
__global__ void __launch_bounds__(threads_of(D, NT), 1) chunk_kernel(const Params P) {
  constexpr int kAhead = NT == 2 ? 1 : 2;             // score tiles issued ahead of their PV, per row tile
  constexpr int kChunks = D / 64;                     // 64-channel chunks of a Q row
  constexpr int kParts = D > 128 ? D / 128 : 1;       // slots of a K or V tile
  constexpr int kSlotCh = kChunks / kParts;
  constexpr int kSlot = slot_bytes(D), kSlots = slots_of(D, NT);
  constexpr int kThreads = threads_of(D, NT), kDq = teams_of(D);
  constexpr int kSoftWarps = 4 * NT, kDqWarps = 4 * kDq;
  // (warps by role: chunk_attn.h)
  enum { kCopies, kProducts, kSegments };
  const int other = ((int)threadIdx.x >> 5) - kSoftWarps;
  const int role = other >= 0 && (other & 3) == 3 ? other >> 2 : -1;
  const int dq = other >= 0 && (other & 3) != 3 ? (other >> 2) * 3 + (other & 3) : -1;  // dequantising warp
  // A team waits for a slot's release by the parity of its round, so the
  // round before last must be known to be over: it has waited for slot
  // (u - kDq + 1) kParts - 1 - kSlots before (its last unit), which must not
  // be older than u kParts - 2 kSlots.
  static_assert(kSlots >= (kDq - 1) * kParts + 1, "operand slots");
  const RowAttnParams& p = P.r;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* q_s = smem;
  unsigned char* ring = smem + q_bytes(D, NT);
  Aux* aux = reinterpret_cast<Aux*>(ring + kSlots * kSlot);
  unsigned char* tables = reinterpret_cast<unsigned char*>(aux) + kAuxBytes;  // [kDq][2]
  unsigned char* raw = tables + kDq * 2 * P.table_bytes;
  volatile int* fail = &aux->fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok_tile = kTile / p.gq, tok_cta = tok_tile * NT;
  const int tries = (p.flags & KVQ_FLAG_TEST_STALL) ? rows::kTestTries : rows::kTries;
  const int nsz = kBlockTokens * D >> P.gshift;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may be launched; it waits for this grid
  if (role == kCopies && lane == 0) {
    for (int i = 0; i < P.units; ++i) {
      mbar_init(&aux->raw_full[i], 1);
      mbar_init(&aux->raw_empty[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&aux->full[i], 4);
      mbar_init(&aux->empty[i], 1);
      mbar_init(&aux->seg_full[i], 1);
      mbar_init(&aux->seg_empty[i], kSoftWarps + kDqWarps + 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&aux->s[i], 1);
      mbar_init(&aux->p[i], 4);
    }
    mbar_init(&aux->q, kSoftWarps);
    mbar_init(&aux->sums, 1);
    mbar_init(&aux->done, 1);
    mbar_init(&aux->s_free, 4);
    mbar_init(&aux->join, 4);
    aux->fail = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (role == kSegments) {
    tmem_alloc(&aux->tmem, 512);
    tmem_relinquish();
  }
  // (the ring is not in use yet: the scan's scratch)
  find_place<kThreads>(p, tok_cta, blockIdx.x, gridDim.x, reinterpret_cast<long long*>(ring), &aux->start, aux->range,
                       blockIdx.x == 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = aux->tmem;
  const long long s0 = aux->range[0], s1 = aux->range[1];

  if (s1 > s0) {
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return rows::bounded_wait(bar, parity, fail, tries);
    };
    // Copies of the rows in a tile of `rows_n` rows (see above).
    auto copies_of = [&](int rows_n) { return NT == 2 || rows_n > 64 ? 1 : rows_n > 32 ? 2 : 4; };
    constexpr int kPCol = D > 128 ? 128 : 384;  // with copies: two buffers of probabilities, apart from the scores
    // The same after a failure too: what is in flight must land.
    auto drain = [&](uint64_t* bar, uint32_t parity) {
      for (int i = 0; i < tries && !mbar_try_wait_sleep(bar, parity, 20000u); ++i) {}
    };
    // The next segment, read by every lane of a consuming warp.
    auto next_segment = [&](int k, Segment& g) -> bool {
      if (!__all_sync(0xffffffffu, wait(&aux->seg_full[k & 3], (k >> 2) & 1))) return false;
      g = aux->seg[k & 3];
      __syncwarp();
      if (lane == 0) mbar_arrive(&aux->seg_empty[k & 3]);
      return g.tiles >= 0;
    };

    if (warp < kSoftWarps) {
      // ------------------------------------------------------------ softmax
      // (registers at launch: 6 warpgroups x 80 of two row tiles, 5 x 96 of one;
      // head dim 256: 4 x 128, enough as they are)
      if (D <= 128) setmaxnreg_inc<NT == 2 ? 128 : 144>();
      const int i = warp >> 2, r = tid & 127;
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;
      const uint32_t t_o = tmem + lanes + 256 + i * D;
      int uses = 0;         // score tiles of this row tile so far
      uint32_t s_phase = 0, joins = 0;  // next phases of s[], of join
      Segment g;
      for (int k = 0; next_segment(k, g); ++k) {
        const int tok0 = g.tile * tok_cta, ntok = min(tok_cta, g.n - tok0);
        const int rows_i = max(0, min(tok_tile, ntok - i * tok_tile)) * p.gq;
        const int copies = copies_of(rows_i), share = kTile / copies;  // rows of a copy, and columns that it has
        const int row_i = r & (share - 1), copy = r / share;
        const bool mine = row_i < rows_i, any = ((warp & 3) * 32 & (share - 1)) < rows_i;
        const int tok = tok0 + i * tok_tile + row_i / p.gq, head = g.kvh * p.gq + row_i % p.gq;
        const int pos = g.len - g.n + tok;
        auto unit_at = [&](int rr, int u) { return unit_of(q_s + i * kChunks * 16384, rr, u); };
        // Q rows -> fp16 (stage_rows).  With two row tiles by whole warps; with one, the
        // thread's own row, by less code, is the better of the two (four chunks of
        // 2,048 tokens 1212 -> 1176 us with the output's below, but 64 ragged
        // sequences of a few tokens 956 -> 988 us).
        float c = p.scale_log2;
        if (g.tiles > 0) {
          if constexpr (NT == 2) {
            if (any)
              c *= stage_rows<BITS, D>(static_cast<const uint16_t*>(p.q.data),
                                       (long long)(g.first + tok) * p.q.st + (long long)head * p.q.sh, mine, p.fp16 != 0,
                                       q_s + i * kChunks * 16384);
          } else {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.data) +
                                                              (long long)(g.first + tok) * p.q.st + head * p.q.sh);
            float mul = 1.f;
            if (mine && !p.fp16) {
              uint32_t most = 0;
#pragma unroll 16
              for (int e = 0; e < D / 8; ++e) {
                const uint4 v = src[e];
                most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                               __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
              }
              const int ex = (int)(max(most & 0xffffu, most >> 16) >> 7);  // biased exponent
              if (ex > 0 && ex < 255) {
                const int up = min(13 + 127 - ex, 100);
                mul = __uint_as_float((uint32_t)(up + 127) << 23);
                c *= __uint_as_float((uint32_t)(127 - up) << 23);
              }
            }
            if (any) {
#pragma unroll 4
              for (int e = 0; e < D / 16; ++e) {
                float f[16];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  const uint4 v = mine ? src[2 * e + hf] : make_uint4(0u, 0u, 0u, 0u);
                  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    if (p.fp16) {
                      const float2 h = __half22float2(as_h2(w[j]));
                      f[8 * hf + 2 * j] = h.x;
                      f[8 * hf + 2 * j + 1] = h.y;
                    } else {
                      f[8 * hf + 2 * j] = __uint_as_float(w[j] << 16) * mul;
                      f[8 * hf + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * mul;
                    }
                  }
                }
                unsigned char* dst = q_s + (i * kChunks + e / 4) * 16384 + r * 128;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  uint32_t o[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    o[j] = rows::round2<true>(f[element_at<BITS>(8 * hf + 2 * j)], f[element_at<BITS>(8 * hf + 2 * j + 1)]);
                  *reinterpret_cast<uint4*>(dst + (((e % 4 * 2 + hf) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
              }
            }
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux->q);
        RowState st;
        bool ok = true;
        if (copies > 1 && g.tiles > 0) {  // the other copies' columns stay zero
          uint32_t none[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) none[e] = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) tmem_st_32x32b_x32p(tmem + lanes + kPCol + 32 * e, none);
          tc_wait_st();
        }
        if (rows_i > 0) {
          for (int j = 0; j < g.tiles && ok; ++j, ++uses) {
            const int buf = NT == 2 ? i : copies > 1 ? 0 : j & 1;
            ok = __all_sync(0xffffffffu, wait(&aux->s[buf], s_phase >> buf & 1));
            if (!ok) break;
            s_phase ^= 1u << buf;
            tc_fence_after();
            auto scores_read = [&] {
              if (copies > 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&aux->s_free);
              }
            };
            if (any) {
              const int seen = !mine ? kTile : (p.causal ? min(g.len, pos + 1) : g.len) - (g.top - j) * kTile;
              rows::softmax_tile_rolled<D, true>(tmem + lanes + 128 * buf,
                                                 copies > 1 ? tmem + lanes + kPCol + 64 * (j & 1) : tmem + lanes + 128 * buf,
                                                 t_o, copy * share, copy * share + share, c, seen, j == 0, st,
                                                 [](int x) { return element_at<BITS>(x); },
                                                 [&] {
                                                   if (NT == 1) {
                                                     wait(&aux->sums, (uses - 1) & 1);
                                                     __syncwarp();
                                                     tc_fence_after();
                                                   }
                                                 },
                                                 scores_read);
            } else {
              scores_read();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux->p[NT == 2 ? i : j & 1]);
          }
        }
        ok = ok && __all_sync(0xffffffffu, wait(&aux->done, k & 1));
        if (!ok) break;
        tc_fence_after();
        const bool seen_any = st.l > 0.f || isnan(st.l);
        float f = seen_any ? 1.f / st.l : 0.f;  // of this row's sums in its output
        float lse2 = seen_any ? st.m * c + log2f(st.l) - rows::shift_log2<true>() : -INFINITY;
        const long long row = (long long)(g.first + tok) * p.num_q_heads + head;
        const size_t prow = (size_t)max(g.slot, 0) * (NT * kTile) + i * kTile + row_i;
        auto rounded = [&](const float* x) {  // 8 channels
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = p.fp16 ? rows::round2<true>(x[2 * j], x[2 * j + 1]) : rows::round2<false>(x[2 * j], x[2 * j + 1]);
          return make_uint4(w[0], w[1], w[2], w[3]);
        };
        auto put = [&](int col, const float* x) {  // 8 channels of this thread's row
          if (g.slot >= 0) {
            float4* dst = reinterpret_cast<float4*>(P.part_o + prow * D + col);
#pragma unroll
            for (int e = 0; e < 2; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + col) = rounded(x);
          }
        };
        auto sums = [&](int col, float (&x)[32]) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(t_o + col, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = seen_any ? __uint_as_float(o[e]) * f : 0.f;
        };
        if (copies == 1) {
          // Rows go out: with two row tiles through Q's place, so that neighbouring
          // lanes write neighbouring units (the rows are this warp's own there too,
          // and the next segment's are put there by it); with one as above.
          if (NT == 2 && any) {
            const int passes = g.slot >= 0 ? 2 : 1, chans = D / passes;  // fp32: half of the channels at a time
            const int rows_w = min(32, rows_i - (warp & 3) * 32);
            constexpr int kUnits = D / 8, kAtOnce = 32 / kUnits;
            const unsigned long long own =
                g.slot >= 0 ? (unsigned long long)(P.part_o + prow * D)
                            : (unsigned long long)(static_cast<uint16_t*>(p.out) + row * D);
#pragma unroll 1
            for (int pass = 0; pass < passes; ++pass) {
#pragma unroll 1
              for (int col = 0; col < chans; col += 32) {
                float x[32];
                sums(pass * chans + col, x);
                if (g.slot >= 0) {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<float4*>(unit_at(lane, col / 4 + e)) =
                        make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                } else {
#pragma unroll
                  for (int e = 0; e < 4; ++e) *unit_at(lane, col / 8 + e) = rounded(x + 8 * e);
                }
              }
              __syncwarp();
#pragma unroll 4
              for (int i0 = 0; i0 < 32; i0 += kAtOnce) {
                const int rr = i0 + lane / kUnits, u = lane % kUnits;
                uint4* dst = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, own, rr)) + pass * kUnits + u;
                if (rr < rows_w) *dst = *unit_at(rr, u);
              }
              __syncwarp();
            }
          }
          if (NT == 1 && any) {
#pragma unroll 1
            for (int col = 0; col < D; col += 32) {
              float x[32];
              sums(col, x);
              if (mine) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) put(col + e, x + e);
              }
            }
          }
        } else {
          // Joined over the copies through Q's place in shared memory, half of
          // the channels at a time; every copy's warps add up a share of them.
          auto join = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux->join);
            ok = __all_sync(0xffffffffu, wait(&aux->join, joins++ & 1)) && ok;
          };
          float* xs = reinterpret_cast<float*>(q_s);  // [copy, row] log-sum-exps, then [channel][copy, row]
          xs[r] = lse2;
          join();
          float m = -INFINITY, w = 0.f;
          for (int e = 0; e < copies; ++e) m = fmaxf(m, xs[e * share + row_i]);
          for (int e = 0; e < copies; ++e) {
            const float l = xs[e * share + row_i];
            w += l == -INFINITY ? 0.f : exp2f(l - m);  // (NaN stays, m passes it over)
          }
          f = seen_any ? f * exp2f(lse2 - m) / w : 0.f;
          lse2 = w > 0.f || isnan(w) ? m + log2f(w) : -INFINITY;
          join();
          constexpr int kHalf = D / 2;
          const int each = kHalf / copies;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll 1
            for (int col = 0; col < kHalf; col += 32) {
              float x[32];
              sums(half * kHalf + col, x);
#pragma unroll
              for (int e = 0; e < 32; ++e) xs[(col + e) * kTile + r] = x[e];
            }
            join();
#pragma unroll 1
            for (int col = copy * each; col < (copy + 1) * each; col += 8) {
              const float* at = xs + col * kTile + row_i;
              float x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = at[e * kTile];
              for (int c = 1; c < copies; ++c) {
                at += share;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] += at[e * kTile];
              }
              if (mine) put(half * kHalf + col, x);
            }
            join();
          }
          if (!ok) break;
        }
        if (mine && copy == 0) {
          if (g.slot >= 0) P.part_lse[prow] = lse2;
          else if (p.lse != nullptr) p.lse[row] = lse2 * 0.6931471805599453f;
        }
        tc_fence_before();  // the accumulators are read before the next segment's products
      }
    } else {
      // One instruction for all of these warps: a warpgroup's four have to reach
      // the same one, and three of them dequantise while the last has another role.
      if (D <= 128) setmaxnreg_dec<NT == 2 ? 56 : 80>();
      if (dq >= 0) {
        // ------------------------------------------------ dequantisation
        const int me = dq >> 2, t = (dq & 3) * 32 + lane;  // this team takes units me, me + kDq, ...
        if (me < kDq) {
          const bool k_col = p.k_scheme == KVQ_CHANNELWISE, v_col = p.v_scheme == KVQ_TOKENWISE;
          // The team's own barrier, with a vote.  Every warp of it comes here after
          // each segment is read and after each unit's table is written, whatever
          // its waits returned, so that all of them go on or leave together.
          auto together = [&](bool ok) -> bool {
            uint32_t all;
            asm volatile(
                "{\n\t.reg .pred q, r;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.and.pred r, %2, 128, q;\n\t"
                "selp.u32 %0, 1, 0, r;\n\t}"
                : "=r"(all)
                : "r"((uint32_t)ok), "r"(me + 1)
                : "memory");
            return all != 0;
          };
          // Units of a segment of n key tiles: K_0 V_0 K_1 V_1 ... with one score
          // tile ahead, else K_0 K_1 V_0 K_2 V_1 ... K_n-1 V_n-2 V_n-1.
          auto is_value = [](int i, int n) { return kAhead == 1 ? (i & 1) != 0 : (i >= 2 && !(i & 1)) || i == 2 * n - 1; };
          int u = me, first = 0, did = 0;  // next unit, units of the segments before, units done
          int slot_r = me, round_r = 0;    // its place in the ring of packed blocks
          Segment g;
          for (int k = 0; together(next_segment(k, g)); ++k) {
            const int end = first + 2 * g.tiles;
            bool ok = true;
            for (; u < end; u += kDq) {
              unsigned char* src = raw + slot_r * P.unit_bytes;
              unsigned char* table = tables + (me * 2 + (did & 1)) * P.table_bytes;
              const bool value = is_value(u - first, g.tiles), by_column = value ? v_col : k_col;
              ok = ok && __all_sync(0xffffffffu, wait(&aux->raw_full[slot_r], round_r & 1));
              if (ok) {
                const uint16_t* s = reinterpret_cast<const uint16_t*>(src + kBlockTokens * D * BITS / 8);
                prepare_table<BITS>(t, s, s + nsz, nsz, by_column, value, D, P.gshift, aux->raw_bad[slot_r] != 0, table,
                                    p.dev_status);
              }
              ok = together(ok);
              if (!ok) break;
  #pragma unroll 1
              for (int part = 0; part < kParts && ok; ++part) {
                const int n = u * kParts + part, sl = n % kSlots, round = n / kSlots;
                if (round > 0) ok = __all_sync(0xffffffffu, wait(&aux->empty[sl], (round - 1) & 1));
                if (!ok) break;
                const uint32_t dst = smem_u32(ring) + sl * kSlot;
                if (value) {
                  if (by_column) dequant_part<BITS, D, true, true>(t, smem_u32(src), smem_u32(table), nsz, part, P.gshift, dst);
                  else dequant_part<BITS, D, true, false>(t, smem_u32(src), smem_u32(table), nsz, part, P.gshift, dst);
                } else {
                  if (by_column) dequant_part<BITS, D, false, true>(t, smem_u32(src), smem_u32(table), nsz, part, P.gshift, dst);
                  else dequant_part<BITS, D, false, false>(t, smem_u32(src), smem_u32(table), nsz, part, P.gshift, dst);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&aux->full[sl]);
              }
              if (ok && lane == 0) mbar_arrive(&aux->raw_empty[slot_r]);
              ++did;
              slot_r += kDq;
              if (slot_r >= P.units) {
                slot_r = me;
                ++round_r;
              }
            }
            first = end;
          }
        }
      } else if (role == kCopies) {
        // ---------------------------------------------------------- copies
        int u = 0;
        bool ok = true;
        Segment g;
        for (int k = 0; ok && next_segment(k, g); ++k) {
          int base = 0x7fffffff, ids = 0;  // page ids of key tiles base ... base + 31, one per lane
          auto page_of = [&](int j) {
            if (j < base || j >= base + 32) {
              base = max(0, j - 29);  // K runs up to two tiles ahead (below) of V
              const int t = min(base + lane, p.max_blocks - 1);
              ids = p.page_table ? p.page_table[(size_t)g.b * p.max_blocks + t] : g.b * p.max_blocks + t;
            }
            return __shfl_sync(0xffffffffu, ids, j - base);
          };
          auto unit = [&](bool value, int j) {
            const int sl = u % P.units, round = u / P.units;
            const int page = page_of(j);
            if (round > 0) ok = __all_sync(0xffffffffu, wait(&aux->raw_empty[sl], (round - 1) & 1));
            const bool stall = (p.flags & KVQ_FLAG_TEST_STALL) && s0 == 0 && u == 0;  // test hook: the first is withheld
            if (ok && lane == 0 && !stall) {
              const bool bad = page < 0 || page >= p.num_pages;
              if (bad) report(p.dev_status, KVQ_DEV_BAD_PAGE);
              aux->raw_bad[sl] = bad;
              const size_t blk = (size_t)(bad ? 0 : page) * p.num_kv_heads + g.kvh;
              constexpr int kCodes = kBlockTokens * D * BITS / 8;
              unsigned char* dst = raw + sl * P.unit_bytes;
              mbar_arrive_expect_tx(&aux->raw_full[sl], kCodes + nsz * 4);
              bulk_g2s(dst, (value ? p.v_codes : p.k_codes) + blk * kCodes, kCodes, &aux->raw_full[sl]);
              bulk_g2s(dst + kCodes, (value ? p.v_scale : p.k_scale) + blk * nsz, nsz * 2, &aux->raw_full[sl]);
              bulk_g2s(dst + kCodes + nsz * 2, (value ? p.v_zero : p.k_zero) + blk * nsz, nsz * 2, &aux->raw_full[sl]);
            }
            if (ok) ++u;
          };
          for (int j = -kAhead; j < g.tiles && ok; ++j) {
#pragma unroll 1
            for (int v = 1; v >= 0 && ok; --v)
              if (v ? j >= 0 : j + kAhead < g.tiles) unit(v != 0, g.top - (v ? j : j + kAhead));
          }
        }
        // copies in flight land before this CTA's shared memory is given up
        for (int n = u > P.units ? u - P.units : 0; n < u; ++n) {
          if ((p.flags & KVQ_FLAG_TEST_STALL) && s0 == 0 && n == 0) continue;
          drain(&aux->raw_full[n % P.units], (n / P.units) & 1);
        }
      } else if (role == kProducts) {
        // -------------------------------------------------------- products
        constexpr uint32_t idesc_s = make_idesc(0, 0, 0, 0, 128, 128);
        constexpr int kN = D < 128 ? D : 128;
        constexpr uint32_t idesc_o = make_idesc(0, 0, 0, 0, 128, kN);
        const uint32_t q_a = smem_u32(q_s), ring_a = smem_u32(ring);
        auto scores = [&](int i, int buf, int n) {  // n: running number of the K tile's first slot
#pragma unroll 1
          for (int part = 0; part < kParts; ++part)
            rows::issue_scores<kSlotCh>(tmem + 128 * buf,
                                        make_desc_sw128_lo(q_a + (i * kChunks + part * kSlotCh) * 16384, 0),
                                        make_desc_sw128_lo(ring_a + (n + part) % kSlots * kSlot, 0), idesc_s, part > 0);
        };
        auto values = [&](int i, int pcol, int n, bool add) {  // pcol: column of the probabilities
#pragma unroll 1
          for (int part = 0; part < kParts; ++part)  // V rows are channels: 64 tokens to a chunk of kN rows
            rows::issue_values(tmem + 256 + i * D + part * 128, tmem + pcol,
                               make_desc_sw128_lo(ring_a + (n + part) % kSlots * kSlot, 0), 2, kN * 8, idesc_o, add);
        };
        int n = 0;  // slots taken so far
        uint32_t p_phase = 0, free_phase = 0;  // next phases of p[], of s_free
        bool ok = true;
        auto take = [&]() {
          const int at = n;
          for (int part = 0; part < kParts && ok; ++part, ++n) ok = wait(&aux->full[n % kSlots], (n / kSlots) & 1);
          return at;
        };
        auto release = [&](int at) {
          for (int part = 0; part < kParts; ++part) tc_commit(&aux->empty[(at + part) % kSlots]);
        };
        auto probabilities = [&](int buf) {  // written
          ok = wait(&aux->p[buf], p_phase >> buf & 1);
          p_phase ^= 1u << buf;
          tc_fence_after();
          return ok;
        };
        Segment g;
        for (int k = 0; ok && next_segment(k, g); ++k) {
          if (lane == 0) {
            const int ntok = min(tok_cta, g.n - g.tile * tok_cta);
            const int act = NT == 2 && ntok > tok_tile ? 2 : 1;
            const bool split = copies_of(ntok * p.gq) > 1;  // one buffer of scores, probabilities apart
            ok = wait(&aux->q, k & 1);
            tc_fence_after();
            auto first_scores = [&](int j) {  // tile j's, for every row tile
              const int ks = take();
              if (!ok) return;
#pragma unroll 1
              for (int i = 0; i < act; ++i) {
                const int buf = NT == 2 ? i : j;
                scores(i, buf, ks);
                tc_commit(&aux->s[buf]);
              }
              release(ks);
            };
            for (int j = 0; j < (split ? 1 : kAhead) && j < g.tiles && ok; ++j) first_scores(j);
#pragma unroll 1
            for (int j = 0; j < g.tiles && ok; ++j) {
              if (NT == 1 && split) {
                // S of tile j + 1 as soon as tile j's scores are read
                if (j + 1 < g.tiles) {
                  ok = wait(&aux->s_free, free_phase & 1);
                  tc_fence_after();
                  if (ok) first_scores(0);
                }
                ++free_phase;
                const int vs = ok ? take() : 0;
                if (!ok || !probabilities(j & 1)) break;
                values(0, kPCol + 64 * (j & 1), vs, j > 0);
                tc_commit(&aux->sums);
                release(vs);
                continue;
              }
              const int vs = take();
              const bool more = j + kAhead < g.tiles;
              int ks = 0;
#pragma unroll 1
              for (int i = 0; i < act && ok; ++i) {
                const int buf = NT == 2 ? i : j & 1;
                if (!probabilities(buf)) break;
                values(i, 128 * buf, vs, j > 0);
                if (NT == 1) tc_commit(&aux->sums);
                if (i == act - 1) release(vs);
                if (more) {
                  if (i == 0) ks = take();  // after the first PV: with head dim 256 K needs slots that V gives up
                  if (!ok) break;
                  scores(i, buf, ks);
                  tc_commit(&aux->s[buf]);
                }
              }
              if (ok && more) release(ks);
            }
            tc_commit(&aux->done);
            drain(&aux->done, k & 1);  // also: nothing in flight at the end
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        __syncwarp();
      } else if (role == kSegments && lane == 0) {
        // ---------------------------------------------------------- segments
        Place at = aux->start;
        uint32_t bad = 0;
        Seq s = load_seq(p, at.b, &bad);
        long long left = s1 - s0;
        bool first = true, ok = true;
        for (int k = 0; ok;) {
          Segment g;
          g.tiles = -1;
          bool some = true;  // else: none of the tile's work, only steps that stand for its cost
          if (left > 0) {
            const int w = key_tiles(s, at.t, tok_cta, p.causal), work = work_steps(w);
            const int take = (int)min(left, (long long)(work + tile_cost(D) - at.x));
            some = at.x < work;
            g.kvh = at.h; g.first = s.first; g.n = s.n; g.len = s.len; g.tile = at.t; g.b = at.b;
            g.top = w - 1 - at.x;
            g.tiles = min(take, w - at.x);  // 0: nothing to see
            g.slot = at.x == 0 && take >= work ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1);
            left -= take;
            first = false;
          }
          if (some) {
            if (k >= 4) ok = wait(&aux->seg_empty[k & 3], ((k >> 2) - 1) & 1);
            if (!ok) break;
            aux->seg[k & 3] = g;
            mbar_arrive(&aux->seg_full[k & 3]);
            if (g.tiles < 0) break;
            ++k;
          }
          if (left > 0) {  // the next tile with rows
            at.x = 0;
            ++at.t;
            while (at.t * tok_cta >= s.n) {
              at.t = 0;
              if (++at.b == p.batch) { at.b = 0; ++at.h; }
              s = load_seq(p, at.b, &bad);
            }
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (role == kSegments) tmem_dealloc(tmem, 512);
  if (tid == 0 && aux->fail) report(p.dev_status, KVQ_DEV_TIMEOUT);
}

template <int BITS, int D, int NT>
cudaError_t launch_instance(const Params& p, int grid, size_t smem, cudaStream_t stream) {
  cudaError_t e =
      cudaFuncSetAttribute(chunk_kernel<BITS, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  chunk_kernel<BITS, D, NT><<<grid, threads_of(D, NT), smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace chunk
}  // namespace kvq
