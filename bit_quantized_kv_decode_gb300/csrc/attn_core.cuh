// What the attention kernels over rows of new tokens share: bounded waits,
// arithmetic on pairs, one softmax step of a 128 x 128 score tile in tensor
// memory, and the loops that issue a tile's MMAs.
//
// Rows of a tile are (token, query head of one KV group) pairs, token-major:
// all heads of the group ride in one tile, so K and V are read once for them
// and a chunk of a few tokens still fills rows.  Row r of a tile is tensor-
// memory lane r; one thread owns it, so the softmax needs no exchange between
// threads and any group size works (the last 128 mod G_q rows stay unused).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_rows.h"
#include "kvq_ptx.cuh"

namespace kvq {
namespace rows {

constexpr int kTile = 128;          // rows of a tile, and keys of a tile
constexpr float kRescaleLog2 = 8.f;  // a row's reference maximum moves when its scores exceed it by this (log2 units)

// Waits for a barrier's phase, at most `tries` times a suspended try (20 us at
// most each, counted and not timed: the waits are in every role's inner loop,
// and their code has to stay small), or until *fail is set; sets *fail when it
// gives up.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* fail, int tries) {
  if (mbar_try_wait(bar, parity)) return true;  // (a first try without the hint: 7% on long prompts)
  while (!mbar_try_wait_sleep(bar, parity, 20000u))
    if (*fail != 0 || --tries < 0) {
      *fail = 1;
      return false;
    }
  return true;
}
constexpr int kTries = 1 << 19, kTestTries = 1 << 12;  // under the stall flag: a test's patience

// fp32 pairs in one register pair: the FMA pipe takes both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two values rounded to 16 bits, lo in the low half.
template <bool FP16>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  uint32_t r;
  if (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row's softmax state: the reference maximum m (in score units), the sum l
// of exp2(c (s - m) + kShift) so far.
struct RowState {
  float m = -INFINITY, l = 0.f;
};

// 16-bit floating point with 5 exponent bits (fp16) loses probabilities below
// 2^-24; raised by 2^7 they keep their bits down to 2^-31, and with the 2^8
// that the reference maximum may lag they stay below 2^15.
template <bool FP16>
__host__ __device__ constexpr float shift_log2() { return FP16 ? 7.f : 0.f; }

// Multiplies this warp's lanes of the D accumulator columns at t_o by alpha.
template <int D>
__device__ __forceinline__ void scale_rows(uint32_t t_o, float alpha) {
  const uint64_t a2 = pair(alpha, alpha);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(t_o + 32 * c, o);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x, y;
      unpair(mul2(pair(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), x, y);
      o[i] = __float_as_uint(x);
      o[i + 1] = __float_as_uint(y);
    }
    tmem_st_32x32b_x32p(t_o + 32 * c, o);
  }
}

// One softmax step of this warp's 32 rows: scores in columns t_s, columns at
// or past `seen` hidden (seen >= 128: none), probabilities written over the
// scores as 16-bit pairs.  PERM(i) gives the score column of operand position
// i (a permutation within the tile).  c: scale times log2(e).
//
// The output sums are rescaled only when a row's maximum has grown by more
// than 2^8 since its reference was taken: until then exp2 stays below 2^8 and
// nothing is lost in fp32, and nearly every tile is spared the pass over D
// accumulator columns.  Each row decides for itself, so that a row's result
// does not depend on its neighbours.
// sums_ready() returns when the output sums hold every earlier tile.
template <int D, bool FP16, class Perm, class Ready>
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, float c, int seen, bool first, RowState& st,
                                             Perm perm, Ready sums_ready) {
  uint32_t s[kTile];
  float mx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mx[i] = tmem_ld_max_32x32b_x32(t_s + 32 * i, s + 32 * i);
  tc_wait_ld();
  if (__builtin_expect(__any_sync(0xffffffffu, seen < kTile), 0)) {  // hidden scores: out of the row and of its maximum
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      s[i] = i < seen ? s[i] : 0xff800000u;
      mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
    }
  }
  const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  const bool grow = (mt - st.m) * c > kRescaleLog2;  // also the row's first finite score (m = -inf)
  float alpha = 1.f;
  if (grow) {
    alpha = ex2((st.m - mt) * c);
    st.m = mt;
    st.l *= alpha;
  }
  if (__builtin_expect(!first && __any_sync(0xffffffffu, grow), 0)) {
    sums_ready();
    scale_rows<D>(t_o, alpha);
  }
  const float off = (st.m == -INFINITY ? 0.f : -st.m * c) + shift_log2<FP16>();
  const uint64_t c2 = pair(c, c), off2 = pair(off, off);
  uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int a = perm(64 * q + 2 * i), b = perm(64 * q + 2 * i + 1);
      float x, y;
      unpair(fma2(pair(__uint_as_float(s[a]), __uint_as_float(s[b])), c2, off2), x, y);
      x = ex2(x);
      y = ex2(y);
      if (i & 1) sum1 = add2(sum1, pair(x, y));
      else sum0 = add2(sum0, pair(x, y));
      p[i] = round2<FP16>(x, y);
    }
    tmem_st_32x32b_x32p(t_s + 32 * q, p);
  }
  float x, y;
  unpair(add2(sum0, sum1), x, y);
  st.l += x + y;
  tc_wait_st();
}

// softmax_tile in a rolled form, over the columns [col0, col1) (multiples of
// 32): the scores are read 32 columns at a time, twice (the maxima of all,
// downwards, then upwards for the probabilities), by loops of a few hundred
// bytes of code.  For kernels whose other warps run code of their own at the
// same time: the straight-line form then keeps missing the instruction cache.
// Probabilities go to the columns from t_p on, which may be t_s: those of 32
// scores take the place of 16 that were read before.  scores_read() is called
// once the scores may be overwritten.
template <int D, bool FP16, class Perm, class Ready, class Read>
__device__ __forceinline__ void softmax_tile_rolled(uint32_t t_s, uint32_t t_p, uint32_t t_o, int col0, int col1, float c,
                                                    int seen, bool first, RowState& st, Perm perm, Ready sums_ready,
                                                    Read scores_read) {
  const bool hidden = __any_sync(0xffffffffu, seen < col1);
  uint32_t s[32];
  float mt = -INFINITY;
#pragma unroll 1
  for (int b = col1 - 32; b >= col0; b -= 32) {
    float m = tmem_ld_max_32x32b_x32(t_s + b, s);
    tc_wait_ld();
    if (__builtin_expect(hidden, 0)) {
      m = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        s[i] = b + i < seen ? s[i] : 0xff800000u;
        m = fmaxf(m, __uint_as_float(s[i]));
      }
    }
    mt = fmaxf(mt, m);
  }
  const bool grow = (mt - st.m) * c > kRescaleLog2;
  float alpha = 1.f;
  if (grow) {
    alpha = ex2((st.m - mt) * c);
    st.m = mt;
    st.l *= alpha;
  }
  if (__builtin_expect(!first && __any_sync(0xffffffffu, grow), 0)) {
    sums_ready();
    scale_rows<D>(t_o, alpha);
  }
  const float off = (st.m == -INFINITY ? 0.f : -st.m * c) + shift_log2<FP16>();
  const uint64_t c2 = pair(c, c), off2 = pair(off, off);
  uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
  for (int b = col0; b < col1; b += 32) {
    uint32_t p[16];
    if (b != col0) {  // (the first columns are still here)
      tmem_ld_32x32b_x32(t_s + b, s);
      tc_wait_ld();
      if (__builtin_expect(hidden, 0)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = b + i < seen ? s[i] : 0xff800000u;
      }
    }
    if (b + 32 == col1) scores_read();
    // neighbouring columns lie in register pairs, as the packed arithmetic wants
    // them; the operand's order is made as they are rounded
    float e[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      unpair(fma2(pair(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, off2), e[2 * i], e[2 * i + 1]);
      e[2 * i] = ex2(e[2 * i]);
      e[2 * i + 1] = ex2(e[2 * i + 1]);
      if (i & 1) sum1 = add2(sum1, pair(e[2 * i], e[2 * i + 1]));
      else sum0 = add2(sum0, pair(e[2 * i], e[2 * i + 1]));
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = round2<FP16>(e[perm(2 * i)], e[perm(2 * i + 1)]);
    tmem_st_32x32b_x16(t_p + (b >> 1), p);
  }
  float x, y;
  unpair(add2(sum0, sum1), x, y);
  st.l += x + y;
  tc_wait_st();
}

// The MMAs of one product of 128-row tiles, issued by one thread.  (Loops and
// not straight-line code: the issuing thread runs through it alone, and each
// line of code that it has to fetch delays the tensor cores.)
//
// S = Q K^T: `chunks` chunks of 64 channels of Q (16 KB each) and K; a, b: low
// descriptor words.
template <int CHUNKS>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
#pragma unroll 1
  for (int c = 0; c < CHUNKS; ++c, a += 1024, b += 1024) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16_ss_sw128(d, a + 2 * k, b + 2 * k, idesc, add || c + k > 0);
  }
}
// O += P V: P (tensor-memory columns from a) times V in 8 steps of 16 tokens,
// four steps `step` descriptor units apart and then `half` on to the next four.
__device__ __forceinline__ void issue_values(uint32_t d, uint32_t a, uint32_t b, uint32_t step, uint32_t half,
                                             uint32_t idesc, bool add) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c, a += 32, b += half) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f16_ts_sw128(d, a + 8 * k, b + step * k, idesc, add || c + k > 0);
  }
}

// lse in natural units.
template <bool FP16>
__device__ __forceinline__ float row_lse(const RowState& st, float c) {
  return st.l > 0.f || isnan(st.l) ? (st.m * c + log2f(st.l) - shift_log2<FP16>()) * 0.6931471805599453f : -INFINITY;
}

}  // namespace rows
}  // namespace kvq
