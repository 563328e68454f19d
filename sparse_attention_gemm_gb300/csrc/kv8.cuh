// kv8.cuh -- the 8-bit block cache: where a token's row lives, and the
// conversions between bf16 values, E4M3 codes and their block scales.
//
// Codes uint8 [n_blocks, block, Hc, D], scale fp32 [n_blocks, Hc]; the value
// of a code is e4m3(code) * scale[its block, its head].
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dsa {

// Where the rows of a batch live.  Sequence b holds packed tokens cu[b] ..
// cu[b+1]-1 at positions pos[b] + (t - cu[b]); position p is row
// table[b, p >> lb] * block + (p & (block - 1)), or row p without a table.
struct Kv8Geom {
  const int32_t* cu;
  const int32_t* pos;    // NULL: 0 with a table, cu[b] without
  const int32_t* table;  // [n_seqs, max_blocks] or NULL
  int n_seqs, T, lb, n_blocks, max_blocks;
  // Sequence b is cu[b * step] .. cu[(b + 1) * step] - 1.  With neither table nor pos, row t
  // of the batch is row t of the cache whatever its sequence: n_seqs is 1 then, and
  // step the number of sequences.
  int step = 1;
};

// The sequence's first position.
__device__ __forceinline__ int64_t kv8_pos0(const Kv8Geom& g, int b, int cu_b) {
  return g.pos ? __ldg(g.pos + b) : (g.table ? 0 : cu_b);
}

// Physical block of logical block `page` of sequence b, -1 where there is none.
__device__ __forceinline__ int kv8_block(const Kv8Geom& g, int b, int64_t page) {
  if (page < 0) return -1;
  int64_t phys = page;
  if (g.table) {
    if (page >= g.max_blocks) return -1;
    phys = __ldg(g.table + static_cast<int64_t>(b) * g.max_blocks + page);
  }
  return phys >= 0 && phys < g.n_blocks ? static_cast<int>(phys) : -1;
}

// Row of position p of sequence b, -1 where there is none.
__device__ __forceinline__ int kv8_row(const Kv8Geom& g, int b, int64_t p) {
  const int blk = kv8_block(g, b, p >> g.lb);
  return blk < 0 ? -1 : (blk << g.lb) + static_cast<int>(p & ((1 << g.lb) - 1));
}

// Largest b with cu[b] <= t (binary search); the caller checks t < cu[n_seqs].
__device__ __forceinline__ int kv8_seq(const int32_t* __restrict__ cu, int n_seqs, int t) {
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The same by a converged warp, 32 probes a step: a load's latency per factor of 32 in n_seqs.
__device__ __forceinline__ int kv8_seq_warp(const int32_t* __restrict__ cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at < n && __ldg(cu + lo + at) <= t);
    const int k = le ? (31 - __clz(le)) * step : 0;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

// Cache row of packed token t; -1 not mapped, -2 behind the last sequence.
__device__ __forceinline__ int row_of_token(const Kv8Geom& g, int64_t t) {
  if (t >= g.T || t < __ldg(g.cu) || t >= __ldg(g.cu + g.n_seqs * g.step)) return -2;
  const int b = kv8_seq(g.cu, g.n_seqs, static_cast<int>(t));
  const int c = __ldg(g.cu + b);
  return kv8_row(g, b, kv8_pos0(g, b, c) + (t - c));
}

// Sequences of packed tokens as a converged warp looks them up: up to 32 are loaded at once, with
// their positions, and a token's is a ballot away; of more, every step-th, then a search between two.
struct SeqFinder {
  int n, step, c, p, end;

  __device__ __forceinline__ explicit SeqFinder(const Kv8Geom& g) : n(g.n_seqs), step((g.n_seqs + 31) >> 5) {
    const int at = static_cast<int>(threadIdx.x & 31) * step;
    c = at < n ? __ldg(g.cu + static_cast<int64_t>(at) * g.step) : INT32_MAX;
    end = __ldg(g.cu + static_cast<int64_t>(n) * g.step);
    p = g.pos && step == 1 && at < n ? __ldg(g.pos + at) : 0;
  }
  // The sequence of token t (the same in all lanes), its cu and its pos (0 without one); false: in none.
  __device__ __forceinline__ bool find(const Kv8Geom& g, int64_t t, int* b, int* cu_b, int* pos_b) const {
    const uint32_t le = __ballot_sync(0xffffffffu, c <= t && t < end);
    if (!le || t >= g.T) return false;
    const int k = 31 - __clz(le);
    *b = k;
    *cu_b = __shfl_sync(0xffffffffu, c, k), *pos_b = __shfl_sync(0xffffffffu, p, k);
    if (step > 1) {
      const int lo = k * step;
      *b = lo + kv8_seq_warp(g.cu + lo, min(step, n - lo), static_cast<int>(t));
      *cu_b = __ldg(g.cu + *b);
      *pos_b = g.pos ? __ldg(g.pos + *b) : 0;
    }
    return true;
  }
};

// The cache rows of `tokens` packed tokens from t0 on: -1 not mapped, -2 in no sequence.  A warp a token
// where there are few; a thread a token where there are more (14 tokens of a CTA, 4 sequences: writing
// and reading 16384 rows takes 15.1 us together, and 16.9 with the warps going through two tokens each).
template <int kThreads>
__device__ __forceinline__ void rows_of_tokens(const Kv8Geom& g, int64_t t0, int tokens, int* rows) {
  if (tokens > kThreads / 32) {
    for (int k = threadIdx.x; k < tokens; k += kThreads) rows[k] = row_of_token(g, t0 + k);
    return;
  }
  const int k = threadIdx.x >> 5;
  if (k >= tokens) return;
  int b, c, p;
  const bool found = SeqFinder(g).find(g, t0 + k, &b, &c, &p);
  const int row = found ? kv8_row(g, b, (g.pos ? p : (g.table ? 0 : c)) + (t0 + k - c)) : -2;
  if ((threadIdx.x & 31) == 0) rows[k] = row;
}

// n / d for n * d < 2^32, magic = magic_of(d): n * (2^32 / d + 1) exceeds n / d *
// 2^32 by at most n, less than the 2^32 / d that would reach the next quotient.
// 0 stands for d = 1, and 1 gives 0 for every n.
__device__ __forceinline__ int fast_div(int n, uint32_t magic) {
  return magic ? static_cast<int>(__umulhi(n, magic)) : n;
}
inline uint32_t magic_of(int d) { return d == 1 ? 0 : static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint32_t>(d)) + 1; }

// Scale of values up to `amax` (>= 0, finite): 2^e with the smallest e that
// keeps amax <= 448 * 2^e, at least 2^-126.  448 = 1.75 * 2^8, so e follows
// from the exponent and from whether the significand exceeds 1.75.  Powers
// of two keep x / s and code * s exact, so that the only rounding is the one to E4M3.
__device__ __forceinline__ float kv8_scale_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// 1 / s of a power of two s in [2^-126, 2^126], exactly.
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Larger of two pairs of 16-bit unsigned numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitudes of the eight bf16 values of a piece, kept in two lanes as
// bits without the sign (monotonic; 0x7F80 and above: infinity or NaN).
__device__ __forceinline__ uint32_t amax_bf16x8(uint4 v, uint32_t m) {
  m = max_u16x2(m, v.x & 0x7FFF7FFFu);
  m = max_u16x2(m, v.y & 0x7FFF7FFFu);
  m = max_u16x2(m, v.z & 0x7FFF7FFFu);
  return max_u16x2(m, v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t larger_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// Two values -> two E4M3 codes (x0 in the low byte), to nearest even, beyond
// +-448 the largest code of that sign, NaN stays NaN.
__device__ __forceinline__ uint16_t e4m3x2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
__device__ __forceinline__ uint16_t e4m3x2_h2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
// The same to E5M2.
__device__ __forceinline__ uint16_t e5m2x2_h2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
// Two codes -> two halves, exactly.
__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ float2 f2_of_e4m3x2(uint16_t c) {
  const uint32_t h = h2_of_e4m3x2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace dsa
