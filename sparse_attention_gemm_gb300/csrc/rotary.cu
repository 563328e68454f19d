// rotary.cu -- rotary positions of query and key rows.
//
// A row's R values are pairs (a, b): elements (2i, 2i + 1), or (i, i + R / 2).
// At position p, pair i turns by p * f_i:
//   (a, b) -> mul * (a cos - b sin, a sin + b cos),
// and by the opposite angle in the adjoint, which is the gradient's pass.
//
// Angles: f_i / (2 pi) is taken as a fraction of a turn in 64-bit fixed point, so that
// p times it modulo a turn is one integer product: the angle of position p is off
// by p * 2^-61 of f_i and p * 2^-64 of a turn, and by 2^-25 of half a turn when it becomes fp32.
//
// A CTA works out its tokens' cosines and sines once, for all their heads, while the first loads
// are under way.  The rows' bytes bound it: 16,384 tokens of 64 + 1 rows of 64, halves, 272 MB, take
// 45 us (6.1 TB/s), pairs 47; rows that are the last 64 of 576 the same 48 and 50; 4096 tokens of
// 24 + 1 heads of 256 21 us (4.9 TB/s).  32 tokens take 2.6 us: the chain from the sequence's
// offsets to the angles, not the bytes.
#include <algorithm>
#include <climits>
#include <cmath>

#include "kv8.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;   // of a CTA
constexpr int kMaxAngles = 2048;  // cosines and sines that a CTA keeps
constexpr int kAhead = 4;        // units of a thread in flight

struct Side {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  int64_t xt, xh, yt, yh;  // strides of a token and a head, in elements
};

struct Params {
  Side a, b;
  const double* f;
  dsa::Kv8Geom g;
  int H, H2, R, tokens;
  int rows;              // of a token, that a CTA takes: all of them, or with one token a part
  int per;               // units of a row
  uint32_t m_token, m_row, m_half;  // dsa::fast_div by a token's units, a row's and R / 2
  float mul, sign;
  uint32_t* status;
};

// f / (2 pi) modulo 1, in units of 2^-64.  Of f = m 2^(e - 52): m times 2^11 / (2 pi), its
// whole part, is shifted by e + 1 (FP64 units are few here, and this is exact to 2^-61 of f).
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>(bits >> 52 & 0x7FF) - 1023;
  if (e == -1023) return 0;  // below 2^-1022
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (1ull << 52);
  const uint64_t x = __umul64hi(m << 11, 0x28BE60DB9391054Aull);  // 2^64 / (2 pi)
  const int s = e + 1;
  const uint64_t r = s >= 64 || s <= -64 ? 0 : s >= 0 ? x << s : x >> -s;
  return bits >> 63 ? 0 - r : r;
}

// A unit: 16 bytes of 4 pairs, or two times 16 bytes, half a row apart, of 8 pairs.
template <bool PAIRS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Params p) {
  constexpr int kWords = PAIRS ? 1 : 2;
  // mul * cos, mul * sin of [token][pair of a unit][unit]: neighbouring units read neighbouring words
  // (unit by unit they met in the same banks: R = 256 took 36 us where it takes 21)
  __shared__ float2 turn[kMaxAngles];
  __shared__ int64_t place[kMaxTokens];  // position, or kNone
  constexpr int64_t kNone = INT64_MIN;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int half = p.R >> 1, row0 = blockIdx.y * p.rows, rows = min(p.rows, p.H + p.H2 - row0);
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.g.T - t0));
  const int n = n_tok * rows * p.per;
  uint4 v[kAhead][kWords];
  auto where = [&](int i, int* token, int* u, const Side** s, int* h) {
    const int k = dsa::fast_div(i, p.m_token), rest = i - k * rows * p.per;
    const int in = dsa::fast_div(rest, p.m_row), r = row0 + in;
    *token = k;
    *u = rest - in * p.per;
    *s = r < p.H ? &p.a : &p.b;
    *h = r < p.H ? r : r - p.H;
  };
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      if (i < n) {
        int k, u, h;
        const Side* s;
        where(i, &k, &u, &s, &h);
        const __nv_bfloat16* src = s->x + (t0 + k) * s->xt + h * s->xh + u * 8;
#pragma unroll
        for (int w = 0; w < kWords; ++w) v[j][w] = __ldcs(reinterpret_cast<const uint4*>(src + w * half));
      }
    }
  };
  load(threadIdx.x);  // under way while the angles are worked out
  {
    const dsa::SeqFinder seqs(p.g);
    for (int k = threadIdx.x >> 5; k < n_tok; k += kThreads / 32) {
      int b, c, pos;
      const bool inside = seqs.find(p.g, t0 + k, &b, &c, &pos);
      if ((threadIdx.x & 31) == 0 && dsa::check(k < kMaxTokens, p.status)) place[k] = inside ? pos + (t0 + k - c) : kNone;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
    const int k = dsa::fast_div(i, p.m_half), j = i - k * half;
    const uint64_t angle = static_cast<uint64_t>(place[k]) * turns_of(__ldg(p.f + j)) + 0x80000000ull;
    float sn, cs;  // the upper half as a signed number is the angle in 2^-31 half turns
    sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &sn, &cs);
    constexpr int kPairs = PAIRS ? 4 : 8;  // of a unit
    if (dsa::check(k < n_tok && (k + 1) * half <= kMaxAngles && j / kPairs < p.per, p.status))
      turn[k * half + j % kPairs * p.per + j / kPairs] = make_float2(cs * p.mul, sn * p.mul * p.sign);
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kAhead) {
    if (i0 != threadIdx.x) load(i0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      if (i >= n) continue;
      int k, u, h;
      const Side* s;
      where(i, &k, &u, &s, &h);
      if (!dsa::check(k < n_tok && u < p.per && h < (s == &p.a ? p.H : p.H2), p.status) || place[k] == kNone) continue;
      const float2* at = turn + k * half + u;
      __nv_bfloat16* dst = s->y + (t0 + k) * s->yt + h * s->yh + u * 8;
      uint32_t* w0 = reinterpret_cast<uint32_t*>(&v[j][0]);
      auto pack2 = [](float lo, float hi) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
      };
      auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
      auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = lo(w0[e]), b = hi(w0[e]);
          const float2 c = at[e * p.per];
          w0[e] = pack2(a * c.x - b * c.y, a * c.y + b * c.x);
        }
      } else {
        uint32_t* w1 = reinterpret_cast<uint32_t*>(&v[j][kWords - 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = at[2 * e * p.per], d = at[(2 * e + 1) * p.per];
          const float a0 = lo(w0[e]), a1 = hi(w0[e]), b0 = lo(w1[e]), b1 = hi(w1[e]);
          w0[e] = pack2(a0 * c.x - b0 * c.y, a1 * d.x - b1 * d.y);
          w1[e] = pack2(a0 * c.y + b0 * c.x, a1 * d.y + b1 * d.x);
        }
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) *reinterpret_cast<uint4*>(dst + w * half) = v[j][w];
    }
  }
}

// Whether n0 x n1 rows of R values, s0 and s1 apart, have no value in common.
bool apart(int64_t s0, int n0, int64_t s1, int n1, int R) {
  if (n0 <= 1) return n1 <= 1 || s1 >= R;
  if (n1 <= 1) return s0 >= R;
  const bool first = s0 < s1;
  const int64_t in = first ? s0 : s1, out = first ? s1 : s0, n = first ? n0 : n1;
  return in >= R && (out - R) / (n - 1) >= in;
}

}  // namespace

extern "C" int dsa_rotary_inv_freq(int R, double base, int scaling, double factor, int64_t first, double beta_fast,
                                   double beta_slow, double* inv_freq, float* mul) {
  dsa::clear_error();
  const char* fn = "dsa_rotary_inv_freq";
  if (R < 2 || R > DSA_ROTARY_MAX_DIM || R % 2 != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: R must be even, in [2, %d]", fn, DSA_ROTARY_MAX_DIM);
  if (!(base > 1.0) || !std::isfinite(base)) return dsa::set_error(DSA_ERR_VALUE, "%s: base must be finite and > 1", fn);
  if (scaling != DSA_ROTARY_PLAIN && scaling != DSA_ROTARY_LINEAR && scaling != DSA_ROTARY_NTK &&
      scaling != DSA_ROTARY_YARN)
    return dsa::set_error(DSA_ERR_VALUE, "%s: unknown scaling %d", fn, scaling);
  if (scaling != DSA_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: factor must be finite and >= 1", fn);
  if (scaling == DSA_ROTARY_NTK && R < 4) return dsa::set_error(DSA_ERR_VALUE, "%s: NTK scaling needs R >= 4", fn);
  if (scaling == DSA_ROTARY_YARN &&
      (first < 1 || !(beta_fast > beta_slow) || !(beta_slow > 0.0) || !std::isfinite(beta_fast)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: YaRN needs first >= 1 and beta_fast > beta_slow > 0", fn);
  if (!inv_freq || !mul) return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  const int half = R / 2;
  double b = base;
  if (scaling == DSA_ROTARY_NTK) b *= std::pow(factor, static_cast<double>(R) / (R - 2));
  double lo = 0, hi = 0;
  if (scaling == DSA_ROTARY_YARN) {
    // the pair that makes `turns` turns over the first positions
    auto pair_of = [&](double turns) {
      return half * std::log(static_cast<double>(first) / (turns * 6.283185307179586477)) / std::log(base);
    };
    lo = std::max(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::min(std::ceil(pair_of(beta_slow)), static_cast<double>(R - 1));
    if (pair_of(beta_slow) < 0.0) lo = hi = -1.0;  // no pair makes as many turns: the blend ends before the first
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(b, -static_cast<double>(i) / half);
    if (scaling == DSA_ROTARY_LINEAR) {
      inv_freq[i] = f / factor;
    } else if (scaling == DSA_ROTARY_YARN) {
      const double keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      inv_freq[i] = f * keep + f / factor * (1.0 - keep);
    } else {
      inv_freq[i] = f;
    }
  }
  *mul = scaling == DSA_ROTARY_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return DSA_OK;
}

extern "C" int dsa_rotary(const void* x, int64_t x_token, int64_t x_head, int H, const void* x2, int64_t x2_token,
                          int64_t x2_head, int H2, const double* inv_freq, const int32_t* cu_seqlens,
                          const int32_t* pos, int n_seqs, int T, int R, int interleaved, int inverse, float mul,
                          void* y, int64_t y_token, int64_t y_head, void* y2, int64_t y2_token, int64_t y2_head,
                          cudaStream_t stream) {
  dsa::clear_error();
  const char* fn = "dsa_rotary";
  if (T < 0 || n_seqs < 1 || H < 1 || H2 < 0 || static_cast<int64_t>(H) + H2 > DSA_ROTARY_MAX_HEADS)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need T >= 0, n_seqs >= 1, H >= 1, H2 >= 0 and H + H2 <= %d", fn,
                          DSA_ROTARY_MAX_HEADS);
  if (R < 16 || R > DSA_ROTARY_MAX_DIM || R % 16 != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: R must be a multiple of 16 in [16, %d]", fn, DSA_ROTARY_MAX_DIM);
  if (!(mul > -INFINITY && mul < INFINITY)) return dsa::set_error(DSA_ERR_VALUE, "%s: mul must be finite", fn);
  if (!inv_freq || !cu_seqlens || (T > 0 && (!x || !y || (H2 > 0 && (!x2 || !y2)))))
    return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  const int64_t strides[8] = {x_token, x_head, y_token, y_head, x2_token, x2_head, y2_token, y2_head};
  for (int i = 0; i < (H2 > 0 ? 8 : 4); ++i)
    if (strides[i] % 8 != 0) return dsa::set_error(DSA_ERR_VALUE, "%s: strides must be multiples of 8 elements", fn);
  if (!apart(y_token, T, y_head, H, R) || (H2 > 0 && !apart(y2_token, T, y2_head, H2, R)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: rows of the result must not overlap", fn);
  if ((x == y && (x_token != y_token || x_head != y_head)) ||
      (H2 > 0 && x2 == y2 && (x2_token != y2_token || x2_head != y2_head)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: in place, the strides of both sides must be equal", fn);
  if (H2 > 0 && T > 0 && (y == y2 || y == x2 || y2 == x))
    return dsa::set_error(DSA_ERR_VALUE, "%s: y and y2 must not be one tensor, nor the other tensor's input", fn);
  if (!dsa::aligned(x, 16) || !dsa::aligned(y, 16) || !dsa::aligned(inv_freq, 8) ||
      (H2 > 0 && (!dsa::aligned(x2, 16) || !dsa::aligned(y2, 16))))
    return dsa::set_error(DSA_ERR_VALUE, "%s: rows must be 16-byte aligned, inv_freq 8-byte aligned", fn);
  int sms = 0;
  int rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  Params p{};
  p.a = Side{static_cast<const __nv_bfloat16*>(x), static_cast<__nv_bfloat16*>(y), x_token, x_head, y_token, y_head};
  if (H2 > 0)
    p.b = Side{static_cast<const __nv_bfloat16*>(x2), static_cast<__nv_bfloat16*>(y2), x2_token, x2_head, y2_token, y2_head};
  p.f = inv_freq;
  p.g = dsa::Kv8Geom{cu_seqlens, pos, nullptr, n_seqs, T, 0, 0, 0};
  p.H = H, p.H2 = H2, p.R = R;
  p.per = interleaved ? R / 8 : R / 16;
  p.mul = mul, p.sign = inverse ? -1.f : 1.f;
  p.status = dsa::device_status_ptr();
  // Tokens of a CTA: one round of its threads' units, or two rounds where one token takes more than
  // half of one (16,384 tokens of 65 rows of 64, pairs: 47 us, and 57 with one token a CTA; rounds
  // of 20 rows, where three tokens share one, gain nothing from two: 17.0 us), and two CTAs an SM at
  // least.
  const int per_token = (H + H2) * p.per, round = kAhead * kThreads;
  const int units = per_token > round / 2 ? 2 * round : round;
  int tokens = std::min({kMaxTokens, kMaxAngles / (R / 2), std::max(1, units / per_token)});
  tokens = std::max(1, std::min(tokens, T / (2 * sms)));
  p.tokens = tokens;
  // Few tokens: a token's rows go to several CTAs, a unit a thread, up to four CTAs an SM (32 tokens of 129
  // rows of 64, pairs: 2.6 us, and 3.5 in one CTA a token; 19 of 129 rows of 256: 2.8, and 6.8; 150 of them: 5.1,
  // with one or eight CTAs an SM 6.9 and 6.2).
  int parts = 1;
  if (tokens == 1) parts = std::max(1, std::min(per_token / kThreads, 4 * sms / T));
  p.rows = (H + H2 + parts - 1) / parts;
  p.m_token = tokens == 1 ? 1 : dsa::magic_of(per_token);
  p.m_row = dsa::magic_of(p.per);
  p.m_half = dsa::magic_of(R / 2);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(T) + tokens - 1) / tokens),
                  static_cast<unsigned>((H + H2 + p.rows - 1) / p.rows));
  if (interleaved)
    rotary_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    rotary_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return dsa::launch_error("rotary_kernel");
}
