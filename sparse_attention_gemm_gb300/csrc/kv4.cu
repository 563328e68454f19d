// kv4.cu -- writing bf16 rows into the 4-bit block cache and reading them back.
//
// Write.  Per 32 elements of a row, with a = max |x| over their finite values:
// e the smallest integer with a <= 6 * 2^e, in [-126, 125]; codes e2m1(x / 2^e).
// With a NaN among the 32 the scale byte is 255 and the codes 0.
// Read.  out = e2m1(code) * 2^e, a bf16 value; NaN for byte 255.
//
// A lane of the writer takes 16 elements (32 bytes of bf16, 8 of codes), two lanes the
// 32 of a scale: with 8 elements a lane, and its scale worked out by four lanes, it
// took 22.6 us for 65,536 rows of 576 where it takes 16.4 (96 MB, 5.8 TB/s).  A lane
// of the reader takes 8 (18.4 us, 5.2 TB/s).  Calls of a few tokens are one chain of
// loads -- sequence, page, row -- 5 us from end to end.  Nothing of a row depends on another, so rows of a block are written
// in any order by any call.
#include <algorithm>
#include <climits>

#include "kv4.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // pieces of a thread in flight
constexpr int kMaxTokens = 64;

__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const __nv_bfloat16* __restrict__ src, const dsa::Kv8Geom g, int Hc, int D, int tokens,
                     uint32_t magic_row, uint8_t* __restrict__ cache, uint8_t* __restrict__ scale, uint32_t* status) {
  constexpr int kAhead = 2;  // pieces here are 16 values: two lanes have a scale's 32
  __shared__ int rows[kMaxTokens];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int per = Hc * (D >> 4);  // pieces of a token
  const int n = static_cast<int>(min(static_cast<int64_t>(tokens), g.T - t0)) * per;
  const uint4* s0 = reinterpret_cast<const uint4*>(src) + t0 * per * 2;
  uint4 v[kAhead][2];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
#pragma unroll
      for (int h = 0; h < 2; ++h) v[j][h] = i < n ? __ldg(s0 + 2 * i + h) : make_uint4(0, 0, 0, 0);
    }
  };
  load(threadIdx.x);
  dsa::rows_of_tokens<kThreads>(g, t0, tokens, rows);
  __syncthreads();
  // n is even: the two lanes of a scale are in or out together.  Every lane of a warp makes the
  // same trips, for the shuffles.
  for (int i0 = threadIdx.x; i0 - static_cast<int>(threadIdx.x) < n; i0 += kThreads * kAhead) {
    if (i0 != threadIdx.x) load(i0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      uint32_t m = dsa::amax_bf16x8(v[j][1], dsa::amax_bf16x8(v[j][0], 0));
      m = dsa::larger_half(dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1)));
      float x[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {v[j][h].x, v[j][h].y, v[j][h].z, v[j][h].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[h][2 * k] = __uint_as_float(w[k] << 16);
          x[h][2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
      const bool nan = m > 0x7F80u;  // of one of the 32: in both lanes
      if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
        uint32_t f = 0;  // the largest finite one
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t u = (__float_as_uint(x[k >> 3][k & 7]) >> 16) & 0x7FFFu;
          f = max(f, u < 0x7F80u ? u : 0u);
        }
        m = max(f, __shfl_xor_sync(0xffffffffu, f, 1));
      }
      if (i >= n) continue;
      const int t = dsa::fast_div(i, magic_row);
      if (!dsa::check(t < tokens, status)) continue;
      const int row = rows[t];
      if (row < 0 || !dsa::check(row < (g.n_blocks << g.lb), status)) continue;
      const uint32_t e = dsa::kv4_scale_of(m);
      const float inv = dsa::kv4_inverse(e);
      const int64_t at = static_cast<int64_t>(row) * per + (i - t * per);
      reinterpret_cast<uint2*>(cache)[at] =
          nan ? make_uint2(0, 0) : make_uint2(dsa::e2m1x8(x[0], inv), dsa::e2m1x8(x[1], inv));
      if ((i & 1) == 0) scale[at >> 1] = static_cast<uint8_t>(nan ? dsa::kMxNan : e);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const uint8_t* __restrict__ cache, const uint8_t* __restrict__ scale, const dsa::Kv8Geom g, int Hc,
                    int D, int tokens, uint32_t magic_row, __nv_bfloat16* __restrict__ out, uint32_t* status) {
  __shared__ int rows[kMaxTokens];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  dsa::rows_of_tokens<kThreads>(g, t0, tokens, rows);
  __syncthreads();
  const int per = Hc * (D >> 3);
  const int n = static_cast<int>(min(static_cast<int64_t>(tokens), g.T - t0)) * per;
  uint4* o0 = reinterpret_cast<uint4*>(out) + t0 * per;
  for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kAhead) {
    uint32_t w[kAhead], e[kAhead], live = 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      w[j] = 0, e[j] = 127;
      if (i < n) {
        const int t = dsa::fast_div(i, magic_row), row = dsa::check(t < tokens, status) ? rows[t] : -2;
        if (row != -2) live |= 1u << j;
        if (row >= 0 && dsa::check(row < (g.n_blocks << g.lb), status)) {
          const int64_t at = static_cast<int64_t>(row) * per + (i - t * per);
          w[j] = __ldcs(reinterpret_cast<const uint32_t*>(cache) + at);
          e[j] = __ldg(scale + (at >> 2));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      uint32_t o[4];
      dsa::bf8_of_e2m1(w[j], e[j], o);
      if (live >> j & 1) o0[i0 + j * kThreads] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Tokens per CTA: one round of its threads' pieces, fewer where the batch would not fill the device
// twice, two rounds where that leaves six CTAs an SM (32,768 rows of 576 written and read: 17.8 us, and 19.1 with
// one round; 16,384: 11.6 with one, 11.9 with two).  fast_div: several tokens have 2048 pieces at most.
int tokens_per_cta(int T, int Hc, int D, int sms) {
  const int round = kThreads * kAhead / (Hc * (D / 8));
  const int n = std::max(1, std::min(kMaxTokens, T / std::max(1, 2 * round) >= 6 * sms ? 2 * round : round));
  return std::max(1, std::min(n, T / (2 * sms)));
}

unsigned ctas_of(int T, int tokens) { return static_cast<unsigned>((static_cast<int64_t>(T) + tokens - 1) / tokens); }

int check_args(const char* fn, const void* rows, const void* cache, const void* scale, const int32_t* cu,
               const int32_t* pos, const int32_t* table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
               int max_blocks, dsa::Kv8Geom* g) {
  if (n_seqs < 1 || T < 0 || Hc < 1 || n_blocks < 1)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need n_seqs >= 1, T >= 0, Hc >= 1, n_blocks >= 1", fn);
  if (D < 32 || D > DSA_KV8_MAX_DIM || D % 32 != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: D must be a multiple of 32 in [32, %d]", fn, DSA_KV8_MAX_DIM);
  if (Hc > DSA_KV8_MAX_HEADS)
    return dsa::set_error(DSA_ERR_VALUE, "%s: Hc must be at most %d", fn, DSA_KV8_MAX_HEADS);
  if (block < 1 || block > DSA_KV8_MAX_BLOCK || (block & (block - 1)) != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: block must be a power of two in [1, %d]", fn, DSA_KV8_MAX_BLOCK);
  if (static_cast<int64_t>(n_blocks) * block > INT_MAX)
    return dsa::set_error(DSA_ERR_VALUE, "%s: n_blocks * block exceeds the int32 row range", fn);
  if (table && max_blocks < 1) return dsa::set_error(DSA_ERR_VALUE, "%s: a block table needs max_blocks >= 1", fn);
  if (!cu || !cache || !scale || (T > 0 && !rows)) return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  if (!dsa::aligned(rows, 16) || !dsa::aligned(cache, 16))
    return dsa::set_error(DSA_ERR_VALUE, "%s: the bf16 rows and the cache must be 16-byte aligned", fn);
  int lb = 0;
  while ((1 << lb) < block) ++lb;
  const bool one = !pos && !table;
  *g = dsa::Kv8Geom{cu, pos, table, one ? 1 : n_seqs, T, lb, n_blocks, max_blocks, one ? n_seqs : 1};
  return DSA_OK;
}

}  // namespace

extern "C" int dsa_kv4_write(const void* src, const int32_t* cu_seqlens, const int32_t* pos,
                             const int32_t* block_table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
                             int max_blocks, void* cache, uint8_t* scale, cudaStream_t stream) {
  dsa::clear_error();
  dsa::Kv8Geom g;
  int rc = check_args("dsa_kv4_write", src, cache, scale, cu_seqlens, pos, block_table, n_seqs, T, Hc, D, block,
                      n_blocks, max_blocks, &g);
  if (rc != DSA_OK) return rc;
  int sms = 0;
  rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  const int tokens = tokens_per_cta(T, Hc, D, sms);
  kv4_write_kernel<<<ctas_of(T, tokens), kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(src), g, Hc, D, tokens, tokens == 1 ? 1 : dsa::magic_of(Hc * (D / 16)),
      static_cast<uint8_t*>(cache), scale, dsa::device_status_ptr());
  return dsa::launch_error("kv4_write_kernel");
}

extern "C" int dsa_kv4_read(const void* cache, const uint8_t* scale, const int32_t* cu_seqlens, const int32_t* pos,
                            const int32_t* block_table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
                            int max_blocks, void* out, cudaStream_t stream) {
  dsa::clear_error();
  dsa::Kv8Geom g;
  int rc = check_args("dsa_kv4_read", out, cache, scale, cu_seqlens, pos, block_table, n_seqs, T, Hc, D, block,
                      n_blocks, max_blocks, &g);
  if (rc != DSA_OK) return rc;
  int sms = 0;
  rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  const int tokens = tokens_per_cta(T, Hc, D, sms);
  kv4_read_kernel<<<ctas_of(T, tokens), kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(cache), scale, g, Hc, D, tokens, tokens == 1 ? 1 : dsa::magic_of(Hc * (D / 8)),
      static_cast<__nv_bfloat16*>(out), dsa::device_status_ptr());
  return dsa::launch_error("kv4_read_kernel");
}
