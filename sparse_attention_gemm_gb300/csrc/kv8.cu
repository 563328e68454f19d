// kv8.cu -- writing bf16 rows into the 8-bit block cache and reading them back.
//
// Write.  For each (block, head) that receives rows, with a = max |x| over
// their finite values: s_new = 2^e, e the smallest integer with a <= 448 * 2^e.
// A block whose first new row is its first row takes s = s_new; otherwise s =
// max(s_old, s_new), and where that grew the rows before the new ones are
// rounded again as code * (s_old / s).  code = e4m3(x / s).
// Read.  out = bf16(e4m3(code) * s).
#include <algorithm>
#include <climits>

#include "kv8.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowPieces = 4;  // 16-byte pieces in flight per lane of the row writer

constexpr uint32_t kInfinity = 0x7F80u;  // bf16 bits

// Largest finite magnitude of a piece, as bf16 bits (dsa::amax_bf16x8 takes a
// third of the instructions: this is for the rare block that holds infinity or NaN).
__device__ __forceinline__ uint32_t finite_max(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = w[k] & 0x7FFFu, b = (w[k] >> 16) & 0x7FFFu;
    m = max(m, a < 0x7F80u ? a : 0u);
    m = max(m, b < 0x7F80u ? b : 0u);
  }
  return m;
}

// Codes of x / s: a product for a power of two s (every scale that the writer makes), else
// divided.  A block may come with a scale of 2^127, whose inverse is below the normal range.
template <bool kPow2>
__device__ __forceinline__ uint2 codes_of(uint4 v, float s) {
  const bool exact = kPow2 || (__float_as_uint(s) & 0x7FFFFFu) == 0;
  const float inv = kPow2 || s != 0x1p127f ? dsa::pow2_inverse(s) : 0x1p-127f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint16_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xFFFF0000u);
    o[k] = exact ? dsa::e4m3x2(a * inv, b * inv) : dsa::e4m3x2(a / s, b / s);
  }
  return make_uint2(o[0] | (static_cast<uint32_t>(o[1]) << 16), o[2] | (static_cast<uint32_t>(o[3]) << 16));
}

// What one CTA of the block writer works on: a block that receives rows.
struct WriteItem {
  int seq, t0;  // sequence, packed token of the first new row
  int rows;     // new rows
  int first;    // their first row inside the block
  int64_t page; // logical block
};

// The item-th block that receives rows, counted through the sequences.  Every
// warp looks for itself, 32 sequences at a time: no barrier before the rows are read.
__device__ bool find_item(const dsa::Kv8Geom& g, int item, WriteItem* out) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < g.n_seqs; b0 += 32) {
    const int b = b0 + lane;
    int c0 = 0, n = 0, count = 0;
    int64_t p0 = 0;
    if (b < g.n_seqs) {
      c0 = max(__ldg(g.cu + b * g.step), 0);
      n = min(__ldg(g.cu + (b + 1) * g.step), g.T) - c0;
      p0 = kv8_pos0(g, b, c0);
      if (n > 0) count = static_cast<int>(((p0 + n - 1) >> g.lb) - (p0 >> g.lb)) + 1;
    }
    int inc = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    inc += base;
    const uint32_t hit = __ballot_sync(0xffffffffu, item >= inc - count && item < inc);
    if (hit) {
      const int from = __ffs(hit) - 1;
      const int64_t first_pos = __shfl_sync(0xffffffffu, p0, from);
      const int64_t page = (first_pos >> g.lb) + (item - __shfl_sync(0xffffffffu, inc - count, from));
      const int64_t lo = max(first_pos, page << g.lb);
      const int64_t hi = min(first_pos + __shfl_sync(0xffffffffu, n, from), (page + 1) << g.lb);
      out->seq = b0 + from;
      out->t0 = __shfl_sync(0xffffffffu, c0, from) + static_cast<int>(lo - first_pos);
      out->rows = static_cast<int>(hi - lo);
      out->first = static_cast<int>(lo - (page << g.lb));
      out->page = page;
      return true;
    }
    base = __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// One CTA per (block that receives rows, head): a warp per row, the rows' pieces
// read once and kept in registers until the block's scale is known (rows
// beyond what fits are read again).  NP: pieces of a lane and row, kRows: rows
// that a warp keeps -- few for small blocks, so that more CTAs are resident.
// Bound: memory, 3 bytes a value; with few blocks the chain cu_seqlens -> rows ->
// maximum -> codes.  16384 latent rows in pages of 64: 9.6 us (264 CTAs, all resident, 2.9 TB/s), 64
// single rows: 3.6 us.
template <int NP, int kRows>
__global__ void __launch_bounds__(kThreads)
    kv8_write_kernel(const __nv_bfloat16* __restrict__ src, const dsa::Kv8Geom g, int Hc, int D,
                     uint8_t* __restrict__ cache, float* __restrict__ scale) {
  __shared__ uint32_t wmax[kWarps];
  WriteItem it;
  if (!find_item(g, blockIdx.x, &it)) return;
  const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p8 = D >> 3;
  const int64_t ld = static_cast<int64_t>(Hc) * D;
  const __nv_bfloat16* s0 = src + it.t0 * ld + static_cast<int64_t>(h) * D;
  const int block = dsa::kv8_block(g, it.seq, it.page);
  auto load = [&](int r, int k) {
    const int c = k * 32 + lane;
    return c < p8 ? __ldg(reinterpret_cast<const uint4*>(s0 + r * ld) + c) : make_uint4(0, 0, 0, 0);
  };
  uint4 v[kRows][NP];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    if (r < it.rows) {
#pragma unroll
      for (int k = 0; k < NP; ++k) v[i][k] = load(r, k);
    }
  }
  float* sp = scale + static_cast<int64_t>(block < 0 ? 0 : block) * Hc + h;
  const float s_old = it.first > 0 && block >= 0 ? *sp : 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (warp + i * kWarps < it.rows) {
#pragma unroll
      for (int k = 0; k < NP; ++k) m = dsa::amax_bf16x8(v[i][k], m);
    }
  }
  for (int r = warp + kRows * kWarps; r < it.rows; r += kWarps) {
#pragma unroll
    for (int k = 0; k < NP; ++k) m = dsa::amax_bf16x8(load(r, k), m);
  }
  auto block_max = [&](uint32_t x) {
    x = __reduce_max_sync(0xffffffffu, x);
    if (lane == 0) wmax[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = max(x, wmax[w]);
    return x;
  };
  m = block_max(dsa::larger_half(m));  // (behind its barrier every thread has read the old scale)
  if (block < 0) return;
  if (m >= kInfinity) {
    m = 0;
    for (int r = warp; r < it.rows; r += kWarps) {
#pragma unroll
      for (int k = 0; k < NP; ++k) m = finite_max(load(r, k), m);
    }
    __syncthreads();
    m = block_max(m);
  }
  const float s = fmaxf(s_old, dsa::kv8_scale_of(__uint_as_float(m << 16)));
  if (threadIdx.x == 0) *sp = s;
  uint8_t* c0 = cache + (static_cast<int64_t>(block) << g.lb) * ld + static_cast<int64_t>(h) * D;
  if (it.first > 0 && s > s_old) {
    const float ratio = s_old / s;
    for (int r = warp; r < it.first; r += kWarps) {
      for (int c = lane; c < D >> 4; c += 32) {
        uint4* p = reinterpret_cast<uint4*>(c0 + r * ld) + c;
        uint4 u = *p;
        uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 a = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k])),
                       b = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k] >> 16));
          w[k] = dsa::e4m3x2(a.x * ratio, a.y * ratio) | (static_cast<uint32_t>(dsa::e4m3x2(b.x * ratio, b.y * ratio)) << 16);
        }
        *p = u;
      }
    }
  }
  uint8_t* o0 = c0 + it.first * ld;
  auto store = [&](int r, int k, uint4 u) {
    const int c = k * 32 + lane;
    if (c < p8) *(reinterpret_cast<uint2*>(o0 + r * ld) + c) = codes_of<false>(u, s);
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    if (r < it.rows) {
#pragma unroll
      for (int k = 0; k < NP; ++k) store(r, k, v[i][k]);
    }
  }
  for (int r = warp + kRows * kWarps; r < it.rows; r += kWarps) {
#pragma unroll
    for (int k = 0; k < NP; ++k) store(r, k, load(r, k));
  }
}

// Cache row of packed token t; -1 not mapped, -2 behind the last sequence.
__device__ __forceinline__ int row_of_token(const dsa::Kv8Geom& g, int64_t t) {
  if (t >= g.T || t < __ldg(g.cu) || t >= __ldg(g.cu + g.n_seqs * g.step)) return -2;
  const int b = dsa::kv8_seq(g.cu, g.n_seqs, static_cast<int>(t));
  const int c = __ldg(g.cu + b);
  return dsa::kv8_row(g, b, kv8_pos0(g, b, c) + (t - c));
}

// n / d for n * d < 2^32, magic = magic_of(d): n * (2^32 / d + 1) exceeds n / d *
// 2^32 by at most n, less than the 2^32 / d that would reach the next quotient.
// 0 stands for d = 1, and 1 gives 0 for every n.
__device__ __forceinline__ int fast_div(int n, uint32_t magic) {
  return magic ? static_cast<int>(__umulhi(n, magic)) : n;
}
uint32_t magic_of(int d) { return d == 1 ? 0 : static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint32_t>(d)) + 1; }

// block = 1: a (token, head) row has its own scale.  G lanes per row, NP pieces
// each, kRowPieces / NP rows at a time; `tokens` tokens per CTA, whose cache
// rows are looked up first.  Bound: memory, 3 bytes a value; 8192 x 64 rows of
// 128: 36 us, 5.7 TB/s where a copy reaches 6.8.
constexpr int kMaxTokens = 64;

template <int G, int NP>
__global__ void __launch_bounds__(kThreads)
    kv8_write_rows_kernel(const __nv_bfloat16* __restrict__ src, const dsa::Kv8Geom g, int Hc, int D, int tokens,
                          uint32_t magic_hc, uint8_t* __restrict__ cache, float* __restrict__ scale) {
  constexpr int kRows = kRowPieces / NP, kGroups = kThreads / G;
  __shared__ int rows[kMaxTokens];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  if (threadIdx.x < tokens) rows[threadIdx.x] = row_of_token(g, t0 + threadIdx.x);
  __syncthreads();
  const int sub = threadIdx.x % G, p8 = D >> 3;
  const int n = min(static_cast<int64_t>(tokens), g.T - t0) * Hc;
  const __nv_bfloat16* s0 = src + t0 * Hc * D;
  // every lane takes part in the reductions: all groups make the same trips
  const int first = threadIdx.x / G;
  for (int i0 = 0; i0 < n; i0 += kGroups * kRows) {
    uint4 v[kRows][NP];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int i = i0 + first + r * kGroups;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int c = k * G + sub;
        v[r][k] = i < n && c < p8 ? __ldcs(reinterpret_cast<const uint4*>(s0 + static_cast<int64_t>(i) * D) + c)
                                  : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int i = i0 + first + r * kGroups;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < NP; ++k) m = dsa::amax_bf16x8(v[r][k], m);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) m = dsa::max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = dsa::larger_half(m);
      if (__any_sync(0xffffffffu, m >= kInfinity)) {
        m = 0;
#pragma unroll
        for (int k = 0; k < NP; ++k) m = finite_max(v[r][k], m);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      if (i >= n) continue;
      const int t = fast_div(i, magic_hc);
      const int row = rows[t];
      if (row < 0) continue;
      const float s = dsa::kv8_scale_of(__uint_as_float(m << 16));
      const int64_t rh = static_cast<int64_t>(row) * Hc + (i - t * Hc);
      if (sub == 0) scale[rh] = s;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int c = k * G + sub;
        if (c < p8) *(reinterpret_cast<uint2*>(cache + rh * D) + c) = codes_of<true>(v[r][k], s);
      }
    }
  }
}

// `tokens` packed tokens per CTA: their cache rows are looked up once, then the
// threads stream the rows' pieces of 8 codes (a warp's store covers 512
// consecutive bytes), kReadPieces of them in flight each.  Bound: memory,
// 3 bytes a value; 65536 latent rows: 20.6 us with the launch, 5.5 TB/s.
constexpr int kReadPieces = 8;

__global__ void __launch_bounds__(kThreads)
    kv8_read_kernel(const uint8_t* __restrict__ cache, const float* __restrict__ scale, const dsa::Kv8Geom g, int Hc,
                    int D, int tokens, uint32_t magic_row, uint32_t magic_head, __nv_bfloat16* __restrict__ out) {
  __shared__ int rows[kMaxTokens];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  if (threadIdx.x < tokens) rows[threadIdx.x] = row_of_token(g, t0 + threadIdx.x);
  __syncthreads();
  const int p8 = D >> 3, per = Hc * p8;
  const int64_t ld = static_cast<int64_t>(Hc) * D;
  const int n = min(static_cast<int64_t>(tokens), g.T - t0) * per;
  uint4* o0 = reinterpret_cast<uint4*>(out + t0 * ld);
  for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kReadPieces) {
    uint2 v[kReadPieces];
    float s[kReadPieces];
    uint32_t live = 0;  // pieces that are written
#pragma unroll
    for (int j = 0; j < kReadPieces; ++j) {
      const int i = i0 + j * kThreads;
      v[j] = make_uint2(0, 0);
      s[j] = 0.f;
      if (i < n) {
        const int k = fast_div(i, magic_row), c = i - k * per;
        const int row = rows[k];
        if (row != -2) live |= 1u << j;
        if (row >= 0) {
          v[j] = __ldcs(reinterpret_cast<const uint2*>(cache + row * ld) + c);
          s[j] = __ldg(scale + static_cast<int64_t>(row >> g.lb) * Hc + fast_div(c, magic_head));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kReadPieces; ++j) {
      const uint32_t w[2] = {v[j].x, v[j].y};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k])),
                     y = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k] >> 16));
        const __nv_bfloat162 l = __floats2bfloat162_rn(x.x * s[j], x.y * s[j]), u = __floats2bfloat162_rn(y.x * s[j], y.y * s[j]);
        o[2 * k] = *reinterpret_cast<const uint32_t*>(&l);
        o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&u);
      }
      if (live >> j & 1) o0[i0 + j * kThreads] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Tokens per CTA: enough for 16 KB of codes, fewer where the batch would not
// fill the device twice.  What fast_div needs of them holds: several tokens have
// 2048 pieces at most, and the 131072 that one token can have are divided by a
// head's pieces alone, 128 at most.
int tokens_per_cta(int T, int Hc, int D, int sms) {
  int n = std::max(1, std::min(kMaxTokens, 16384 / (Hc * D)));
  n = std::max(1, std::min(n, T / (2 * sms)));
  return n;
}

// (T + tokens may pass the int range)
unsigned ctas_of(int T, int tokens) { return static_cast<unsigned>((static_cast<int64_t>(T) + tokens - 1) / tokens); }

// Checks of the two calls; fills the geometry.
int check_args(const char* fn, const void* rows, const void* cache, const void* scale, const int32_t* cu,
               const int32_t* pos, const int32_t* table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
               int max_blocks, dsa::Kv8Geom* g) {
  if (n_seqs < 1 || T < 0 || Hc < 1 || n_blocks < 1)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need n_seqs >= 1, T >= 0, Hc >= 1, n_blocks >= 1", fn);
  if (D < 16 || D > DSA_KV8_MAX_DIM || D % 16 != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: D must be a multiple of 16 in [16, %d]", fn, DSA_KV8_MAX_DIM);
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

extern "C" int dsa_kv8_write(const void* src, const int32_t* cu_seqlens, const int32_t* pos,
                             const int32_t* block_table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
                             int max_blocks, void* cache, float* scale, cudaStream_t stream) {
  dsa::clear_error();
  dsa::Kv8Geom g;
  int rc = check_args("dsa_kv8_write", src, cache, scale, cu_seqlens, pos, block_table, n_seqs, T, Hc, D, block,
                      n_blocks, max_blocks, &g);
  if (rc != DSA_OK) return rc;
  int sms = 0;
  rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  const auto* x = static_cast<const __nv_bfloat16*>(src);
  auto* c = static_cast<uint8_t*>(cache);
  if (block == 1) {
    const int tokens = tokens_per_cta(T, Hc, D, sms);
    const unsigned grid = ctas_of(T, tokens);
    const uint32_t magic = magic_of(Hc);
    if (D <= 128)
      kv8_write_rows_kernel<16, 1><<<grid, kThreads, 0, stream>>>(x, g, Hc, D, tokens, magic, c, scale);
    else if (D <= 256)
      kv8_write_rows_kernel<32, 1><<<grid, kThreads, 0, stream>>>(x, g, Hc, D, tokens, magic, c, scale);
    else if (D <= 512)
      kv8_write_rows_kernel<32, 2><<<grid, kThreads, 0, stream>>>(x, g, Hc, D, tokens, magic, c, scale);
    else
      kv8_write_rows_kernel<32, 4><<<grid, kThreads, 0, stream>>>(x, g, Hc, D, tokens, magic, c, scale);
    return dsa::launch_error("kv8_write_rows_kernel");
  }
  // a sequence of n rows touches at most n / block + 2 blocks, and at most n
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(T, T / block + 2ll * g.n_seqs)), Hc);
  const int np = (D + 255) / 256;
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(x, g, Hc, D, c, scale); };
  if (block <= 16)
    launch(np == 1 ? kv8_write_kernel<1, 2> : np == 2 ? kv8_write_kernel<2, 2> : np == 3 ? kv8_write_kernel<3, 2> : kv8_write_kernel<4, 2>);
  else
    launch(np == 1 ? kv8_write_kernel<1, 8> : np == 2 ? kv8_write_kernel<2, 8> : np == 3 ? kv8_write_kernel<3, 8> : kv8_write_kernel<4, 6>);
  return dsa::launch_error("kv8_write_kernel");
}

extern "C" int dsa_kv8_read(const void* cache, const float* scale, const int32_t* cu_seqlens, const int32_t* pos,
                            const int32_t* block_table, int n_seqs, int T, int Hc, int D, int block, int n_blocks,
                            int max_blocks, void* out, cudaStream_t stream) {
  dsa::clear_error();
  dsa::Kv8Geom g;
  int rc = check_args("dsa_kv8_read", out, cache, scale, cu_seqlens, pos, block_table, n_seqs, T, Hc, D, block,
                      n_blocks, max_blocks, &g);
  if (rc != DSA_OK) return rc;
  int sms = 0;
  rc = dsa::check_device(&sms);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  const int tokens = tokens_per_cta(T, Hc, D, sms);
  kv8_read_kernel<<<ctas_of(T, tokens), kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(cache), scale, g, Hc, D, tokens, tokens == 1 ? 1 : magic_of(Hc * (D / 8)), magic_of(D / 8),
      static_cast<__nv_bfloat16*>(out));
  return dsa::launch_error("kv8_read_kernel");
}
