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

constexpr int kWriteThreads = 256;
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;

// What one CTA of the write kernel works on: a block that receives rows.
struct WriteItem {
  int t0;     // packed token of the first new row
  int rows;   // new rows
  int first;  // their first row inside the block
  int block;  // physical block, -1 when there is none
};

// The item-th block that receives rows, counted through the sequences.
__device__ bool find_item(const dsa::Kv8Geom& g, int item, WriteItem* out) {
  __shared__ int wsum[kWriteThreads / 32];
  __shared__ int s_found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = 1 << g.lb;
  if (tid == 0) s_found = 0;
  int base = 0;
  for (int b0 = 0; b0 < g.n_seqs; b0 += kWriteThreads) {
    const int b = b0 + tid;
    int c0 = 0, n = 0, count = 0;
    int64_t p0 = 0;
    if (b < g.n_seqs) {
      c0 = max(__ldg(g.cu + b), 0);
      n = min(__ldg(g.cu + b + 1), g.T) - c0;
      p0 = kv8_pos0(g, b, c0);
      if (n > 0) count = static_cast<int>(((p0 + n - 1) >> g.lb) - (p0 >> g.lb)) + 1;
    }
    int inc = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = base, total = 0;
#pragma unroll
    for (int w = 0; w < kWriteThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    inc += before;
    if (item >= inc - count && item < inc) {
      const int64_t page = (p0 >> g.lb) + (item - (inc - count));
      const int64_t lo = max(p0, page << g.lb), hi = min(p0 + n, (page << g.lb) + size);
      out->t0 = c0 + static_cast<int>(lo - p0);
      out->rows = static_cast<int>(hi - lo);
      out->first = static_cast<int>(lo - (page << g.lb));
      out->block = kv8_block(g, b, page);
      s_found = 1;
    }
    base += total;
    if (base > item) break;
  }
  __syncthreads();
  return s_found != 0;
}

__global__ void __launch_bounds__(kWriteThreads)
    kv8_write_kernel(const __nv_bfloat16* __restrict__ src, const dsa::Kv8Geom g, int Hc, int D,
                     uint8_t* __restrict__ cache, float* __restrict__ scale) {
  __shared__ WriteItem it;
  __shared__ uint32_t wmax[kWriteThreads / 32];
  if (!find_item(g, blockIdx.x, &it) || it.block < 0) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int p8 = D >> 3;  // 16-byte pieces of a bf16 row
  const int64_t ld = static_cast<int64_t>(Hc) * D;
  const __nv_bfloat16* s0 = src + it.t0 * ld + static_cast<int64_t>(h) * D;
  // largest finite magnitude, as bf16 bits without the sign (monotonic)
  uint32_t m = 0;
  for (int i = tid; i < it.rows * p8; i += kWriteThreads) {
    const int r = i / p8, c = i - r * p8;
    const uint4 v = *reinterpret_cast<const uint4*>(s0 + r * ld + c * 8);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = w[k] & 0x7FFFu, b = (w[k] >> 16) & 0x7FFFu;
      m = max(m, a < 0x7F80u ? a : 0u);
      m = max(m, b < 0x7F80u ? b : 0u);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) wmax[tid >> 5] = m;
  float* sp = scale + static_cast<int64_t>(it.block) * Hc + h;
  const float s_old = it.first > 0 ? *sp : 0.f;
  __syncthreads();  // every thread has read the old scale before it is replaced
#pragma unroll
  for (int w = 0; w < kWriteThreads / 32; ++w) m = max(m, wmax[w]);
  const float s = fmaxf(s_old, dsa::kv8_scale_of(__uint_as_float(m << 16)));
  if (tid == 0) *sp = s;
  uint8_t* c0 = cache + (static_cast<int64_t>(it.block) << g.lb) * ld + static_cast<int64_t>(h) * D;
  const int p16 = D >> 4;
  if (it.first > 0 && s > s_old) {
    const float ratio = s_old / s;
    for (int i = tid; i < it.first * p16; i += kWriteThreads) {
      const int r = i / p16, c = i - r * p16;
      uint4* p = reinterpret_cast<uint4*>(c0 + r * ld + c * 16);
      uint4 v = *p;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k])),
                     b = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[k] >> 16));
        w[k] = dsa::e4m3x2(a.x * ratio, a.y * ratio) | (static_cast<uint32_t>(dsa::e4m3x2(b.x * ratio, b.y * ratio)) << 16);
      }
      *p = v;
    }
  }
  for (int i = tid; i < it.rows * p8; i += kWriteThreads) {
    const int r = i / p8, c = i - r * p8;
    const uint4 v = *reinterpret_cast<const uint4*>(s0 + r * ld + c * 8);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = dsa::e4m3x2(__uint_as_float(w[k] << 16) / s, __uint_as_float(w[k] & 0xFFFF0000u) / s);
    uint2 q;
    q.x = o[0] | (static_cast<uint32_t>(o[1]) << 16);
    q.y = o[2] | (static_cast<uint32_t>(o[3]) << 16);
    *reinterpret_cast<uint2*>(c0 + (it.first + r) * ld + c * 8) = q;
  }
}

// One CTA per kReadTokens packed tokens: their rows and sequences are looked
// up once, then the threads stream the rows' 16-byte pieces.
__global__ void __launch_bounds__(kReadThreads)
    kv8_read_kernel(const uint8_t* __restrict__ cache, const float* __restrict__ scale, const dsa::Kv8Geom g, int Hc,
                    int D, __nv_bfloat16* __restrict__ out) {
  __shared__ int rows[kReadTokens];  // cache row, -1 unmapped, -2 behind the last sequence
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int64_t t = t0 + threadIdx.x;
    int row = -2;
    if (t < g.T && t >= __ldg(g.cu) && t < __ldg(g.cu + g.n_seqs)) {
      const int b = dsa::kv8_seq(g.cu, g.n_seqs, static_cast<int>(t));
      const int c = __ldg(g.cu + b);
      row = dsa::kv8_row(g, b, kv8_pos0(g, b, c) + (t - c));
    }
    rows[threadIdx.x] = row;
  }
  __syncthreads();
  const int p16 = D >> 4, per = Hc * p16;
  const int64_t ld = static_cast<int64_t>(Hc) * D;
  for (int i = threadIdx.x; i < kReadTokens * per; i += kReadThreads) {
    const int k = i / per, c = i - k * per;
    const int row = rows[k];
    if (row == -2) continue;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (row >= 0) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(cache + row * ld) + c);
      const float s = __ldg(scale + static_cast<int64_t>(row >> g.lb) * Hc + c / p16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[j])),
                     y = dsa::f2_of_e4m3x2(static_cast<uint16_t>(w[j] >> 16));
        const __nv_bfloat162 l = __floats2bfloat162_rn(x.x * s, x.y * s), u = __floats2bfloat162_rn(y.x * s, y.y * s);
        o[2 * j] = *reinterpret_cast<const uint32_t*>(&l);
        o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&u);
      }
      a = make_uint4(o[0], o[1], o[2], o[3]);
      b = make_uint4(o[4], o[5], o[6], o[7]);
    }
    uint4* p = reinterpret_cast<uint4*>(out + (t0 + k) * ld) + 2 * c;
    p[0] = a;
    p[1] = b;
  }
}

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
  *g = dsa::Kv8Geom{cu, pos, table, n_seqs, T, lb, n_blocks, max_blocks};
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
  rc = dsa::check_device(nullptr);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  // a sequence of n rows touches at most n / block + 2 blocks, and at most n
  const int64_t items = std::min<int64_t>(T, T / block + 2ll * n_seqs);
  kv8_write_kernel<<<dim3(static_cast<unsigned>(items), Hc), kWriteThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(src), g, Hc, D, static_cast<uint8_t*>(cache), scale);
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
  rc = dsa::check_device(nullptr);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  kv8_read_kernel<<<(T + kReadTokens - 1) / kReadTokens, kReadThreads, 0, stream>>>(
      static_cast<const uint8_t*>(cache), scale, g, Hc, D, static_cast<__nv_bfloat16*>(out));
  return dsa::launch_error("kv8_read_kernel");
}
