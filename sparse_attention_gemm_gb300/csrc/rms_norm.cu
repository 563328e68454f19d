// rms_norm.cu -- root-mean-square norm of rows, with the residual's addition
// and an output in 8 bits, and its backward pass.
//
// Forward, per row of D:
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w.
// Backward, with xh = h * rstd and g = dy * w:
//   dx = rstd * (g - xh * mean(g * xh)) + d_sum,  dw = sum over rows of dy * xh.
//
// A group of G threads holds a whole row in registers, NP pieces of 8 values
// a thread, so that each value is read once; sums are fp32.
//
// The bytes bound it.  16,384 rows of 4096 with a residual: 82 us, 6.6 TB/s.  64 rows of 4096
// to 8 bits: 2.7 us, the chain of a load, two barriers and a store; 1,048,576 rows of 128 to 8 bits 125 us, 3.3 TB/s, where
// the issue of instructions bounds it (70% of the slots).  Backward, 8192 rows of 4096:
// 45 us, 5.9 TB/s, of which the join of dw's partial sums (one row of them a CTA, added in a fixed
// order) takes 6; 24,216 rows of 256 9.4 us.  One row ahead is under way while a row is summed (66 us
// without it, 53 with more CTAs than are resident).  Above 8192 wide it spills and loads no row ahead (2048 rows of
// 16,384: 96 us, 2.1 TB/s).
#include <algorithm>
#include <climits>

#include "kv8.cuh"

namespace {

constexpr int kBf16 = 0, kE4m3 = 1, kMx = 2;  // forms of the output

struct Piece {
  float v[8];
};

__device__ __forceinline__ Piece unpack(uint4 u) {
  Piece p;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.v[2 * i] = __uint_as_float(w[i] << 16);
    p.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return p;
}
__device__ __forceinline__ uint4 pack(const Piece& p) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.v[2 * i], p.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Piece load_weight(const float* w) {
  Piece p;
  const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  p.v[0] = a.x, p.v[1] = a.y, p.v[2] = a.z, p.v[3] = a.w;
  p.v[4] = b.x, p.v[5] = b.y, p.v[6] = b.z, p.v[7] = b.w;
  return p;
}

// Threads of a CTA: several groups where a group is a warp or less, else one.
template <int G>
struct Cta {
  static constexpr int kThreads = G <= 32 ? 256 : G;
  static constexpr int kGroups = kThreads / G;
};

// Sum over a group, the same in each of its threads.  `red`: one float per
// warp; a CTA that calls this again in its next row takes another.
template <int G>
__device__ __forceinline__ float group_sum(float x, float* red) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w) x += red[w];
  }
  return x;
}

struct FwdParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* r;  // residual or NULL
  const float* w;
  __nv_bfloat16* sum;  // or NULL
  void* y;
  void* scale;
  float* rstd;  // or NULL
  int64_t ld_x, ld_r, ld_sum, ld_y;
  int T, D;
  float eps;
};

template <int G, int NP, int FMT>
__global__ void __launch_bounds__(Cta<G>::kThreads) rms_fwd_kernel(const FwdParams p) {
  __shared__ float red[2][G > 32 ? G / 32 : 1];
  const int sub = threadIdx.x % G, p8 = p.D >> 3;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * Cta<G>::kGroups + threadIdx.x / G;
  const bool live = t < p.T;  // (all lanes take part in the reductions)
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 xr[NP], rr[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c = k * G + sub;
    xr[k] = live && c < p8 ? __ldcs(reinterpret_cast<const uint4*>(p.x + t * p.ld_x) + c) : zero;
  }
  if (p.r) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = k * G + sub;
      rr[k] = live && c < p8 ? __ldcs(reinterpret_cast<const uint4*>(p.r + t * p.ld_r) + c) : zero;
    }
  }
  Piece h[NP];
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    h[k] = unpack(xr[k]);
    if (p.r) {
      const Piece b = unpack(rr[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k].v[i] += b.v[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(h[k].v[i], h[k].v[i], sq);
  }
  sq = group_sum<G>(sq, red[0]);
  const float mean = sq / static_cast<float>(p.D) + p.eps;
  float rstd = 1.f / sqrtf(mean);
  // Out of fp32's range the squares are summed again, of values 2^100 times smaller or larger.
  // * beyond it: of 16,384 values below 2^128 the sum is then below 2^70; those whose squares underflow are below 2^26
  //   beside one of 2^57 at least (or an eps of the size);
  // * below it: a mean and an eps that together are under 2^-100 leave a sum under 2^114, and squares that would have
  //   lost bits (under 2^-126) are whole.  From 2^-100 on what they lose is under 2^-49 of the mean.
  // (one comparison for both and NaN: bits from those of 2^-100 on, below infinity's)
  constexpr uint32_t kLow = 27u << 23;
  const bool out = __float_as_uint(mean) - kLow >= 0x7F800000u - kLow;
  if (__any_sync(0xffffffffu, out)) {
    const float by = mean < INFINITY ? 0x1p100f : 0x1p-100f;
    float again = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = h[k].v[i] * by;
        again = fmaf(v, v, again);
      }
    again = group_sum<G>(again, red[1]) / static_cast<float>(p.D);
    if (out) rstd = by / sqrtf(again + p.eps * by * by);
  }
  if (live && sub == 0 && p.rstd) p.rstd[t] = rstd;
  if (live && p.sum) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = k * G + sub;
      if (c < p8) reinterpret_cast<uint4*>(p.sum + t * p.ld_sum)[c] = pack(h[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c = k * G + sub;
    const bool have = live && c < p8;
    if (have) {
      const Piece w = load_weight(p.w + c * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k].v[i] = h[k].v[i] * rstd * w.v[i];
    }
    if constexpr (FMT == kBf16) {
      if (have) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.y) + t * p.ld_y)[c] = pack(h[k]);
    } else {
      // the largest finite magnitude of the lanes that share a scale
      constexpr int kLanes = FMT == kE4m3 ? 16 : 4;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(h[k].v[i]) & 0x7FFFFFFFu;
        m = max(m, have && u < 0x7F800000u ? u : 0u);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = dsa::kv8_scale_of(__uint_as_float(m)), inv = dsa::pow2_inverse(s);
      uint32_t o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        o[i] = dsa::e4m3x2(h[k].v[4 * i] * inv, h[k].v[4 * i + 1] * inv) |
               (static_cast<uint32_t>(dsa::e4m3x2(h[k].v[4 * i + 2] * inv, h[k].v[4 * i + 3] * inv)) << 16);
      if (have) {
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + t * p.ld_y)[c] = make_uint2(o[0], o[1]);
        if (c % kLanes == 0) {
          const int64_t at = t * (p8 / kLanes) + c / kLanes;
          if (FMT == kE4m3)
            static_cast<float*>(p.scale)[at] = s;
          else
            static_cast<uint8_t*>(p.scale)[at] = static_cast<uint8_t>(__float_as_uint(s) >> 23);
        }
      }
    }
  }
}

struct BwdParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* x;
  const float* w;
  const float* rstd;
  const __nv_bfloat16* d_sum;  // or NULL
  __nv_bfloat16* dx;
  float* part;  // [CTAs, D] or NULL
  int64_t ld_dy, ld_x, ld_ds, ld_dx;
  int T, D;
};

// Groups go through the rows in steps of all groups of the grid, a row's loads
// under way while the row before it is worked on; a thread keeps dw's terms of its
// columns, the CTA adds its groups' and writes one row of `part`.
// Resident CTAs an SM: what 64 registers a thread leave room for, 2 of 128 with two pieces a lane (3 of 85
// spill: 24,000 rows of 288 took 23.9 us where they take 12.9), 3 with groups of 8 (4 spill: 5.1 us for 24,000
// rows of 40, and 4.7 with 3).
template <int G, int NP>
__host__ __device__ constexpr int bwd_per_sm() {
  return G == 8 ? 3 : G == 32 && NP == 2 ? 2 : 1024 / Cta<G>::kThreads;
}

template <int G, int NP>
__global__ void __launch_bounds__(Cta<G>::kThreads, (bwd_per_sm<G, NP>())) rms_bwd_kernel(const BwdParams p) {
  constexpr bool kAhead = NP * G <= 1024;  // two pieces of 1024 threads leave no registers for the next row
  constexpr int kGroups = Cta<G>::kGroups;
  __shared__ float red[2][G > 32 ? G / 32 : 1];
  extern __shared__ float cols[];  // [groups][D], with several groups a CTA
  const int sub = threadIdx.x % G, group = threadIdx.x / G, p8 = p.D >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  Piece dw[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k].v[i] = 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const float inv_d = 1.f / static_cast<float>(p.D);
  int par = 0;
  uint4 xr[NP], yr[NP], sr[NP];
  float rstd = 0.f;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = k * G + sub;
      const bool have = t < p.T && c < p8;
      xr[k] = have ? __ldcs(reinterpret_cast<const uint4*>(p.x + t * p.ld_x) + c) : zero;
      yr[k] = have ? __ldcs(reinterpret_cast<const uint4*>(p.dy + t * p.ld_dy) + c) : zero;
      sr[k] = have && p.d_sum ? __ldcs(reinterpret_cast<const uint4*>(p.d_sum + t * p.ld_ds) + c) : zero;
    }
    rstd = t < p.T ? __ldg(p.rstd + t) : 0.f;
  };
  load(static_cast<int64_t>(blockIdx.x) * kGroups + group);
  // all groups of a CTA make the same trips: their lanes meet in the reductions
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGroups; t0 < p.T; t0 += step, par ^= 1) {
    const int64_t t = t0 + group;
    Piece x[NP], g[NP];  // x * rstd, and dy * w
    uint4 s[NP];
    const float r = rstd;
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = k * G + sub;
      x[k] = unpack(xr[k]), g[k] = unpack(yr[k]), s[k] = sr[k];
      if (c < p8) {
        const Piece w = load_weight(p.w + c * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[k].v[i] *= r;
          dw[k].v[i] = fmaf(g[k].v[i], x[k].v[i], dw[k].v[i]);
          g[k].v[i] *= w.v[i];
          dot = fmaf(g[k].v[i], x[k].v[i], dot);
        }
      }
    }
    if (kAhead && t0 + step < p.T) load(t + step);
    const float mean = group_sum<G>(dot, red[par]) * inv_d;
    if (t < p.T) {
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int c = k * G + sub;
        if (c >= p8) continue;
        Piece o = unpack(s[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = fmaf(r, fmaf(-mean, x[k].v[i], g[k].v[i]), o.v[i]);
        reinterpret_cast<uint4*>(p.dx + t * p.ld_dx)[c] = pack(o);
      }
    }
    if (!kAhead && t0 + step < p.T) load(t + step);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!p.part) return;
  float* row = p.part + static_cast<int64_t>(blockIdx.x) * p.D;
  float* to = kGroups > 1 ? cols + group * p.D : row;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c = k * G + sub;
    if (c >= p8) continue;
    reinterpret_cast<float4*>(to + c * 8)[0] = make_float4(dw[k].v[0], dw[k].v[1], dw[k].v[2], dw[k].v[3]);
    reinterpret_cast<float4*>(to + c * 8)[1] = make_float4(dw[k].v[4], dw[k].v[5], dw[k].v[6], dw[k].v[7]);
  }
  if (kGroups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += Cta<G>::kThreads) {
      float v = cols[c];
      for (int g = 1; g < kGroups; ++g) v += cols[g * p.D + c];  // in order: the same sums in every run
      row[c] = v;
    }
  }
}

// dw = the sum of `n` rows of partial sums, in a fixed order: a warp takes 8 columns (32 bytes) of 4
// rows at a time, a CTA's warps the same columns of others, with five loads of a thread under way (24,216
// rows of 256: 9.4 us; 32 columns a warp and four loads 10.7, eight loads 11.8).
constexpr int kDwWarps = 16, kDwCols = 8;
__global__ void __launch_bounds__(kDwWarps * 32) rms_dw_kernel(const float* __restrict__ part, int n, int D,
                                                               float* __restrict__ dw) {
  constexpr int kRows = 32 / kDwCols, kStep = kDwWarps * kRows, kAhead = 5;
  __shared__ float s[kDwWarps][kDwCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums' kernel has finished
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * kDwCols + lane % kDwCols;
  float v = 0.f;
  if (c < D) {
    for (int i0 = warp * kRows + lane / kDwCols; i0 < n; i0 += kStep * kAhead) {
      float x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + kStep * k;
        x[k] = i < n ? __ldcg(part + static_cast<int64_t>(i) * D + c) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v += x[k];
    }
  }
#pragma unroll
  for (int o = kDwCols; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane < kDwCols) s[warp][lane] = v;
  __syncthreads();
  if (threadIdx.x < kDwCols && c < D) {
    float x = s[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kDwWarps; ++w) x += s[w][threadIdx.x];
    dw[c] = x;
  }
}

template <int N>
using Int = std::integral_constant<int, N>;

// Threads a row and pieces a thread, by the row's length.
template <class F>
void by_width(int D, F f) {
  if (D <= 64) f(Int<8>{}, Int<1>{});
  else if (D <= 128) f(Int<16>{}, Int<1>{});
  else if (D <= 256) f(Int<32>{}, Int<1>{});
  else if (D <= 512) f(Int<32>{}, Int<2>{});
  else if (D <= 1024) f(Int<32>{}, Int<4>{});
  else if (D <= 2048) f(Int<128>{}, Int<2>{});
  else if (D <= 4096) f(Int<256>{}, Int<2>{});
  else if (D <= 8192) f(Int<512>{}, Int<2>{});
  else f(Int<512>{}, Int<4>{});
}

constexpr int kPlanSms = 152;

// The backward pass keeps dw's terms and the next row beside a row: fewer pieces a thread.
template <class F>
void by_width_bwd(int D, F f) {
  if (D <= 64) f(Int<8>{}, Int<1>{});
  else if (D <= 128) f(Int<16>{}, Int<1>{});
  else if (D <= 256) f(Int<32>{}, Int<1>{});
  else if (D <= 512) f(Int<32>{}, Int<2>{});
  else if (D <= 1024) f(Int<128>{}, Int<1>{});
  else if (D <= 2048) f(Int<256>{}, Int<1>{});
  else if (D <= 4096) f(Int<512>{}, Int<1>{});
  else if (D <= 8192) f(Int<1024>{}, Int<1>{});
  else f(Int<1024>{}, Int<2>{});
}

// CTAs of the backward pass: what is resident at once, fewer for few rows.
int bwd_ctas(int T, int D) {
  int n = 0;
  by_width_bwd(D, [&](auto g, auto np) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, kGroups = Cta<G>::kGroups;
    n = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(T) + kGroups - 1) / kGroups, bwd_per_sm<G, NP>() * kPlanSms));
  });
  return n;
}

bool width_ok(int D) { return D >= 8 && D <= DSA_NORM_MAX_DIM && D % 8 == 0; }
bool stride_ok(int64_t ld, int D) { return ld >= D && ld % 8 == 0; }

}  // namespace

extern "C" int dsa_rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, const float* weight,
                                int T, int D, float eps, int fmt, void* y, int64_t ld_y, void* y_scale, void* sum,
                                int64_t ld_sum, float* rstd, cudaStream_t stream) {
  dsa::clear_error();
  const char* fn = "dsa_rms_norm_fwd";
  if (fmt != DSA_NORM_BF16 && fmt != DSA_NORM_E4M3 && fmt != DSA_NORM_MXFP8)
    return dsa::set_error(DSA_ERR_VALUE, "%s: fmt must be DSA_NORM_BF16, DSA_NORM_E4M3 or DSA_NORM_MXFP8", fn);
  const int group = fmt == DSA_NORM_E4M3 ? 128 : fmt == DSA_NORM_MXFP8 ? 32 : 8;
  if (T < 0 || !width_ok(D) || D % group != 0)
    return dsa::set_error(DSA_ERR_VALUE, "%s: need T >= 0 and D a multiple of %d in [%d, %d]", fn, group, group,
                          DSA_NORM_MAX_DIM);
  if (!(eps > 0.f) || !(eps < INFINITY)) return dsa::set_error(DSA_ERR_VALUE, "%s: eps must be finite and > 0", fn);
  if (!stride_ok(ld_x, D) || !stride_ok(ld_y, D) || (residual && !stride_ok(ld_r, D)) || (sum && !stride_ok(ld_sum, D)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: row strides must be at least D and multiples of 8", fn);
  if (T > 0 && ((y == x && (fmt != DSA_NORM_BF16 || ld_y != ld_x)) || (sum == x && sum && ld_sum != ld_x) ||
      (residual && ((y == residual && (fmt != DSA_NORM_BF16 || ld_y != ld_r)) || (sum == residual && ld_sum != ld_r))) ||
      (sum && y == sum)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: in place, y or sum takes the rows and the stride of x or residual", fn);
  if (!weight || (T > 0 && (!x || !y || (fmt != DSA_NORM_BF16 && !y_scale))))
    return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  if (!dsa::aligned(x, 16) || !dsa::aligned(residual, 16) || !dsa::aligned(weight, 16) || !dsa::aligned(sum, 16) ||
      !dsa::aligned(y, fmt == DSA_NORM_BF16 ? 16 : 8) || !dsa::aligned(rstd, 4) ||
      !dsa::aligned(y_scale, fmt == DSA_NORM_E4M3 ? 4 : 1))
    return dsa::set_error(DSA_ERR_VALUE, "%s: x, residual, weight, sum and y must be 16-byte aligned (8-bit y: 8)", fn);
  int rc = dsa::check_device(nullptr);
  if (rc != DSA_OK) return rc;
  if (T == 0) return DSA_OK;
  const FwdParams p{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(residual), weight,
                    static_cast<__nv_bfloat16*>(sum), y, y_scale, rstd, ld_x, ld_r, ld_sum, ld_y, T, D, eps};
  by_width(D, [&](auto g, auto np) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(T) + Cta<G>::kGroups - 1) / Cta<G>::kGroups);
    if (fmt == DSA_NORM_BF16)
      rms_fwd_kernel<G, NP, kBf16><<<grid, Cta<G>::kThreads, 0, stream>>>(p);
    else if (fmt == DSA_NORM_MXFP8)
      rms_fwd_kernel<G, NP, kMx><<<grid, Cta<G>::kThreads, 0, stream>>>(p);
    else if constexpr (G >= 16)
      rms_fwd_kernel<G, NP, kE4m3><<<grid, Cta<G>::kThreads, 0, stream>>>(p);
  });
  return dsa::launch_error("rms_fwd_kernel");
}

extern "C" size_t dsa_rms_norm_bwd_workspace_size(int T, int D) {
  if (T < 1 || !width_ok(D)) return 0;
  return static_cast<size_t>(bwd_ctas(T, D)) * D * sizeof(float);
}

extern "C" int dsa_rms_norm_bwd(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, const float* weight,
                                const float* rstd, const void* d_sum, int64_t ld_ds, int T, int D, void* dx,
                                int64_t ld_dx, float* dweight, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  dsa::clear_error();
  const char* fn = "dsa_rms_norm_bwd";
  if (T < 0 || !width_ok(D))
    return dsa::set_error(DSA_ERR_VALUE, "%s: need T >= 0 and D a multiple of 8 in [8, %d]", fn, DSA_NORM_MAX_DIM);
  if (!stride_ok(ld_dy, D) || !stride_ok(ld_x, D) || !stride_ok(ld_dx, D) || (d_sum && !stride_ok(ld_ds, D)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: row strides must be at least D and multiples of 8", fn);
  if (T > 0 && ((dx == dy && ld_dx != ld_dy) || (dx == x && ld_dx != ld_x) || (dx == d_sum && ld_dx != ld_ds)))
    return dsa::set_error(DSA_ERR_VALUE, "%s: in place, dx takes the stride of its rows", fn);
  if (!weight || (T > 0 && (!dy || !x || !rstd || !dx))) return dsa::set_error(DSA_ERR_VALUE, "%s: NULL pointer", fn);
  if (!dsa::aligned(dy, 16) || !dsa::aligned(x, 16) || !dsa::aligned(weight, 16) || !dsa::aligned(d_sum, 16) ||
      !dsa::aligned(dx, 16) || !dsa::aligned(rstd, 4) || !dsa::aligned(dweight, 4))
    return dsa::set_error(DSA_ERR_VALUE, "%s: dy, x, weight, d_sum and dx must be 16-byte aligned", fn);
  const size_t need = dweight ? dsa_rms_norm_bwd_workspace_size(T, D) : 0;
  if (need > 0 && (!workspace || ws_bytes < need || !dsa::aligned(workspace, 256)))
    return dsa::set_error(DSA_ERR_WORKSPACE, "%s: needs a 256-byte aligned workspace of %zu bytes, got %zu", fn, need,
                          workspace ? ws_bytes : static_cast<size_t>(0));
  int rc = dsa::check_device(nullptr);
  if (rc != DSA_OK) return rc;
  if (T == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(D) * sizeof(float), stream) != cudaSuccess)
      return dsa::launch_error("dsa_rms_norm_bwd zero dweight");
    return DSA_OK;
  }
  const int ctas = bwd_ctas(T, D);
  const BwdParams p{static_cast<const __nv_bfloat16*>(dy), static_cast<const __nv_bfloat16*>(x), weight, rstd,
                    static_cast<const __nv_bfloat16*>(d_sum), static_cast<__nv_bfloat16*>(dx),
                    dweight ? static_cast<float*>(workspace) : nullptr, ld_dy, ld_x, ld_ds, ld_dx, T, D};
  by_width_bwd(D, [&](auto g, auto np) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value;
    rms_bwd_kernel<G, NP><<<ctas, Cta<G>::kThreads, Cta<G>::kGroups > 1 ? Cta<G>::kGroups * D * sizeof(float) : 0,
                                                    stream>>>(p);
  });
  rc = dsa::launch_error("rms_bwd_kernel");
  if (rc != DSA_OK || !dweight) return rc;
  // launched while the pass drains, so that its start-up hides behind it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((D + kDwCols - 1) / kDwCols);
  cfg.blockDim = dim3(kDwWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, rms_dw_kernel, static_cast<const float*>(p.part), ctas, D, dweight) != cudaSuccess)
    return dsa::launch_error("rms_dw_kernel");
  return DSA_OK;
}
