// attention_kv8.cuh -- what the two kernels of the attention over the 8-bit
// block cache share: the arguments, the weights' range and small helpers.
#pragma once

#include <atomic>
#include <climits>

#include "kv8.cuh"

namespace dsa {
namespace kv8_attn {

constexpr int kKeys = 64;  // keys per tile
constexpr uint32_t kChunkBytes = kKeys * 128;  // 64 keys x 64 dims
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPlanSms = 152;

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* k8;
  const float* k_scale;
  const uint8_t* v8;  // separate V, or unused
  const float* v_scale;
  const uint8_t* k_exp;  // 4-bit cache: a scale byte per 32 elements of a row
  const uint8_t* v_exp;
  const int32_t* idx;
  const int32_t* topk_length;
  const float* sink;
  dsa::Kv8Geom g;
  __nv_bfloat16* out;
  float* lse;
  float* lse_kv;
  float* max_logits;
  float* part_o;   // [T, H, splits, Dv]: mean values of splits > 1
  float4* part_s;  // [T, H, splits]: reference, sum, maximum
  uint32_t* status;
  int H, Hc, G, K, splits, n_items;  // G: 64-head groups per KV head
  float scale_log2;
  bool steal;  // more items than CTAs that fit: a CTA takes over those of CTAs not yet started
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two products, sums or fused ones at a time, each rounded as alone.
__device__ __forceinline__ uint64_t bits2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 of_bits2(uint64_t r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return of_bits2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return of_bits2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return of_bits2(r);
}

__device__ __forceinline__ bool elect_sync() {
  uint32_t is = 0;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}" : "=r"(is));
  return is != 0;
}

// 16-byte global -> shared copy; src_bytes = 0 fills zeros without reading.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// This thread's arrival at a barrier once its copies so far have landed.  (A tensor
// core that reads them is behind a proxy fence of the thread that waited.)
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void l2_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 h2_of(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint2 pack4(const uint16_t (&c)[4]) {
  return make_uint2(c[0] | (static_cast<uint32_t>(c[1]) << 16), c[2] | (static_cast<uint32_t>(c[3]) << 16));
}

// Smallest power of two >= x (x >= 0 finite), within [2^-126, 2^126].
__device__ __forceinline__ float pow2_ceil(float x) {
  const uint32_t u = __float_as_uint(x);
  uint32_t e = (u >> 23) + ((u & 0x7FFFFFu) ? 1u : 0u);
  e = e < 1u ? 1u : (e > 253u ? 253u : e);
  return __uint_as_float(e << 23);
}

// Byte offset of 16-byte unit `u` of row `r` in rows of 64 bytes, 64-byte swizzle.
__device__ __forceinline__ uint32_t sw64_offset(uint32_t r, uint32_t u) { return r * 64u + ((u ^ ((r >> 1) & 3u)) << 4); }

// The two terms of a pair of query values (bf16x2): x / s = hi + lo / 16, inv = 1 / s.
__device__ __forceinline__ void split_query(uint32_t u, float inv, uint16_t& hi, uint16_t& lo) {
  const __half2 h = __floats2half2_rn(__uint_as_float(u << 16) * inv, __uint_as_float(u & 0xFFFF0000u) * inv);
  hi = e4m3x2_h2(h2_bits(h));
  lo = e4m3x2_h2(h2_bits(__hmul2(__hsub2(h, h2_of(h2_of_e4m3x2(hi))), __float2half2_rn(16.f))));
}

// Two codes -> two bf16 values, exactly: a code's 4 significant bits leave
// the lower half of its fp32 form zero, so the upper halves are the bf16 ones
// (NaN too), and a byte permute takes them.
__device__ __forceinline__ uint32_t bf2_of_e4m3x2(uint32_t c) {
  const float2 f = f2_of_e4m3x2(static_cast<uint16_t>(c));
  return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A piece of 16 codes (of 8 in 128 dims, lane & 7) to two units of 16 bytes of
// row `key` of a chunk of 64 dims.  Lanes of the upper pieces store the second
// unit first: eight lanes (a row) touch all banks once.
__device__ __forceinline__ void widen(const uint4& c, uint8_t* chunk, int key, int piece) {
  const bool up = (piece & 4) != 0;
  const uint32_t w[4] = {up ? c.z : c.x, up ? c.w : c.y, up ? c.x : c.z, up ? c.y : c.w};
  uint32_t o[8];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    o[2 * n] = bf2_of_e4m3x2(w[n]);
    o[2 * n + 1] = bf2_of_e4m3x2(w[n] >> 16);
  }
  const int unit = (piece & 3) * 2 + (up ? 1 : 0);
  *reinterpret_cast<uint4*>(chunk + sw128_offset(key, unit * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(chunk + sw128_offset(key, (unit ^ 1) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
}

// The two terms of a pair of weights: E4M3, and what it leaves in E5M2.
__device__ __forceinline__ void split_weights(float w0, float w1, uint16_t& hi, uint16_t& lo) {
  const __half2 h = __floats2half2_rn(w0, w1);
  hi = e4m3x2_h2(h2_bits(h));
  lo = e5m2x2_h2(h2_bits(__hsub2(h, h2_of(h2_of_e4m3x2(hi)))));
}
// max_logits of a head with slots, whose weights' sum is l and whose largest score is mx (in powers of two; a
// maximum passes over NaN): NaN where the sum is.
__device__ __forceinline__ float max_logit(float l, float mx) { return l == l ? mx * kLn2 : l; }

// x (> 0, finite) as 2^e * f, f in (1/2, 1].
__device__ __forceinline__ float2 scale_parts(float x) {
  const bool small = x < 1.17549435e-38f;  // below 2^-126
  const uint32_t u = __float_as_uint(small ? x * 4294967296.f : x);
  const bool one = (u & 0x7FFFFFu) == 0;
  return make_float2(static_cast<float>(static_cast<int>(u >> 23) - (one ? 127 : 126) - (small ? 32 : 0)),
                     __uint_as_float(one ? 0x3F800000u : 0x3F000000u | (u & 0x7FFFFFu)));
}

// The gather of a tile of 64 keys by eight warps: thread gt takes piece (gt &
// 7) (16 codes) of keys (gt >> 3) and (gt >> 3) + 32 of every 128 dims.  The
// codes of a tile are loaded into registers a tile ahead and widened as they
// are stored: chunks of 64 dims, rows of 128 bytes, 128-byte swizzle.
template <int DQK, int DV, bool SEP>
struct Gather {
  static constexpr int kWarps = 8, kThreads = kWarps * 32, kStep = kThreads / 8;
  static constexpr bool kScaled = true;   // codes whose scales come beside the tile
  static constexpr bool kPlaced = false;  // eight dims lie as 0, 4, 1, 5, 2, 6, 3, 7 in shared memory
  static constexpr int kFull = DQK / 128, kNv = SEP ? DV / 128 : 0;
  static constexpr bool kTail = DQK % 128 != 0;
  static_assert(2 * kStep == kKeys, "a thread gathers two keys of a tile");
  uint4 k[kFull][2], v[SEP ? kNv : 1][2], tail;
  float scale;  // of one of the two keys (pieces 0 and 1) or values (pieces 2 and 3)

  // Rows r[0], r[1] of the cache (-1: none, zeros without reading).
  __device__ __forceinline__ void load_keys(const Params& p, const int (&r)[2], int kvh, int piece) {
    const int rows = p.g.n_blocks << p.g.lb;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool have = r[s] >= 0 && dsa::check(r[s] < rows, p.status);
      const uint8_t* src = p.k8 + (static_cast<int64_t>(have ? r[s] : 0) * p.Hc + kvh) * DQK + piece * 16;
#pragma unroll
      for (int c = 0; c < kFull; ++c)
        k[c][s] = have ? __ldcg(reinterpret_cast<const uint4*>(src + c * 128)) : make_uint4(0, 0, 0, 0);
    }
    if (kTail) {  // its four pieces: threads with piece 0..3 take the first key's, the others the second's
      const int x = piece >= 4 ? r[1] : r[0];
      const bool have = x >= 0 && dsa::check(x < rows, p.status);
      const uint8_t* src = p.k8 + (static_cast<int64_t>(have ? x : 0) * p.Hc + kvh) * DQK + kFull * 128 + (piece & 3) * 16;
      tail = have ? __ldcg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    }
    scale = 0.f;
    if (piece < (SEP ? 4 : 2)) {
      const int x = piece & 1 ? r[1] : r[0];
      if (x >= 0 && dsa::check(x < rows, p.status))
        scale = __ldg((SEP && piece >= 2 ? p.v_scale : p.k_scale) + static_cast<int64_t>(x >> p.g.lb) * p.Hc + kvh);
    }
  }
  __device__ __forceinline__ void load_values(const Params& p, const int (&r)[2], int kvh, int piece) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool have = r[s] >= 0 && dsa::check(r[s] < (p.g.n_blocks << p.g.lb), p.status);
      const uint8_t* src = p.v8 + (static_cast<int64_t>(have ? r[s] : 0) * p.Hc + kvh) * DV + piece * 16;
#pragma unroll
      for (int c = 0; c < kNv; ++c)
        v[c][s] = have ? __ldcg(reinterpret_cast<const uint4*>(src + c * 128)) : make_uint4(0, 0, 0, 0);
    }
  }
  // meta: the scale of each slot's key and, behind them, value; 0: no slot.
  __device__ __forceinline__ void store_keys(uint8_t* buf, float* meta, int key0, int piece) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < kFull; ++c)
        widen(k[c][s], buf + (2 * c + (piece >> 2)) * kChunkBytes, key0 + s * kStep, piece);
    if (kTail) widen(tail, buf + 2 * kFull * kChunkBytes, key0 + (piece >> 2) * kStep, piece);
    if (piece < (SEP ? 4 : 2)) meta[(piece >> 1) * kKeys + (piece & 1) * kStep + key0] = scale;
  }
  __device__ __forceinline__ void store_values(uint8_t* buf, int key0, int piece) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < kNv; ++c)
        widen(v[c][s], buf + (2 * c + (piece >> 2)) * kChunkBytes, key0 + s * kStep, piece);
  }
};

// Attention in groups of 16 heads (attention_kv8_narrow.cu): whether it takes
// a call, and the launch.
bool narrow_takes(int T, int H, int Hc, int K);
int launch_narrow(Params p, int T, int Dqk, cudaStream_t stream);

}  // namespace kv8_attn
}  // namespace dsa
