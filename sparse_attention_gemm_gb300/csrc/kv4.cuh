// kv4.cuh -- the 4-bit block cache: E2M1 codes with a power of two per 32.
//
// Codes uint8 [n_blocks, block, Hc, D / 2] (element 2i in the low half of byte
// i), scale uint8 [n_blocks, block, Hc, D / 32] (E8M0); a value is
// e2m1(code) * 2^(scale - 127).  Rows live where the 8-bit cache's do (kv8.cuh).
#pragma once

#include "kv8.cuh"

namespace dsa {

constexpr uint32_t kMxNan = 255;  // scale byte of 32 values one of which is NaN

// Scale byte of 32 values whose largest magnitude is `bits` (bf16, finite):
// e + 127 with the smallest e that keeps it <= 6 * 2^e, 6 = 1.5 * 2^2, within
// [-126, 125]: the smallest code, 2^(e - 1), and the largest, 6 * 2^e, are bf16 values.
__device__ __forceinline__ uint32_t kv4_scale_of(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 2 + ((bits & 0x7Fu) > 0x40u ? 1 : 0);
  return static_cast<uint32_t>(min(max(e, 1), 252));
}

// 2^(127 - byte), of a byte in [1, 252], exactly.
__device__ __forceinline__ float kv4_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight values times inv -> eight E2M1 codes, to nearest even, beyond +-6 the
// largest code of that sign; element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8], float inv) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv), "f"(x[4] * inv), "f"(x[5] * inv),
        "f"(x[6] * inv), "f"(x[7] * inv));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A code's three bits at bits 6..8 of a bf16 are its value times 2^-126: exponents 0 to 3, of which 0 is
// subnormal in both.  Eight codes of a word as such: x[i] holds elements i and i + 4, which lie 16 bits apart.  One product
// puts the three bits and, six places on, the sign where they belong (shifts and an OR for each take one
// instruction more a pair: 2048 rows of 64 heads over the cache 919 us, and 890 like this).
__device__ __forceinline__ void e2m1_raw(uint32_t w, uint32_t (&x)[4]) {
  const uint32_t v = w >> 8;
  x[0] = ((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
  x[1] = ((w & 0x00F000F0u) * 0x104u) & 0x81C081C0u;
  x[2] = ((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
  x[3] = ((v & 0x00F000F0u) * 0x104u) & 0x81C081C0u;
}

// Their factor, twice, as bf16: 2^126 times 2^(byte - 127), for bytes up to kMxDirect; of
// larger ones it is 2^127 and another follows: 2^(byte - 128), NaN for kMxNan.
constexpr uint32_t kMxDirect = 128;
__device__ __forceinline__ uint32_t mx_factor(uint32_t byte) { return (min(byte, kMxDirect) + 126u) * 0x00800080u; }
__device__ __forceinline__ uint32_t mx_factor2(uint32_t byte) {
  return byte == kMxNan ? 0x7FC07FC0u : (max(byte, kMxDirect) - 1u) * 0x00800080u;
}

// The second factor, 1 where there is none.
__device__ __forceinline__ uint32_t mx_second(uint32_t byte) { return byte > kMxDirect ? mx_factor2(byte) : 0x3F803F80u; }

// Eight codes -> eight bf16 values, exactly, those beyond the range infinite; in order.
__device__ __forceinline__ void bf8_of_e2m1(uint32_t w, uint32_t byte, uint32_t (&o)[4]) {
  uint32_t x[4];
  e2m1_raw(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = mul_bf16x2(x[i], mx_factor(byte));
    if (byte > kMxDirect) x[i] = mul_bf16x2(x[i], mx_factor2(byte));
  }
  o[0] = __byte_perm(x[0], x[1], 0x5410);
  o[1] = __byte_perm(x[2], x[3], 0x5410);
  o[2] = __byte_perm(x[0], x[1], 0x7632);
  o[3] = __byte_perm(x[2], x[3], 0x7632);
}

}  // namespace dsa
