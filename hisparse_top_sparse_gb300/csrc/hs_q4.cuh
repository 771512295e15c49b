// The q4 latent row (HS_Q4_ROW_BYTES bytes) and the conversions its kernels share.
//
//   [0, 256)    e2m1 codes of dims 0..511, a word of four bytes for eight dims:
//               dim 2 i of the eight in nibble i, dim 2 i + 1 in nibble 4 + i
//   [256, 384)  dims 512..575 (rope) in bf16, as they are
//   [384, 416)  one scale byte for each 16 dims of the first 512: five bits of
//               exponent x, three of fraction f, (8 + f) * 2^(x - 19)
//
// The value of a code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) is code *
// scale. A group's scale is the smallest whose largest code, 6 * scale, reaches
// the group's largest magnitude. A code has two significant bits and a scale
// four, so every value is a bf16 number and reading a row back rounds nothing.
// Sixteen dims a scale and three bits of its fraction leave rows of normally
// distributed dims, alike or unlike in size, a squared error of 1.0 % of theirs;
// 32 dims and a power of two, 16 bytes less a row, 1.3 to 2.0 %. Scales run from
// 2^-16 to 1.75 * 2^15; byte 255 marks a group that held a NaN or an infinity,
// all of whose values are NaN.
// The order of the nibbles is that of a pair of bf16 values: nibble i and nibble
// 4 + i lie 16 bits apart, so a shift and a mask take a pair out of a word.
#pragma once

#include "hs_internal.cuh"

constexpr int Q4_GROUP = 16;
constexpr int Q4_ROPE_OFF = HS_VALUE_DIM / 2;                                    // 256
constexpr int Q4_SCALE_OFF = Q4_ROPE_OFF + 2 * (HS_LATENT_DIM - HS_VALUE_DIM);   // 384
static_assert(Q4_SCALE_OFF + HS_VALUE_DIM / Q4_GROUP == HS_Q4_ROW_BYTES, "q4 row");
constexpr int Q4_BYTE_MAX = 254;           // the largest scale
constexpr uint32_t Q4_BYTE_NAN = 255;
constexpr int Q4_BIAS = (127 - 16) << 3;   // a scale byte and a float's top 12 bits (sign 0)

// Scale byte of a group whose largest magnitude has the bits `amax` (infinities and
// NaNs are the largest of all).
__device__ __forceinline__ uint32_t q4_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return Q4_BYTE_NAN;
  const float a = __uint_as_float(amax);
  // a / 6 from above (1/6 rounded up, the product rounded up), cut to three bits
  // of fraction: the scale wanted or the one below it
  const uint32_t t = __float_as_uint(__fmul_ru(a, 0.166666671633720397949f)) >> 20;
  const int b = (int)t - Q4_BIAS + (6.f * __uint_as_float(t << 20) < a);
  return (uint32_t)min(max(b, 0), Q4_BYTE_MAX);
}
__device__ __forceinline__ float q4_scale(uint32_t byte) { return __uint_as_float((byte + Q4_BIAS) << 20); }

// Codes. A value's quotient by the scale has to fall on the right side of the
// middles between codes, and on a middle exactly when it is there (a tie goes to
// the even code); the product with a reciprocal is off by a unit or two. One step
// of the product's remainder, which an fma gives exactly, mends it (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor,
// 1990): the result's error before its rounding is the reciprocal's times the
// correction, some 2^-45, where a middle is exact and any other quotient of a float
// by a four-bit scale is further than half a unit from it. (tests/test_q4_codes.py
// goes through the eight fractions, reciprocals off by up to two units, and the 20000
// floats on either side of every middle.)
__device__ __forceinline__ float q4_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(s));
  return r;
}
__device__ __forceinline__ uint64_t q4_pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
// Two values over the scale, with every sign the other way round (so that a zero's
// comes out right: Q4_SIGNS).
__device__ __forceinline__ float2 q4_minus_over(float x, float y, uint64_t s, uint64_t minus_inv) {
  const uint64_t a = q4_pair(x, y);
  uint64_t b, e;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(b) : "l"(a), "l"(minus_inv));
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(e) : "l"(s), "l"(b), "l"(a));
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(b) : "l"(e), "l"(minus_inv), "l"(b));
  float2 f;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f.x), "=f"(f.y) : "l"(b));
  return f;
}
// Four bytes of two codes each, x in the low nibble: to nearest, ties to even,
// saturated.
__device__ __forceinline__ uint32_t q4_codes(float2 a, float2 b, float2 c, float2 d) {
  uint32_t w;
  asm("{\n.reg .b8 p, q, r, s;\n"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n"
      "mov.b32 %0, {p, q, r, s};\n}\n"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}
constexpr uint32_t Q4_SIGNS = 0x88888888u;

// Decoding, two codes at a time. The three bits of a magnitude, moved to where a
// bf16 number has its last exponent bits and its first fraction bit, are the code
// times 2^-126 (0.5 a subnormal one); a product with the scale times 2^111 gives
// the value times 2^-15, exactly, and no scale overflows.
constexpr int Q4_SHIFT = 15;               // q4_decode2's values are 2^-15 of theirs
__device__ __forceinline__ uint32_t q4_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// a scale byte to the multiplier of q4_decode2, in both halves
__device__ __forceinline__ uint32_t q4_scale2(uint32_t byte) {
  const uint32_t s = byte == Q4_BYTE_NAN ? 0x7fc0u : (byte << 4) + ((127 - 16 + 126 - Q4_SHIFT) << 7);
  return s * 0x10001u;
}
// dims 2 I and 2 I + 1 of a word's eight: one product with a sum of two powers of two
// brings a nibble's sign and its magnitude where they belong at once
template <int I>
__device__ __forceinline__ uint32_t q4_decode2(uint32_t word, uint32_t scale2) {
  const uint32_t w = I < 2 ? word : word >> 8;
  const uint32_t n = I & 1 ? (w & 0x00f000f0u) * 0x104u : (w & 0x000f000fu) * 0x1040u;
  return q4_mul(n & 0x81c081c0u, scale2);
}
// 2^15 and 2^-15 in both halves
constexpr uint32_t Q4_UP2 = ((127 + Q4_SHIFT) << 7) * 0x10001u, Q4_DOWN2 = ((127 - Q4_SHIFT) << 7) * 0x10001u;
