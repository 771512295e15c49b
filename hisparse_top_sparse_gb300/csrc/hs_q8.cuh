// The q8 latent row (HS_Q8_ROW_BYTES bytes) and the conversions its kernels share.
//
//   [0, 512)    e4m3 codes of dims 0..511
//   [512, 640)  dims 512..575 (rope) in bf16, as they are
//   [640, 656)  one byte e + 127 for each 32 dims of the first 512
//
// The value of a code is code * 2^e. e is the smallest integer whose largest
// code, 448 * 2^e, reaches the group's largest magnitude, so no finite value
// saturates; a power of two (rather than amax / 448) makes the products of
// code and scale exact: an e4m3 code has four significant bits, so every
// value of a q8 row is a bf16 number, and reading a row back, in bf16 inside
// the attention or in either type by hs_dequant_rows, rounds nothing. e stays
// within [-112, 120]: below, the smallest step is 2^-121 and every non-zero
// value is still a normal number; at 120 the largest code is past the largest
// finite float, which is how an infinity is kept (see q8_exponent).
#pragma once

#include <cuda_fp8.h>

#include "hs_internal.cuh"

constexpr int Q8_GROUP = 32;
constexpr int Q8_ROPE_OFF = HS_VALUE_DIM;                                   // 512
constexpr int Q8_SCALE_OFF = Q8_ROPE_OFF + 2 * (HS_LATENT_DIM - HS_VALUE_DIM);   // 640
static_assert(Q8_SCALE_OFF + HS_VALUE_DIM / Q8_GROUP == HS_Q8_ROW_BYTES, "q8 row");
constexpr int Q8_E_MIN = -112, Q8_E_MAX = 120;

// Biased exponent byte of a group whose largest magnitude is amax (NaNs left
// out). 448 = 1.75 * 2^8, so with amax = f * 2^k (1 <= f < 2) it is k - 8, or
// k - 7 when f > 1.75. amax = inf gives Q8_E_MAX: the infinity saturates to
// code 448, and 448 * 2^120 is infinite again in f32 and bf16.
__device__ __forceinline__ uint32_t q8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  if (e < Q8_E_MIN) e = Q8_E_MIN;
  if (e > Q8_E_MAX) e = Q8_E_MAX;
  return (uint32_t)(e + 127);
}
// 2^-e of a byte that q8_exponent returned (15 .. 247)
__device__ __forceinline__ float q8_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// 2^e; byte 0 (a row never written) gives 0
__device__ __forceinline__ float q8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two values to two codes, to nearest even; NaN -> 0x7F.
__device__ __forceinline__ uint32_t q8_encode2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Codes i and i + 1 (i = 0 or 2) of a word, times scale, in f32: exact.
__device__ __forceinline__ float2 q8_decode2(uint32_t word, int i, float scale) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (8 * i)), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return make_float2(f.x * scale, f.y * scale);
}
// The four codes of a word, times (scale, scale) packed, as two bf16 pairs:
// exact. Five instructions a pair (one to f16, two to f32, one product of
// two, one to bf16); taking the bits apart instead costs as many.
__device__ __forceinline__ uint64_t q8_scale2(uint32_t byte) {
  const uint32_t s = byte << 23;
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(r) : "r"(s));
  return r;
}
__device__ __forceinline__ uint2 q8_decode4_bf16(uint32_t word, uint64_t scale2) {
  uint32_t out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 f = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * k)), __NV_E4M3)));
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(f.x), "f"(f.y));
    asm("mul.rn.f32x2 %0, %0, %1;\n" : "+l"(v) : "l"(scale2));
    float a, b;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    out[k] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint2(out[0], out[1]);
}
