// gdn_kv8.cuh -- the 8-bit cache's number format, shared by its write and by
// the attention that reads it.
//
// A code is an e4m3 number (3 bits after the leading one, largest value
// 448 = 1.75 2^8, smallest step 2^-9); a page's values of one head are its
// codes times 2^e, with one e for K and one for V.  e is the least exponent
// that keeps the page's largest magnitude within 448 2^e, and at least -60, so
// that differences of two exponents stay inside the range of fp32.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdnkv {

constexpr int kExpMin = -60;

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Least e >= kExpMin with amax <= 448 2^e.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kExpMin ? kExpMin : e;
}
// Least exponent e, -60 to 126, with 2^e not below a scale; for those that an append
// wrote (powers of two) the scale is 2^e.
__device__ __forceinline__ int exponent_over(float scale) {
  const uint32_t u = __float_as_uint(scale) & 0x7fffffffu;
  const int e = (int)(u >> 23) - 127 + ((u & 0x7fffffu) ? 1 : 0);
  return e < kExpMin ? kExpMin : e > 126 ? 126 : e;
}

// Two numbers rounded to e4m3 (to nearest, ties to even; beyond 448, and
// infinities, to 448): `lo` in bits 0-7, `hi` in bits 8-15.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes as an f16x2 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  const uint16_t c = (uint16_t)codes;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four codes as two f16x2 pairs.
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t codes, uint32_t &lo, uint32_t &hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  float2 r;
  asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
// Four codes multiplied by f and rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float f) {
  const float2 a = f16x2_f32(e4m3x2_f16x2(c)), b = f16x2_f32(e4m3x2_f16x2(c >> 16));
  return cvt_e4m3x2(a.x * f, a.y * f) | (cvt_e4m3x2(b.x * f, b.y * f) << 16);
}

}  // namespace gdnkv
