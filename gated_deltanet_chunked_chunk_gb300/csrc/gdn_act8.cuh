// gdn_act8.cuh -- activations as 8-bit codes: e4m3 numbers (gdn_kv8.cuh) with one
// power-of-two scale for each kGroup consecutive elements of a row, the least one (2^-60
// at least) that keeps the group's largest finite magnitude within 448 scales.  What is
// not finite becomes NaN.
#pragma once

#include "gdn_kv8.cuh"
#include "gdn_sm103.cuh"

namespace gdn8 {

constexpr int kGroup = 128;

// Largest finite magnitude of 8 bf16, as their bits (without signs the order is theirs),
// and whether all are finite.
__device__ __forceinline__ uint32_t largest(const uint4 &v, bool &finite) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
  m = max(m & 0xffffu, m >> 16);
  finite = m < 0x7f80u;
  if (!finite) {
    m = 0;
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = w[i / 2] >> (16 * (i & 1)) & 0xffffu;
      if (x < 0x7f80u) m = max(m, x);
    }
  }
  return m;
}
// The exponent of a group whose largest magnitude has these bits.
__device__ __forceinline__ int exponent_of(uint32_t m) { return gdnkv::scale_exponent(__uint_as_float(m << 16)); }
// Codes of 8 bf16 times f = 2^-e.
__device__ __forceinline__ uint2 codes8(const uint4 &v, float f, bool finite) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = gdnkv::cvt_e4m3x2(gdn::bf16lo_f(w[i]) * f, gdn::bf16hi_f(w[i]) * f);
  if (!finite) {  // the conversion takes infinities to 448
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) c[i] |= 0x7fu;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) c[i] |= 0x7f00u;
    }
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

}  // namespace gdn8
