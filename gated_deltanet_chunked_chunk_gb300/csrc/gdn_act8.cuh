// gdn_act8.cuh -- activations as 8-bit codes: e4m3 numbers (gdn_kv8.cuh) with one
// power-of-two scale for each kGroup consecutive elements of a row, the least one (2^-60
// at least) that keeps the group's largest finite magnitude within 448 scales.  What is
// not finite becomes NaN.
#pragma once

#include "gdn_kv8.cuh"
#include "gdn_sm103.cuh"

namespace gdn8 {

constexpr int kGroup = 128;

struct Codes {
  uint2 bits;
  float scale;
};
// Largest finite magnitude of 8 bf16 (of bf16 without their signs, the order is that of
// the bits), and whether all are finite.
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
// Codes of a lane's 8 bf16; GL lanes (a power of two, the whole warp in step) hold a group.
template <int GL> __device__ __forceinline__ Codes encode(const uint4 &v) {
  bool finite;
  uint32_t m = largest(v, finite);
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = gdnkv::scale_exponent(__uint_as_float(m << 16));
  const float f = gdnkv::pow2(-e);
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
  Codes r;
  r.bits = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  r.scale = gdnkv::pow2(e);
  return r;
}

}  // namespace gdn8
