// gdn_rope.cu -- rotary positions for the queries and keys of the attention
// layers: both pair layouts, a part of the head, any token stride.
//
//   (a, b) -> f (a cos t - b sin t, a sin t + b cos t),   t = position inv_freq[i]
//
// for pair i < rot / 2: elements (i, i + rot / 2), or (2 i, 2 i + 1) when
// interleaved; elements from rot on pass unchanged.  The inverse (the
// backward: the matrix is f times a rotation, and its transpose turns the
// other way) takes -t.
//
// The angle.  position inv_freq in fp32 loses 2^-24 of an angle that reaches
// 10^5 and more, so it is reduced exactly: inv_freq / 2 pi, in turns, is taken
// in fp64 once a thread and held as a 64-bit binary fraction of a turn; the
// product with the position modulo 2^64 is then one integer multiplication
// whose overflow drops whole turns, and its top 32 bits are the angle with an
// error below 2^-32 turns + 2^-53 |angle|.
//
// Bound: HBM, q and k are read and written once.  A block takes a tile of
// tokens, writes the tile's cosines and sines to shared memory once, and
// applies them to every head of q and k; a thread keeps one place in the head
// (one vector of 8, or two 8-vectors half a rotation apart) and walks over
// (token, head).
#include "gdn_common.cuh"

namespace {

using gdn::bf2f;
using gdn::f2bf;

struct RopeArgs {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  int64_t ldq, ldk;  // token strides of the inputs, in elements; the outputs are dense
  const int32_t *pos;
  const float *inv_freq;
  int64_t T;
  int HQ, HK, D, rot, inverse, interleaved;
  float factor;
  int tile;  // tokens a block
};

__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

__device__ __forceinline__ void tile_angles(const RopeArgs &a, float2 *cs, int64_t t0, int n) {
  const int half = a.rot / 2;
  for (int e = threadIdx.x; e < n * half; e += blockDim.x) {
    const int t = e / half, i = e - t * half;
    const uint64_t ph = (uint64_t)(int64_t)a.pos[t0 + t] * turn_fraction(__ldg(a.inv_freq + i));
    const float x = (float)(int32_t)(uint32_t)(ph >> 32) * 4.656612873077393e-10f;  // half turns, in [-1, 1)
    float s, c;
    sincospif(x, &s, &c);
    cs[e] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
}

__device__ __forceinline__ void unpack8(const uint4 &v, float *f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// 16-byte accesses: rot / 2 (or rot, interleaved) and D are multiples of 8.
// Places in a head: rotated ones first (a pair of vectors each in the half
// layout, a vector each when interleaved), then the vectors that pass.
template <bool INTER>
__global__ void __launch_bounds__(256, 8) rope_vec_kernel(const RopeArgs a, int places, int rows_at_once) {
  gdn::grid_release();
  gdn::grid_wait();
  extern __shared__ float2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int n = (int)(a.T - t0 < a.tile ? a.T - t0 : a.tile);
  tile_angles(a, cs, t0, n);
  __syncthreads();
  const int half = a.rot / 2, H = a.HQ + a.HK;
  const int turned = INTER ? a.rot / 8 : a.rot / 16;
  const int r0 = threadIdx.x / places, u = threadIdx.x - r0 * places;
  if (r0 >= rows_at_once) return;
  int t = r0 / H, h = r0 - t * H;
  const int dt = rows_at_once / H, dh = rows_at_once - dt * H;
  const bool pass = u >= turned;  // this thread's place is not turned
  const int e0 = pass ? a.rot + (u - turned) * 8 : u * 8, e1 = e0 + half;
  // Two (token, head) rows a trip, both loads issued before either is used:
  // eight blocks of 32 registers a thread on a SM measured 184 us for 65536 x 36
  // heads of 128, one row a trip 198, three (more registers) 199.
  constexpr int U = 2;
  while (t < n) {
    const uint16_t *in[U];
    uint16_t *out[U];
    int tt[U];
    uint4 v0[U], v1[U];
    bool on[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      on[i] = t < n;
      tt[i] = t;
      const int64_t tok = t0 + t;
      const bool isq = h < a.HQ;
      in[i] = isq ? a.q + tok * a.ldq + (int64_t)h * a.D : a.k + tok * a.ldk + (int64_t)(h - a.HQ) * a.D;
      out[i] = isq ? a.qo + (tok * a.HQ + h) * a.D : a.ko + (tok * a.HK + h - a.HQ) * a.D;
      if (on[i]) {
        if (!pass || in[i] != out[i]) v0[i] = __ldcs(reinterpret_cast<const uint4 *>(in[i] + e0));
        if (!INTER && !pass) v1[i] = __ldcs(reinterpret_cast<const uint4 *>(in[i] + e1));
      }
      t += dt;
      h += dh;
      if (h >= H) {
        h -= H;
        ++t;
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!on[i]) continue;
      if (pass) {
        if (in[i] != out[i]) __stcs(reinterpret_cast<uint4 *>(out[i] + e0), v0[i]);
        continue;
      }
      float x[8], y[8];
      unpack8(v0[i], x);
      if (INTER) {
        const float2 *c = cs + tt[i] * half + u * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 w = c[j];
          y[2 * j] = x[2 * j] * w.x - x[2 * j + 1] * w.y;
          y[2 * j + 1] = x[2 * j] * w.y + x[2 * j + 1] * w.x;
        }
        __stcs(reinterpret_cast<uint4 *>(out[i] + e0), pack8(y));
      } else {
        float z[8], v[8];
        unpack8(v1[i], z);
        const float2 *c = cs + tt[i] * half + u * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 w = c[j];
          y[j] = x[j] * w.x - z[j] * w.y;
          v[j] = x[j] * w.y + z[j] * w.x;
        }
        __stcs(reinterpret_cast<uint4 *>(out[i] + e0), pack8(y));
        __stcs(reinterpret_cast<uint4 *>(out[i] + e1), pack8(v));
      }
    }
  }
}

// Any even rot, any D, any alignment: one pair, or one element that passes, a step.
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeArgs a) {
  extern __shared__ float2 cs[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int n = (int)(a.T - t0 < a.tile ? a.T - t0 : a.tile);
  tile_angles(a, cs, t0, n);
  __syncthreads();
  const int half = a.rot / 2, H = a.HQ + a.HK, places = a.D - half;
  for (int64_t e = threadIdx.x; e < (int64_t)n * H * places; e += blockDim.x) {
    const int64_t r = e / places;
    const int u = (int)(e - r * places), t = (int)(r / H), h = (int)(r - (int64_t)t * H);
    const bool isq = h < a.HQ;
    const uint16_t *in = isq ? a.q + (t0 + t) * a.ldq + (int64_t)h * a.D : a.k + (t0 + t) * a.ldk + (int64_t)(h - a.HQ) * a.D;
    uint16_t *out = isq ? a.qo + ((t0 + t) * a.HQ + h) * a.D : a.ko + ((t0 + t) * a.HK + h - a.HQ) * a.D;
    if (u >= half) {
      out[half + u] = in[half + u];
      continue;
    }
    const int i = a.interleaved ? 2 * u : u, j = a.interleaved ? 2 * u + 1 : u + half;
    const float x = bf2f(in[i]), z = bf2f(in[j]);
    const float2 w = cs[t * half + u];
    out[i] = f2bf(x * w.x - z * w.y);
    out[j] = f2bf(x * w.y + z * w.x);
  }
}

}  // namespace

namespace gdn_host {

cudaError_t launch_rope(const uint16_t *q, const uint16_t *k, const int32_t *pos, const float *inv_freq, int64_t T, int HQ,
                        int HK, int D, int rot, int interleaved, int inverse, float factor, int64_t ldq, int64_t ldk,
                        uint16_t *qo, uint16_t *ko, cudaStream_t s) {
  const int sms = sm_count();
  RopeArgs a{q, k, qo, ko, ldq, ldk, pos, inv_freq, T, HQ, HK, D, rot, inverse, interleaved, factor, 1};
  // Tokens a block: 8 once the grid fills the SMs several times over (16: 193
  // against 184 us), fewer below that; the tile's angles (rot / 2 pairs of 8 bytes a token) stay
  // within 32 KB.
  int64_t tile = T / ((int64_t)sms * 8);
  const int64_t most = (32 << 10) / ((int64_t)(rot / 2) * 8 + 1);
  if (tile > 8) tile = 8;
  if (tile > most) tile = most;
  if (tile < 1) tile = 1;
  if ((T + tile - 1) / tile > 2147483647LL) return cudaErrorInvalidValue;
  a.tile = (int)tile;
  const int grid = (int)((T + tile - 1) / tile);
  const size_t smem = (size_t)tile * (size_t)(rot / 2) * sizeof(float2);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(qo) |
                         reinterpret_cast<uintptr_t>(ko);
  const bool vec = !(bits & 15) && D % 8 == 0 && rot % (interleaved ? 8 : 16) == 0 && ldq % 8 == 0 && ldk % 8 == 0;
  const int places = vec ? (interleaved ? D / 8 : D / 8 - rot / 16) : 0;
  if (vec && places <= 256) {
    return interleaved ? launch_dependent(rope_vec_kernel<true>, dim3(grid), 256, smem, s, a, places, 256 / places)
                       : launch_dependent(rope_vec_kernel<false>, dim3(grid), 256, smem, s, a, places, 256 / places);
  }
  rope_any_kernel<<<grid, 256, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn_host
