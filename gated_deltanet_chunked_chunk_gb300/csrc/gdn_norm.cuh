// gdn_norm.cuh -- the norm kernels for rows in 16-byte accesses: gdn_norm.cu's, and
// with 8-bit codes of what the backward needs gdn_norm8.cu's.  What they compute, and
// why so, stands in gdn_norm.cu.
#pragma once

#include <initializer_list>

#include "gdn_act8.cuh"
#include "gdn_common.cuh"

namespace {

using namespace gdn;

struct NormArgs {
  const uint16_t *x, *res, *z;
  const float *w;
  float res_scale, eps;
  int64_t rows;
  int D;
  int64_t z_group, z_stride;  // row r of z starts at (r / z_group) z_stride + (r % z_group) D; z_group 0: dense
  uint16_t *y, *h;
  // backward (x holds the normed stream h)
  const uint16_t *dy, *dh;
  uint16_t *dx, *dres, *dz;
  float *part;  // [blocks][D] partial weight gradients
  // 8-bit codes of h and z (dense) and their scales [rows][groups]: outputs of the
  // forward, or what the backward reads in place of x and z
  uint8_t *h8, *z8;
  float *hs, *zs;
  int groups;
};

__device__ __forceinline__ uint4 ld16(const uint16_t *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
__device__ __forceinline__ void st16(uint16_t *p, const uint4 &v) { __stcs(reinterpret_cast<uint4 *>(p), v); }

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_SIGMOID = 2 };
// act(z) and act'(z); s = sigmoid(z).
template <int ACT> __device__ __forceinline__ void act_grad(float z, float &f, float &d) {
  const float s = gdn::sigmoid_fast(z);
  if (ACT == ACT_SILU) {
    f = z * s;
    d = s * fmaf(z, 1.f - s, 1.f);
  } else {
    f = s;
    d = s * (1.f - s);
  }
}

__device__ __forceinline__ int64_t z_offset(const NormArgs &a, int64_t row) {
  if (a.z_group == 0) return row * a.D;  // dense
  if (a.z_group == 1) return row * a.z_stride;
  const int64_t g = row <= 0xffffffffll ? (uint32_t)row / (uint32_t)a.z_group : row / a.z_group;
  return g * a.z_stride + (row - g * a.z_group) * a.D;
}

// Sum over the L lanes (a power of two) that share a row.
template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over a block; every thread gets it.  `sh` holds two sets of 32 floats,
// used in turn, so that one barrier a call is enough.
template <int THREADS> __device__ __forceinline__ float block_sum(float v, float (*sh)[32], int &turn) {
  v = gdn::warp_sum(v);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) sh[turn][w] = v;
  __syncthreads();
  v = lane < THREADS / 32 ? sh[turn][lane] : 0.f;
  turn ^= 1;
  return gdn::warp_sum(v);
}

// L lanes a row (L = THREADS: the block), NV vectors of 8 elements a lane:
// lane l holds the vectors l, l + L, ...
template <int L, int NV, int THREADS> struct Shape {
  static constexpr bool kBlock = L > 32;
  static constexpr int kRows = kBlock ? 1 : THREADS / L;  // rows at once in a block
  // Up to 16 weights a thread stay in registers; more are read in each row, as
  // the registers would spill.
  static constexpr int kKept = NV <= 2 ? NV : 1;
};
template <int NV>
__device__ __forceinline__ void keep_weights(const float *w, int l, int L, int nvec, f2 (*kept)[4]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = l + i * L;
#pragma unroll
    for (int j = 0; j < 4; ++j) kept[i][j] = v < nvec ? f2_of(__ldg(w + v * 8 + 2 * j), __ldg(w + v * 8 + 2 * j + 1)) : f2_both(0.f);
  }
}
template <int NV> __device__ __forceinline__ void weights8(const float *w, const f2 (*kept)[4], int i, int v, f2 *o) {
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = NV <= 2 ? kept[NV <= 2 ? i : 0][j] : f2_of(__ldg(w + v * 8 + 2 * j), __ldg(w + v * 8 + 2 * j + 1));
}
__device__ __forceinline__ void unpack8(const uint4 &v, f2 *f) {
  f[0] = f2_bf16(v.x);
  f[1] = f2_bf16(v.y);
  f[2] = f2_bf16(v.z);
  f[3] = f2_bf16(v.w);
}
// The 8 numbers of a 16-byte place: bf16, or codes and their scale.
template <bool C8> __device__ __forceinline__ void values8(const uint4 &v, f2 *f) {
  if (!C8) {
    unpack8(v, f);
  } else {
    const f2 s = f2_both(__uint_as_float(v.z));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = gdnkv::f16x2_f32(gdnkv::e4m3x2_f16x2((j < 2 ? v.x : v.y) >> (16 * (j & 1))));
      f[j] = f2_mul(f2_of(x.x, x.y), s);
    }
  }
}
__device__ __forceinline__ uint4 pack8(const f2 *f) {
  return make_uint4(f2_to_bf16(f[0]), f2_to_bf16(f[1]), f2_to_bf16(f[2]), f2_to_bf16(f[3]));
}
__device__ __forceinline__ float f2_sum(f2 a) {
  const float2 x = f2_get(a);
  return x.x + x.y;
}

// The codes of a lane's 8 bf16 of h and (GATE) of z, whose groups' other elements are with
// the GL lanes around it, and the groups' scales; `on`: it has some.
template <int GL, bool GATE>
__device__ __forceinline__ void encode_row(const uint4 &h, const uint4 &z, bool on, bool first, uint8_t *h8, float *hs, uint8_t *z8, float *zs) {
  bool h_finite, z_finite = true;
  uint32_t m = gdn8::largest(h, h_finite);
  if (GATE) m |= gdn8::largest(z, z_finite) << 16;  // both maxima in one word
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!on) return;
  const int eh = gdn8::exponent_of(m & 0xffffu);
  __stcs(reinterpret_cast<uint2 *>(h8), gdn8::codes8(h, gdnkv::pow2(-eh), h_finite));
  if (first) __stcs(hs, gdnkv::pow2(eh));
  if (GATE) {
    const int ez = gdn8::exponent_of(m >> 16);
    __stcs(reinterpret_cast<uint2 *>(z8), gdn8::codes8(z, gdnkv::pow2(-ez), z_finite));
    if (first) __stcs(zs, gdnkv::pow2(ez));
  }
}

// C8: codes of h and of z are written as well.  (262144 rows of 128 with a SiLU gate: 53 us,
// 5.0 TB/s, at four blocks an SM; 63 at three, 56 at five, whose registers are too few.)
template <int L, int NV, int THREADS, int ACT, bool RES, bool C8>
__global__ void __launch_bounds__(THREADS, C8 && NV == 1 ? 1024 / THREADS : 1) norm_fwd_kernel(const NormArgs a) {
  using S = Shape<L, NV, THREADS>;
  __shared__ float sh[2][32];
  grid_release();
  grid_wait();
  int turn = 0;
  const int l = S::kBlock ? (int)threadIdx.x : (int)(threadIdx.x % L);
  const int nvec = a.D / 8;
  const float inv_d = 1.f / (float)a.D;
  f2 w[S::kKept][4];
  keep_weights<S::kKept>(a.w, l, L, nvec, w);
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  // every lane of a warp takes every trip, as the shuffles need them all
  for (int64_t row0 = (int64_t)blockIdx.x * S::kRows; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + (S::kBlock ? 0 : threadIdx.x / L);
    const bool in = row < a.rows;
    const int64_t at = row * a.D, zat = (ACT != ACT_NONE && in) ? z_offset(a, row) : 0;
    uint4 xv[NV], zv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      const bool on = in && v < nvec;
      xv[i] = on ? ld16(a.x + at + v * 8) : make_uint4(0, 0, 0, 0);
      if (RES) rv[i] = on ? ld16(a.res + at + v * 8) : make_uint4(0, 0, 0, 0);
      if (ACT != ACT_NONE) zv[i] = on ? ld16(a.z + zat + v * 8) : make_uint4(0, 0, 0, 0);
    }
    f2 h[NV][4], s2 = f2_both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack8(xv[i], h[i]);
      if (RES) {
        f2 r[4];
        unpack8(rv[i], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = f2_fma(f2_both(a.res_scale), h[i][j], r[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = f2_fma(h[i][j], h[i][j], s2);
    }
    float ss = f2_sum(s2);
    ss = S::kBlock ? block_sum<THREADS>(ss, sh, turn) : lanes_sum<S::kBlock ? 32 : L>(ss);
    const f2 rstd = f2_both(rsqrtf(fmaf(ss, inv_d, a.eps)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (!in || v >= nvec) continue;
      f2 z[4], y[4], wi[4];
      weights8<NV>(a.w, w, i, v, wi);
      if (ACT != ACT_NONE) unpack8(zv[i], z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = f2_mul(f2_mul(h[i][j], rstd), wi[j]);
        if (ACT == ACT_SILU) y[j] = f2_mul(y[j], f2_mul(z[j], f2_sigmoid(z[j])));
        if (ACT == ACT_SIGMOID) y[j] = f2_mul(y[j], f2_sigmoid(z[j]));
      }
      st16(a.y + at + v * 8, pack8(y));
      if (RES) st16(a.h + at + v * 8, pack8(h[i]));
    }
    if (C8) {
      constexpr int GL = L < 16 ? L : 16;
#pragma unroll
      for (int i = 0; i < NV; ++i) {  // every lane: the shuffles need them all
        const int v = l + i * L;
        const bool on = in && v < nvec;
        const int64_t s = row * a.groups + v / 16;
        // the stream as it is stored
        encode_row<GL, ACT != ACT_NONE>(RES ? pack8(h[i]) : xv[i], zv[i], on, v % 16 == 0, a.h8 + at + v * 8, a.hs + s, a.z8 + at + v * 8,
                                        a.zs + s);
      }
    }
  }
}

// A row's vectors come through a ring in shared memory by asynchronous copies,
// kAhead rows ahead; a thread copies and reads places of its own only, so no
// barrier is needed.  262144 rows of 128 with a SiLU gate: 56.4 us for both
// kernels (5.95 TB/s), three rows ahead 57.6; loads to registers took 10 us more.
__device__ __forceinline__ void copy16(void *dst, const uint16_t *src, bool on) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(on ? 16 : 0) : "memory");
}

template <int BYTES> __device__ __forceinline__ void copy_small(void *dst, const void *src, bool on) {  // 4 or 8
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(on ? BYTES : 0) : "memory");
}
// A stage of the ring: kTensors 16-byte places of each vector of each thread and, with codes,
// kCoded 8-byte ones, behind which the groups' scales stand (one for each 8 lanes at most).
template <int NV, int THREADS, int ACT, bool RES, bool C8> struct Stage {
  static constexpr int kGate = ACT != ACT_NONE ? 1 : 0;
  static constexpr int kTensors = C8 ? 1 + (RES ? 1 : 0) : 2 + kGate + (RES ? 1 : 0);
  static constexpr int kCoded = C8 ? 1 + kGate : 0;
  static constexpr int kCodes = kTensors * NV * THREADS * 16, kScales = kCodes + kCoded * NV * THREADS * 8;
  static constexpr int kBytes = kScales + kCoded * NV * (THREADS / 8) * 4;
  static constexpr int kAhead = NV <= 2 ? 2 : 1;
};

// C8: h and z come as codes, a group's scale by the copy of its first lane.  (262144 rows of
// 128 with a SiLU gate: 60 us, 4.5 TB/s, 70 % of the issue slots; 81 with loads to registers a
// row ahead, 60 with three or four rows ahead.)
template <int L, int NV, int THREADS, int ACT, bool RES, bool C8>
__global__ void __launch_bounds__(THREADS, (NV == 1 && L <= 32) ? 4 : 1) norm_bwd_kernel(const NormArgs a) {
  using S = Shape<L, NV, THREADS>;
  using R = Stage<NV, THREADS, ACT, RES, C8>;
  constexpr int kAhead = R::kAhead, kTensors = R::kTensors;
  extern __shared__ uint4 ring[];  // [kAhead] stages, then the blocks' sums
  __shared__ float sh[2][32];
  grid_wait();
  int turn = 0;
  const int l = S::kBlock ? (int)threadIdx.x : (int)(threadIdx.x % L);
  const int nvec = a.D / 8;
  const float inv_d = 1.f / (float)a.D;
  f2 w[S::kKept][4], dw[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = f2_both(0.f);
  keep_weights<S::kKept>(a.w, l, L, nvec, w);
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  const int rg = S::kBlock ? 0 : (int)threadIdx.x / L;
  auto place = [&](int stage, int tensor, int i) { return ring + stage * (R::kBytes / 16) + (tensor * NV + i) * THREADS + threadIdx.x; };
  auto code = [&](int stage, int which, int i) {
    return reinterpret_cast<uint2 *>(reinterpret_cast<char *>(ring) + stage * R::kBytes + R::kCodes) + (which * NV + i) * THREADS + threadIdx.x;
  };
  auto scale = [&](int stage, int which, int i) {  // the group's: of 16 lanes, or of the 8 of a short row
    return reinterpret_cast<float *>(reinterpret_cast<char *>(ring) + stage * R::kBytes + R::kScales) + (which * NV + i) * (THREADS / 8) +
           threadIdx.x / (L < 16 ? 8 : 16);
  };
  auto call = [&](int64_t row, int stage) {
    const bool in = row < a.rows;
    const int64_t at = in ? row * a.D : 0, zat = (ACT != ACT_NONE && !C8 && in) ? z_offset(a, row) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      const bool on = in && v < nvec;
      const int e = on ? v * 8 : 0;
      const int64_t g = C8 && on ? row * a.groups + v / 16 : 0;
      if (C8) {
        copy_small<8>(code(stage, 0, i), a.h8 + at + e, on);
        if (l % (L < 16 ? 8 : 16) == 0) copy_small<4>(scale(stage, 0, i), a.hs + g, on);
        if (ACT != ACT_NONE) {
          copy_small<8>(code(stage, 1, i), a.z8 + at + e, on);
          if (l % (L < 16 ? 8 : 16) == 0) copy_small<4>(scale(stage, 1, i), a.zs + g, on);
        }
        copy16(place(stage, 0, i), a.dy + at + e, on);
      } else {
        copy16(place(stage, 0, i), a.x + at + e, on);
        copy16(place(stage, 1, i), a.dy + at + e, on);
        if (ACT != ACT_NONE) copy16(place(stage, 2, i), a.z + zat + e, on);
      }
      if (RES) copy16(place(stage, kTensors - 1, i), a.dh + at + e, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int64_t first = (int64_t)blockIdx.x * S::kRows;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) call(first + k * step + rg, k);
  int stage = 0;
  // every lane of a warp takes every trip, as the shuffles need them all
  for (int64_t row0 = first; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + rg;
    const bool in = row < a.rows;
    const int64_t at = row * a.D;
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    if (C8) __syncwarp();  // a group's scale is its first lane's copy
    uint4 xc[NV], yc[NV], zc[NV], gc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (C8) {
        auto coded = [&](int which) {
          const uint2 c = *code(stage, which, i);
          return make_uint4(c.x, c.y, __float_as_uint(*scale(stage, which, i)), 0);
        };
        xc[i] = coded(0);
        if (ACT != ACT_NONE) zc[i] = coded(1);
        yc[i] = *place(stage, 0, i);
      } else {
        xc[i] = *place(stage, 0, i);
        yc[i] = *place(stage, 1, i);
        if (ACT != ACT_NONE) zc[i] = *place(stage, 2, i);
      }
      if (RES) gc[i] = *place(stage, kTensors - 1, i);
    }
    if (C8) __syncwarp();  // all have read it before the next one comes
    call(row + kAhead * step, stage);
    stage = stage + 1 == kAhead ? 0 : stage + 1;
    // First pass: the sums of h^2 and of p h, p = dy w act(z).  The sigmoid stays
    // where a lane's registers hold it (16 numbers at most); the rest is formed
    // again in the second pass, which costs less than the registers would.
    constexpr bool kKeep = NV <= 2;
    f2 sg[kKeep ? NV : 1][4];
    f2 s2 = f2_both(0.f), p2 = f2_both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      f2 h[4], dy[4], z[4], wi[4];
      if (v < nvec) weights8<NV>(a.w, w, i, v, wi);
      else continue;
      values8<C8>(xc[i], h);
      unpack8(yc[i], dy);
      if (ACT != ACT_NONE) values8<C8>(zc[i], z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f2 p = f2_mul(dy[j], wi[j]);
        if (ACT != ACT_NONE) {
          const f2 s = f2_sigmoid(z[j]);
          if (kKeep) sg[i][j] = s;
          p = f2_mul(p, ACT == ACT_SILU ? f2_mul(z[j], s) : s);
        }
        s2 = f2_fma(h[j], h[j], s2);
        p2 = f2_fma(p, h[j], p2);
      }
    }
    float ss = f2_sum(s2), sp = f2_sum(p2);
    if (S::kBlock) {
      ss = block_sum<THREADS>(ss, sh, turn);
      sp = block_sum<THREADS>(sp, sh, turn);
    } else {
      ss = lanes_sum<S::kBlock ? 32 : L>(ss);
      sp = lanes_sum<S::kBlock ? 32 : L>(sp);
    }
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
    // dH = r (p - n mean(p n)) = r p - h r^3 mean(p h)
    const f2 r2 = f2_both(rstd), c2 = f2_both(-sp * inv_d * rstd * rstd * rstd), scale2 = f2_both(a.res_scale);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (!in || v >= nvec) continue;
      f2 h[4], dy[4], z[4], wi[4], g[4], dx[4], dr[4], dz[4];
      weights8<NV>(a.w, w, i, v, wi);
      values8<C8>(xc[i], h);
      unpack8(yc[i], dy);
      if (ACT != ACT_NONE) values8<C8>(zc[i], z);
      if (RES) unpack8(gc[i], g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 n = f2_mul(h[j], r2);
        f2 u = dy[j], p = f2_mul(dy[j], wi[j]);
        if (ACT != ACT_NONE) {
          const f2 s = kKeep ? sg[kKeep ? i : 0][j] : f2_sigmoid(z[j]);
          const f2 r = f2_fma(s, f2_both(-1.f), f2_both(1.f));  // 1 - sigmoid
          const f2 f = ACT == ACT_SILU ? f2_mul(z[j], s) : s;
          dz[j] = f2_mul(f2_mul(p, n), ACT == ACT_SILU ? f2_fma(f, r, s) : f2_mul(s, r));
          u = f2_mul(u, f);
          p = f2_mul(p, f);
        }
        dw[i][j] = f2_fma(u, n, dw[i][j]);
        f2 t = f2_fma(p, r2, f2_mul(h[j], c2));
        if (RES) t = f2_add(t, g[j]);
        dr[j] = t;
        dx[j] = f2_mul(scale2, t);
      }
      st16(a.dx + at + v * 8, pack8(dx));
      if (RES) st16(a.dres + at + v * 8, pack8(dr));
      if (ACT != ACT_NONE) st16(a.dz + at + v * 8, pack8(dz));
    }
  }
  // the kernel that adds the partial rows may come in; it waits for this grid
  grid_release();
  float *part = a.part + (int64_t)blockIdx.x * a.D;
  if (S::kBlock) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (v >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = f2_get(dw[i][j]);
        *reinterpret_cast<float2 *>(part + v * 8 + 2 * j) = x;
      }
    }
  } else {
    // the row groups' sums, added in order
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float *sums = reinterpret_cast<float *>(ring);  // [kRows][L NV 8]
    constexpr int W = L * NV * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<float2 *>(sums + rg * W + (l + i * L) * 8 + 2 * j) = f2_get(dw[i][j]);
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += THREADS) {
      float s = 0.f;
      for (int r = 0; r < S::kRows; ++r) s += sums[r * W + e];
      part[e] = s;
    }
  }
}

// dw[e] = sum over the partial rows: 32 columns a block, 32 shares of the rows
// (share s has the rows s, s + 32, ..), added in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *__restrict__ part, int blocks, int D,
                                                       float *__restrict__ dw) {
  __shared__ float sh[32][33];
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  grid_wait();
  float v = 0.f;
  if (e < D) {
#pragma unroll 8
    for (int b = s; b < blocks; b += 32) v += part[(int64_t)b * D + e];
  }
  sh[s][c] = v;
  __syncthreads();
  if (s == 0 && e < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][c];
    dw[e] = t;
  }
}

template <int L, int NV, int THREADS, int ACT, bool RES, bool C8>
cudaError_t launch_bwd(const NormArgs &a, int blocks, cudaStream_t s) {
  using S = Shape<L, NV, THREADS>;
  using R = Stage<NV, THREADS, ACT, RES, C8>;
  constexpr int ring = R::kAhead * R::kBytes, sums = S::kBlock ? 0 : S::kRows * L * NV * 32;
  constexpr int bytes = ring > sums ? ring : sums;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = gdn_host::allow_smem(norm_bwd_kernel<L, NV, THREADS, ACT, RES, C8>, bytes, done);
  if (e != cudaSuccess) return e;
  return gdn_host::launch_dependent(norm_bwd_kernel<L, NV, THREADS, ACT, RES, C8>, dim3(blocks), THREADS, bytes, s, a);
}
template <bool BWD, bool C8, int L, int NV, int THREADS, int ACT>
cudaError_t launch_one(const NormArgs &a, int blocks, cudaStream_t s) {
  const bool res = BWD ? a.dh != nullptr : a.res != nullptr;
  if (BWD) return res ? launch_bwd<L, NV, THREADS, ACT, true, C8>(a, blocks, s) : launch_bwd<L, NV, THREADS, ACT, false, C8>(a, blocks, s);
  return res ? gdn_host::launch_dependent(norm_fwd_kernel<L, NV, THREADS, ACT, true, C8>, dim3(blocks), THREADS, 0, s, a)
             : gdn_host::launch_dependent(norm_fwd_kernel<L, NV, THREADS, ACT, false, C8>, dim3(blocks), THREADS, 0, s, a);
}
template <bool BWD, bool C8, int L, int NV, int THREADS>
cudaError_t launch_act(const NormArgs &a, int act, int blocks, cudaStream_t s) {
  if (act == ACT_NONE) return launch_one<BWD, C8, L, NV, THREADS, ACT_NONE>(a, blocks, s);
  if (act == ACT_SILU) return launch_one<BWD, C8, L, NV, THREADS, ACT_SILU>(a, blocks, s);
  return launch_one<BWD, C8, L, NV, THREADS, ACT_SIGMOID>(a, blocks, s);
}

// Lanes a row, vectors a lane and threads a block for a width; L = 0: none.
struct Plan { int L, NV, threads, rows; };
Plan plan_of(int D, bool aligned) {
  const int v = D / 8;
  if (!aligned || D % 8 || D > 16384) return {0, 0, 256, 1};
  if (v <= 8) return {8, 1, 256, 32};
  if (v <= 16) return {16, 1, 256, 16};
  if (v <= 32) return {32, 1, 256, 8};
  if (v <= 64) return {32, 2, 256, 8};
  if (v <= 128) return {32, 4, 256, 8};
  if (v <= 256) return {256, 1, 256, 1};
  if (v <= 512) return {256, 2, 256, 1};
  if (v <= 1024) return {512, 2, 512, 1};
  return {512, 4, 512, 1};
}
template <bool BWD, bool C8> cudaError_t dispatch(const NormArgs &a, int act, const Plan &p, int blocks, cudaStream_t s) {
  if (p.L == 8) return launch_act<BWD, C8, 8, 1, 256>(a, act, blocks, s);
  if (p.L == 16) return launch_act<BWD, C8, 16, 1, 256>(a, act, blocks, s);
  if (p.L == 32 && p.NV == 1) return launch_act<BWD, C8, 32, 1, 256>(a, act, blocks, s);
  if (p.L == 32 && p.NV == 2) return launch_act<BWD, C8, 32, 2, 256>(a, act, blocks, s);
  if (p.L == 32) return launch_act<BWD, C8, 32, 4, 256>(a, act, blocks, s);
  if (p.L == 256 && p.NV == 1) return launch_act<BWD, C8, 256, 1, 256>(a, act, blocks, s);
  if (p.L == 256) return launch_act<BWD, C8, 256, 2, 256>(a, act, blocks, s);
  if (p.L == 512 && p.NV == 2) return launch_act<BWD, C8, 512, 2, 512>(a, act, blocks, s);
  if (p.L == 512) return launch_act<BWD, C8, 512, 4, 512>(a, act, blocks, s);
  return cudaErrorInvalidValue;  // p.L = 0: not for these kernels
}

bool vec_ok(std::initializer_list<const void *> ptrs, bool has_z, int64_t z_stride) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return !has_z || z_stride % 8 == 0;
}

constexpr int kPartBlocks = 152 * 4;  // most blocks (partial rows) of the backward

// Blocks of the backward.
inline int bwd_blocks(const Plan &p, int64_t rows, int D) {
  const int64_t want = (rows + p.rows - 1) / p.rows;
  // A block leaves a partial row of the weight's gradient, 4 D bytes written and
  // read again: wide rows, which few blocks fill an SM with, take as few blocks as
  // that (4 an SM against 1: 1000 rows of 4096 24.6 us against 15.4, 30000 rows 233
  // against 220; 2 at 8192 rows of 2048: 43.1 against 40.7).  All blocks take
  // the same number of turns, or one less.
  const int64_t cap = p.L < 256 ? kPartBlocks : D > 2048 ? kPartBlocks / 4 : kPartBlocks / 2;
  const int64_t turns = (want + cap - 1) / cap;
  return turns > 0 ? (int)((want + turns - 1) / turns) : 0;
}

}  // namespace
