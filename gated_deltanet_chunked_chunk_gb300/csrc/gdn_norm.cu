// gdn_norm.cu -- RMS norm of a block's output or of the residual stream, fused
// with the gate, the residual addition and its scale; forward and backward.
//
//   h = x                         or  residual + res_scale x
//   r = 1 / sqrt(mean(h^2) + eps)      (one value a row of D elements)
//   y = h r w act(z)              act: 1, z sigmoid(z) or sigmoid(z)
//
// Backward, given dy and (with a residual) the gradient dh of the stream, with
// n = h r, u = dy act(z), p = u w:
//   dH = dh + r (p - n mean(p n)),  dx = res_scale dH,  dresidual = dH
//   dz = dy n w act'(z),            dw = sum over rows of u n
//
// Every tensor is read and written once and the arithmetic is a few operations
// an element, so the bound is HBM.  A row stays in registers between its
// reduction and its output.  Rows of up to 1024 elements (the heads after a
// recurrence) belong to 2^k lanes of a warp, so that a warp covers several
// short rows with 16-byte loads and the reduction is shuffles alone; longer
// rows (the model width) belong to a whole block.  Sums are fp32.
// The weight's gradient: a thread meets the same columns in every row that it
// takes, so it keeps their sums in registers over all its rows; a block adds
// its row groups in shared memory in a fixed order and writes one partial row,
// and a second kernel adds the partial rows in order: no atomics, so two runs
// agree bit for bit.
// Rows whose width or addresses do not allow 16-byte accesses take a plain
// loop over elements.
#include <initializer_list>

#include "gdn_common.cuh"

namespace {

using gdn::bf2f;
using gdn::f2bf;

struct NormArgs {
  const uint16_t *x, *res, *z;
  const float *w;
  float res_scale, eps;
  int64_t rows;
  int D;
  int64_t z_group, z_stride;  // row r of z starts at (r / z_group) z_stride + (r % z_group) D
  uint16_t *y, *h;
  // backward (x holds the normed stream h)
  const uint16_t *dy, *dh;
  uint16_t *dx, *dres, *dz;
  float *part;  // [blocks][D] partial weight gradients
};

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
__device__ __forceinline__ uint4 ld16(const uint16_t *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
__device__ __forceinline__ void st16(uint16_t *p, const uint4 &v) { __stcs(reinterpret_cast<uint4 *>(p), v); }

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_SIGMOID = 2 };
// act(z) and act'(z); s = sigmoid(z).
template <int ACT> __device__ __forceinline__ float act_f(float z) {
  if (ACT == ACT_NONE) return 1.f;
  const float s = gdn::sigmoid_fast(z);
  return ACT == ACT_SILU ? z * s : s;
}
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
  const int64_t g = row / a.z_group;
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
template <int NV> __device__ __forceinline__ void weights8(const float *w, const float (*kept)[8], int i, int v, float *o) {
  if (NV <= 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = kept[i][j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __ldg(w + v * 8 + j);
  }
}

template <int L, int NV, int THREADS, int ACT, bool RES>
__global__ void __launch_bounds__(THREADS) norm_fwd_kernel(const NormArgs a) {
  using S = Shape<L, NV, THREADS>;
  __shared__ float sh[2][32];
  int turn = 0;
  const int l = S::kBlock ? (int)threadIdx.x : (int)(threadIdx.x % L);
  const int nvec = a.D / 8;
  const float inv_d = 1.f / (float)a.D;
  float w[S::kKept][8];
#pragma unroll
  for (int i = 0; i < S::kKept; ++i) {
    const int v = l + i * L;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = v < nvec ? __ldg(a.w + v * 8 + j) : 0.f;
  }
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
    float h[NV][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack8(xv[i], h[i]);
      if (RES) {
        float r[8];
        unpack8(rv[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = fmaf(a.res_scale, h[i][j], r[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    ss = S::kBlock ? block_sum<THREADS>(ss, sh, turn) : lanes_sum<S::kBlock ? 32 : L>(ss);
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (!in || v >= nvec) continue;
      float z[8], y[8], wi[8];
      weights8<NV>(a.w, w, i, v, wi);
      if (ACT != ACT_NONE) unpack8(zv[i], z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = h[i][j] * rstd * wi[j];
        if (ACT != ACT_NONE) y[j] *= act_f<ACT>(z[j]);
      }
      st16(a.y + at + v * 8, pack8(y));
      if (RES) st16(a.h + at + v * 8, pack8(h[i]));
    }
  }
}

template <int L, int NV, int THREADS, int ACT, bool RES>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const NormArgs a) {
  using S = Shape<L, NV, THREADS>;
  __shared__ float sh[2][32];
  __shared__ float dwsh[S::kBlock ? 1 : S::kRows][S::kBlock ? 1 : L * NV * 8];
  int turn = 0;
  const int l = S::kBlock ? (int)threadIdx.x : (int)(threadIdx.x % L);
  const int nvec = a.D / 8;
  const float inv_d = 1.f / (float)a.D;
  float w[S::kKept][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
#pragma unroll
  for (int i = 0; i < S::kKept; ++i) {
    const int v = l + i * L;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = v < nvec ? __ldg(a.w + v * 8 + j) : 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * S::kRows;
  for (int64_t row0 = (int64_t)blockIdx.x * S::kRows; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + (S::kBlock ? 0 : threadIdx.x / L);
    const bool in = row < a.rows;
    const int64_t at = row * a.D, zat = (ACT != ACT_NONE && in) ? z_offset(a, row) : 0;
    uint4 xv[NV], yv[NV], zv[NV], gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      const bool on = in && v < nvec;
      xv[i] = on ? ld16(a.x + at + v * 8) : make_uint4(0, 0, 0, 0);
      yv[i] = on ? ld16(a.dy + at + v * 8) : make_uint4(0, 0, 0, 0);
      if (ACT != ACT_NONE) zv[i] = on ? ld16(a.z + zat + v * 8) : make_uint4(0, 0, 0, 0);
      if (RES) gv[i] = on ? ld16(a.dh + at + v * 8) : make_uint4(0, 0, 0, 0);
    }
    float ss = 0.f, sp = 0.f;  // sums of h^2 and of dy act(z) w h
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float h[8], dy[8], z[8], wi[8];
      const int v = l + i * L;
      if (v < nvec) weights8<NV>(a.w, w, i, v, wi);
      else continue;
      unpack8(xv[i], h);
      unpack8(yv[i], dy);
      if (ACT != ACT_NONE) unpack8(zv[i], z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(h[j], h[j], ss);
        float u = dy[j];
        if (ACT != ACT_NONE) u *= act_f<ACT>(z[j]);
        sp = fmaf(u * wi[j], h[j], sp);
      }
    }
    if (S::kBlock) {
      ss = block_sum<THREADS>(ss, sh, turn);
      sp = block_sum<THREADS>(sp, sh, turn);
    } else {
      ss = lanes_sum<S::kBlock ? 32 : L>(ss);
      sp = lanes_sum<S::kBlock ? 32 : L>(sp);
    }
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
    const float c = sp * inv_d * rstd * rstd;  // mean(p n) r, to be multiplied by h
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (!in || v >= nvec) continue;
      float h[8], dy[8], z[8], g[8], dx[8], dr[8], dz[8], wi[8];
      weights8<NV>(a.w, w, i, v, wi);
      unpack8(xv[i], h);
      unpack8(yv[i], dy);
      if (ACT != ACT_NONE) unpack8(zv[i], z);
      if (RES) unpack8(gv[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = h[j] * rstd;
        float u = dy[j];
        if (ACT != ACT_NONE) {
          float f, d;
          act_grad<ACT>(z[j], f, d);
          dz[j] = dy[j] * n * wi[j] * d;
          u *= f;
        }
        dw[i][j] = fmaf(u, n, dw[i][j]);
        float t = rstd * fmaf(-c, h[j], u * wi[j]);
        if (RES) t += g[j];
        dr[j] = t;
        dx[j] = a.res_scale * t;
      }
      st16(a.dx + at + v * 8, pack8(dx));
      if (RES) st16(a.dres + at + v * 8, pack8(dr));
      if (ACT != ACT_NONE) st16(a.dz + at + v * 8, pack8(dz));
    }
  }
  float *part = a.part + (int64_t)blockIdx.x * a.D;
  if (S::kBlock) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      if (v >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) part[v * 8 + j] = dw[i][j];
    }
  } else {
    const int rg = threadIdx.x / L;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) dwsh[rg][(l + i * L) * 8 + j] = dw[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += THREADS) {
      float s = 0.f;
      for (int r = 0; r < S::kRows; ++r) s += dwsh[r][e];
      part[e] = s;
    }
  }
}

// dw[e] = sum over the partial rows, in order within each of 32 strided shares
// and then over the shares: a warp's lane l of column e adds the rows l, l + 32, ...
__global__ void __launch_bounds__(256) norm_dw_kernel(const float *__restrict__ part, int blocks, int D,
                                                      float *__restrict__ dw) {
  __shared__ float sh[8][33];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  float s = 0.f;
  if (e < D)
    for (int b = w; b < blocks; b += 8) s += part[(int64_t)b * D + e];
  sh[w][c] = s;
  __syncthreads();
  if (w == 0 && e < D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sh[i][c];
    dw[e] = t;
  }
}

// Any width and any alignment: one block a row, elements read again for the
// second pass.  A thread meets the same columns in every row.
template <bool BWD>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormArgs a, int act) {
  __shared__ float sh[2][32];
  int turn = 0;
  const float inv_d = 1.f / (float)a.D;
  if (BWD)
    for (int e = threadIdx.x; e < a.D; e += 256) a.part[(int64_t)blockIdx.x * a.D + e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t at = row * a.D, zat = act != ACT_NONE ? z_offset(a, row) : 0;
    auto gate = [&](int e, float &f, float &d) {
      f = 1.f;
      d = 0.f;
      if (act == ACT_SILU) act_grad<ACT_SILU>(bf2f(a.z[zat + e]), f, d);
      if (act == ACT_SIGMOID) act_grad<ACT_SIGMOID>(bf2f(a.z[zat + e]), f, d);
    };
    auto stream = [&](int e) {
      const float x = bf2f(a.x[at + e]);
      return (!BWD && a.res) ? fmaf(a.res_scale, x, bf2f(a.res[at + e])) : x;
    };
    float ss = 0.f, sp = 0.f, f, d;
    for (int e = threadIdx.x; e < a.D; e += 256) {
      const float h = stream(e);
      ss = fmaf(h, h, ss);
      if (BWD) {
        gate(e, f, d);
        sp = fmaf(bf2f(a.dy[at + e]) * f * a.w[e], h, sp);
      }
    }
    ss = block_sum<256>(ss, sh, turn);
    if (BWD) sp = block_sum<256>(sp, sh, turn);
    const float rstd = rsqrtf(fmaf(ss, inv_d, a.eps));
    const float c = sp * inv_d * rstd * rstd;
    for (int e = threadIdx.x; e < a.D; e += 256) {
      const float h = stream(e);
      gate(e, f, d);
      if (!BWD) {
        a.y[at + e] = f2bf(h * rstd * a.w[e] * f);
        if (a.res) a.h[at + e] = f2bf(h);
      } else {
        const float dy = bf2f(a.dy[at + e]), n = h * rstd, u = dy * f;
        if (act != ACT_NONE) a.dz[at + e] = f2bf(dy * n * a.w[e] * d);
        a.part[(int64_t)blockIdx.x * a.D + e] += u * n;
        float t = rstd * fmaf(-c, h, u * a.w[e]);
        if (a.dh) {
          t += bf2f(a.dh[at + e]);
          a.dres[at + e] = f2bf(t);
        }
        a.dx[at + e] = f2bf(a.res_scale * t);
      }
    }
    __syncthreads();  // the sums' buffers are written again in the next row
  }
}

template <bool BWD, int L, int NV, int THREADS, int ACT>
void launch_one(const NormArgs &a, int blocks, cudaStream_t s) {
  const bool res = BWD ? a.dh != nullptr : a.res != nullptr;
  if (BWD) {
    if (res) norm_bwd_kernel<L, NV, THREADS, ACT, true><<<blocks, THREADS, 0, s>>>(a);
    else norm_bwd_kernel<L, NV, THREADS, ACT, false><<<blocks, THREADS, 0, s>>>(a);
  } else {
    if (res) norm_fwd_kernel<L, NV, THREADS, ACT, true><<<blocks, THREADS, 0, s>>>(a);
    else norm_fwd_kernel<L, NV, THREADS, ACT, false><<<blocks, THREADS, 0, s>>>(a);
  }
}
template <bool BWD, int L, int NV, int THREADS>
void launch_act(const NormArgs &a, int act, int blocks, cudaStream_t s) {
  if (act == ACT_NONE) launch_one<BWD, L, NV, THREADS, ACT_NONE>(a, blocks, s);
  else if (act == ACT_SILU) launch_one<BWD, L, NV, THREADS, ACT_SILU>(a, blocks, s);
  else launch_one<BWD, L, NV, THREADS, ACT_SIGMOID>(a, blocks, s);
}

// Lanes a row, vectors a lane and threads a block for a width; L = 0: the plain loop.
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
template <bool BWD> void dispatch(const NormArgs &a, int act, const Plan &p, int blocks, cudaStream_t s) {
  if (p.L == 8) launch_act<BWD, 8, 1, 256>(a, act, blocks, s);
  else if (p.L == 16) launch_act<BWD, 16, 1, 256>(a, act, blocks, s);
  else if (p.L == 32 && p.NV == 1) launch_act<BWD, 32, 1, 256>(a, act, blocks, s);
  else if (p.L == 32 && p.NV == 2) launch_act<BWD, 32, 2, 256>(a, act, blocks, s);
  else if (p.L == 32) launch_act<BWD, 32, 4, 256>(a, act, blocks, s);
  else if (p.L == 256 && p.NV == 1) launch_act<BWD, 256, 1, 256>(a, act, blocks, s);
  else if (p.L == 256) launch_act<BWD, 256, 2, 256>(a, act, blocks, s);
  else if (p.L == 512 && p.NV == 2) launch_act<BWD, 512, 2, 512>(a, act, blocks, s);
  else if (p.L == 512) launch_act<BWD, 512, 4, 512>(a, act, blocks, s);
  else norm_any_kernel<BWD><<<blocks, 256, 0, s>>>(a, act);
}

bool vec_ok(std::initializer_list<const void *> ptrs, bool has_z, int64_t z_stride) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return !has_z || z_stride % 8 == 0;
}

constexpr int kPartBlocks = 152 * 4;  // most blocks (partial rows) of the backward

}  // namespace

namespace gdn_host {

size_t norm_bwd_workspace_bytes(int64_t rows, int D) {
  const int64_t blocks = rows < kPartBlocks ? rows : kPartBlocks;
  return (size_t)blocks * (size_t)D * sizeof(float);
}

cudaError_t launch_norm_fwd(const uint16_t *x, const uint16_t *res, const uint16_t *z, const float *w, float res_scale,
                            float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride, uint16_t *y,
                            uint16_t *h, cudaStream_t s) {
  NormArgs a{};
  a.x = x; a.res = res; a.z = z; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.z_group = z_group; a.z_stride = z_stride; a.y = y; a.h = h;
  const Plan p = plan_of(D, vec_ok({x, res, z, y, h}, z != nullptr, z_stride));
  const int64_t want = (rows + p.rows - 1) / p.rows, cap = (int64_t)sm_count() * (2048 / p.threads);
  dispatch<false>(a, act, p, (int)(want < cap ? want : cap), s);
  return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const uint16_t *dy, const uint16_t *h, const uint16_t *z, const uint16_t *dh, const float *w,
                            float res_scale, float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride,
                            uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s) {
  NormArgs a{};
  a.x = h; a.dy = dy; a.z = z; a.dh = dh; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.z_group = z_group; a.z_stride = z_stride; a.dx = dx; a.dres = dres; a.dz = dz; a.part = static_cast<float *>(ws);
  const Plan p = plan_of(D, vec_ok({dy, h, z, dh, dx, dres, dz}, z != nullptr, z_stride));
  const int64_t want = (rows + p.rows - 1) / p.rows;
  const int blocks = (int)(want < kPartBlocks ? want : kPartBlocks);
  if (rows > 0) dispatch<true>(a, act, p, blocks, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_dw_kernel<<<(D + 31) / 32, 256, 0, s>>>(a.part, blocks, D, dw);
  return cudaGetLastError();
}

}  // namespace gdn_host
