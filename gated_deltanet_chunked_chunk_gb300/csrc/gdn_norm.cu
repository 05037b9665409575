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
__device__ __forceinline__ uint4 pack8(const f2 *f) {
  return make_uint4(f2_to_bf16(f[0]), f2_to_bf16(f[1]), f2_to_bf16(f[2]), f2_to_bf16(f[3]));
}
__device__ __forceinline__ float f2_sum(f2 a) {
  const float2 x = f2_get(a);
  return x.x + x.y;
}

template <int L, int NV, int THREADS, int ACT, bool RES>
__global__ void __launch_bounds__(THREADS) norm_fwd_kernel(const NormArgs a) {
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
  }
}

// A row's vectors come through a ring in shared memory by asynchronous copies,
// kAhead rows ahead; a thread copies and reads places of its own only, so no
// barrier is needed.  262144 rows of 128 with a SiLU gate: 56.4 us for both
// kernels (5.95 TB/s), three rows ahead 57.6; loads to registers took 10 us more.
template <int NV> struct Ahead { static constexpr int kRows = NV <= 2 ? 2 : 1; };
__device__ __forceinline__ void copy16(void *dst, const uint16_t *src, bool on) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(on ? 16 : 0) : "memory");
}

template <int L, int NV, int THREADS, int ACT, bool RES>
__global__ void __launch_bounds__(THREADS, (NV == 1 && L <= 32) ? 4 : 1) norm_bwd_kernel(const NormArgs a) {
  using S = Shape<L, NV, THREADS>;
  constexpr int kAhead = Ahead<NV>::kRows;
  constexpr int kTensors = 2 + (ACT != ACT_NONE ? 1 : 0) + (RES ? 1 : 0);
  extern __shared__ uint4 ring[];  // [kAhead][kTensors][NV][THREADS], then the blocks' sums
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
  auto place = [&](int stage, int tensor, int i) { return ring + ((stage * kTensors + tensor) * NV + i) * THREADS + threadIdx.x; };
  auto call = [&](int64_t row, int stage) {
    const bool in = row < a.rows;
    const int64_t at = in ? row * a.D : 0, zat = (ACT != ACT_NONE && in) ? z_offset(a, row) : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = l + i * L;
      const bool on = in && v < nvec;
      const int e = on ? v * 8 : 0;
      copy16(place(stage, 0, i), a.x + at + e, on);
      copy16(place(stage, 1, i), a.dy + at + e, on);
      if (ACT != ACT_NONE) copy16(place(stage, 2, i), a.z + zat + e, on);
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
    uint4 xc[NV], yc[NV], zc[NV], gc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xc[i] = *place(stage, 0, i);
      yc[i] = *place(stage, 1, i);
      if (ACT != ACT_NONE) zc[i] = *place(stage, 2, i);
      if (RES) gc[i] = *place(stage, kTensors - 1, i);
    }
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
      unpack8(xc[i], h);
      unpack8(yc[i], dy);
      if (ACT != ACT_NONE) unpack8(zc[i], z);
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
      unpack8(xc[i], h);
      unpack8(yc[i], dy);
      if (ACT != ACT_NONE) unpack8(zc[i], z);
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

template <int L, int NV, int THREADS, int ACT, bool RES>
cudaError_t launch_bwd(const NormArgs &a, int blocks, cudaStream_t s) {
  using S = Shape<L, NV, THREADS>;
  constexpr int kTensors = 2 + (ACT != ACT_NONE ? 1 : 0) + (RES ? 1 : 0);
  constexpr int ring = Ahead<NV>::kRows * kTensors * NV * THREADS * 16, sums = S::kBlock ? 0 : S::kRows * L * NV * 32;
  constexpr int bytes = ring > sums ? ring : sums;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = gdn_host::allow_smem(norm_bwd_kernel<L, NV, THREADS, ACT, RES>, bytes, done);
  if (e != cudaSuccess) return e;
  return gdn_host::launch_dependent(norm_bwd_kernel<L, NV, THREADS, ACT, RES>, dim3(blocks), THREADS, bytes, s, a);
}
template <bool BWD, int L, int NV, int THREADS, int ACT>
cudaError_t launch_one(const NormArgs &a, int blocks, cudaStream_t s) {
  const bool res = BWD ? a.dh != nullptr : a.res != nullptr;
  if (BWD) return res ? launch_bwd<L, NV, THREADS, ACT, true>(a, blocks, s) : launch_bwd<L, NV, THREADS, ACT, false>(a, blocks, s);
  return res ? gdn_host::launch_dependent(norm_fwd_kernel<L, NV, THREADS, ACT, true>, dim3(blocks), THREADS, 0, s, a)
             : gdn_host::launch_dependent(norm_fwd_kernel<L, NV, THREADS, ACT, false>, dim3(blocks), THREADS, 0, s, a);
}
template <bool BWD, int L, int NV, int THREADS>
cudaError_t launch_act(const NormArgs &a, int act, int blocks, cudaStream_t s) {
  if (act == ACT_NONE) return launch_one<BWD, L, NV, THREADS, ACT_NONE>(a, blocks, s);
  if (act == ACT_SILU) return launch_one<BWD, L, NV, THREADS, ACT_SILU>(a, blocks, s);
  return launch_one<BWD, L, NV, THREADS, ACT_SIGMOID>(a, blocks, s);
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
template <bool BWD> cudaError_t dispatch(const NormArgs &a, int act, const Plan &p, int blocks, cudaStream_t s) {
  if (p.L == 8) return launch_act<BWD, 8, 1, 256>(a, act, blocks, s);
  if (p.L == 16) return launch_act<BWD, 16, 1, 256>(a, act, blocks, s);
  if (p.L == 32 && p.NV == 1) return launch_act<BWD, 32, 1, 256>(a, act, blocks, s);
  if (p.L == 32 && p.NV == 2) return launch_act<BWD, 32, 2, 256>(a, act, blocks, s);
  if (p.L == 32) return launch_act<BWD, 32, 4, 256>(a, act, blocks, s);
  if (p.L == 256 && p.NV == 1) return launch_act<BWD, 256, 1, 256>(a, act, blocks, s);
  if (p.L == 256) return launch_act<BWD, 256, 2, 256>(a, act, blocks, s);
  if (p.L == 512 && p.NV == 2) return launch_act<BWD, 512, 2, 512>(a, act, blocks, s);
  if (p.L == 512) return launch_act<BWD, 512, 4, 512>(a, act, blocks, s);
  norm_any_kernel<BWD><<<blocks, 256, 0, s>>>(a, act);
  return cudaGetLastError();
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
  return dispatch<false>(a, act, p, (int)(want < cap ? want : cap), s);
}

cudaError_t launch_norm_bwd(const uint16_t *dy, const uint16_t *h, const uint16_t *z, const uint16_t *dh, const float *w,
                            float res_scale, float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride,
                            uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s) {
  NormArgs a{};
  a.x = h; a.dy = dy; a.z = z; a.dh = dh; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.z_group = z_group; a.z_stride = z_stride; a.dx = dx; a.dres = dres; a.dz = dz; a.part = static_cast<float *>(ws);
  const Plan p = plan_of(D, vec_ok({dy, h, z, dh, dx, dres, dz}, z != nullptr, z_stride));
  const int64_t want = (rows + p.rows - 1) / p.rows;
  // A block leaves a partial row of the weight's gradient, 4 D bytes written and
  // read again: wide rows, which few blocks fill an SM with, take as few blocks as
  // that (4 an SM against 1: 1000 rows of 4096 24.6 us against 15.4, 30000 rows 233
  // against 220; 2 at 8192 rows of 2048: 43.1 against 40.7).  All blocks take
  // the same number of turns, or one less.
  const int64_t cap = p.L < 256 ? kPartBlocks : D > 2048 ? kPartBlocks / 4 : kPartBlocks / 2;
  const int64_t turns = (want + cap - 1) / cap;
  const int blocks = turns > 0 ? (int)((want + turns - 1) / turns) : 0;
  if (rows > 0) {
    const cudaError_t e = dispatch<true>(a, act, p, blocks, s);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3((D + 31) / 32), 1024, 0, s, static_cast<const float *>(a.part), blocks, D, dw);
}

}  // namespace gdn_host
