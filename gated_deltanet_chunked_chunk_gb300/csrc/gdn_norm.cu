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
#include "gdn_norm.cuh"

namespace {

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

template <bool BWD> cudaError_t plain_or(const NormArgs &a, int act, const Plan &p, int blocks, cudaStream_t s) {
  if (p.L) return dispatch<BWD, false>(a, act, p, blocks, s);
  norm_any_kernel<BWD><<<blocks, 256, 0, s>>>(a, act);
  return cudaGetLastError();
}

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
  return plain_or<false>(a, act, p, (int)(want < cap ? want : cap), s);
}

cudaError_t launch_norm_bwd(const uint16_t *dy, const uint16_t *h, const uint16_t *z, const uint16_t *dh, const float *w,
                            float res_scale, float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride,
                            uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s) {
  NormArgs a{};
  a.x = h; a.dy = dy; a.z = z; a.dh = dh; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.z_group = z_group; a.z_stride = z_stride; a.dx = dx; a.dres = dres; a.dz = dz; a.part = static_cast<float *>(ws);
  const Plan p = plan_of(D, vec_ok({dy, h, z, dh, dx, dres, dz}, z != nullptr, z_stride));
  const int blocks = bwd_blocks(p, rows, D);
  if (rows > 0) {
    const cudaError_t e = plain_or<true>(a, act, p, blocks, s);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3((D + 31) / 32), 1024, 0, s, static_cast<const float *>(a.part), blocks, D, dw);
}

}  // namespace gdn_host
