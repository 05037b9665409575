// gdn_norm8.cu -- the norm of gdn_norm.cu whose forward also writes 8-bit codes of what
// the backward needs (the normed stream h, the gate z), and the backward that reads those
// codes in place of h and z.
//
// The codes are made from registers that the forward holds anyway, and the backward reads
// a byte where it read two, so that beside the memory that the step keeps (half) the
// backward moves 8 bytes an element instead of 10 (with a gate, without a residual).
// Bound: HBM, as in gdn_norm.cu.
#include "gdn_norm.cuh"

namespace gdn_host {

bool norm8_takes(int D) { return plan_of(D, true).L != 0; }

cudaError_t launch_norm8_fwd(const uint16_t *x, const uint16_t *res, const uint16_t *z, const float *w, float res_scale,
                             float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride, uint16_t *y,
                             uint16_t *h, uint8_t *h8, float *hs, uint8_t *z8, float *zs, cudaStream_t s) {
  NormArgs a{};
  a.x = x; a.res = res; a.z = z; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.z_group = z_group; a.z_stride = z_stride; a.y = y; a.h = h;
  a.h8 = h8; a.hs = hs; a.z8 = z8; a.zs = zs; a.groups = (D + gdn8::kGroup - 1) / gdn8::kGroup;
  const Plan p = plan_of(D, true);
  const int64_t want = (rows + p.rows - 1) / p.rows, cap = (int64_t)sm_count() * (2048 / p.threads);
  return dispatch<false, true>(a, act, p, (int)(want < cap ? want : cap), s);
}

cudaError_t launch_norm8_bwd(const uint16_t *dy, const uint8_t *h8, const float *hs, const uint8_t *z8, const float *zs,
                             const uint16_t *dh, const float *w, float res_scale, float eps, int act, int64_t rows, int D,
                             uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s) {
  NormArgs a{};
  a.dy = dy; a.dh = dh; a.w = w; a.res_scale = res_scale; a.eps = eps; a.rows = rows; a.D = D;
  a.h8 = const_cast<uint8_t *>(h8); a.hs = const_cast<float *>(hs);
  a.z8 = const_cast<uint8_t *>(z8); a.zs = const_cast<float *>(zs);
  a.groups = (D + gdn8::kGroup - 1) / gdn8::kGroup;
  a.dx = dx; a.dres = dres; a.dz = dz; a.part = static_cast<float *>(ws);
  const Plan p = plan_of(D, true);
  const int blocks = bwd_blocks(p, rows, D);
  if (rows > 0) {
    const cudaError_t e = dispatch<true, true>(a, act, p, blocks, s);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3((D + 31) / 32), 1024, 0, s, static_cast<const float *>(a.part), blocks, D, dw);
}

}  // namespace gdn_host
