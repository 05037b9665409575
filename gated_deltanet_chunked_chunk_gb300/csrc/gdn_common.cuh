// gdn_common.cuh -- small device helpers shared by the libgdn kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdn.h"

#define GDN_CHUNK 64
#define GDN_L2_EPS 1e-6f

namespace gdn {

__device__ __forceinline__ float bf2f(uint16_t x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}

__device__ __forceinline__ uint16_t f2bf(float x) {
  __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<uint16_t *>(&h);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// softplus(x) = log1p(exp(x)), and x itself above 20 (where the two agree
// to well under one fp32 ulp).
__device__ __forceinline__ float softplus_f(float x) {
  return x > 20.f ? x : log1pf(expf(x));
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }

// The same two functions in a few fused multiply-adds, for the streaming gate
// kernels.  softplus(x) = max(x, 0) + log1p(e^-|x|), and for y = e^-|x| in
// (0, 1], log1p(y) = 2 artanh(s) with s = y / (2 + y) in (0, 1/3], taken as
// the odd Taylor series of artanh, 2 s (1 + s^2/3 + s^4/5 + ... + s^14/15):
// the first omitted term is below 1e-9 of the sum.  The exponential is the
// hardware one and the divisions are the fast ones (errors of a few ulp, far
// inside the 1e-5 relative budget of the gates).  gdn_gating and the fused
// gating of the prefill both use these, so their gates agree bit for bit.
__device__ __forceinline__ float log1p_unit(float y) {  // y in [0, 1]
  const float s = __fdividef(y, 2.f + y);
  const float t = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, t, 1.f / 13.f);
  p = fmaf(p, t, 1.f / 11.f);
  p = fmaf(p, t, 1.f / 9.f);
  p = fmaf(p, t, 1.f / 7.f);
  p = fmaf(p, t, 1.f / 5.f);
  p = fmaf(p, t, 1.f / 3.f);
  p = fmaf(p, t, 1.f);
  return 2.f * s * p;
}
__device__ __forceinline__ float softplus_fast(float x) {
  return x > 20.f ? x : fmaxf(x, 0.f) + log1p_unit(__expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Programmatic dependent launch.  A kernel launched with launch_dependent()
// below may have its blocks in place while the kernel before it on the stream
// still runs; grid_wait() waits until that kernel is done and its writes are
// visible, and every thread calls it before it touches global memory (also where
// it then has nothing to do: a grid that ended early would let the next one pass
// the one before).  grid_release() lets such a successor's blocks come in.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two fp32 numbers and operations on both.
struct f2 {
  float x, y;
};
__device__ __forceinline__ f2 f2_of(float lo, float hi) { return f2{lo, hi}; }
__device__ __forceinline__ float2 f2_get(f2 a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ f2 f2_both(float x) { return f2{x, x}; }
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) { return f2{a.x * b.x, a.y * b.y}; }
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) { return f2{a.x + b.x, a.y + b.y}; }
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) { return f2{fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
// From and to the bits of two bf16.
__device__ __forceinline__ f2 f2_bf16(uint32_t u) { return f2_of(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
__device__ __forceinline__ uint32_t f2_to_bf16(f2 a) {
  const float2 x = f2_get(a);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}
// sigmoid of both: 1 / (1 + 2^(-z log2 e)) with the hardware's 2^x and 1/x.
__device__ __forceinline__ f2 f2_sigmoid(f2 z) {
  const float2 t = f2_get(f2_mul(z, f2_both(-1.4426950408889634f)));
  float a, b;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(t.y));
  const float2 e = f2_get(f2_add(f2_of(a, b), f2_both(1.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(e.y));
  return f2_of(a, b);
}

__device__ __forceinline__ void set_status(int32_t *st, int bits) {
  if (st) atomicOr(st, bits);
}

}  // namespace gdn

// Host-side launchers implemented in the kernel translation units.
namespace gdn_host {
cudaError_t launch_gating(const float *A_log, const uint16_t *a,
                          const uint16_t *b, const float *dt_bias,
                          int64_t Ttok, int HV, float *g, float *beta,
                          cudaStream_t s);
// Recurrent decode over N requests: request n owns tokens [cu[n], cu[n+1])
// (token n when cu is NULL), starts from pool[read_idx[n*ld + num_acc[n]-1]]
// (column 0 when num_acc is NULL) and stores the state after its i-th token
// into pool[write_idx[n*ld + i]].  pool is float* or bf16 (uint16_t*).
struct DecodeArgs {
  const uint16_t *q, *k, *v;
  const float *g, *beta, *A_log;
  const uint16_t *a, *b;
  const float *dt_bias;
  float scale;
  int l2;
  void *pool;
  int pool_bf16;
  int P;
  const int32_t *cu;
  int N, Ttot;
  const int32_t *read_idx, *write_idx;
  int ld;
  const int32_t *num_acc;
  int H, HV, K, V;
  uint16_t *o;
  int32_t *dev_status;
  int force_expiry;  // testing hook: the first bounded wait of every block runs out
};
cudaError_t launch_decode_general(const DecodeArgs &a, cudaStream_t s);
struct ChunkArgs {
  const uint16_t *q, *k, *v;
  const float *g, *beta;
  float scale;
  const float *h0;
  const int32_t *cu;
  int N, B, T, H, HV, K, V, l2;
  uint16_t *o;   // may be NULL (no output written)
  float *ht;
  float *hsave;  // NULL, or [chunk slots][HV][K][V]: the state entering every chunk
  // Fused gating (A_log != NULL; g, beta then NULL): the prep kernel computes
  // g = -e^{A_log} softplus(a + dt_bias), beta = sigmoid(b) itself and, when
  // g_out / beta_out are set, stores them ([B, T, HV] fp32).
  const float *A_log;
  const uint16_t *ga, *gb;
  const float *dt_bias;
  float *g_out, *beta_out;
  void *ws;
  size_t ws_bytes;
  int32_t *dev_status;
  int force_expiry;  // testing hook: the first bounded wait of every chain runs out
};
size_t chunk_workspace_bytes(int B, int T, int H, int HV, int K, int V, int N,
                             int varlen);
cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t s);
// Kernel launches of launch_chunk for these sizes on the current device (-1: no device).
int chunk_fwd_launches(int B, int T, int H, int HV, int K, int V, int N, int varlen);
struct ChunkBwdArgs {
  const uint16_t *q, *k, *v;
  const float *g, *beta;
  float scale;
  const float *h0;
  const int32_t *cu;
  int N, B, T, H, HV, K, V, l2;
  const uint16_t *dout;
  const float *dht;
  float *dq, *dk, *dv, *dg, *dbeta, *dh0;
  void *ws;
  size_t ws_bytes;
  int32_t *dev_status;
};
size_t chunk_bwd_workspace_bytes(int B, int T, int H, int HV, int K, int V, int N, int varlen);
cudaError_t launch_chunk_bwd(const ChunkBwdArgs &a, cudaStream_t s);
// SMs of the current device, and leave for a kernel to use `bytes` of dynamic
// shared memory, each asked of the runtime once a device (a query costs as
// much as a small launch's checks).  `done`: a static of the caller, a bit a device.
inline int sm_count() {
  static std::atomic<int> count[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    n = 152;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
template <class F> cudaError_t allow_smem(F *kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// A launch whose blocks may come in before the stream's last kernel is done; the
// kernel begins with gdn::grid_wait().
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A &&...args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
// Norms, rotary positions and the paged 8-bit cache (gdn_norm.cu, gdn_rope.cu,
// gdn_paged.cu, gdn_kv8_attn.cu).  Row r of z starts at (r / z_group) z_stride +
// (r % z_group) D elements; act: 0 none, 1 SiLU, 2 sigmoid.
size_t norm_bwd_workspace_bytes(int64_t rows, int D);
cudaError_t launch_norm_fwd(const uint16_t *x, const uint16_t *res, const uint16_t *z, const float *w, float res_scale,
                            float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride, uint16_t *y,
                            uint16_t *h, cudaStream_t s);
cudaError_t launch_norm_bwd(const uint16_t *dy, const uint16_t *h, const uint16_t *z, const uint16_t *dh, const float *w,
                            float res_scale, float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride,
                            uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s);
cudaError_t launch_rope(const uint16_t *q, const uint16_t *k, const int32_t *pos, const float *inv_freq, int64_t T, int HQ,
                        int HK, int D, int rot, int interleaved, int inverse, float factor, int64_t ldq, int64_t ldk,
                        uint16_t *qo, uint16_t *ko, cudaStream_t s);
cudaError_t launch_paged_plan(const int32_t *cached, const int32_t *cu, int N, int T, int32_t *table, int width,
                              const int32_t *free_pages, int F, const int32_t *num_free, int bs, int32_t *seq_lens,
                              int32_t *slots, int32_t *positions, int32_t *num_free_out, int32_t *dev_status,
                              cudaStream_t s);
cudaError_t launch_kv8_append(const uint16_t *k, const uint16_t *v, int64_t ldk, int64_t ldv, uint8_t *kc, uint8_t *vc,
                              float *ks, float *vs, const int32_t *slots, int64_t T, int P, int HK, int D, int bs,
                              int32_t *dev_status, cudaStream_t s);
struct Kv8AttnArgs {
  const uint16_t *q;
  int64_t ldq;  // token stride in elements
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *table;
  int width;
  const int32_t *seq_lens, *cu;
  int N, T, P, HQ, HK, D, bs, max_q, max_seq;
  float scale;
  uint16_t *o;
  float *lse;
  void *ws;
  int32_t *dev_status;
  int force_expiry;  // testing hook: the first bounded wait of every block runs out
};
size_t kv8_attn_workspace_bytes(int N, int T, int G, int D, int max_q);
cudaError_t launch_kv8_attn(const Kv8AttnArgs &a, cudaStream_t s);
// The norm with 8-bit codes of h and z (gdn_norm8.cu), scales [rows][ceil(D / 128)], and
// activations as such codes (gdn_act8.cu).
bool norm8_takes(int D);
cudaError_t launch_norm8_fwd(const uint16_t *x, const uint16_t *res, const uint16_t *z, const float *w, float res_scale,
                             float eps, int act, int64_t rows, int D, int64_t z_group, int64_t z_stride, uint16_t *y,
                             uint16_t *h, uint8_t *h8, float *hs, uint8_t *z8, float *zs, cudaStream_t s);
cudaError_t launch_norm8_bwd(const uint16_t *dy, const uint8_t *h8, const float *hs, const uint8_t *z8, const float *zs,
                             const uint16_t *dh, const float *w, float res_scale, float eps, int act, int64_t rows, int D,
                             uint16_t *dx, uint16_t *dres, uint16_t *dz, float *dw, void *ws, cudaStream_t s);
cudaError_t launch_act8_save(const uint16_t *x, int64_t rows, int D, int64_t x_group, int64_t x_stride, uint8_t *codes,
                             float *scale, cudaStream_t s);
cudaError_t launch_act8_load(const uint8_t *codes, const float *scale, int64_t rows, int D, uint16_t *y, cudaStream_t s);
// Attention of packed sequences for training (gdn_attn_fwd.cu, gdn_attn_bwd.cu).
struct TrainAttnArgs {
  const uint16_t *q, *k, *v;
  int64_t ldq, ldk, ldv;  // token strides in elements
  const int32_t *cu, *cu_k;
  int N, Tq, Tk, HQ, HK, D, causal;
  float scale;
  uint16_t *o;
  float *lse;
  // backward (o and lse are inputs)
  const uint16_t *dout;
  uint16_t *dq, *dk, *dv;
  void *ws;
  int32_t *dev_status;
  int force_expiry;  // testing hook: the first bounded wait of every block runs out
};
cudaError_t launch_attn_fwd(const TrainAttnArgs &a, cudaStream_t s);
bool attn_bwd_takes(int N, int Tq, int Tk, int HQ, int HK);  // fewer tiles than 2^31
size_t attn_bwd_workspace_bytes(int N, int Tq, int Tk, int HQ, int HK, int D);
cudaError_t launch_attn_bwd(const TrainAttnArgs &a, cudaStream_t s);
}  // namespace gdn_host
