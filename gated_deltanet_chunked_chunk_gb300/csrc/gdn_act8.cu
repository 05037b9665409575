// gdn_act8.cu -- activations to 8-bit codes and back (gdn_act8.cuh).
//
// Two bytes in and one out an element, or the other way, and a few operations: HBM.  A
// lane has 16 elements of a row (8, where a row is no multiple of 16), the lanes of a group
// find its largest magnitude by shuffles, and kAhead 16-byte loads of a lane are in flight
// together.  Rows whose width,
// stride or address do not allow 16-byte accesses take a warp a group, element by element.
#include <algorithm>

#include "gdn_act8.cuh"
#include "gdn_common.cuh"

namespace {

using namespace gdn;

constexpr int kThreads = 256, kAhead = 4;  // kAhead: vectors of 8 elements of a lane in flight

struct SaveArgs {
  const uint16_t *x;
  int64_t rows, x_group, x_stride;  // row r of x starts at (r / x_group) x_stride + (r % x_group) D; x_group 0: dense
  int D, groups;
  uint8_t *codes;
  float *scale;
};
__device__ __forceinline__ int64_t row_start(const SaveArgs &a, int64_t row) {
  if (a.x_group == 0) return row * a.D;
  if (a.x_group == 1) return row * a.x_stride;
  const int64_t g = row / a.x_group;
  return g * a.x_stride + (row - g * a.x_group) * a.D;
}

// V vectors of 8 elements a lane, 16 / V lanes a group; FLAT: the rows are whole groups one
// after another.  (8192 rows of 4096, a slice of wider ones: 19.7 us, 5.2 TB/s; 27.6 with
// one vector a lane, whose arithmetic took 69 % of the issue slots.)
template <int V, bool FLAT> __global__ void __launch_bounds__(kThreads) act8_save_kernel(const SaveArgs a) {
  constexpr int GL = 16 / V, AHEAD = kAhead / V;
  grid_wait();
  const int64_t total = a.rows * a.groups;  // groups of all rows
  const int64_t step = (int64_t)gridDim.x * (kThreads / GL);
  const int l = threadIdx.x % GL;
  // every lane of a warp takes every trip, as the shuffles need them all
  for (int64_t g0 = (int64_t)blockIdx.x * (kThreads / GL); g0 < total; g0 += step * AHEAD) {
    uint4 v[AHEAD][V];
    int64_t out[AHEAD];
    bool on[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t g = g0 + i * step + threadIdx.x / GL;
      int64_t from;
      if (FLAT) {
        on[i] = g < total;
        from = out[i] = g * gdn8::kGroup + l * (8 * V);
      } else {
        const int64_t row = g < 0x7fffffff ? (uint32_t)g / (uint32_t)a.groups : g / a.groups;
        const int at = (int)(g - row * a.groups) * gdn8::kGroup + l * (8 * V);
        on[i] = g < total && at < a.D;
        out[i] = row * a.D + at;
        from = on[i] ? row_start(a, row) + at : 0;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = on[i] ? __ldcs(reinterpret_cast<const uint4 *>(a.x + from) + j) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      bool finite[V];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) m = max(m, gdn8::largest(v[i][j], finite[j]));
#pragma unroll
      for (int o = GL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int e = gdn8::exponent_of(m);
      const float f = gdnkv::pow2(-e);
      uint2 c[V];
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = gdn8::codes8(v[i][j], f, finite[j]);
      if (on[i]) {
        if (V == 2) __stcs(reinterpret_cast<uint4 *>(a.codes + out[i]), make_uint4(c[0].x, c[0].y, c[V - 1].x, c[V - 1].y));
        else __stcs(reinterpret_cast<uint2 *>(a.codes + out[i]), c[0]);
        if (l == 0) __stcs(a.scale + (g0 + i * step + threadIdx.x / GL), gdnkv::pow2(e));
      }
    }
  }
}
// Any width and any alignment: a warp a group, four elements a lane.
__global__ void __launch_bounds__(kThreads) act8_save_any_kernel(const SaveArgs a) {
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = a.rows * a.groups;
  for (int64_t g = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; g < total; g += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row = g / a.groups, from = row_start(a, row);
    const int at = (int)(g - row * a.groups) * gdn8::kGroup;
    uint32_t v[4], m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = at + lane + 32 * i;
      v[i] = e < a.D ? a.x[from + e] : 0u;
      if ((v[i] & 0x7fffu) < 0x7f80u) m = max(m, v[i] & 0x7fffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const int e2 = gdnkv::scale_exponent(__uint_as_float(m << 16));
    const float f = gdnkv::pow2(-e2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = at + lane + 32 * i;
      uint32_t c = gdnkv::cvt_e4m3x2(__uint_as_float(v[i] << 16) * f, 0.f) & 0xffu;
      if ((v[i] & 0x7f80u) == 0x7f80u) c |= 0x7fu;
      if (e < a.D) a.codes[row * a.D + e] = (uint8_t)c;
    }
    if (lane == 0) a.scale[g] = gdnkv::pow2(e2);
  }
}

struct LoadArgs {
  const uint8_t *codes;
  const float *scale;
  int64_t rows;
  int D, groups;
  uint16_t *y;
};
__device__ __forceinline__ uint2 decode4(uint32_t c, float s) {
  const float2 a = gdnkv::f16x2_f32(gdnkv::e4m3x2_f16x2(c)), b = gdnkv::f16x2_f32(gdnkv::e4m3x2_f16x2(c >> 16));
  return make_uint2(pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s));
}
// A lane has 16 codes (V = 2) or 8 (V = 1).
template <int V> __global__ void __launch_bounds__(kThreads) act8_load_kernel(const LoadArgs a) {
  constexpr int AHEAD = kAhead / V;
  grid_wait();
  const int nvec = a.D / (8 * V);
  const int64_t total = a.rows * nvec, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += step * AHEAD) {
    uint4 c[AHEAD];
    float s[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t at = i0 + i * step;
      if (at >= total) continue;
      const int64_t row = at < 0x7fffffff ? (uint32_t)at / (uint32_t)nvec : at / nvec;
      if (V == 2) {
        c[i] = __ldcs(reinterpret_cast<const uint4 *>(a.codes) + at);
      } else {
        const uint2 x = __ldcs(reinterpret_cast<const uint2 *>(a.codes) + at);
        c[i] = make_uint4(x.x, x.y, 0, 0);
      }
      s[i] = __ldg(a.scale + row * a.groups + (at - row * nvec) / (16 / V));
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int64_t at = i0 + i * step;
      if (at >= total) continue;
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint2 lo = decode4(w[2 * j], s[i]), hi = decode4(w[2 * j + 1], s[i]);
        __stcs(reinterpret_cast<uint4 *>(a.y) + at * V + j, make_uint4(lo.x, lo.y, hi.x, hi.y));
      }
    }
  }
}
__global__ void __launch_bounds__(kThreads) act8_load_any_kernel(const LoadArgs a) {
  grid_wait();
  const int64_t total = a.rows * a.D;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / a.D;
    const float s = a.scale[row * a.groups + (i - row * a.D) / gdn8::kGroup];
    a.y[i] = (uint16_t)decode4(a.codes[i], s).x;
  }
}

bool whole(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
// Blocks for `want` shares of a thread block, `each` of them a trip: as many as the SMs hold
// at once at most, and all with the same number of trips.
int blocks_for(int64_t want, int each = 1) {
  const int64_t most = (int64_t)gdn_host::sm_count() * (2048 / kThreads);
  const int64_t trips = std::max<int64_t>(1, (want + most * each - 1) / (most * each));
  return (int)std::max<int64_t>(1, std::min(most, (want + trips * each - 1) / (trips * each)));
}

}  // namespace

namespace gdn_host {

cudaError_t launch_act8_save(const uint16_t *x, int64_t rows, int D, int64_t x_group, int64_t x_stride, uint8_t *codes,
                             float *scale, cudaStream_t s) {
  SaveArgs a{x, rows, x_group, x_stride, D, (D + gdn8::kGroup - 1) / gdn8::kGroup, codes, scale};
  const int64_t groups = rows * a.groups;
  const bool wide = D % 16 == 0 && whole(codes, 16);
  if (D % 8 || !whole(x, 16) || !whole(codes, 8) || (x_group && x_stride % 8))
    return launch_dependent(act8_save_any_kernel, dim3(blocks_for((groups + 7) / 8)), kThreads, 0, s, a);
  if (wide && D % gdn8::kGroup == 0 && x_group == 0)
    return launch_dependent(act8_save_kernel<2, true>, dim3(blocks_for((groups + 31) / 32, kAhead / 2)), kThreads, 0, s, a);
  if (wide) return launch_dependent(act8_save_kernel<2, false>, dim3(blocks_for((groups + 31) / 32, kAhead / 2)), kThreads, 0, s, a);
  return launch_dependent(act8_save_kernel<1, false>, dim3(blocks_for((groups + 15) / 16, kAhead)), kThreads, 0, s, a);
}

cudaError_t launch_act8_load(const uint8_t *codes, const float *scale, int64_t rows, int D, uint16_t *y, cudaStream_t s) {
  LoadArgs a{codes, scale, rows, D, (D + gdn8::kGroup - 1) / gdn8::kGroup, y};
  if (D % 8 || !whole(codes, 8) || !whole(y, 16))
    return launch_dependent(act8_load_any_kernel, dim3(blocks_for((rows * D + kThreads - 1) / kThreads)), kThreads, 0, s, a);
  if (D % 16 == 0 && whole(codes, 16))
    return launch_dependent(act8_load_kernel<2>, dim3(blocks_for((rows * (D / 16) + kThreads - 1) / kThreads, kAhead / 2)), kThreads, 0, s, a);
  return launch_dependent(act8_load_kernel<1>, dim3(blocks_for((rows * (D / 8) + kThreads - 1) / kThreads, kAhead)), kThreads, 0, s, a);
}

}  // namespace gdn_host
