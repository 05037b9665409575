// gdn_kv8_attn.cu -- attention over the paged 8-bit cache, for a few rows a
// request: single tokens, drafted tokens (kv8_decode_kernel).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j),  j <= L - m + i
//
// for the m new tokens i of a request whose context, the new tokens among it,
// is L long.  A key is its page's code times the page's scale, so its logit is
// the codes' product times (scale x page scale), and a value's page scale joins
// the exponent: with lv = log2(v scale) the kernel forms
//   t_ij = log2(e) scale ks (q_i . kcode_j) + lv,   p'_ij = 2^(t_ij - m_i),
//   O_i = sum_j p'_ij vcode_j,   l_i = sum_j p'_ij 2^-lv
// with m_i the running maximum of t.  So p' is in [0, 1] whatever the scales
// are, codes enter the products as they are (e4m3 is exact in f16), and
// o = O / l, logsumexp = (m + log2 l) ln 2.  Maxima and sums are fp32, products
// f16 with fp32 accumulation: p' rounds to 11 bits, and q, brought to a largest
// magnitude of 1 to 2 by a power of two for each row, loses nothing (bf16 has 8
// bits) but elements under 2^-24 of the row's largest.
//
// Bound: HBM, 2 D bytes for each (token, kv head), read once for all the query
// rows of the head's group.  One block works on one split (a stretch of keys)
// of one (request, kv head); the rows of a block are (token, head of the
// group) pairs.  A producer warp brings pages by TMA into a ring of 64-key
// stages (128-byte swizzle, so that the fragment reads below meet no bank
// twice), four consumer warps take stages in turn, each with a softmax of its
// own that they join at the end; a second kernel joins splits.
// mma.sync rather than tcgen05: a tile has 16 to 64 rows, not 128, and its
// products take a quarter of the time that its bytes do.
//
// Fragments.  S = Q K^T (m16n8k16): thread (g, t) = (lane / 4, lane % 4) holds
// for key n = g 16-byte chunks t, t + 4, .. of its row; the order of d inside a
// product is free as long as Q has the same, so no element moves.  Keys of an
// 8-key tile are taken in the order 0 4 1 5 2 6 3 7: then the 8 lanes that read
// shared memory together hit 8 different 16-byte places.  O = P V: the
// accumulators of S are the A operand as they stand, and a byte permutation
// pairs the two keys of a thread for each d.
#include <cuda.h>
#include <math.h>

#include "gdn_chunk_shared.cuh"
#include "gdn_common.cuh"
#include "gdn_kv8_attn.cuh"
#include "gdn_sm103.cuh"

namespace {

using namespace gdn;
using namespace gdnkv;

constexpr int kKeys = 64;       // keys a stage
constexpr int kConsumers = 4;   // consumer warps
constexpr int kThreads = 32 * (kConsumers + 1);

template <int D, int MT>
struct DecodeLay {
  static constexpr int TILE = kKeys * D;        // bytes of K (or V) a stage
  static constexpr int STAGE = 2 * TILE;
  static constexpr int NS = D == 128 ? 6 : 10;  // stages
  static constexpr int OFF_PAR = NS * STAGE;    // float4 {kmul, lv, 2^-lv, 0} x 4 pages a stage
  static constexpr int OFF_BAR = OFF_PAR + NS * 64;
  static constexpr int BYTES = OFF_BAR + (2 * NS + 1) * 8 + 16;
  static constexpr int WM = MT;                 // warps over rows
  static constexpr int WK = kConsumers / MT;    // warps over keys
  // joining the warps at the end, in the ring's memory: O [WK][16 MT][D + 4] and m, l
  static constexpr int JROW = D + 4;
  static constexpr int JOIN = WK * 16 * MT * JROW * 4 + WK * 16 * MT * 8;
  static_assert(JOIN <= NS * STAGE, "join fits the ring");
};

__device__ __forceinline__ void mma_f16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_add(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows as TMA
// leaves it (128-byte swizzle for D = 128, 64-byte swizzle for D = 64).
template <int D> __device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t c) {
  return D == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2)
    kv8_decode_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Ly = DecodeLay<D, MT>;
  constexpr int NCH = D / 64;  // 16-byte chunks of a key row that a thread holds
  constexpr int KS = D / 16;   // k-steps of S
  constexpr int NO = D / 8;    // n-tiles of O
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.z, h = blockIdx.y, sp = blockIdx.x;
  // The joining kernel's blocks may come in as soon as every block here has
  // started; they wait for this grid's results.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Span s;
  if (!request_span(a, n, 0, 16 * MT, s)) {
    if (tid == 0 && s.bits) set_status(a.dev_status, s.bits);
    return;
  }
  if (s.m * a.G > a.row_most || sp >= s.splits) return;
  const int L = s.L, m = s.m;
  constexpr int row0 = 0;
  const int k_begin = sp * a.split, k_end = min(s.keys, k_begin + a.split);
  const int stages = (max(0, k_end - k_begin) + kKeys - 1) / kKeys;

  const uint32_t bar = sb + Ly::OFF_BAR;
  const uint32_t never = bar + 16 * Ly::NS;
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_BAR + (2 * Ly::NS + 1) * 8);
  auto full = [&](int st) { return bar + 8 * st; };
  auto empty = [&](int st) { return bar + 8 * (Ly::NS + st); };
  if (tid == 0) {
    for (int st = 0; st < Ly::NS; ++st) {
      mbar_init(full(st), 1);
      mbar_init(empty(st), Ly::WM);
    }
    mbar_init(never, 1);
    mbar_fence_init();
    *failed = 0;
  }
  __syncthreads();

  float o[NO][4];
  float mx[2] = {-INFINITY, -INFINITY}, ls[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NO; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int g = lane >> 2, t = lane & 3;
  const int mt = warp % Ly::WM, kg = warp / Ly::WM;
  int issued = 0;  // stages that the producer has issued

  if (warp == kConsumers) {
    // ------------------------------------------------------------- producer
    const int ppt = a.bs >= kKeys ? 1 : kKeys / a.bs;  // copies a stage (of K, and of V)
    const int box = kKeys / ppt;                       // keys a copy
    const int pg0 = k_begin / a.bs;
    int batch = -1, page = -1;
    float ks = 0.f, lv = 0.f, iv = 1.f;
    for (int it = 0; it < stages; ++it) {
      const int st = it % Ly::NS, use = it / Ly::NS;
      const int first = (k_begin + it * kKeys) / a.bs - pg0;
      if (first / 32 != batch) {
        // table entries and scales, 32 pages at a time, a page a lane.  A page
        // that is not there counts as keys that nothing sees: logits of -inf.
        batch = first / 32;
        const int pi = pg0 + batch * 32 + lane;
        page = -1;
        ks = 0.f;
        lv = -INFINITY;
        iv = 1.f;
        if ((int64_t)pi * a.bs < k_end) {
          const int32_t p = a.table[(int64_t)n * a.width + pi];
          if (p < 0 || p >= a.P) {
            set_status(a.dev_status, GDN_DEV_BAD_SLOT);
          } else {
            page = p;
            const int64_t at = (int64_t)p * a.HK + h;
            ks = a.ks[at];
            const float v = a.vs[at];
            lv = log2f(v);
            iv = 1.f / v;
          }
        }
      }
      if (use > 0) {  // until the stage is free, or a consumer has given up
        const long long from = clock64();
        while (!mbar_try_wait(empty(st), (use - 1) & 1)) {
          if (*failed) break;
          if (clock64() - from > gdnc::kWaitLimit) {
            if (lane == 0) set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
            *failed = 1;
            break;
          }
        }
      }
      if (__any_sync(0xffffffffu, *failed)) break;
      const int src = (first - batch * 32 + (lane & (ppt - 1))) & 31;
      const int pg = __shfl_sync(0xffffffffu, page, src);
      const float4 par = make_float4(__shfl_sync(0xffffffffu, ks, src), __shfl_sync(0xffffffffu, lv, src),
                                     __shfl_sync(0xffffffffu, iv, src), 0.f);
      if (lane < ppt) *reinterpret_cast<float4 *>(smem + Ly::OFF_PAR + st * 64 + lane * 16) = par;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full(st), Ly::STAGE);
      __syncwarp();
      if (lane < ppt) {
        // pages that are not there lie outside the tensor: TMA fills in zeros
        const int z = pg >= 0 ? pg * a.HK + h : a.P * a.HK;
        const int y = (k_begin + it * kKeys) % a.bs;
        const uint32_t dst = sb + st * Ly::STAGE + lane * box * D;
        tma_load_3d(dst, &mk, full(st), 0, y, z);
        tma_load_3d(dst + Ly::TILE, &mv, full(st), 0, y, z);
      }
      issued = it + 1;
    }
  } else {
    // ------------------------------------------------------------ consumers
    // Queries: row g and row g + 8 of this warp's 16; thread t holds d =
    // 16 (t + 4 i) + 0..15, k-step 4 i + w taking 4 w + {0, 1 | 2, 3} of them.
    uint32_t qf[KS][4];
    float krow[2];
    int limit[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = row0 + 16 * mt + g + 8 * r;
      const bool on = row < m * a.G;
      limit[r] = on ? L - m + row / a.G : -1;
      float x[NCH][16], top = 0.f, bad = 0.f;
      const uint16_t *src = a.q + (int64_t)(s.t0 + row / a.G) * a.ldq + (int64_t)(h * a.G + row % a.G) * D;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint4 u = on ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * (t + 4 * i)) + v) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[i][8 * v + 2 * e] = bf16lo_f(w[e]);
            x[i][8 * v + 2 * e + 1] = bf16hi_f(w[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          top = fmaxf(top, fabsf(x[i][e]));
          bad = fmaf(x[i][e], 0.f, bad);  // NaN once an element is not finite
        }
      }
      top = quad_max(top);
      bad = quad_add(bad);
      int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      e2 = e2 < -100 ? -100 : e2 > 120 ? 120 : e2;
      const float down = gdnkv::pow2(-e2);
      krow[r] = gdnkv::pow2(e2) * a.scale_log2e + bad;
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          qf[4 * i + w][r] = pack_f16(x[i][4 * w] * down, x[i][4 * w + 1] * down);
          qf[4 * i + w][r + 2] = pack_f16(x[i][4 * w + 2] * down, x[i][4 * w + 3] * down);
        }
    }
    const int low = L - m + (row0 + 16 * mt) / a.G;  // what the tile's first row sees last
    const int kperm = (g >> 1) | ((g & 1) << 2);     // row of key n = g in an 8-key tile
    const uint32_t sel0 = (g & 1) ? 0x1504u : 0x5140u, sel1 = (g & 1) ? 0x3726u : 0x7362u;
    const int va = t + 4 * (g & 1), vb = t + 4 * ((g & 1) ^ 1);

    for (int it = kg; it < stages; it += Ly::WK) {
      const int st = it % Ly::NS, use = it / Ly::NS;
      bool ok = true;
      if (a.force_expiry) ok = mbar_wait_bounded(never, 0, gdnc::kTestWaitLimit);
      if (ok) ok = mbar_wait_bounded(full(st), use & 1, gdnc::kWaitLimit);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
        *failed = 1;
        break;
      }
      const uint32_t kt = sb + st * Ly::STAGE, vt = kt + Ly::TILE, par = sb + Ly::OFF_PAR + st * 64;
      const int k0 = k_begin + it * kKeys;

      float p[kKeys / 8][4];
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j) {
        p[j][0] = p[j][1] = p[j][2] = p[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const uint4 u = lds128(kt + tile_at<D>(8 * j + kperm, t + 4 * i));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_f16(p[j], qf[4 * i + e], gdnkv::e4m3x2_f16x2(w[e]), gdnkv::e4m3x2_f16x2(w[e] >> 16));
        }
      }
      const bool masked = k0 + kKeys - 1 > low;
      float top[2] = {-INFINITY, -INFINITY}, iv[kKeys / 16];
#pragma unroll
      for (int jj = 0; jj < kKeys / 16; ++jj) {  // a page holds 16 keys at least
        const float4 f = lds_f4(par + (a.bs >= kKeys ? 0 : 16 * jj / a.bs) * 16);
        iv[jj] = f.z;
        const float c0 = krow[0] * f.x, c1 = krow[1] * f.x;
#pragma unroll
        for (int jx = 0; jx < 2; ++jx) {
          const int j = 2 * jj + jx;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[j][e] = fmaf(p[j][e], c0, f.y);
            p[j][2 + e] = fmaf(p[j][2 + e], c1, f.y);
            if (masked) {
              const int key = k0 + 8 * j + t + 4 * e;
              if (key > limit[0]) p[j][e] = -INFINITY;
              if (key > limit[1]) p[j][2 + e] = -INFINITY;
            }
            top[0] = fmaxf(top[0], p[j][e]);
            top[1] = fmaxf(top[1], p[j][2 + e]);
          }
        }
      }
      float base[2], down[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float now = fmaxf(mx[r], quad_max(top[r]));
        base[r] = now == -INFINITY ? 0.f : now;
        down[r] = ex2f(mx[r] - base[r]);
        mx[r] = now;
        ls[r] *= down[r];
      }
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[j][e] = ex2f(p[j][e] - base[e >> 1]);
          ls[e >> 1] = fmaf(p[j][e], iv[j >> 1], ls[e >> 1]);
        }
      if (__any_sync(0xffffffffu, down[0] != 1.f || down[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= down[e >> 1];
      }
      uint32_t nan_seen = 0;
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk) {
        const uint32_t pa[4] = {pack_f16(p[2 * kk][0], p[2 * kk][1]), pack_f16(p[2 * kk][2], p[2 * kk][3]),
                                pack_f16(p[2 * kk + 1][0], p[2 * kk + 1][1]), pack_f16(p[2 * kk + 1][2], p[2 * kk + 1][3])};
        uint32_t wa[2][D / 32], wb[2][D / 32];
#pragma unroll
        for (int jx = 0; jx < 2; ++jx) {
          const int j = 2 * kk + jx;
          if (D == 128) {
            const uint4 u = lds128(vt + tile_at<D>(8 * j + va, g)), w = lds128(vt + tile_at<D>(8 * j + vb, g));
            wa[jx][0] = u.x; wa[jx][1] = u.y; wa[jx][D / 64] = u.z; wa[jx][D / 32 - 1] = u.w;
            wb[jx][0] = w.x; wb[jx][1] = w.y; wb[jx][D / 64] = w.z; wb[jx][D / 32 - 1] = w.w;
          } else {
            const uint2 u = lds64(vt + tile_at<D>(8 * j + va, g >> 1) + 8 * (g & 1));
            const uint2 w = lds64(vt + tile_at<D>(8 * j + vb, g >> 1) + 8 * (g & 1));
            wa[jx][0] = u.x; wa[jx][1] = u.y;
            wb[jx][0] = w.x; wb[jx][1] = w.y;
          }
          if (masked) {
            // Keys past the context hold whatever the page held before, and a
            // key that only later rows see may be NaN: p' is 0 there, but
            // 0 x NaN is not.  Such codes become 0; NaN that a row does see is
            // put back below.
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              if (k0 + 8 * j + va >= L) wa[jx][x] = 0;
              if (k0 + 8 * j + vb >= L) wb[jx][x] = 0;
              nan_seen |= any_nan(wa[jx][x]) | any_nan(wb[jx][x]);
              wa[jx][x] = drop_nan(wa[jx][x]);
              wb[jx][x] = drop_nan(wb[jx][x]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const uint32_t l0 = __byte_perm(wa[0][x], wb[0][x], sel0), l1 = __byte_perm(wa[0][x], wb[0][x], sel1);
          const uint32_t h0 = __byte_perm(wa[1][x], wb[1][x], sel0), h1 = __byte_perm(wa[1][x], wb[1][x], sel1);
          mma_f16(o[4 * x], pa, gdnkv::e4m3x2_f16x2(l0), gdnkv::e4m3x2_f16x2(h0));
          mma_f16(o[4 * x + 1], pa, gdnkv::e4m3x2_f16x2(l0 >> 16), gdnkv::e4m3x2_f16x2(h0 >> 16));
          mma_f16(o[4 * x + 2], pa, gdnkv::e4m3x2_f16x2(l1), gdnkv::e4m3x2_f16x2(h1));
          mma_f16(o[4 * x + 3], pa, gdnkv::e4m3x2_f16x2(l1 >> 16), gdnkv::e4m3x2_f16x2(h1 >> 16));
        }
      }
      if (masked && __any_sync(0xffffffffu, nan_seen != 0)) {
        const unsigned char *vs = smem + st * Ly::STAGE + Ly::TILE;
        for (int key = 0; key < kKeys && k0 + key < L; ++key)
#pragma unroll
          for (int i = 0; i < NO; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = (2 * t + e) * (D / 8) + i;
              if ((vs[tile_at<D>(key, d >> 4) + (d & 15)] & 0x7f) != 0x7f) continue;
              if (k0 + key <= limit[0]) o[i][e] = NAN;
              if (k0 + key <= limit[1]) o[i][2 + e] = NAN;
            }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }
  }

  __syncthreads();
  if (*failed) {
    // A wait ran out: write nothing, and stay until this block's copies are in.
    if (warp == kConsumers && lane == 0) {
      for (int st = 0; st < Ly::NS && st < issued; ++st) {
        const int last = (issued - 1 - st) / Ly::NS;
        if (!mbar_wait_bounded(full(st), last & 1, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
      }
    }
    return;
  }

  // Join the warps over keys.
  float *js = reinterpret_cast<float *>(smem);
  float2 *jml = reinterpret_cast<float2 *>(smem + Ly::WK * 16 * MT * Ly::JROW * 4);
  if (warp < kConsumers) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ls[r] = quad_add(ls[r]);
      const int row = kg * 16 * MT + 16 * mt + g + 8 * r;
      if (t == 0) jml[row] = make_float2(mx[r], ls[r]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < NO; i += 4)
          *reinterpret_cast<float4 *>(js + row * Ly::JROW + (2 * t + e) * (D / 8) + i) =
              make_float4(o[i][2 * r + e], o[i + 1][2 * r + e], o[i + 2][2 * r + e], o[i + 3][2 * r + e]);
    }
  }
  __syncthreads();
  const int mine = min(16 * MT, m * a.G - row0);
  for (int e = tid; e < mine * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = (e - r * (D / 4)) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < Ly::WK; ++k) top = fmaxf(top, jml[k * 16 * MT + r].x);
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < Ly::WK; ++k) {
      const float2 ml = jml[k * 16 * MT + r];
      const float w = ex2f(ml.x - base);
      const float4 v = *reinterpret_cast<const float4 *>(js + (k * 16 * MT + r) * Ly::JROW + c);
      l = fmaf(w, ml.y, l);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    const int row = row0 + r;
    if (s.splits == 1) {
      store_row4(a, s.t0 + row / a.G, h * a.G + row % a.G, D, c, acc, top, l);
    } else {
      const int64_t at = (((int64_t)n * a.HK + h) * a.row_cap + row) * a.max_splits + sp;
      *reinterpret_cast<float4 *>(a.part_o + at * D + c) = acc;
      if (c == 0) a.part_ml[at] = make_float2(top, l);
    }
  }
}

// Joins the splits of a row, in order: one block a (request, kv head, row).
// D / 4 lanes hold four columns each; the block's other threads take further
// splits and are added at the end.
constexpr int kJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
  __shared__ float4 so[GROUPS][LANES];
  __shared__ float sl[GROUPS], sm[GROUPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = blockIdx.z, h = blockIdx.y, row = blockIdx.x;
  Span s;
  if (!request_span(a, n, 0, a.row_cap, s) || s.m * a.G > a.row_most || row >= s.m * a.G || s.splits == 1) return;
  const int64_t at = (((int64_t)n * a.HK + h) * a.row_cap + row) * a.max_splits;
  const int c = threadIdx.x % LANES, gr = threadIdx.x / LANES;
  float top = -INFINITY;
  for (int i = gr; i < s.splits; i += GROUPS) top = fmaxf(top, a.part_ml[at + i].x);
  const float base = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = gr; i < s.splits; i += GROUPS) {
    const float2 ml = a.part_ml[at + i];
    const float4 v = *reinterpret_cast<const float4 *>(a.part_o + (at + i) * D + 4 * c);
    const float w = ex2f(ml.x - base);
    l = fmaf(w, ml.y, l);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  so[gr][c] = acc;
  if (c == 0) {
    sl[gr] = l;
    sm[gr] = top;
  }
  __syncthreads();
  if (gr != 0) return;
  float best = -INFINITY;
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) best = fmaxf(best, sm[k]);
  const float b2 = best == -INFINITY ? 0.f : best;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) {
    const float w = ex2f(sm[k] - b2);
    const float4 v = so[k][c];
    l = fmaf(w, sl[k], l);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  store_row4(a, s.t0 + row / a.G, h * a.G + row % a.G, D, 4 * c, acc, best, l);
}

// ---------------------------------------------------------------- host side
// How a call's requests are worked on, from its host bounds.  Requests of up to
// row_most rows (tokens x heads of a group) go to kv8_decode_kernel, with 16,
// 32 or 64 rows a block, the others to kv8_prefill_kernel.  A call whose bounds
// allow more than 64 rows may mix long and short requests (a serving step that
// prefills some and decodes others): then those of at most 16 rows (64 where
// the group itself is larger) stay with the first kernel, where a long context
// of few rows is split over many blocks.
struct DecodePlan {
  int mt, split, max_splits, row_cap, row_most;
};
DecodePlan plan_decode(int N, int HK, int G, int max_q, int max_seq) {
  DecodePlan p{};
  const int64_t rows = (int64_t)max_q * G;
  if (rows <= 64) p.row_most = (int)rows;
  else if (N == 1 || G > 64) p.row_most = 0;
  else p.row_most = G <= 16 ? 16 : 64;
  if (p.row_most == 0) return p;
  p.mt = p.row_most <= 16 ? 1 : p.row_most <= 32 ? 2 : 4;
  p.row_cap = 16 * p.mt;
  const int64_t keys = ((int64_t)max_seq + kKeys - 1) / kKeys * kKeys;
  int64_t want = (152 * 2 * 6) / ((int64_t)N * HK);  // six blocks for each place on the GPU
  if (want < 1) want = 1;
  int64_t split = (keys + want - 1) / want;
  split = (split + kKeys - 1) / kKeys * kKeys;
  if (split < 4 * kKeys) split = 4 * kKeys;
  if (split > 2048) split = 2048;
  p.split = (int)(split < keys ? split : keys < kKeys ? kKeys : keys);
  p.max_splits = (int)((keys + p.split - 1) / p.split);
  if (p.max_splits < 1) p.max_splits = 1;
  return p;
}

template <int D, int MT>
cudaError_t launch_decode(const AttnArgs &a, const DecodePlan &p, cudaStream_t s) {
  using Ly = DecodeLay<D, MT>;
  CUtensorMap mk, mv;
  const int keys = a.bs < kKeys ? a.bs : kKeys;
  if (!cache_map(&mk, a.kc, D, a.bs, (int64_t)a.P * a.HK, keys, true) ||
      !cache_map(&mv, a.vc, D, a.bs, (int64_t)a.P * a.HK, keys, true))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::BYTES);
  if (e != cudaSuccess) return e;
  kv8_decode_kernel<D, MT><<<dim3(p.max_splits, a.HK, a.N), kThreads, Ly::BYTES, s>>>(a, mk, mv);
  if ((e = cudaGetLastError()) != cudaSuccess || p.max_splits == 1) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.row_cap, a.HK, a.N);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_join_kernel<D>, a);
}

}  // namespace

namespace gdn_host {

size_t kv8_attn_workspace_bytes(int N, int HK, int G, int D, int max_q, int max_seq) {
  if (N <= 0 || max_q <= 0) return 0;
  const DecodePlan p = plan_decode(N, HK, G, max_q, max_seq);
  if (p.max_splits <= 1) return 0;
  return (size_t)N * HK * p.row_cap * p.max_splits * (size_t)(D + 2) * sizeof(float);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs &c, cudaStream_t s) {
  const DecodePlan p = plan_decode(c.N, c.HK, c.HQ / c.HK, c.max_q, c.max_seq);
  AttnArgs a{};
  static_cast<Kv8AttnArgs &>(a) = c;
  a.G = c.HQ / c.HK;
  a.scale_log2e = c.scale * gdnc::kLog2e;
  a.split = p.split;
  a.max_splits = p.max_splits;
  a.row_cap = p.row_cap;
  a.row_most = p.row_most;
  if (a.split < 1) a.split = kKeys;
  a.part_o = static_cast<float *>(c.ws);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)c.N * c.HK * p.row_cap * p.max_splits * c.D);
  if ((int64_t)c.max_q * a.G > p.row_most) {
    const cudaError_t e = launch_prefill(a, p.row_most + 1, s);
    if (e != cudaSuccess || p.row_most == 0) return e;
  }
  if (c.D == 128) {
    if (p.mt == 1) return launch_decode<128, 1>(a, p, s);
    if (p.mt == 2) return launch_decode<128, 2>(a, p, s);
    return launch_decode<128, 4>(a, p, s);
  }
  if (p.mt == 1) return launch_decode<64, 1>(a, p, s);
  if (p.mt == 2) return launch_decode<64, 2>(a, p, s);
  return launch_decode<64, 4>(a, p, s);
}

}  // namespace gdn_host
