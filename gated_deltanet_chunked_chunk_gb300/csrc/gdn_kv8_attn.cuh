// gdn_kv8_attn.cuh -- what the two attention kernels over the paged 8-bit cache
// share: arguments, the work of a tile of rows, the row's end, the cache's
// tensor map.
#pragma once

#include <cuda.h>
#include <math.h>

#include "gdn_chunk_shared.cuh"
#include "gdn_common.cuh"
#include "gdn_kv8.cuh"
#include "gdn_sm103.cuh"

namespace gdnkv {

using gdn::set_status;

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2f(float x) { return gdnc::ex2(x); }

// What a row's exponents are taken against when `top` is the largest of them: `lift`
// below it, so that its weight is 2^lift and one of f16 still has a bit at 2^-24.
// `lift` is at most 15 (2^16 is past f16), and exponents so large that their difference
// rounds to more have top itself.
__device__ __forceinline__ float reference_of(float top, float lift) {
  const float r = top - lift;
  return top - r > 15.f ? top : r;
}

// Whether any of four codes is NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t any_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
  const uint32_t m = any_nan(w);       // bit 7 of every NaN byte
  return w & ~((m >> 7) * 0xffu);
}

struct AttnArgs : gdn_host::Kv8AttnArgs {
  int G;  // query heads a kv head
  float scale_log2e;
  int row_cap;      // rows of a team of the kernels for few rows (8, 16 or 32)
  int stage_bits;   // log2 of the keys of their stages
  int row_most;     // requests with more rows are the prefill kernel's
  float *part_o;    // [team][2][row_cap][D] partial results
  float2 *part_ml;  // [team][2][row_cap]: maximum, sum
  int64_t *place;   // [N + 1] where a request's stages begin on the line of all
  float *tile_o;    // the prefill kernel's partial results: [slot][256][D]
  float2 *tile_ml;  // [slot][256]: maximum, sum
  int4 *owners;     // [slot] request, head, tile and pieces of the item that begins there
};

// What one tile of rows [row0, row0 + count) of a request works on; rows are
// (token, head of the group), token first.
struct Span {
  int t0, m;   // the request's tokens
  int L;       // its context
  int keys;    // keys that some row of the tile sees
  int bits;    // status bits of what is wrong with the request
};
// False: there is nothing to do.
__device__ __forceinline__ bool request_span(const AttnArgs &a, int n, int row0, int count, Span &s) {
  s.bits = 0;
  s.t0 = n;
  s.m = 1;
  s.L = a.seq_lens[n];
  if (a.cu) {
    const int c0 = a.cu[n], c1 = a.cu[n + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.T || (n == 0 && c0 != 0) || c1 - c0 > a.max_q) {
      s.bits = GDN_DEV_BAD_CU_SEQLENS;
      return false;
    }
    s.t0 = c0;
    s.m = c1 - c0;
  }
  if (row0 >= s.m * a.G) return false;
  if (s.L < 0 || s.L > a.max_seq) {
    s.bits = GDN_DEV_BAD_SEQ_LEN;
    return false;
  }
  const int last = min(row0 + count, s.m * a.G) - 1;
  s.keys = max(0, s.L - s.m + last / a.G + 1);
  return true;
}

// Four columns of a finished row: o = acc / l, and the row's logsumexp.
__device__ __forceinline__ void store_row4(const AttnArgs &a, int tok, int head, int D, int c, float4 acc, float top, float l) {
  const int64_t row = (int64_t)tok * a.HQ + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is 0
  *reinterpret_cast<uint2 *>(a.o + row * D + c) =
      make_uint2(gdn::pack_bf16(acc.x * inv, acc.y * inv), gdn::pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// ------------------------------------------------------- the line of stages
constexpr int kSMs = 152;
constexpr int kMinStages = 2;  // stages a team takes at least

// Stages of request n, 0 where the kernels for few rows have nothing to do for
// it; s is its span.  A request whose rows see no key has one stage, which writes its zeros.
__device__ __forceinline__ int stages_of(const AttnArgs &a, int n, Span &s) {
  if (!request_span(a, n, 0, a.row_cap, s) || s.m * a.G > a.row_most) return 0;
  return max(1, (s.keys + (1 << a.stage_bits) - 1) >> a.stage_bits);
}
// Stages that a team takes.
__device__ __forceinline__ int64_t stretch_of(int64_t total, int teams) {
  const int64_t per = (total + teams - 1) / teams;
  return per < kMinStages ? kMinStages : per;
}

// Where a walk along the line of stages stands.
struct Place {
  int n, h;       // request, kv head
  int stage, of;  // stage of the pair, stages that it has
  Span s;
};
__device__ __forceinline__ void next_request(const AttnArgs &a, Place &p) {
  p.stage = 0;
  p.h = 0;
  do {
    ++p.n;
    p.of = p.n < a.N ? stages_of(a, p.n, p.s) : 1;
  } while (p.of == 0);
}
// A team's stretch of the line, found by a warp: where it begins; returns its
// stages (0: none).  `first` for one warp of each team.
__device__ __forceinline__ int find_place(const AttnArgs &a, int team, int teams, bool first, Place &at) {
  const int lane = threadIdx.x & 31;
  int left;
  // Up to 32 requests, a lane each; else lane l sums the stages of requests
  // [l seg, (l + 1) seg) and the requests of the lane that holds the start are
  // looked at again.  The last team also writes every request's place on the
  // line for the joining kernel, which forms the places of few requests itself.
  if (a.N <= 32) {
    Span s{};
    const int of = lane < a.N ? stages_of(a, lane, s) : 0;
    if (s.bits && team == 0 && first) set_status(a.dev_status, s.bits);
    // below 2^31: 32 contexts of up to 2^25 stages would be 2^36 keys
    const uint32_t mine = (uint32_t)of * (uint32_t)a.HK;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
    const uint32_t per = (uint32_t)stretch_of(total, teams), start = per * (uint32_t)team;
    if (start >= total) return 0;
    left = (int)min(per, total - start);
    const int n = __ffs((int)__ballot_sync(0xffffffffu, incl > start)) - 1;
    at.n = n;
    at.of = __shfl_sync(0xffffffffu, of, n);
    at.s.t0 = __shfl_sync(0xffffffffu, s.t0, n);
    at.s.m = __shfl_sync(0xffffffffu, s.m, n);
    at.s.L = __shfl_sync(0xffffffffu, s.L, n);
    at.s.keys = __shfl_sync(0xffffffffu, s.keys, n);
    const uint32_t in = start - (__shfl_sync(0xffffffffu, incl, n) - (uint32_t)at.of * (uint32_t)a.HK);
    at.h = (int)(in / (uint32_t)at.of);
    at.stage = (int)(in - (uint32_t)at.h * (uint32_t)at.of);
  } else {
    Span s;
    const int seg = (a.N + 31) / 32;
    int64_t mine = 0;
    int bits = 0;
    for (int n = lane * seg; n < min(a.N, (lane + 1) * seg); ++n) {
      mine += (int64_t)stages_of(a, n, s) * a.HK;
      bits |= s.bits;
    }
    if (bits && team == 0 && first) set_status(a.dev_status, bits);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    const int64_t per = stretch_of(total, teams), start = per * team;
    if (team == teams - 1 && first) {
      int64_t run = incl - mine;
      for (int n = lane * seg; n < min(a.N, (lane + 1) * seg); ++n) {
        a.place[n] = run;
        run += (int64_t)stages_of(a, n, s) * a.HK;
      }
      if (lane == 0) a.place[a.N] = total;
    }
    if (start >= total) return 0;
    left = (int)min(per, total - start);
    const int owner = __ffs((int)__ballot_sync(0xffffffffu, incl > start)) - 1;
    int64_t run = __shfl_sync(0xffffffffu, incl - mine, owner);
    for (int base = owner * seg;; base += 32) {
      const int n = base + lane;
      const int64_t c = n < a.N ? (int64_t)stages_of(a, n, s) * a.HK : 0;
      int64_t sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + sum > start);
      if (past) {
        const int l = __ffs((int)past) - 1;
        at.n = base + l;
        const int64_t in = start - (run + __shfl_sync(0xffffffffu, sum - c, l));
        at.of = stages_of(a, at.n, at.s);
        at.h = (int)(in / at.of);
        at.stage = (int)(in - (int64_t)at.h * at.of);
        break;
      }
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  return left;
}

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}
// Map over a cache [P HK][bs][D] of bytes, box {D, keys, 1}.
inline bool cache_map(CUtensorMap *mp, const void *ptr, int D, int bs, int64_t planes, int keys, bool swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)bs, (cuuint64_t)planes};
  const cuuint64_t str[2] = {(cuuint64_t)D, (cuuint64_t)D * (cuuint64_t)bs};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)keys, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(mp, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dim, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Attention of the requests that have at least min_rows rows (gdn_kv8_prefill.cu).
cudaError_t launch_prefill(const AttnArgs &a, int min_rows, cudaStream_t s);
// Attention of the requests of up to 32 rows, stages of 128 keys; partial results
// as the decode kernel's, kSMs teams (gdn_kv8_rows.cu).
cudaError_t launch_kv8_rows(const AttnArgs &a, cudaStream_t s);
// Bytes of workspace that the prefill kernel needs, and their place.
size_t prefill_workspace(int D);
void prefill_place(AttnArgs &a, void *ws);

}  // namespace gdnkv
