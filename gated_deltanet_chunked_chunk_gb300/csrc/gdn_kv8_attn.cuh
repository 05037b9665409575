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

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2f(float x) { return gdnc::ex2(x); }

// Whether any of four codes is NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t any_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t drop_nan(uint32_t w) {
  const uint32_t m = any_nan(w);       // bit 7 of every NaN byte
  return w & ~((m >> 7) * 0xffu);
}

struct AttnArgs : gdn_host::Kv8AttnArgs {
  int G;  // query heads a kv head
  float scale_log2e;
  int row_cap;      // rows of a team of the decode kernel (8, 16, 32 or 64)
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
// Bytes of workspace that it needs, and their place.
size_t prefill_workspace(int D);
void prefill_place(AttnArgs &a, void *ws);

}  // namespace gdnkv
