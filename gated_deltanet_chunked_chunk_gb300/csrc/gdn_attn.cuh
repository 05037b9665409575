// gdn_attn.cuh -- what the kernels of training attention (gdn_attn_fwd.cu,
// gdn_attn_bwd.cu) share: arguments, which rows a block works on, tensor maps.
//
// Packed sequences: sequence n has the rows [cu[n], cu[n + 1]) of q and the keys
// [cu_k[n], cu_k[n + 1]) of k and v.  Rows and keys behind the last sequence count
// as one more sequence that sees nothing, so that every row of an output is written
// (zeros there).
//
// The kernels are persistent, one block an SM.  One warp of a block walks the items (a
// tile of rows or of keys, a head) that are the block's and hands them to the others in a
// ring in shared memory, so that the search and a next item's copies and first products
// run beside the end of the one before: of 24 packed sequences of 200 to 2000 tokens a
// block an item took 441 us, of which some 170 were block starts and ends.
#pragma once

#include "gdn_kv8_tc.cuh"

namespace gdnat {

using namespace gdn;
using gdnkv::elect_one;
using gdnkv::ex2f;
using gdnkv::kLn2;
using gdnkv::tmem_st32;
using gdnkv::tmem_st_wait;
using gdnkv::umma_f16_ta;

constexpr int kTile = 128;  // rows and keys of a tile

__device__ __forceinline__ int lds_i(uint32_t at) {
  int x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float lds_f(uint32_t at) { return __int_as_float(lds_i(at)); }
__device__ __forceinline__ void sts_i(uint32_t at, int x) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }
__device__ __forceinline__ void sts_f(uint32_t at, float x) { sts_i(at, __float_as_int(x)); }
// What a wait may take that lasts as long as an item: its walk is the rows of a group's heads
// or the keys of one, of which 280 GB hold 10^9 at most (D = 64), 8 million tiles at some 1800
// cycles: 1.5e10.
constexpr long long kItemLimit = 16 * gdnc::kWaitLimit;
// Waits for a barrier's phase; gives up after the limit or once another warp has, which
// the word at `failed` in shared memory says.  (Shared memory by 32-bit addresses: the
// loops need the registers.)
template <long long LIMIT = gdnc::kWaitLimit>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint32_t failed, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long from = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (lds_i(failed)) return false;
    if (clock64() - from > LIMIT) {
      sts_i(failed, 1);
      set_status(status, GDN_DEV_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

struct Args : gdn_host::TrainAttnArgs {
  int G;  // query heads a kv head
  float scale_log2e;
};

// A sequence's tiles have places in the workspace without a search.  Sequence n's are from
// floor(cu[n] / R) + n on: with a = R A + r and b = R B + s, ceil((b - a) / R) <= B - A + 1,
// so no two sequences share a place, and with the rows behind the last one there are at
// most T / R + N + 1.  Where there are fewer rows than that (most sequences are empty or
// short) a tile's place is its first row, of which there are T.
__host__ __device__ __forceinline__ bool by_row(int64_t T, int N, int R) { return T < T / R + N + 1; }
// Places, and tiles that T rows of N sequences have at most.
__host__ __device__ __forceinline__ int64_t most_tiles(int64_t T, int N, int R) { return by_row(T, N, R) ? T : T / R + N + 1; }

// One side's sequences: offsets, or one sequence of all rows (cu NULL).
struct Side {
  const int32_t *cu;
  int N, T;
  __device__ __forceinline__ int at(int n) const { return cu ? cu[n] : (n == 0 ? 0 : T); }
  // The place of tile 0 of sequence n, whose first row this is, and from a tile's to the next one's.
  __device__ __forceinline__ int64_t place(int n, int first, int R) const { return by_row(T, N, R) ? first : (int64_t)(first / R) + n; }
  __device__ __forceinline__ int apart(int R) const { return by_row(T, N, R) ? R : 1; }
};
__device__ __forceinline__ Side rows_of(const Args &a) { return Side{a.cu, a.N, a.Tq}; }
// Keys: their own offsets, else the rows'.
__device__ __forceinline__ Side keys_of(const Args &a) { return Side{a.cu_k ? a.cu_k : a.cu, a.N, a.Tk}; }

struct Run {
  int first, count;
};
// The rows of sequence n (n = N: those behind the last one); false where the offsets
// break the rules.
__device__ __forceinline__ bool run_of(const Side &s, int n, Run &r) {
  const int c0 = s.at(n), c1 = n == s.N ? s.T : s.at(n + 1);
  if (c0 < 0 || c1 < c0 || c1 > s.T || (n == 0 && c0 != 0)) return false;
  r.first = c0;
  r.count = c1 - c0;
  return true;
}
// The sequence that owns a place, found by a warp (every lane gets it): 32 sequences are
// looked at in each turn.  Offsets that are not sorted give some sequence.
__device__ __forceinline__ int owner_of(const Side &s, int64_t place, int R) {
  const int lane = threadIdx.x & 31;
  int lo = 0, span = s.N + 1;
  while (span > 1) {
    const int step = (span + 31) / 32, n = lo + lane * step;
    const bool there = lane * step < span && s.place(n, s.at(n), R) <= place;
    const uint32_t m = __ballot_sync(0xffffffffu, there || lane == 0);
    const int top = 31 - __clz((int)m);
    lo += top * step;
    span = min(step, span - top * step);
  }
  return lo;
}

// What the tile of a place works on.
struct Tile {
  int n;           // its sequence
  Run rows, keys;  // the sequence's
  int row0;        // its first row in the sequence (of the place's side)
};
// `by_keys`: places of the keys' side.  False: nothing to do.
__device__ __forceinline__ bool tile_of(const Args &a, int64_t place, int R, bool by_keys, Tile &t) {
  const Side rows = rows_of(a), keys = keys_of(a), mine = by_keys ? keys : rows;
  t.n = owner_of(mine, place, R);
  if (!run_of(rows, t.n, t.rows) || !run_of(keys, t.n, t.keys)) return false;
  if (t.n == a.N) (by_keys ? t.rows : t.keys).count = 0;
  const bool rowwise = by_row(mine.T, mine.N, R);
  const int64_t past = place - mine.place(t.n, mine.at(t.n), R), row0 = rowwise ? past : past * R;
  if (past < 0 || (rowwise && past % R) || row0 >= (by_keys ? t.keys : t.rows).count) return false;
  t.row0 = (int)row0;
  return true;
}
// The items of a call in the order in which blocks take them: chunks of up to 32 sequences,
// in each those of most work first (of all its sequences the u-th tiles from the cheap end,
// u from the largest down).  What a tile walks along (the keys, or the rows of all heads of
// a group) is walked by every other tile of its sequence, so a chunk has no more of it than
// stays in L2: `most` tokens.  All lanes of the walking warp are in step; lane l holds
// sequence chunk + l.
struct Walk {
  int chunk, count, level;  // first sequence, sequences; tiles from the cheap end
  int64_t base;             // index of the level's first item
  Run rows, keys;
  int tiles;                // this lane's sequence's
  int rows_end, keys_end;   // of all sequences before the chunk
};
struct Found {
  int n;           // sequence
  Run rows, keys;  // its rows and keys
  int tile, in;    // tile of R, which of the tile's items
  int of;          // items of the tile
};
constexpr int64_t kStays = 64 << 20;  // bytes: half of L2
__device__ __forceinline__ int tiles_in(int count, int R) { return (count + R - 1) / R; }
__device__ __forceinline__ int64_t most_tokens(int heads, int D) { return kStays / ((int64_t)heads * D * 4); }  // of two bf16 tensors
__device__ __forceinline__ void walk_chunk(const Args &a, Walk &w, int R, bool by_keys, int64_t most) {
  const int lane = threadIdx.x & 31, n = w.chunk + lane;
  w.rows = Run{0, 0};
  w.keys = Run{0, 0};
  w.tiles = 0;
  bool ok = n <= a.N && run_of(rows_of(a), n, w.rows) && run_of(keys_of(a), n, w.keys);
  // One that begins before the end of an earlier one (offsets that decrease somewhere) is left
  // out: no row comes twice, however bad the offsets are.
  int rows_end = ok ? w.rows.first + w.rows.count : 0, keys_end = ok ? w.keys.first + w.keys.count : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, rows_end, o), y = __shfl_up_sync(0xffffffffu, keys_end, o);
    if (lane >= o) {
      rows_end = max(rows_end, x);
      keys_end = max(keys_end, y);
    }
  }
  rows_end = max(rows_end, w.rows_end);
  keys_end = max(keys_end, w.keys_end);
  int rows_from = __shfl_up_sync(0xffffffffu, rows_end, 1), keys_from = __shfl_up_sync(0xffffffffu, keys_end, 1);
  if (lane == 0) {
    rows_from = w.rows_end;
    keys_from = w.keys_end;
  }
  ok = ok && w.rows.first >= rows_from && w.keys.first >= keys_from;
  if (ok && n == a.N) (by_keys ? w.rows : w.keys).count = 0;
  int64_t upto = ok ? (by_keys ? w.rows : w.keys).count : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  w.count = max(1, __popc(__ballot_sync(0xffffffffu, upto <= most)));
  if (ok && lane < w.count) w.tiles = tiles_in((by_keys ? w.keys : w.rows).count, R);
  w.rows_end = __shfl_sync(0xffffffffu, rows_end, w.count - 1);
  w.keys_end = __shfl_sync(0xffffffffu, keys_end, w.count - 1);
  w.level = (int)__reduce_max_sync(0xffffffffu, (unsigned)w.tiles) - 1;
}
__device__ __forceinline__ void walk_begin(const Args &a, Walk &w, int R, bool by_keys, int64_t most) {
  w.chunk = 0;
  w.base = 0;
  w.rows_end = 0;
  w.keys_end = 0;
  walk_chunk(a, w, R, by_keys, most);
}
// Item `index` (not below the one before); false: there are no more.  `first_most`: the
// first tiles of a sequence have most work, else the last ones.  items(tile): how many
// items the tile of this lane's sequence is.
template <class F>
__device__ __forceinline__ bool walk_to(const Args &a, Walk &w, int R, bool by_keys, bool first_most, int64_t most, int64_t index, Found &f,
                                        F items) {
  const int lane = threadIdx.x & 31;
  for (;;) {
    if (w.level >= 0) {
      const int tile = first_most ? w.tiles - 1 - w.level : w.level, mine = w.tiles > w.level ? items(tile) : 0;
      int upto = mine;  // (below 2^31: 32 sequences)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const int all = __shfl_sync(0xffffffffu, upto, 31);
      if (index < w.base + all) {
        const int at = (int)(index - w.base), l = __ffs((int)__ballot_sync(0xffffffffu, at < upto)) - 1;
        f.n = w.chunk + l;
        f.of = __shfl_sync(0xffffffffu, mine, l);
        f.in = at - (__shfl_sync(0xffffffffu, upto, l) - f.of);
        f.rows.first = __shfl_sync(0xffffffffu, w.rows.first, l);
        f.rows.count = __shfl_sync(0xffffffffu, w.rows.count, l);
        f.keys.first = __shfl_sync(0xffffffffu, w.keys.first, l);
        f.keys.count = __shfl_sync(0xffffffffu, w.keys.count, l);
        f.tile = __shfl_sync(0xffffffffu, tile, l);
        return true;
      }
      w.base += all;
      --w.level;
    } else {
      w.chunk += w.count;
      if (w.chunk > a.N) return false;
      walk_chunk(a, w, R, by_keys, most);
    }
  }
}

// The item that a block takes in its k-th turn: every other turn the other way round, so
// that no block has the larger one of every turn.
__device__ __forceinline__ int64_t turn_item(int64_t k) {
  return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Reports offsets that break the rules; by all threads of one block.
__device__ __forceinline__ void check_offsets(const Args &a) {
  const Side rows = rows_of(a), keys = keys_of(a);
  Run r;
  bool bad = false;
  for (int n = threadIdx.x; n < a.N; n += blockDim.x) bad |= !run_of(rows, n, r) || !run_of(keys, n, r);
  if (bad) set_status(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
}

// A 128-row tile of D bf16 in shared memory: D / 64 blocks of 128 rows x 128 bytes,
// 128-byte swizzle, as TMA brings them.
template <int D> __device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, uint32_t bar, int head, int row) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kTile * 128, map, bar, c * 64, head, row);
}
template <int D> constexpr int tile_bytes() { return kTile * D * 2; }
// Zeros the rows [from, 128) of a tile in shared memory (a warp).
template <int D> __device__ __forceinline__ void zero_rows(uint32_t tile, int from) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    for (int i = from * 8 + lane; i < kTile * 8; i += 32) gdnkv::sts128(tile + c * kTile * 128 + i * 16, 0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// Products of 128 x 128 x D (or 128 x D x 128) by one thread.
// D[128 x 128] = A B^T, both rows of D in shared memory.
template <int D> __device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = umma_idesc_bf16(128, 128);
  const uint64_t da = umma_desc_sw128(a), db = umma_desc_sw128(b);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t at = (k / 4) * (kTile * 128 / 16) + (k % 4) * 2;
    umma_bf16(d, da + at, db + at, id, k > 0);
  }
}
// D[128 x D] (+)= A B: A 128 x 128 bf16 in tensor memory, its columns 0-63 packed at a
// and 64-127 at a + 64 (over the halves of the fp32 tile they came from); B 128 rows of
// D in shared memory.
template <int D> __device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t id = umma_idesc_bf16(128, D, 0, 1);
  const uint64_t db = umma_desc_sw128_mn(b, kTile * 128);
#pragma unroll
  for (int k = 0; k < 8; ++k) umma_f16_ta(d, a + (k / 4) * 64 + (k % 4) * 8, db + k * 128, id, add || k > 0);
}

// Half of mma_cols: the columns 0-31 and 64-95 of A (part 0), or the others, added.
template <int D> __device__ __forceinline__ void mma_cols_half(uint32_t d, uint32_t a, uint32_t b, int part, bool add) {
  constexpr uint32_t id = umma_idesc_bf16(128, D, 0, 1);
  const uint64_t db = umma_desc_sw128_mn(b, kTile * 128);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = (i >> 1) * 4 + part * 2 + (i & 1);
    umma_f16_ta(d, a + (k / 4) * 64 + (k % 4) * 8, db + k * 128, id, add || part > 0 || i > 0);
  }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
               "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
               : "memory");
}
// a b + c and a b of two numbers each.
__device__ __forceinline__ float2 fma2v(float2 a, float b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mov.b64 z, {%5, %6}; fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 pair(const uint32_t *r, int i) {
  return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// 64 columns of a row from tensor memory, without the wait.
__device__ __forceinline__ void load64(uint32_t taddr, uint32_t *r) {
  tmem_ld32_issue(taddr, r);
  tmem_ld32_issue(taddr + 32, r + 32);
}
__device__ __forceinline__ void wait64(uint32_t *r) {
  tmem_ld_wait(r);
  gdnkv::tie32(r + 32);
}

// ---------------------------------------------------------------- host side
// Whether a kernel has the registers a thread that its warps' shares add up to: with fewer
// a warp would wait for ever for its own.  `known`: a static of the caller.
template <class F> cudaError_t check_registers(F *kernel, int registers, std::atomic<bool> &known) {
  if (known.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes f;
  const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
  if (e != cudaSuccess) return e;
  if (f.numRegs != registers) return cudaErrorInvalidConfiguration;
  known.store(true, std::memory_order_relaxed);
  return cudaSuccess;
}
// Map over [T][heads][D] bf16 with ld elements between tokens, box of 128 rows of 64
// elements of one head.
inline bool rows_map(CUtensorMap *m, const void *ptr, int D, int heads, int64_t T, int64_t ld) {
  gdnkv::EncodeTiledFn fn = gdnkv::encode_fn();
  if (!fn) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, kTile}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dim, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdnat
