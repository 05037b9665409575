// gdn_kv8_prefill.cu -- attention over the paged 8-bit cache for many rows a
// request (prompts and their chunks), on tcgen05.  The mathematics and the
// number formats are those of gdn_kv8_attn.cu.
//
// Bound: the tensor cores, 4 keys D operations for each (row, key, value) pair
// that a row sees.  One block works on 256 rows of one (request, kv head), rows
// being (token, head of the group) pairs, so that the head's group shares the
// keys and values it loads: two tiles of 128 rows, whose softmaxes take turns
// on the tensor cores' two accumulators.
//
// Products.  S = Q K^T takes the cache's bytes as they stand: kind::f8f6f4 with
// Q, brought to a largest magnitude of 128 to 256 by a power of two for each
// row, as the sum of two e4m3 numbers.  A bf16 number has 8 significant bits
// and an e4m3 number 4, so high part and remainder are exact but for elements
// under 2^-9 of 256.  Two products at twice the 16-bit rate cost what one f16
// product would, and no key is converted.  O = P V is kind::f16: P in f16 from
// tensor memory (11 bits; e4m3 would leave 4), V widened to f16 (exact) by four
// warps, once for both tiles.
//
// Warps: 0-3 and 4-7 softmax of the two tiles (a thread holds one row: its 128
// logits come from tensor memory to registers, no shuffles), 8-11 widen V, 12
// brings pages by TMA, 13 issues the products.  Tensor
// memory (512 columns): S of both tiles, P in place of its S, O of both tiles.
// An S of the next key tile is issued right after the P V that last read its
// columns; products of one thread execute in order, so "S is there" also says
// that O may be touched.  A row's reference is taken 11 under its maximum, so that f16
// holds weights down to 2^-35 of the largest, and O is rescaled, by the softmax warps
// themselves, only when an exponent is more than 15 above it (p' <= 2^15 is safe in f16).
//
// The last items, where they do not come out even with the SMs, are cut along
// their keys (find_work).  4096 tokens over 16384 keys, 32 heads of 128, 4 kv
// heads: 512 items on 152 SMs, 727 us (1.32 PFLOP/s, 70 % of a 16-bit library
// product) on new inputs each time; on the same ones 682 us, and 787 with the last 56
// items whole; 512 tokens over 16384: 130 us, two pieces an item (whole 232).  What a
// block works on stands in shared memory, as every register that the loops spill
// costs (70 bytes more of them: 25 us).  A key tile takes 3500 cycles, of which the
// tensor cores work 2176: S of a tile's next keys waits for its P V, as P stands in
// S's columns, and that for a softmax thread's chain from "S is there" to "P is
// there" (load, maximum, exponentials, store: 2000), longer than the other tile's
// products that hide it; P V begins when the first half of P is there (7 us).  Two threads a
// row (1200 us: with 64 logits each their registers spill), blocks that stay and
// take a stretch of all items' key tiles (822 us: what that adds to the loop costs
// more than the even end gains) and reading the logits twice (1490 us) were
// slower.  A block's own start and end (its item, queries, the result: 28000
// cycles) are what short prompts pay.
#include <limits.h>

#include <algorithm>

#include "gdn_kv8_tc.cuh"

namespace {

using namespace gdn;
using namespace gdnkv;

constexpr int kTileKeys = 128;
constexpr int kPrefThreads = 512;
constexpr int kItemRows = 256;
constexpr int kSlots = kSMs;    // partial results, one for each SM
constexpr int kPieceTiles = 8;  // key tiles that a piece of an item has at least
constexpr float kLift = 11.f, kMost = 15.f;  // exponents of a new maximum, and the largest
constexpr int kParSlots = 8;  // key tiles whose page constants are kept: more than can be in flight

template <int D>
struct PrefLay {
  static constexpr int T8 = 128 * D;   // bytes of a K, V or Q-part tile
  static constexpr int T16 = 256 * D;  // bytes of a widened V tile
  static constexpr int NK = 3, NV = 2, NW = 2;
  static constexpr int OFF_Q = 0;  // tile 0 high, low, tile 1 high, low
  static constexpr int OFF_K = OFF_Q + 4 * T8;
  static constexpr int OFF_W = OFF_K + NK * T8;
  static constexpr int OFF_V = OFF_W + NW * T16;
  static constexpr int OFF_PAR = OFF_V + NV * T8;  // float4 {k scale, lv, 2^-lv, 0} x 8 pages a slot
  static constexpr int OFF_BAR = OFF_PAR + kParSlots * 128;
  static constexpr int BARS = 2 * NK + 2 * NV + 2 * NW + 12 + kParSlots;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 32 + 16 * 8 + 48;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};

// What a block works on.  It stands in shared memory, and each kind of warp
// takes what it needs: the loops need the registers.
struct Work {
  int n, h, row0, rows;  // rows: the request's
  int t0, past, keys;    // past: L - m, what stands before the request's first token
  int base, tiles;       // key tiles: the `tiles` from base on
  int pieces, slot;      // pieces the item has, 0: nothing to do; where this one's result goes
};

// An item is 256 rows of one (request, kv head).  Those of a call stand in one
// order: requests, in each the last rows (which see the most keys) first, heads.
// Where the items do not come out even with the SMs, the last ones are cut along
// their keys, each into as many pieces as leave no SM without one; a small
// kernel joins the pieces.
__device__ __forceinline__ int item_tiles(const AttnArgs &a, int n, int min_rows, bool report) {
  Span s;
  const bool some = n < a.N && request_span(a, n, 0, 1, s);
  if (n < a.N && report && s.bits) set_status(a.dev_status, s.bits);
  return some && s.m * a.G >= min_rows ? (s.m * a.G + kItemRows - 1) / kItemRows : 0;
}
// Finds this block's work, by all its threads.  sums: 16 numbers of shared memory.
__device__ __forceinline__ void find_work(const AttnArgs &a, int min_rows, int sms, int64_t *sums, volatile Work *work) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (a.N + kPrefThreads - 1) / kPrefThreads, n0 = tid * each;
  const bool report = blockIdx.x == 0;
  int64_t mine = 0;
  for (int i = 0; i < each; ++i) mine += (int64_t)a.HK * item_tiles(a, n0 + i, min_rows, report);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  if (tid == 0) work->pieces = 0;
  __syncthreads();
  int64_t total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < kPrefThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  // (more than the host's bound only where cu_seqlens is no such array)
  const int all = (int)min(total, (int64_t)gridDim.x - kSlots);
  const int whole = all / sms * sms, rest = all - whole;
  // Pieces of each of the last items, one an SM.  (Two turns of smaller pieces,
  // 56 items in 5 pieces each, ended 13 us later.)
  const int cut = rest > 0 ? min(sms, kSlots) / rest : 1;
  const int slot = (int)blockIdx.x - whole;
  int item = blockIdx.x, piece = 0, pieces = 1;
  if (slot >= 0 && cut > 1) {
    item = whole + slot / cut;
    piece = slot % cut;
    pieces = cut;
  }
  if (item < all && item >= before && item < before + mine) {
    int n = n0, at = (int)(item - before), tiles;
    for (int t; at >= (t = a.HK * (tiles = item_tiles(a, n, min_rows, false))); ++n) at -= t;
    const int h = at % a.HK, tile = tiles - 1 - at / a.HK;
    Span s;
    request_span(a, n, tile * kItemRows, kItemRows, s);  // true: it has tiles
    const int keys = (s.keys + kTileKeys - 1) / kTileKeys;
    pieces = min(pieces, max(1, keys / kPieceTiles));
    if (piece < pieces) {
      work->n = n;
      work->h = h;
      work->row0 = tile * kItemRows;
      work->rows = s.m * a.G;
      work->t0 = s.t0;
      work->past = s.L - s.m;
      work->keys = s.keys;
      work->base = (int)((int64_t)keys * piece / pieces);
      work->tiles = (int)((int64_t)keys * (piece + 1) / pieces) - work->base;
      work->slot = slot;
      work->pieces = pieces;
    }
    if (slot >= 0 && slot < kSlots) a.owners[slot] = make_int4(n, h, tile, piece == 0 && pieces > 1 ? pieces : 0);
  } else if (tid == 0 && item >= all && slot >= 0 && slot < kSlots) {
    a.owners[slot] = make_int4(0, 0, 0, 0);
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kPrefThreads, 1)
    kv8_prefill_kernel(const AttnArgs a, int min_rows, int sms, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Ly = PrefLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_wait();
  volatile Work *work = reinterpret_cast<volatile Work *>(smem + Ly::OFF_MISC + 32 + 16 * 8);
  find_work(a, min_rows, sms, reinterpret_cast<int64_t *>(smem + Ly::OFF_MISC + 32), work);
  if (work->pieces == 0) return;
  const int page_bits = 31 - __clz(a.bs);

  const uint32_t bar = sb + Ly::OFF_BAR;
  auto KF = [&](int i) { return bar + 8 * i; };
  auto KE = [&](int i) { return bar + 8 * (Ly::NK + i); };
  auto VF = [&](int i) { return bar + 8 * (2 * Ly::NK + i); };
  auto VE = [&](int i) { return bar + 8 * (2 * Ly::NK + Ly::NV + i); };
  auto WF = [&](int i) { return bar + 8 * (2 * Ly::NK + 2 * Ly::NV + i); };
  auto WE = [&](int i) { return bar + 8 * (2 * Ly::NK + 2 * Ly::NV + Ly::NW + i); };
  const uint32_t bx = bar + 8 * (2 * Ly::NK + 2 * Ly::NV + 2 * Ly::NW);
  auto SF = [&](int w) { return bx + 8 * w; };
  auto PF = [&](int w) { return bx + 16 + 8 * w; };
  auto OD = [&](int w) { return bx + 32 + 8 * w; };
  const uint32_t QR = bx + 48, never = bx + 56;
  const uint32_t DR = bx + 64;
  auto PH = [&](int w) { return bx + 72 + 8 * w; };
  auto PR = [&](int i) { return bx + 88 + 8 * i; };
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC);
  volatile int *nan_zone = failed + 1;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  if (tid == 0) {
    for (int i = 0; i < Ly::NK; ++i) { mbar_init(KF(i), 1); mbar_init(KE(i), 1); }
    for (int i = 0; i < Ly::NV; ++i) { mbar_init(VF(i), 1); mbar_init(VE(i), 4); }
    for (int i = 0; i < Ly::NW; ++i) { mbar_init(WF(i), 4); mbar_init(WE(i), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(SF(i), 1); mbar_init(PF(i), 128); mbar_init(PH(i), 128); mbar_init(OD(i), 1); }
    for (int i = 0; i < kParSlots; ++i) mbar_init(PR(i), 1);
    mbar_init(QR, 256);
    mbar_init(DR, 1);
    mbar_init(never, 1);
    mbar_fence_init();
    *failed = 0;
    *nan_zone = 0;
  }
  if (warp == 13) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Of the block's 65536 registers (512 threads x 128) the softmax warps take
  // 184 a thread, the other warps 72: 2 x 128 x 184 + 2 x 128 x 72 = 65536.  (200
  // and 56: 694 us against 682, as above.)
  const int tiles = work->tiles;
  float m_ref = -INFINITY, l_sum = 0.f;
  int issued_k = 0, issued_v = 0;  // key tiles that the producer has issued
  const int wg = warp >> 2;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
  const uint32_t S_col = tmem + lanes + (wg & 1) * 128, O_col = tmem + lanes + 256 + (wg & 1) * D;

  if (wg < 2) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int row = work->row0 + wg * 128 + (tid & 127), base = work->base;
    const bool on = row < work->rows;
    const int low = work->past + work->row0 / a.G;  // what the first row sees last
    const int limit = on ? work->past + row / a.G : -1;
    float krow;
    {
      // the row's query: largest magnitude, then high and low parts
      const uint16_t *src = a.q + (int64_t)(work->t0 + row / a.G) * a.ldq + (int64_t)(work->h * a.G + row % a.G) * D;
      uint4 u[D / 8];
      float top = 0.f, bad = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        u[i] = on ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = bf16lo_f(w[e]), y = bf16hi_f(w[e]);
          top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
          bad = fmaf(x, 0.f, fmaf(y, 0.f, bad));  // NaN once an element is not finite
        }
      }
      int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      e2 = e2 < -100 ? -100 : e2 > 120 ? 120 : e2;
      const float down = pow2(7 - e2);
      krow = pow2(e2 - 7) * a.scale_log2e + bad;
      const uint32_t qh = sb + Ly::OFF_Q + wg * 2 * Ly::T8, ql = qh + Ly::T8;
      const uint32_t r = tid & 127;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 &v = u[2 * c + (e >> 1)];
          const uint32_t w0 = (e & 1) ? v.z : v.x, w1 = (e & 1) ? v.w : v.y;
          const float x0 = bf16lo_f(w0) * down, x1 = bf16hi_f(w0) * down, x2 = bf16lo_f(w1) * down, x3 = bf16hi_f(w1) * down;
          const uint32_t h0 = cvt_e4m3x2(x0, x1), h1 = cvt_e4m3x2(x2, x3);
          const float2 b0 = f16x2_f32(e4m3x2_f16x2(h0)), b1 = f16x2_f32(e4m3x2_f16x2(h1));
          hi[e] = h0 | (h1 << 16);
          lo[e] = cvt_e4m3x2(x0 - b0.x, x1 - b0.y) | (cvt_e4m3x2(x2 - b1.x, x3 - b1.y) << 16);
        }
        const uint32_t at = D == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
        sts128(qh + at, hi[0], hi[1], hi[2], hi[3]);
        sts128(ql + at, lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(QR);
    }
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(never, 0, gdnc::kTestWaitLimit)) {
      *failed = 1;
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    for (int j = 0; j < tiles; ++j) {
      if (ok) ok = wait_bar(PR(j % kParSlots), (j / kParSlots) & 1, failed, a.dev_status);
      if (ok) ok = wait_bar(SF(wg), j & 1, failed, a.dev_status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t r[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32_issue(S_col + 32 * i, r + 32 * i);
      tmem_ld_wait(r);
#pragma unroll
      for (int i = 1; i < 4; ++i) tie32(r + 32 * i);

      const uint32_t par = sb + Ly::OFF_PAR + (j % kParSlots) * 128;
      const int k0 = (base + j) * kTileKeys;
      const bool masked = k0 + kTileKeys - 1 > low;
      float c[8], b[8], iv[8], top = -INFINITY;  // constants of 16 keys each
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float4 f = lds_f4(par + ((16 * g) >> page_bits) * 16);
        c[g] = krow * f.x;
        b[g] = f.y;
        iv[g] = f.z;
      }
      if (masked) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float t = fmaf(__uint_as_float(r[16 * g + i]), c[g], b[g]);
            if (k0 + 16 * g + i > limit) t = -INFINITY;
            top = fmaxf(top, t);
            r[16 * g + i] = __float_as_uint(t);
          }
          c[g] = 1.f;  // t itself from here on
          b[g] = 0.f;
        }
      } else {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          float x[5];
#pragma unroll
          for (int i = 0; i < 5; ++i)
            x[i] = max3(__uint_as_float(r[16 * g + 3 * i]), __uint_as_float(r[16 * g + 3 * i + 1]), __uint_as_float(r[16 * g + 3 * i + 2]));
          x[0] = max3(x[0], x[1], x[2]);
          x[3] = max3(x[3], x[4], __uint_as_float(r[16 * g + 15]));
          top = fmaxf(top, fmaf(fmaxf(x[0], x[3]), c[g], b[g]));
        }
      }
      float grow = 1.f;
      if (top - m_ref > kMost) {  // (of -inf both, NaN: no)
        const float now = reference_of(top, kLift);
        grow = ex2f(m_ref - now);
        m_ref = now;
        l_sum *= grow;
      }
      if (j > 0 && __any_sync(0xffffffffu, grow != 1.f)) {
#pragma unroll 1
        for (int i = 0; i < D; i += 8) {  // few at a time: the logits hold 128 registers
          uint32_t o[8];
          tmem_ld8(O_col + i, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * grow);
          tmem_st8(O_col + i, o);
        }
      }
      const float ref = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float2 sum = make_float2(0.f, 0.f);
        const float bb = b[g] - ref;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 t = fma2(make_float2(__uint_as_float(r[16 * g + 2 * i]), __uint_as_float(r[16 * g + 2 * i + 1])), c[g], bb);
          t.x = ex2f(t.x);
          t.y = ex2f(t.y);
          sum = add2(sum, t);
          r[8 * g + i] = pack_f16(t.x, t.y);
        }
        l_sum = fmaf(sum.x + sum.y, iv[g], l_sum);
        if (g == 3) {  // the first keys' products may begin
          tmem_st32(S_col, r);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(PH(wg));
        }
      }
      tmem_st32(S_col + 32, r + 32);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(PF(wg));
    }
    if (ok && tiles > 0) ok = wait_bar(OD(wg), 0, failed, a.dev_status);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (wg == 2) {
      // ------------------------------------------------------------ widen V
      const int ct = tid - 256, base = work->base, past = work->past, low = past + work->row0 / a.G;
      const int L = past + work->rows / a.G;
      for (int j = 0; j < tiles; ++j) {
        const int iv = j % Ly::NV, iw = j % Ly::NW;
        bool ok = wait_bar(VF(iv), (j / Ly::NV) & 1, failed, a.dev_status);
        if (ok && j >= Ly::NW) ok = wait_bar(WE(iw), (j / Ly::NW - 1) & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t src = sb + Ly::OFF_V + iv * Ly::T8, dst = sb + Ly::OFF_W + iw * Ly::T16;
        const int k0 = (base + j) * kTileKeys;
        const bool zone = k0 + kTileKeys - 1 > low;
        uint32_t seen = 0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int e = i * 128 + ct, key = e / (D / 16), ch = e % (D / 16);
          uint4 u = lds128(src + key * D + ch * 16);
          if (zone) {
            // keys past the context, and NaN that only later rows may see: see
            // gdn_kv8_attn.cu
            if (k0 + key >= L) u = make_uint4(0, 0, 0, 0);
            seen |= any_nan(u.x) | any_nan(u.y) | any_nan(u.z) | any_nan(u.w);
            u = make_uint4(drop_nan(u.x), drop_nan(u.y), drop_nan(u.z), drop_nan(u.w));
          }
          const uint32_t base = dst + (ch >> 2) * 16384 + key * 128;
          const uint32_t c0 = (((ch & 3) * 2) ^ (key & 7)) << 4, c1 = (((ch & 3) * 2 + 1) ^ (key & 7)) << 4;
          const uint32_t x0 = e4m3x2_f16x2(u.x), x1 = e4m3x2_f16x2(u.x >> 16), x2 = e4m3x2_f16x2(u.y), x3 = e4m3x2_f16x2(u.y >> 16);
          const uint32_t y0 = e4m3x2_f16x2(u.z), y1 = e4m3x2_f16x2(u.z >> 16), y2 = e4m3x2_f16x2(u.w), y3 = e4m3x2_f16x2(u.w >> 16);
          // the upper 64 columns write their halves in the other order: the
          // eight lanes of a row then meet eight different places
          const bool sw = (ch >> 2) & 1;
          sts128(base + (sw ? c1 : c0), sw ? y0 : x0, sw ? y1 : x1, sw ? y2 : x2, sw ? y3 : x3);
          sts128(base + (sw ? c0 : c1), sw ? x0 : y0, sw ? x1 : y1, sw ? x2 : y2, sw ? x3 : y3);
        }
        if (seen) *nan_zone = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(VE(iv));
          mbar_arrive(WF(iw));
        }
      }
    } else if (warp == 12) {
      // ----------------------------------------------------------- producer
      const int ppt = a.bs >= kTileKeys ? 1 : kTileKeys / a.bs, box = kTileKeys / ppt;
      const int n = work->n, h = work->h, keys = work->keys, base = work->base;
      int batch = -1, page = -1;
      float ks = 0.f, lv = 0.f, iv = 1.f;
      for (int j = 0; j < tiles; ++j) {
        const int first = (base + j) * ppt;
        if (first / 32 != batch) {
          batch = first / 32;
          const int pi = batch * 32 + lane;
          page = -1;
          ks = 0.f;
          lv = -INFINITY;
          iv = 1.f;
          if ((int64_t)pi * a.bs < keys) {
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
        const int ik = j % Ly::NK, vi = j % Ly::NV;
        bool ok = true;
        if (j >= Ly::NK) ok = wait_bar(KE(ik), (j / Ly::NK - 1) & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int src = (first - batch * 32 + (lane & (ppt - 1))) & 31;
        const int pg = __shfl_sync(0xffffffffu, page, src);
        const float4 par = make_float4(__shfl_sync(0xffffffffu, ks, src), __shfl_sync(0xffffffffu, lv, src),
                                       __shfl_sync(0xffffffffu, iv, src), 0.f);
        if (lane < ppt) *reinterpret_cast<float4 *>(smem + Ly::OFF_PAR + (j % kParSlots) * 128 + lane * 16) = par;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(PR(j % kParSlots));
          mbar_arrive_expect_tx(KF(ik), Ly::T8);
        }
        __syncwarp();
        const int z = pg >= 0 ? pg * a.HK + h : a.P * a.HK;  // outside the tensor: zeros
        if (lane < ppt) tma_load_3d(sb + Ly::OFF_K + ik * Ly::T8 + lane * box * D, &mk, KF(ik), 0, 0, z);
        issued_k = j + 1;
        if (j >= Ly::NV) ok = wait_bar(VE(vi), (j / Ly::NV - 1) & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) mbar_arrive_expect_tx(VF(vi), Ly::T8);
        __syncwarp();
        if (lane < ppt) tma_load_3d(sb + Ly::OFF_V + vi * Ly::T8 + lane * box * D, &mv, VF(vi), 0, 0, z);
        issued_v = j + 1;
      }
    } else if (warp == 13) {
      // ----------------------------------------------------------- products
      // One thread issues for both tiles, P V and then the next S of one tile
      // before the other's: the tensor cores work in that order, so a tile's
      // softmax runs while they have the other tile.  (Two issuing warps share
      // the tensor cores evenly, so that both tiles wait, and compute, at the
      // same time: 1.05 ms against 0.80 for 4096 tokens over 16384 keys.)
      if (tiles > 0 && elect_one()) {
        constexpr uint32_t id_s = idesc_f32(128, 128, 0), id_o = idesc_f32(128, D, 1);
        const uint64_t q0 = desc_rows<D>(sb + Ly::OFF_Q);
        auto logits = [&](int w, int j) {
          const int ik = j % Ly::NK;
          if (w == 0) {
            if (!wait_bar(KF(ik), (j / Ly::NK) & 1, failed, a.dev_status)) return false;
            tc_fence_after();
          }
          const uint64_t kd = desc_rows<D>(sb + Ly::OFF_K + ik * Ly::T8);
          const uint64_t qh = q0 + w * (2 * Ly::T8 / 16), ql = qh + Ly::T8 / 16;
          const uint32_t S = tmem + w * 128;
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) umma_f8(S, qh + 2 * kk, kd + 2 * kk, id_s, kk > 0);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) umma_f8(S, ql + 2 * kk, kd + 2 * kk, id_s, 1);
          umma_commit(SF(w));
          if (w == 1) umma_commit(KE(ik));
          return true;
        };
        bool ok = wait_bar(QR, 0, failed, a.dev_status) && logits(0, 0) && logits(1, 0);
        for (int j = 0; ok && j < tiles; ++j) {
          const int iw = j % Ly::NW;
          const uint64_t vd = umma_desc_sw128_mn(sb + Ly::OFF_W + iw * Ly::T16, 16384);
          ok = wait_bar(WF(iw), (j / Ly::NW) & 1, failed, a.dev_status);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            ok = ok && wait_bar(PH(w), j & 1, failed, a.dev_status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t P = tmem + w * 128, O = tmem + 256 + w * D;
#pragma unroll
            for (int kk = 0; kk < kTileKeys / 32; ++kk) umma_f16_ta(O, P + 8 * kk, vd + 128 * kk, id_o, j > 0 || kk > 0);
            ok = wait_bar(PF(w), j & 1, failed, a.dev_status);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = kTileKeys / 32; kk < kTileKeys / 16; ++kk) umma_f16_ta(O, P + 8 * kk, vd + 128 * kk, id_o, 1);
            if (w == 1) umma_commit(WE(iw));
            if (j + 1 < tiles) ok = logits(w, j + 1);
            else umma_commit(OD(w));
          }
        }
        if (!ok) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
      __syncwarp();
    }
  }

  __syncthreads();
  if (*failed) {
    if (warp == 12 && lane == 0) {  // copies in flight
      bool ok = true;
      for (int i = 0; i < Ly::NK && i < issued_k; ++i)
        ok &= mbar_wait_bounded(KF(i), ((issued_k - 1 - i) / Ly::NK) & 1, gdnc::kWaitLimit);
      for (int i = 0; i < Ly::NV && i < issued_v; ++i)
        ok &= mbar_wait_bounded(VF(i), ((issued_v - 1 - i) / Ly::NV) & 1, gdnc::kWaitLimit);
      if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
    }
    __syncthreads();
    if (warp == 13) tmem_dealloc(tmem, 512);
    return;
  }
  if (wg < 2) {
    // ---------------------------------------------------------------- output
    tc_fence_after();
    const int n = work->n, h = work->h, row = work->row0 + wg * 128 + (tid & 127);
    const bool on = row < work->rows, part = work->pieces > 1;
    const int low = work->past + work->row0 / a.G, limit = work->past + row / a.G;
    const int tok = work->t0 + row / a.G, head = h * a.G + row % a.G;
    const float inv = part ? 1.f : l_sum == 0.f ? 0.f : 1.f / l_sum;
    const int64_t at = (int64_t)work->slot * kItemRows + (row - work->row0);
    uint16_t *dst = a.o + ((int64_t)tok * a.HQ + head) * D;
    const bool zone = *nan_zone != 0;
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld32_issue(O_col + i, o);
        tmem_ld_wait(o);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = tiles > 0 && l_sum != 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
      if (zone && on) {  // NaN values in the keys of the masked zone that this row does see
        for (int key = max(0, low + 1 - kTileKeys) / kTileKeys * kTileKeys; key <= limit; ++key) {
          const int32_t p = a.table[(int64_t)n * a.width + key / a.bs];
          if (p < 0 || p >= a.P) continue;
          const uint8_t *v = a.vc + (((int64_t)p * a.HK + h) * a.bs + key % a.bs) * D + i;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((v[e] & 0x7f) == 0x7f) o[e] = 0x7fc00000u;
        }
      }
      if (on && part) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<uint4 *>(a.tile_o + at * D + i + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else if (on) {
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4 *>(dst + i + e) =
              make_uint4(pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                         pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
      }
    }
    if (on && part) a.tile_ml[at] = make_float2(m_ref, l_sum);
    else if (on && a.lse) a.lse[(int64_t)tok * a.HQ + head] = l_sum == 0.f ? -INFINITY : (m_ref + log2f(l_sum)) * kLn2;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the items that were cut: a warp a row, a lane four columns.
template <int D>
__global__ void __launch_bounds__(256) kv8_join_items_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4;
  grid_wait();
  const int4 w = a.owners[blockIdx.x];
  if (w.w == 0) return;
  Span s;
  const int row0 = w.z * kItemRows;
  if (!request_span(a, w.x, row0, kItemRows, s)) return;
  const int lane = threadIdx.x & 31, c = lane % LANES, rows = min(kItemRows, s.m * a.G - row0);
  for (int r = 8 * blockIdx.y + (threadIdx.x >> 5); r < rows; r += 8 * gridDim.y) {
    auto at = [&](int i) { return (int64_t)(blockIdx.x + i) * kItemRows + r; };
    float top = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < w.w; b += 32) {
      const int cnt = min(32, w.w - b);
      const float2 ml = lane < cnt ? a.tile_ml[at(b + lane)] : make_float2(-INFINITY, 0.f);
      float now = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
      now = fmaxf(now, top);
      const float ref = now == -INFINITY ? 0.f : now;
      const float wt = ex2f(ml.x - ref), old = ex2f(top - ref);
      top = now;
      l = fmaf(l, old, warp_sum(wt * ml.y));
      acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll 4
      for (int i = 0; i < cnt; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(a.tile_o + at(b + i) * D + 4 * c);
        const float wi = __shfl_sync(0xffffffffu, wt, i);
        acc.x = fmaf(wi, v.x, acc.x);
        acc.y = fmaf(wi, v.y, acc.y);
        acc.z = fmaf(wi, v.z, acc.z);
        acc.w = fmaf(wi, v.w, acc.w);
      }
    }
    const int row = row0 + r;
    if (lane < LANES) store_row4(a, s.t0 + row / a.G, w.y * a.G + row % a.G, D, 4 * c, acc, top, l);
  }
}

template <int D>
cudaError_t launch(const AttnArgs &a, int min_rows, cudaStream_t s) {
  using Ly = PrefLay<D>;
  CUtensorMap mk, mv;
  const int keys = a.bs < kTileKeys ? a.bs : kTileKeys;
  if (!cache_map(&mk, a.kc, D, a.bs, (int64_t)a.P * a.HK, keys, true) || !cache_map(&mv, a.vc, D, a.bs, (int64_t)a.P * a.HK, keys, false))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = gdn_host::allow_smem(kv8_prefill_kernel<D>, Ly::BYTES, done);
  if (e != cudaSuccess) return e;
  // no more items than this, and a slot's block for each SM
  const int64_t rows = (int64_t)a.T * a.G, most = a.HK * (rows / kItemRows + std::min<int64_t>(a.N, rows / min_rows));
  if (most > INT_MAX - kSlots) return cudaErrorInvalidConfiguration;
  e = gdn_host::launch_dependent(kv8_prefill_kernel<D>, dim3((unsigned)most + kSlots), kPrefThreads, Ly::BYTES, s, a, min_rows,
                                 gdn_host::sm_count(), mk, mv);
  if (e != cudaSuccess) return e;
  return gdn_host::launch_dependent(kv8_join_items_kernel<D>, dim3(kSlots, 8), 256, 0, s, a);
}

}  // namespace

namespace gdnkv {
cudaError_t launch_prefill(const AttnArgs &a, int min_rows, cudaStream_t s) {
  return a.D == 128 ? launch<128>(a, min_rows, s) : launch<64>(a, min_rows, s);
}
size_t prefill_workspace(int D) {
  return (size_t)kSlots * (kItemRows * (size_t)(D + 2) * sizeof(float) + sizeof(int4));
}
void prefill_place(AttnArgs &a, void *ws) {
  a.tile_o = static_cast<float *>(ws);
  a.tile_ml = reinterpret_cast<float2 *>(a.tile_o + (size_t)kSlots * kItemRows * a.D);
  a.owners = reinterpret_cast<int4 *>(a.tile_ml + (size_t)kSlots * kItemRows);
}
}  // namespace gdnkv
