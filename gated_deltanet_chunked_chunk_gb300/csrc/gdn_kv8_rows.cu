// gdn_kv8_rows.cu -- attention over the paged 8-bit cache for 17 to 32 rows a
// (request, kv head): drafted tokens of a group of heads, on tcgen05.  The
// mathematics, the number formats and the line of stages (here of 128 keys, one
// team an SM) are those of gdn_kv8_attn.cu.
//
// Bound: HBM, 2 D bytes for each (token, kv head).
//
// Products, transposed as there: S^T = K Q^T has the keys as the 128 rows of a
// tcgen05 tile and the query rows as its columns, O^T = V^T P^T the values'
// columns as its rows.  Both take the cache's bytes as they stand (kind::f8f6f4),
// so no code is widened and a tile's 32 KB pass through shared memory as they
// are (V widened to f16 by eight warps: 115 us where this takes 103, shared
// memory busy with 168 KB a tile).  Q is the sum of two e4m3 numbers, side by
// side as 64 columns of one product.  P is an f16 number taken apart into four
// e5m2 ones, exactly: an e5m2 number is the upper byte of an f16 one, each part
// takes three of the 11 significant bits, and the remainders are f16 numbers
// again; the parts are 4 x 32 columns of one product, whose sum is formed when a
// pair ends.  e5m2 ends at 2^-16, so exponents are held up high: weights reach
// 2^13 when a reference is taken and 2^15 before the next one is, and what is lost
// is under 2^-29 of the largest (f16 weights of up to 1 lose 2^-25).
//
// Softmax.  Two groups of four warps take the tiles in turn, a thread a key, each
// with sums, references and an O^T of its own that join when the pair ends.  What
// a row's exponents are taken against stands in shared memory and changes only
// where some logit of the tile is too far above it, which one barrier with a vote
// finds; then the rows' maxima are formed by halving exchanges, and O^T is
// rescaled column by column.  A thread keeps its own keys' part of every row's sum
// until the pair ends.  One group: 137 us; three, whose registers spill: 117.  At a
// pair's end the second group prepares the next pair's queries while the first one
// writes.
//
// Warps: 0-7 softmax, 8-11 clear what must not be seen in a context's last tiles,
// 12 brings pages by TMA, 13 issues the products.  Tensor memory: two S^T of 64
// columns, two O^T of 128.  Once a wait has run out nothing is waited for any more
// and nothing written, but the softmax warps go through all their tiles, as they
// meet at barriers there.
//
// 4 requests of 4 tokens, 131072 keys, 32 heads of 128, 4 kv heads: 103 us, 77 % of
// HBM (mma.sync in gdn_kv8_attn.cu: 144, 55 %); 256 such requests of 64 to 2048
// keys: 132 (144).  At 16 rows that kernel is the better one (100 us against 105).
// What is left: a group's chain from S^T to P^T, 2500 cycles a tile, against 2 x
// 1400 that two tiles' bytes take.
#include <float.h>

#include "gdn_kv8_tc.cuh"

namespace {

using namespace gdn;
using namespace gdnkv;

constexpr int kTile = 128;     // keys a stage
constexpr int kRows = 32;
constexpr int kParts = 4;      // e5m2 numbers that make up a weight
constexpr int kFirstCleaner = 8, kProducer = 12, kIssuer = 13;
constexpr int kThreads = 512;  // whole warpgroups: two warps idle
constexpr float kLarge = 15.f, kLift = 13.f;  // exponents are at most the first, of a new maximum the second
constexpr int kZones = 8;      // tiles of the masked zone that are on their way at once, or more
constexpr int kParSlots = 16;  // stages whose page constants are kept: more than can be in flight

template <int D>
struct RowsLay {
  static constexpr int T8 = kTile * D;        // bytes of a K or V tile
  static constexpr int QB = kRows * D;        // of a part of Q
  static constexpr int PB = kTile * kRows * kParts;
  static constexpr int NK = 5, NV = 5;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + NK * T8;
  static constexpr int OFF_Z = OFF_V + NV * T8;   // zeros: what stands for columns 64 .. 127 where D is 64
  static constexpr int OFF_Q = OFF_Z + (D == 64 ? T8 : 0);  // high, low
  static constexpr int OFF_P = OFF_Q + 2 * QB;
  static constexpr int OFF_PAR = OFF_P + 2 * PB;  // float4 {k scale, lv, 2^-lv, 0} x 8 pages a slot
  static constexpr int OFF_ROW = OFF_PAR + kParSlots * 128;  // float[32]: factors, the groups' references (negated) and rescales
  static constexpr int OFF_TOP = OFF_ROW + 5 * kRows * 4;    // float[8 warps][32]
  static constexpr int OFF_OUT = OFF_TOP + 8 * kRows * 4;    // int64[32]: where a row's result goes, -1: nowhere
  static constexpr int OFF_BAR = OFF_OUT + kRows * 8;
  static constexpr int BARS = 2 * NK + 2 * NV + 8 + 3 + 2 * kZones + kParSlots;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 160;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};

// MN-major descriptor of a tile [key][B bytes], B 128 or 64 and its swizzle; lbo:
// bytes to the tile of the next B columns.
template <int B> __device__ __forceinline__ uint64_t desc_keys(uint32_t saddr, uint32_t lbo) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16;
  d |= static_cast<uint64_t>((8 * B) >> 4) << 32;  // 8 keys
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(B == 128 ? 2 : 4) << 61;
  return d;
}
// Two fp32 numbers in one instruction.
__device__ __forceinline__ float2 fma22(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 x, x, y, z; "
      "mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul22(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 bits2(const uint32_t *x) { return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])); }
// What two f16 numbers leave beyond their upper bytes.
__device__ __forceinline__ uint32_t remainder2(uint32_t a) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(a & 0xff00ff00u));
  return r;
}
__device__ __forceinline__ bool vote128(int id, bool x) {  // whether any of a group's threads says so; they meet here
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"(x ? 1u : 0u), "r"(id)
               : "memory");
  return r != 0;
}
// Lane l gets the combination over the warp of all lanes' x[l].
template <class F> __device__ __forceinline__ float fold32(const float *x, F f) {
  const int lane = threadIdx.x & 31;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const bool up = lane & 16;
    const float other = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 16], 16);
    y[i] = f(up ? x[i + 16] : x[i], other);
  }
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float other = __shfl_xor_sync(0xffffffffu, up ? y[i] : y[i + o], o);
      y[i] = f(up ? y[i + o] : y[i], other);
    }
  return y[0];
}

// A block's walk over its stretch, pair by pair: each kind of warp has its own.
struct Walk {
  Place at;
  int left, count;  // stages of the stretch, of it in this pair
  __device__ __forceinline__ void enter() { count = min(left, at.of - at.stage); }
  __device__ __forceinline__ bool next(const AttnArgs &a) {  // on to the next pair
    left -= count;
    if (left <= 0) return false;
    at.stage = 0;
    if (++at.h == a.HK) next_request(a, at);
    enter();
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_rows_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Ly = RowsLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto KF = [&](int i) { return bar + 8 * i; };
  auto KE = [&](int i) { return bar + 8 * (Ly::NK + i); };
  auto VF = [&](int i) { return bar + 8 * (2 * Ly::NK + i); };
  auto VE = [&](int i) { return bar + 8 * (2 * Ly::NK + Ly::NV + i); };
  const uint32_t bx = bar + 8 * (2 * Ly::NK + 2 * Ly::NV);
  auto SF = [&](int i) { return bx + 8 * i; };
  auto SE = [&](int i) { return bx + 16 + 8 * i; };
  auto PF = [&](int i) { return bx + 32 + 8 * i; };
  auto PE = [&](int i) { return bx + 48 + 8 * i; };
  const uint32_t QR = bx + 64, never = bx + 72, DR = bx + 80;
  auto ZS = [&](int i) { return bx + 88 + 8 * (i % kZones); };
  auto ZF = [&](int i) { return bx + 88 + 8 * kZones + 8 * (i % kZones); };
  auto PR = [&](int i) { return bx + 88 + 16 * kZones + 8 * i; };
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 4);
  volatile int *nan_zone = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC + 8);  // [16], by pair
  Walk *begin = reinterpret_cast<Walk *>(smem + Ly::OFF_MISC + 80);
  static_assert(sizeof(Walk) <= 80, "room for it");
  if (tid == 0) {
    for (int i = 0; i < Ly::NK; ++i) { mbar_init(KF(i), 1); mbar_init(KE(i), 1); }
    for (int i = 0; i < Ly::NV; ++i) { mbar_init(VF(i), 1); mbar_init(VE(i), 1); }
    for (int i = 0; i < kZones; ++i) { mbar_init(ZS(i), 1); mbar_init(ZF(i), 4); }
    for (int i = 0; i < 2; ++i) { mbar_init(SF(i), 1); mbar_init(SE(i), 4); mbar_init(PF(i), 128); mbar_init(PE(i), 1); }
    for (int i = 0; i < kParSlots; ++i) mbar_init(PR(i), 1);
    mbar_init(QR, 128);  // the second group's threads
    mbar_init(never, 1);
    mbar_init(DR, 1);
    mbar_fence_init();
    *failed = 0;
    for (int i = 0; i < 16; ++i) nan_zone[i] = 0;
  }
  grid_wait();
  // Only now: the joining kernel reads lengths and offsets before its own wait.
  grid_release();
  if (warp == 0) {
    Walk w{};
    w.left = find_place(a, blockIdx.x, gridDim.x, true, w.at);
    w.enter();
    if (lane == 0) *begin = w;
  }
  if (D == 64)
    for (int i = tid; i < Ly::T8 / 16; i += kThreads) sts128(sb + Ly::OFF_Z + i * 16, 0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  if (begin->left == 0) return;
  if (warp == kIssuer) tmem_alloc(sb + Ly::OFF_MISC + 4, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int page_bits = 31 - __clz(a.bs);
  int issued_k = 0, issued_v = 0;  // stages that the producer has issued

  // Of the block's 65536 registers (512 threads x 128) the softmax warps take 192 a
  // thread, the others 64: 256 x 192 + 256 x 64 = 65536.  (168: 106 us against 103.)
  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int wg = warp >> 2, key = tid & 127;  // group, key of the tile
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t S_col = tmem + lanes + wg * 64, O_col = tmem + lanes + 128 + wg * 128;
    float *fac = reinterpret_cast<float *>(smem + Ly::OFF_ROW), *ref = fac + (1 + wg) * kRows, *res = fac + (3 + wg) * kRows;
    float *tops = reinterpret_cast<float *>(smem + Ly::OFF_TOP) + wg * 4 * kRows;
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(never, 0, gdnc::kTestWaitLimit)) {
      *failed = 1;
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    int64_t *outs = reinterpret_cast<int64_t *>(smem + Ly::OFF_OUT);
    // A pair's queries, by the second group: four threads a row.
    const int row = key >> 2, part = key & 3;
    uint4 u[D / 32];
    auto read_queries = [&](const Place &at) {
      const bool on = row < at.s.m * a.G;
      const uint16_t *src = a.q + (int64_t)(at.s.t0 + row / a.G) * a.ldq + (int64_t)(at.h * a.G + row % a.G) * D + part * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) u[i] = on ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
    };
    auto put_queries = [&]() {
      float top = 0.f, bad = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf16lo_f(x[e]), hi = bf16hi_f(x[e]);
          top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
          bad = fmaf(lo, 0.f, fmaf(hi, 0.f, bad));  // NaN once an element is not finite
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        bad += __shfl_xor_sync(0xffffffffu, bad, o);
      }
      int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      e2 = e2 < -100 ? -100 : e2 > 120 ? 120 : e2;
      const float down = pow2(7 - e2);
      if (part == 0) fac[row] = pow2(e2 - 7) * a.scale_log2e + bad;
      const uint32_t qh = sb + Ly::OFF_Q, ql = qh + Ly::QB;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t c = part * (D / 64) + i;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 &v = u[2 * i + (e >> 1)];
          const uint32_t w0 = (e & 1) ? v.z : v.x, w1 = (e & 1) ? v.w : v.y;
          const float x0 = bf16lo_f(w0) * down, x1 = bf16hi_f(w0) * down, x2 = bf16lo_f(w1) * down, x3 = bf16hi_f(w1) * down;
          const uint32_t h0 = cvt_e4m3x2(x0, x1), h1 = cvt_e4m3x2(x2, x3);
          const float2 b0 = f16x2_f32(e4m3x2_f16x2(h0)), b1 = f16x2_f32(e4m3x2_f16x2(h1));
          hi[e] = h0 | (h1 << 16);
          lo[e] = cvt_e4m3x2(x0 - b0.x, x1 - b0.y) | (cvt_e4m3x2(x2 - b1.x, x3 - b1.y) << 16);
        }
        const uint32_t r = row, place = D == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
        sts128(qh + place, hi[0], hi[1], hi[2], hi[3]);
        sts128(ql + place, lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(QR);
    };
    Walk w = *begin;
    int j = 0, mine = 0, piece = 0;  // stages before this pair, this group's tiles, pairs so far
    if (wg == 1) {
      read_queries(w.at);
      put_queries();
    }
    if (key < kRows) ref[key] = FLT_MAX;
    named_bar_sync(3, 256);  // factors and references are there
    bool more;
    do {
      const int m = w.at.s.m, L = w.at.s.L;
      float ls[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) ls[r] = 0.f;
#pragma unroll 1
      for (int i = wg; i < w.count; i += 2, ++mine) {
        const int slot = (j + i) % kParSlots;
        if (ok) ok = wait_bar(PR(slot), ((j + i) / kParSlots) & 1, failed, a.dev_status) &&
                     wait_bar(SF(wg), mine & 1, failed, a.dev_status);
        __syncwarp();
        tc_fence_after();
        uint32_t x[kRows], y[kRows];
        tmem_ld32_issue(S_col, x);
        tmem_ld32_issue(S_col + 32, y);  // the products with Q's low parts
        const float4 par = lds_f4(sb + Ly::OFF_PAR + slot * 128 + (key >> page_bits) * 16);
        const int over = (w.at.stage + i) * kTile + key - (L - m);  // > r / G: row r does not see this key
        tmem_ld_wait(x);
        tie32(y);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(SE(wg));
        float t[kRows], high = -INFINITY;
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(fac + r);
          const float2 s2 = make_float2(par.x, par.x), l2 = make_float2(par.y, par.y);
          const float2 v0 = fma22(add2(bits2(x + r), bits2(y + r)), mul22(make_float2(f.x, f.y), s2), l2);
          const float2 v1 = fma22(add2(bits2(x + r + 2), bits2(y + r + 2)), mul22(make_float2(f.z, f.w), s2), l2);
          t[r] = v0.x;
          t[r + 1] = v0.y;
          t[r + 2] = v1.x;
          t[r + 3] = v1.y;
        }
        if (over > 0) {
          const int first = over * a.G;  // the first row that sees the key
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (r < first) t[r] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {  // ref holds the references' negatives
          const float4 f = *reinterpret_cast<const float4 *>(ref + r);
          const float2 v0 = add2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y));
          const float2 v1 = add2(make_float2(t[r + 2], t[r + 3]), make_float2(f.z, f.w));
          high = max3(high, v0.x, v0.y);
          high = max3(high, v1.x, v1.y);
        }
        if (vote128(1 + wg, high > kLarge)) {
          const float most = fold32(t, [](float p, float q) { return fmaxf(p, q); });
          tops[(warp & 3) * kRows + lane] = most;
          named_bar_sync(1 + wg, 128);
          if ((warp & 3) == 0) {
            const float top = fmaxf(fmaxf(tops[lane], tops[kRows + lane]), fmaxf(tops[2 * kRows + lane], tops[3 * kRows + lane]));
            const float old = -ref[lane], now = fmaxf(old, reference_of(top, kLift));
            res[lane] = ex2f(old - now);
            ref[lane] = -now;
          }
          named_bar_sync(1 + wg, 128);
#pragma unroll
          for (int r = 0; r < kRows; ++r) ls[r] *= res[r];
          if (i >= 2) {
            // the group's product before this one has written O^T
            if (ok) ok = wait_bar(PE(wg), (mine - 1) & 1, failed, a.dev_status);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kParts * kRows; c += kRows) {
              tmem_ld32_issue(O_col + c, x);
              tmem_ld_wait(x);
#pragma unroll
              for (int r = 0; r < kRows; ++r) x[r] = __float_as_uint(__uint_as_float(x[r]) * res[r]);
              tmem_st32(O_col + c, x);
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        uint32_t p[kParts][kRows / 4];
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(ref + r);
          float2 p0 = add2(make_float2(t[r], t[r + 1]), make_float2(f.x, f.y));
          float2 p1 = add2(make_float2(t[r + 2], t[r + 3]), make_float2(f.z, f.w));
          p0 = make_float2(ex2f(p0.x), ex2f(p0.y));
          p1 = make_float2(ex2f(p1.x), ex2f(p1.y));
          const float2 l0 = fma22(p0, make_float2(par.z, par.z), make_float2(ls[r], ls[r + 1]));
          const float2 l1 = fma22(p1, make_float2(par.z, par.z), make_float2(ls[r + 2], ls[r + 3]));
          ls[r] = l0.x;
          ls[r + 1] = l0.y;
          ls[r + 2] = l1.x;
          ls[r + 3] = l1.y;
          uint32_t lo = pack_f16(p0.x, p0.y), hi = pack_f16(p1.x, p1.y);
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            p[q][r / 4] = __byte_perm(lo, hi, 0x7531);  // the upper bytes
            lo = remainder2(lo);
            hi = remainder2(hi);
          }
        }
        if (ok && mine > 0) ok = wait_bar(PE(wg), (mine - 1) & 1, failed, a.dev_status);
        const uint32_t dst = sb + Ly::OFF_P + wg * Ly::PB + key * 128;
#pragma unroll
        for (int c = 0; c < 2 * kParts; ++c) {
          const uint32_t *v = &p[c >> 1][4 * (c & 1)];
          sts128(dst + ((c ^ (key & 7)) << 4), v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(PF(wg));
      }
      // ------------------------------------------------------ the pair's result
      // The second group hands over its half and goes on to the next pair's
      // queries, the first one joins the halves and writes.
      Walk ahead = w;
      more = ahead.next(a);
      if (wg == 1 && more) read_queries(ahead.at);
      const bool some = w.count > wg;  // this group has had a tile
      if (ok && some) ok = wait_bar(PE(wg), (mine - 1) & 1, failed, a.dev_status);
      __syncwarp();
      tc_fence_after();
      tops[(warp & 3) * kRows + lane] = fold32(ls, [](float p, float q) { return p + q; });
      uint32_t x[kRows];
      tmem_ld32_issue(O_col, x);
      tmem_ld_wait(x);
#pragma unroll
      for (int c = kRows; c < kParts * kRows; c += kRows) {
        uint32_t y[kRows];
        tmem_ld32_issue(O_col + c, y);
        tmem_ld_wait(y);
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r] = __float_as_uint(__uint_as_float(x[r]) + __uint_as_float(y[r]));
      }
      tc_fence_before();
      named_bar_sync(3, 256);  // both groups' products are done: P's place is free
      float *other = reinterpret_cast<float *>(smem + Ly::OFF_P);  // the second group's [32 rows][128]
      const bool from_start = w.at.stage == 0, whole = from_start && w.count == w.at.of;
      if (wg == 1) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) other[r * 128 + key] = some ? __uint_as_float(x[r]) : 0.f;
      } else if (warp == 0) {
        const float *t1 = tops + 4 * kRows;
        const float l0 = tops[lane] + tops[kRows + lane] + tops[2 * kRows + lane] + tops[3 * kRows + lane];
        const float l1 = t1[lane] + t1[kRows + lane] + t1[2 * kRows + lane] + t1[3 * kRows + lane];
        const float m0 = -ref[lane], m1 = -ref[kRows + lane], top = fmaxf(m0, m1);
        const float w0 = ex2f(m0 - top), w1 = ex2f(m1 - top), l = w0 * l0 + w1 * l1;
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is 0
        res[lane] = w0 * inv;
        res[kRows + lane] = w1 * inv;
        const int64_t out = whole ? (int64_t)(w.at.s.t0 + lane / a.G) * a.HQ + w.at.h * a.G + lane % a.G
                                  : ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * a.row_cap + lane;
        const bool write = lane < m * a.G && !*failed;
        outs[lane] = write ? out : -1;
        if (write) {
          if (!whole) a.part_ml[out] = make_float2(top, l);
          else if (a.lse) a.lse[out] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
        }
      }
      named_bar_sync(3, 256);
      if (key < kRows) ref[key] = FLT_MAX;
      if (wg == 1) {
        if (more) put_queries();
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          x[r] = __float_as_uint(fmaf(__uint_as_float(x[r]), res[r], other[r * 128 + key] * res[kRows + r]));
      }
      named_bar_sync(3, 256);  // the halves are read, the next pair's factors and references there
      if (wg == 0 && key < D) {
        if (nan_zone[piece & 15]) {
          // NaN values in this stretch's keys of the masked zone, for the rows that see them
          const int k1 = min(L, (w.at.stage + w.count) * kTile);
          for (int k = max(w.at.stage * kTile, max(0, L - m + 1 - kTile)); k < k1; ++k) {
            const int32_t pg = a.table[(int64_t)w.at.n * a.width + (k >> page_bits)];
            if (pg < 0 || pg >= a.P) continue;
            const uint8_t v = a.vc[(((int64_t)pg * a.HK + w.at.h) * a.bs + (k & (a.bs - 1))) * D + key];
            if ((v & 0x7f) != 0x7f) continue;
            const int first = (k - (L - m)) * a.G;  // the first row that sees the key
#pragma unroll
            for (int r = 0; r < kRows; ++r)
              if (r >= first) x[r] = 0x7fc00000u;
          }
        }
        if (whole) {  // turned in this group's place of P: 2-byte stores took 8000 cycles
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(sb + Ly::OFF_P + (r * D + key) * 2),
                         "h"((uint16_t)pack_bf16(__uint_as_float(x[r]), 0.f))
                         : "memory");
        } else {
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const int64_t out = outs[r];
            if (out >= 0) a.part_o[out * D + key] = __uint_as_float(x[r]);
          }
        }
        if (tid == 0) nan_zone[(piece + 8) & 15] = 0;  // eight pairs back and ahead: nobody is there
      }
      if (wg == 0 && whole) {
        named_bar_sync(1, 128);  // (and the next vote comes before P is written again)
#pragma unroll
        for (int e = key; e < kRows * D / 8; e += 128) {
          const int64_t out = outs[e / (D / 8)];
          if (out >= 0) *reinterpret_cast<uint4 *>(a.o + out * D + e % (D / 8) * 8) = lds128(sb + Ly::OFF_P + e * 16);
        }
      }
      j += w.count;
      ++piece;
      w = ahead;
    } while (more);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp >= kFirstCleaner && warp < kProducer) {
    // -------------------------------------------- values of the masked zone
    // Keys past the context hold whatever the page held before, and a key that
    // only later rows see may be NaN: its weight is 0 there, but 0 x NaN is not.
    // Such codes become 0; NaN that a row does see is put back at the end.
    const int ct = tid - 32 * kFirstCleaner;
    Walk w = *begin;
    int j = 0, piece = 0, zones = 0;
    bool ok = true;
    do {
      const int L = w.at.s.L, low = L - w.at.s.m;
      for (int i = 0; ok && i < w.count; ++i) {
        const int k0 = (w.at.stage + i) * kTile;
        if (k0 + kTile - 1 <= low) continue;
        const int iv = (j + i) % Ly::NV;
        // called (until then the tile's barrier may be two uses back), and there
        ok = wait_bar(ZS(zones), (zones / kZones) & 1, failed, a.dev_status) &&
             wait_bar(VF(iv), ((j + i) / Ly::NV) & 1, failed, a.dev_status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint32_t seen = 0;
        for (int e = ct; e < Ly::T8 / 16; e += 128) {
          const uint32_t at = sb + Ly::OFF_V + iv * Ly::T8 + e * 16;
          uint4 u = lds128(at);
          if (k0 + e / (D / 16) >= L) u = make_uint4(0, 0, 0, 0);
          seen |= any_nan(u.x) | any_nan(u.y) | any_nan(u.z) | any_nan(u.w);
          sts128(at, drop_nan(u.x), drop_nan(u.y), drop_nan(u.z), drop_nan(u.w));
        }
        if (seen) nan_zone[piece & 15] = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ZF(zones));
        ++zones;
      }
      j += w.count;
      ++piece;
    } while (ok && w.next(a));
  } else if (warp == kProducer) {
    // ------------------------------------------------------------- producer
    const int ppt = a.bs >= kTile ? 1 : kTile / a.bs, box = kTile / ppt;
    Walk w = *begin;
    int j = 0, zones = 0;
    bool ok = true;
    do {
      int batch = -1, page = -1;
      float ks = 0.f, lv = 0.f, iv = 1.f;
      for (int i = 0; ok && i < w.count; ++i, ++j) {
        const int first = (w.at.stage + i) * ppt;
        if (first / 32 != batch) {
          batch = first / 32;
          const int pi = batch * 32 + lane;
          page = -1;
          ks = 0.f;
          lv = -INFINITY;
          iv = 1.f;
          if (((int64_t)pi << page_bits) < w.at.s.keys) {
            const int32_t p = a.table[(int64_t)w.at.n * a.width + pi];
            if (p < 0 || p >= a.P) {
              set_status(a.dev_status, GDN_DEV_BAD_SLOT);
            } else {
              page = p;
              const int64_t at = (int64_t)p * a.HK + w.at.h;
              ks = a.ks[at];
              const float v = a.vs[at];
              lv = log2f(v);
              iv = 1.f / v;
            }
          }
        }
        const int ik = j % Ly::NK, vi = j % Ly::NV;
        if (j >= Ly::NK) ok = wait_bar(KE(ik), (j / Ly::NK - 1) & 1, failed, a.dev_status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
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
        const int z = pg >= 0 ? pg * a.HK + w.at.h : a.P * a.HK;  // outside the tensor: zeros
        if (lane < ppt) tma_load_3d(sb + Ly::OFF_K + ik * Ly::T8 + lane * box * D, &mk, KF(ik), 0, 0, z);
        issued_k = j + 1;
        if (j >= Ly::NV) ok = wait_bar(VE(vi), (j / Ly::NV - 1) & 1, failed, a.dev_status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(VF(vi), Ly::T8);
        __syncwarp();
        if (lane < ppt) tma_load_3d(sb + Ly::OFF_V + vi * Ly::T8 + lane * box * D, &mv, VF(vi), 0, 0, z);
        if ((w.at.stage + i) * kTile + kTile - 1 > w.at.s.L - w.at.s.m) {
          if (lane == 0) mbar_arrive(ZS(zones));
          ++zones;
        }
        issued_v = j + 1;
      }
    } while (ok && w.next(a));
  } else if (warp == kIssuer && elect_one()) {
    // ------------------------------------------------------------- products
    constexpr uint32_t id_s = idesc_f32(128, 2 * kRows, 0);
    constexpr uint32_t id_o = idesc_f32(128, kParts * kRows, 1) | (1u << 15) | (1u << 10);  // V^T turned; P e5m2
    const uint64_t qd = desc_rows<D>(sb + Ly::OFF_Q);
    Walk w = *begin;
    int j = 0, piece = 0, zones = 0;
    int tiles0 = 0, tiles1 = 0;  // each group's tiles before this pair
    bool ok = true;
    auto logits = [&](int i) {  // tile i of the pair
      const int ik = (j + i) % Ly::NK, g = i & 1;
      if (!wait_bar(KF(ik), ((j + i) / Ly::NK) & 1, failed, a.dev_status)) return false;
      const int nth = (g ? tiles1 : tiles0) + (i >> 1);
      if (nth > 0 && !wait_bar(SE(g), (nth - 1) & 1, failed, a.dev_status)) return false;
      tc_fence_after();
      const uint64_t kd = desc_rows<D>(sb + Ly::OFF_K + ik * Ly::T8);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) umma_f8(tmem + g * 64, kd + 2 * kk, qd + 2 * kk, id_s, kk > 0);
      umma_commit(SF(g));
      umma_commit(KE(ik));
      return true;
    };
    do {
      ok = wait_bar(QR, piece & 1, failed, a.dev_status) && logits(0) && (w.count < 2 || logits(1));
      for (int i = 0; ok && i < w.count; ++i) {
        const int iv = (j + i) % Ly::NV, g = i & 1;
        if (i + 2 < w.count) ok = logits(i + 2);
        ok = ok && wait_bar(VF(iv), ((j + i) / Ly::NV) & 1, failed, a.dev_status);
        if ((w.at.stage + i) * kTile + kTile - 1 > w.at.s.L - w.at.s.m) {
          ok = ok && wait_bar(ZF(zones), (zones / kZones) & 1, failed, a.dev_status);
          ++zones;
        }
        ok = ok && wait_bar(PF(g), ((g ? tiles1 : tiles0) + (i >> 1)) & 1, failed, a.dev_status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t v = sb + Ly::OFF_V + iv * Ly::T8;
        const uint64_t vd = desc_keys<D>(v, sb + Ly::OFF_Z - v), pd = desc_keys<128>(sb + Ly::OFF_P + g * Ly::PB, 0);
#pragma unroll
        for (int kk = 0; kk < kTile / 32; ++kk)
          umma_f8(tmem + 128 + g * 128, vd + 2 * D * kk, pd + 256 * kk, id_o, i > 1 || kk > 0);
        umma_commit(PE(g));
        umma_commit(VE(iv));
      }
      j += w.count;
      tiles0 += (w.count + 1) >> 1;
      tiles1 += w.count >> 1;
      ++piece;
    } while (ok && w.next(a));
    if (!ok) {  // let the products in flight finish before the block leaves
      umma_commit(DR);
      if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*failed && warp == kProducer && lane == 0) {  // copies in flight
    bool ok = true;
    for (int i = 0; i < Ly::NK && i < issued_k; ++i) ok &= mbar_wait_bounded(KF((issued_k - 1 - i) % Ly::NK), ((issued_k - 1 - i) / Ly::NK) & 1, gdnc::kWaitLimit);
    for (int i = 0; i < Ly::NV && i < issued_v; ++i) ok &= mbar_wait_bounded(VF((issued_v - 1 - i) % Ly::NV), ((issued_v - 1 - i) / Ly::NV) & 1, gdnc::kWaitLimit);
    if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
  }
  if (*failed) __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  using Ly = RowsLay<D>;
  CUtensorMap mk, mv;
  const int keys = a.bs < kTile ? a.bs : kTile;
  if (!cache_map(&mk, a.kc, D, a.bs, (int64_t)a.P * a.HK, keys, true) || !cache_map(&mv, a.vc, D, a.bs, (int64_t)a.P * a.HK, keys, true))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = gdn_host::allow_smem(kv8_rows_kernel<D>, Ly::BYTES, done);
  if (e != cudaSuccess) return e;
  return gdn_host::launch_dependent(kv8_rows_kernel<D>, dim3(kSMs), kThreads, Ly::BYTES, s, a, mk, mv);
}

}  // namespace

namespace gdnkv {
cudaError_t launch_kv8_rows(const AttnArgs &a, cudaStream_t s) { return a.D == 128 ? launch<128>(a, s) : launch<64>(a, s); }
}  // namespace gdnkv
