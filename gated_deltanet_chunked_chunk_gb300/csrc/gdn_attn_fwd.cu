// gdn_attn_fwd.cu -- attention of packed sequences, forward, on tcgen05.
//
//   S = q K^T,  p_j = 2^(c S_j - c m),  l = sum p_j,  o = sum p_j v_j / l,
//   lse = (c m + log2 l) ln 2,  c = scale log2 e
//
// with m the running maximum of S.  Bound: the tensor cores, 4 D operations a (row,
// key, head).  16384 rows of one sequence, 32 heads, D = 128: 1385 to 1405 us, 1.57
// PFLOP/s, 81 % of a large library matrix product's rate; D = 64: 1048 us, 1.05 PFLOP/s (half
// the products, all of the arithmetic).  24 sequences of 200 to 2000 rows: 331 us.  A pair of tiles takes some 3000 cycles for 128 keys, of which the products alone
// are 2050; the rest is S's wait for the P V that reads the same columns.
//
// An item is two tiles of 128 rows of one head, which share the keys and values
// that TMA brings, and whose softmaxes take turns on the tensor cores (one tile, where
// fewer items than SMs would come out).  Warps 0-7 and 8-15 are the softmax of the two
// tiles: a thread holds half a row, 64 logits; 16 brings the tiles, 17 issues the
// products, 18 clears what a last tile of values holds past the sequence, 19 finds the
// items.
//
// Tensor memory (512 columns): S of both tiles, P in bf16 over its S (each half over
// the half that its threads read), O of both tiles.  Products of one thread execute in
// order, so an S of the next keys, issued after the P V that reads the same columns, is
// safe, and "S is there" also says that O may be touched.
//
// m grows only where an exponent is more than kMost above c m: both threads of a row
// agree on that in one barrier that also joins their votes, and O is then rescaled.
// P has 8 significant bits (bf16 keeps fp32's range, so any m near the maximum is as
// good), l is the sum before that rounding, whose errors (2^-8 of a weight at most, either
// way) mostly cancel in o.
//
// c m is rounded, the same for all weights of a row, which cancels in o and is in lse.  Past
// |c m| = kFar the rounding could reach 2^6 and, twice as far, overflow the weights: there a
// power of two between c / 4 and c / 2 takes the place of c, whose products are exact.  Numbers
// S of that size that differ at all do so by 2^6 / c or more, so the largest has all the weight,
// but 2^-16, either way.
#include <algorithm>
#include <type_traits>

#include "gdn_attn.cuh"

namespace {

using namespace gdnat;

constexpr int kThreads = 640;
constexpr float kMost = 8.f;
constexpr float kFar = 1073741824.f;  // 2^30
constexpr int kItems = 4;  // items between the warp that finds them and the others

// An item, 32-bit words in shared memory: first row of q and of k of the sequence, its
// keys; the item's first row in the sequence; rows and key tiles of both row tiles; the
// head; whether it is one (0: there are no more); what the first row of both row tiles sees
// last.  (What the softmax's loop rarely needs it reads there: the logits take
// the registers.)
enum Word { W_Q = 0, W_K = 4, W_KEYS = 8, W_ROW0 = 12, W_COUNT = 16, W_TILES = 24, W_HEAD = 32, W_ON = 36, W_LOW = 40, W_BYTES = 48 };

template <int D> struct Lay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NS = D == 128 ? 4 : 8;  // stages of the line K0 V0 K1 V1 ..
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TB;
  static constexpr int OFF_X = OFF_KV + NS * TB;  // float [tile][half][row]: what a row's threads tell each other
  static constexpr int OFF_WORK = OFF_X + 2 * 2 * 128 * 4;
  static constexpr int OFF_BAR = OFF_WORK + kItems * W_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (2 * NS + 2 * kItems + 13) * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(OFF_X % 1024 == 0 && BYTES <= 227 * 1024, "one block an SM");
};

__device__ __forceinline__ bool vote_any(int id, bool mine) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.pred q, %1, 256, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"(id), "r"((uint32_t)mine)
               : "memory");
  return r != 0;
}

// The factor of S in the exponents of a row whose reference is m.
__device__ __forceinline__ float factor(float c, float m) {
  return fabsf(__fmul_rn(m, c)) > kFar ? __uint_as_float((__float_as_uint(c) & 0x7f800000u) - 0x00800000u) : c;
}

// Half a row of O, times inv, to dst; flags: 1: it is a row of the sequence, 2: it saw a
// key (if not, what O's columns hold is not used).  Eight columns at a time: more of them
// cost the softmax registers (spills: 60 us more at 16384 rows).
template <int D> __device__ __forceinline__ void store_half(uint32_t O, uint16_t *dst, float inv, int flags) {
#pragma unroll 1
  for (int i = 0; i < D / 2; i += 8) {
    uint32_t o[8];
    gdnkv::tmem_ld8(O + i, o);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = flags & 2 ? pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
    if (flags & 1) *reinterpret_cast<uint4 *>(dst + i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const Args a, int tiles_an_item, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv) {
  using Ly = Lay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_wait();
  const uint32_t failed = sb + Ly::OFF_MISC;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto FULL = [&](int i) { return bar + 8 * i; };
  auto EMPTY = [&](int i) { return bar + 8 * (Ly::NS + i); };
  const uint32_t bw = bar + 16 * Ly::NS, bx = bw + 16 * kItems;
  auto WF = [&](int i) { return bw + 8 * i; };  // an item is there, all have read it
  auto WE = [&](int i) { return bw + 8 * (kItems + i); };
  auto SF = [&](int w) { return bx + 8 * w; };       // S is there
  auto PF = [&](int w) { return bx + 16 + 8 * w; };  // P is there
  auto OD = [&](int w) { return bx + 32 + 8 * w; };  // O is whole
  auto OE = [&](int w) { return bx + 48 + 8 * w; };  // O is read
  const uint32_t QF = bx + 64, QE = bx + 72;         // Q is there, is done with
  const uint32_t VR = bx + 80, VZ = bx + 88;         // the last values are there, and clean behind the keys
  const uint32_t DR = bx + 96;                       // also what the test's wait finds never done
  if (tid == 0) {
    for (int i = 0; i < Ly::NS; ++i) { mbar_init(FULL(i), 1); mbar_init(EMPTY(i), 1); }
    for (int i = 0; i < kItems; ++i) { mbar_init(WF(i), 1); mbar_init(WE(i), 19); }
    for (int w = 0; w < 2; ++w) { mbar_init(SF(w), 1); mbar_init(PF(w), 8); mbar_init(OD(w), 1); mbar_init(OE(w), 8); }
    mbar_init(QF, 1);
    mbar_init(QE, 1);
    mbar_init(VR, 1);
    mbar_init(VZ, 1);
    mbar_init(DR, 1);
    mbar_fence_init();
    sts_i(failed, 0);
  }
  if (blockIdx.x == 0) check_offsets(a);
  if (warp == 17) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2;
  // Waits for the it-th item; its place is given back, after its last use, by item_read.
  auto item = [&](int it, uint32_t &w) {
    w = sb + Ly::OFF_WORK + it % kItems * W_BYTES;
    return wait_bar<kItemLimit>(WF(it % kItems), (it / kItems) & 1, failed, a.dev_status);
  };
  auto item_read = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(WE(it % kItems));
  };

  // 640 threads x 96 registers at the start: 512 x 104 + 128 x 64
  if (wg < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // -------------------------------------------------------------- softmax
    const int w = wg >> 1, half = wg & 1, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t S_col = tmem + lanes + w * 128 + half * 64, O_col = S_col + 256 - half * (64 - D / 2);
    const uint32_t told = sb + Ly::OFF_X + tid * 4;  // the row's other thread's is told ^ 512
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      sts_i(failed, 1);
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    uint32_t phases = 0;  // bit 0: of the tile's next S, bit 1: of its next O
    if (lane == 0) mbar_arrive(OE(w));  // there is no O yet
    for (int it = 0;; ++it) {
      uint32_t work;
      if (ok) ok = item(it, work);
      if (vote_any(1 + w, !ok)) break;  // all 256 threads of a tile leave together, or none
      if (!lds_i(work + W_ON)) break;
      float m_ref = -INFINITY, l_sum = 0.f;
      for (int j = 0; j < lds_i(work + W_TILES + 4 * w); ++j) {
        // (an item before, which this tile has no rows of, may be under way)
        if (ok) ok = wait_bar<kItemLimit>(SF(w), phases & 1, failed, a.dev_status);
        phases ^= 1;
        tc_fence_after();
        uint32_t s[64];
        load64(S_col, s);
        wait64(s);
        const int k0 = j * kTile + half * 64;
        const int low = lds_i(work + W_LOW + 4 * w);
        if (k0 + 63 > low) {
          const int limit = a.causal ? min(low + r, lds_i(work + W_KEYS) - 1) : low;  // what this row sees last
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (k0 + i > limit) s[i] = __float_as_uint(-INFINITY);
        }
        float top = __uint_as_float(s[0]), next = __uint_as_float(s[1]);
#pragma unroll
        for (int i = 2; i < 62; i += 4) {
          top = gdnkv::max3(top, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          next = gdnkv::max3(next, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
        }
        top = gdnkv::max3(top, __uint_as_float(s[62]), __uint_as_float(s[63]));
        top = fmaxf(top, next);
        // (of -inf both, NaN: no.  A wait that gave up votes too.)
        if (vote_any(1 + w, (top - m_ref) * a.scale_log2e > kMost || !ok)) {
          sts_f(told, top);
          if (vote_any(1 + w, !ok)) goto leave;
          top = fmaxf(top, lds_f(told ^ 512));
          float grow = 1.f;
          if ((top - m_ref) * a.scale_log2e > kMost) {
            const float was = __fmul_rn(m_ref, a.scale_log2e), now = __fmul_rn(top, a.scale_log2e);
            grow = ex2f(fmaxf(fabsf(was), fabsf(now)) > kFar ? (m_ref - top) * a.scale_log2e : was - now);
            m_ref = top;
            l_sum *= grow;
          }
          if (j > 0 && __any_sync(0xffffffffu, grow != 1.f)) {
#pragma unroll 1
            for (int i = 0; i < D / 2; i += 8) {  // few at a time: the logits hold 64 registers
              uint32_t o[8];
              gdnkv::tmem_ld8(O_col + i, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * grow);
              gdnkv::tmem_st8(O_col + i, o);
            }
          }
        }
        const float c = factor(a.scale_log2e, m_ref), ref = m_ref == -INFINITY ? 0.f : __fmul_rn(m_ref, c);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float2 t = gdnkv::fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c, -ref);
          t.x = ex2f(t.x);
          t.y = ex2f(t.y);
          sum = gdnkv::add2(sum, t);
          s[i] = pack_bf16(t.x, t.y);
        }
        l_sum += sum.x + sum.y;
        tmem_st32(S_col, s);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PF(w));
      }
      // ------------------------------------------------------------- output
      const int count = lds_i(work + W_COUNT + 4 * w);
      const bool tiles = lds_i(work + W_TILES + 4 * w) > 0;
      const int64_t at = (int64_t)(lds_i(work + W_Q) + lds_i(work + W_ROW0) + w * kTile + r) * a.HQ + lds_i(work + W_HEAD);
      item_read(it);
      if (count == 0) continue;
      if (tiles) {
        ok = wait_bar(OD(w), phases >> 1 & 1, failed, a.dev_status);
        phases ^= 2;
      }
      sts_f(told, l_sum);  // (after O is whole: the row's other thread has read the maximum here before its P)
      if (vote_any(1 + w, !ok)) break;
      tc_fence_after();
      const float l = l_sum + lds_f(told ^ 512), inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t *dst = a.o + at * D + half * (D / 2);
      store_half<D>(O_col, dst, inv, (tiles && l != 0.f ? 2 : 0) + (r < count ? 1 : 0));
      if (tiles) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(OE(w));
      }
      if (r < count && half == 0) {
        const float ref = __fmul_rn(m_ref, a.scale_log2e), more = log2f(l);
        a.lse[at] = l == 0.f ? -INFINITY : fabsf(ref) > kFar ? fmaf(m_ref, a.scale, more * kLn2) : (ref + more) * kLn2;
      }
    }
  leave:;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 16) {
      // ------------------------------------------------------------- copies
      if (elect_one()) {
        int issued = 0, asked = 0;  // stages filled, Q
        bool ok = true;
        for (int it = 0; ok; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + W_ON)) break;
          const int tiles0 = lds_i(work + W_TILES), tiles1 = lds_i(work + W_TILES + 4), tiles = max(tiles0, tiles1);
          const int row = lds_i(work + W_Q) + lds_i(work + W_ROW0), key = lds_i(work + W_K), head = lds_i(work + W_HEAD);
          mbar_arrive(WE(it % kItems));
          if (tiles == 0) continue;
          ok = asked == 0 || wait_bar(QE, (asked - 1) & 1, failed, a.dev_status);
          if (!ok) break;
          mbar_arrive_expect_tx(QF, (tiles0 > 0 && tiles1 > 0 ? 2 : 1) * Ly::TB);
          if (tiles0 > 0) load_tile<D>(sb + Ly::OFF_Q, &mq, QF, head, row);
          if (tiles1 > 0) load_tile<D>(sb + Ly::OFF_Q + Ly::TB, &mq, QF, head, row + kTile);
          ++asked;
          for (int i = 0; i < 2 * tiles; ++i, ++issued) {
            const int st = issued % Ly::NS;
            if (issued >= Ly::NS) ok = wait_bar(EMPTY(st), (issued / Ly::NS - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(FULL(st), Ly::TB);
            load_tile<D>(sb + Ly::OFF_KV + st * Ly::TB, (i & 1) ? &mv : &mk, FULL(st), head / a.G, key + (i >> 1) * kTile);
          }
        }
        if (lds_i(failed)) {  // copies in flight
          ok = asked == 0 || mbar_wait_bounded(QF, (asked - 1) & 1, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NS && i < issued; ++i)
            ok &= mbar_wait_bounded(FULL(i), ((issued - 1 - i) / Ly::NS) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 19) {
      // -------------------------------------------------------------- items
      const int R = tiles_an_item * kTile;
      Walk walk;
      const int64_t most = most_tokens(a.HK, D);
      walk_begin(a, walk, R, false, most);
      for (int it = 0;; ++it) {
        Found f;
        const bool on = walk_to(a, walk, R, false, false, most, turn_item(it), f, [&](int) { return a.HQ; });
        if (it >= kItems && !__all_sync(0xffffffffu, wait_bar<kItemLimit>(WE(it % kItems), (it / kItems - 1) & 1, failed, a.dev_status))) break;
        if (lane == 0) {
          const uint32_t work = sb + Ly::OFF_WORK + it % kItems * W_BYTES;
          sts_i(work + W_ON, on);
          if (on) {
            const int row0 = f.tile * R, past = f.keys.count - f.rows.count;
            sts_i(work + W_Q, f.rows.first);
            sts_i(work + W_K, f.keys.first);
            sts_i(work + W_KEYS, f.keys.count);
            sts_i(work + W_ROW0, row0);
            sts_i(work + W_HEAD, f.in);
            for (int w = 0; w < 2; ++w) {
              const int count = w < tiles_an_item ? max(0, min(kTile, f.rows.count - row0 - w * kTile)) : 0;
              const int seen = a.causal ? min(f.keys.count, past + row0 + w * kTile + count) : f.keys.count;
              sts_i(work + W_LOW + 4 * w, a.causal ? min(f.keys.count - 1, past + row0 + w * kTile) : f.keys.count - 1);
              sts_i(work + W_COUNT + 4 * w, count);
              sts_i(work + W_TILES + 4 * w, count > 0 ? tiles_in(max(0, seen), kTile) : 0);
            }
          }
          mbar_arrive(WF(it % kItems));
        }
        __syncwarp();
        if (!on) break;
      }
    } else if (warp == 17) {
      // ----------------------------------------------------------- products
      // (by one thread throughout, and one that elect.sync names: a warp that waits together
      // and elects one for each product took 1582 us for 16384 tokens, lane 0 by comparison
      // 1866)
      if (elect_one()) {
        uint32_t pair = 0, phases = 0;  // (K, V) pairs of stages before; a bit for each barrier's next phase
        auto wait = [&](uint32_t b, uint32_t phase) { return wait_bar(b, phase & 1, failed, a.dev_status); };
        auto in_turn = [&](uint32_t b, int bit) {  // the next phase of a barrier that is waited for in each turn
          const bool there = wait(b, phases >> bit);
          phases ^= 1u << bit;
          return there;
        };
        constexpr int NP = Ly::NS / 2;
        for (int it = 0;; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + W_ON)) break;
          const int tiles0 = lds_i(work + W_TILES), tiles1 = lds_i(work + W_TILES + 4), tiles = max(tiles0, tiles1);
          const bool clear = tiles * kTile > lds_i(work + W_KEYS);
          mbar_arrive(WE(it % kItems));
          if (tiles == 0) continue;
          // S of row tile x with key tile j; first, last: of the row tiles that j is for
          auto logits = [&](auto x, int j, bool first, bool last) {
            const uint32_t st = 2 * ((pair + j) % NP);
            if (first && !wait(FULL(st), (pair + j) / NP)) return false;
            tc_fence_after();
            mma_rows<D>(tmem + x * 128, sb + Ly::OFF_Q + x * Ly::TB, sb + Ly::OFF_KV + st * Ly::TB);
            umma_commit(SF(x));
            if (last) {
              umma_commit(EMPTY(st));
              if (j == tiles - 1) umma_commit(QE);
            }
            return true;
          };
          // P V of row tile x with key tile j, and the S that may follow it
          auto values = [&](auto x, int j, int mine, int other) {
            const bool first = x == 0 || j >= other, last = x == 1 || j >= other;
            const uint32_t st = 2 * ((pair + j) % NP) + 1;
            if (first) {
              if (!wait(FULL(st), (pair + j) / NP)) return false;
              if (clear && j == tiles - 1) {
                mbar_arrive(VR);
                if (!in_turn(VZ, 0)) return false;
              }
            }
            if (!in_turn(PF(x), 1 + x)) return false;
            if (j == 0 && !in_turn(OE(x), 3 + x)) return false;
            tc_fence_after();
            mma_cols<D>(tmem + 256 + x * 128, tmem + x * 128, sb + Ly::OFF_KV + st * Ly::TB, j > 0);
            if (last) umma_commit(EMPTY(st));
            if (j + 1 == mine) {
              umma_commit(OD(x));
              return true;
            }
            return logits(x, j + 1, x == 0 || j + 1 >= other, x == 1 || j + 1 >= other);
          };
          constexpr std::integral_constant<int, 0> X0{};
          constexpr std::integral_constant<int, 1> X1{};
          bool ok = in_turn(QF, 5);
          if (tiles0 > 0) ok = ok && logits(X0, 0, true, tiles1 == 0);
          if (tiles1 > 0) ok = ok && logits(X1, 0, tiles0 == 0, true);
          for (int j = 0; ok && j < tiles; ++j) {
            if (j < tiles0) ok = values(X0, j, tiles0, tiles1);
            if (ok && j < tiles1) ok = values(X1, j, tiles1, tiles0);
          }
          if (!ok) break;
          pair += tiles;
        }
        if (lds_i(failed)) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 18) {
      // ------------------------------------- values past the sequence's keys
      // P is 0 there, but 0 times what stands there need not be
      int stages = 0, turn = 0;
      for (int it = 0;; ++it) {
        uint32_t work;
        if (!__all_sync(0xffffffffu, item(it, work)) || !lds_i(work + W_ON)) break;
        const int tiles = max(lds_i(work + W_TILES), lds_i(work + W_TILES + 4)), keys = lds_i(work + W_KEYS);
        item_read(it);
        stages += 2 * tiles;
        if (tiles * kTile <= keys) continue;
        bool there = true;  // (no limit of its own: the products' warp gets there, or gives up and says so)
        while (there && !mbar_try_wait(VR, turn & 1)) there = !lds_i(failed);
        if (!__all_sync(0xffffffffu, there)) break;
        ++turn;
        zero_rows<D>(sb + Ly::OFF_KV + (stages - 1) % Ly::NS * Ly::TB, keys % kTile);
        if (lane == 0) mbar_arrive(VZ);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t launch(const Args &a, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const bool keys = a.Tk > 0;  // without keys no tile of them is loaded
  if (!rows_map(&mq, a.q, D, a.HQ, a.Tq, a.ldq) || !rows_map(&mk, keys ? a.k : a.q, D, keys ? a.HK : a.HQ, keys ? a.Tk : a.Tq, keys ? a.ldk : a.ldq) ||
      !rows_map(&mv, keys ? a.v : a.q, D, keys ? a.HK : a.HQ, keys ? a.Tk : a.Tq, keys ? a.ldv : a.ldq))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  static std::atomic<bool> known{false};
  cudaError_t e = gdn_host::allow_smem(attn_fwd_kernel<D>, Lay<D>::BYTES, done);
  if (e == cudaSuccess) e = check_registers(attn_fwd_kernel<D>, 96, known);
  if (e != cudaSuccess) return e;
  const int sms = gdn_host::sm_count();
  const int each = most_tiles(a.Tq, a.N, 2 * kTile) * a.HQ >= sms ? 2 : 1;
  const int64_t blocks = std::min<int64_t>(most_tiles(a.Tq, a.N, each * kTile) * a.HQ, sms);
  return gdn_host::launch_dependent(attn_fwd_kernel<D>, dim3((unsigned)blocks), kThreads, Lay<D>::BYTES, s, a, each, mq, mk, mv);
}

}  // namespace

namespace gdn_host {
cudaError_t launch_attn_fwd(const TrainAttnArgs &c, cudaStream_t s) {
  gdnat::Args a{};
  static_cast<TrainAttnArgs &>(a) = c;
  a.G = c.HQ / c.HK;
  a.scale_log2e = c.scale * gdnc::kLog2e;
  return c.D == 128 ? launch<128>(a, s) : launch<64>(a, s);
}
}  // namespace gdn_host
