// gdn_attn_bwd.cu -- attention of packed sequences, gradients, on tcgen05.
//
//   P = 2^(c S - lse log2 e),  S = q K^T,  c = scale log2 e      (formed again)
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  delta = sum dO o
//   dQ = scale dS K,  dK = scale dS^T Q
//
// Five products, 10 D operations a (row, key, head); bound: the tensor cores, which
// execute seven.  24 packed sequences of 200 to 2000 rows, 32 heads: 963 to 982 us (a pass
// over the rows 71, dK and dV 510, dQ 400).  8192 rows of one sequence: 1210 to 1240 us,
// 1.1 PFLOP/s by the five and 1.55 by the seven, at the power limit.  D = 64: 730 and 915 us,
// with the tensor pipe busy for 35 % and 34 to 38 % of the issue slots taken: a step waits
// in turn for products and for the arithmetic that reads and writes their columns.
//
// Two kernels, one with the keys fixed (dK, dV) and one with the rows fixed (dQ), each
// of which forms S and dP itself: seven products instead of five.  In exchange every
// sum stays in one block's tensor memory from beginning to end: no sum of dQ passes
// through memory tile by tile in fp32, nothing is added by atomics, and two calls agree
// bit for bit.  A small kernel before them writes what both need of a row, -lse log2 e and
// delta, tile by tile (kTile numbers each, with rows past the sequence at -inf and 0:
// their P is 0).
//
// dK, dV: an item is 128 keys of one kv head, which walks over (head of the group, 128
// rows).  S^T = K Q^T and dP^T = V dO^T have the keys as rows, so P^T and dS^T, written
// to tensor memory over what they came from, are the A operands of dV and dK as they
// stand and never pass through shared memory.  Tensor memory: S^T, dP^T, dV, dK, all
// 512 columns at D = 128.  The products' order is dV(i), S(i+1), dK(i), dP(i+1): P(i+1)
// is formed while dK(i) and dP(i+1) run, dS(i) while dV(i) and S(i+1) do.
// Where few (key tile, kv head) pairs exist a pair's walk is cut into pieces, whose sums
// a last kernel adds in order.
//
// dQ: an item is 128 rows of one head, which walks over the keys.  Tensor memory: S, dP,
// dQ, dO (an operand from there costs shared memory nothing) and dS in a place of its own,
// so that the next keys' S and dP are formed while dS is, and the products wait for the
// arithmetic only once a step: with dS over its dP, where they wait in turn, 2120 cycles a
// step against 1541 of products alone.
//
// P and dS enter the products in bf16 (8 significant bits), sums are fp32.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "gdn_attn.cuh"

namespace {

using namespace gdnat;

constexpr int kThreads = 384;  // warps 0-7 P and dS, 8 copies, 9 products, 10 clears rows past the end, 11 items

constexpr int kBlocks = 152;  // SMs
constexpr int kNear = 4;      // steps before its end from which a walk is about to end
constexpr int kItems = 1;  // items between the warp that finds them and the others: it takes the next when all have one

struct BwdArgs : Args {
  float *stats;  // [HQ][q places][2][kTile]: -lse log2 e, delta
  float *part;   // [piece][k places][HK][2][kTile][D]: sums of dK and dV
  struct Shared {
    int cut;               // steps that a piece of a walk has at least
    int next_kv, next_q;   // items that the blocks of the two kernels have taken
  } *shared;
  int64_t q_places, k_places;
  int pieces;  // most pieces of a walk
};

// The row tiles that see some key of the tile from key k0 on are [t0, tn).
__device__ __forceinline__ int first_seen_by(const Args &a, int tn, int rows, int keys, int k0) {
  return min(tn, a.causal ? max(0, k0 - (keys - rows)) / kTile : 0);
}
__device__ __forceinline__ int pieces_for(const BwdArgs &a, int steps, int cut) { return max(1, min(a.pieces, (steps + cut - 1) / cut)); }
// The next item that no block has taken, for a warp: blocks take them as they come free, as
// walks have from one to many thousand steps.  (Which block has an item changes no result.)
__device__ __forceinline__ int64_t take_item(int *next) {
  int i = 0;
  if ((threadIdx.x & 31) == 0) i = atomicAdd(next, 1);
  return __shfl_sync(0xffffffffu, i, 0);
}

// ------------------------------------------------------------ of each row
template <int D> __global__ void __launch_bounds__(256) attn_stats_kernel(const BwdArgs a) {
  constexpr int L = D / 8, PER = 256 / L;  // lanes a row, rows at once
  const int64_t place = blockIdx.x / a.HQ;
  const int head = blockIdx.x % a.HQ, l = threadIdx.x % L;
  grid_wait();
  if (blockIdx.x == 0) {
    check_offsets(a);
    // The walks of dK, dV have some steps in all (to a tile for the diagonal): a piece has a
    // quarter of a block's share at least, and 4.
    __shared__ unsigned long long total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    unsigned long long mine = 0;
    for (int n = threadIdx.x; n < a.N; n += blockDim.x) {
      Run rows, keys;
      if (!run_of(rows_of(a), n, rows) || !run_of(keys_of(a), n, keys)) continue;
      const int64_t tn = tiles_in(rows.count, kTile), kn = tiles_in(keys.count, kTile);
      // under the mask, tiles from `free` on lose one row tile each, two, ..
      const int64_t free = max(0, keys.count - rows.count) / kTile, lost = a.causal ? max((int64_t)0, kn - free) : 0;
      mine += max((int64_t)1, tn * kn - lost * (lost - 1) / 2);
    }
    atomicAdd(&total, mine);
    __syncthreads();
    if (threadIdx.x == 0) {
      a.shared->cut = (int)min((unsigned long long)INT_MAX, max(4ull, total * a.HQ / (4 * kBlocks)));
      a.shared->next_kv = 0;
      a.shared->next_q = 0;
    }
  }
  Tile t;
  if (!tile_of(a, place, kTile, false, t)) return;
  float *out = a.stats + ((int64_t)head * a.q_places + place) * 2 * kTile;
#pragma unroll 4
  for (int r = threadIdx.x / L; r < kTile; r += PER) {
    const bool on = t.row0 + r < t.rows.count;
    const int64_t at = (int64_t)(t.rows.first + t.row0 + r) * a.HQ + head;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    float lse = -INFINITY;
    if (on) {
      x = __ldcs(reinterpret_cast<const uint4 *>(a.dout + at * D) + l);
      y = __ldcs(reinterpret_cast<const uint4 *>(a.o + at * D) + l);
      lse = a.lse[at];
    }
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fmaf(bf16lo_f(xs[i]), bf16lo_f(ys[i]), fmaf(bf16hi_f(xs[i]), bf16hi_f(ys[i]), sum));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (l == 0) {
      // a row that sees nothing (lse -inf) has P = 0 as well
      out[r] = lse == -INFINITY ? -INFINITY : -lse * gdnc::kLog2e;
      out[kTile + r] = sum;
    }
  }
}

// ----------------------------------------------------------------- dK, dV
// An item, 32-bit words in shared memory: first row of q, rows of the sequence, the place of
// its first row tile; first key, keys; the item's first key, keys - rows; the first row tile
// that sees them, how many there are; the piece's first step and its steps (step s is head
// s / nt of the group, row tile t0 + s % nt); kv head; where the sums go (-1: they are whole),
// whether it is an item (0: there are no more).
enum KvWord { K_Q = 0, K_ROWS = 4, K_QPLACE = 8, K_K = 12, K_KEYS = 16, K_K0 = 20, K_PAST = 24, K_T0 = 28, K_NT = 32, K_S0 = 36, K_STEPS = 40,
              K_HK = 44, K_PART = 48, K_ON = 52, K_BYTES = 64 };
template <int D> struct KvLay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NQ = 3, NO = 2, NT = 2;  // stages of Q, dO, the rows' numbers
  static constexpr int OFF_K = 0, OFF_V = TB, OFF_Q = 2 * TB, OFF_O = OFF_Q + NQ * TB;
  static constexpr int OFF_T = OFF_O + NO * TB;
  static constexpr int OFF_WORK = OFF_T + NT * 2 * kTile * 4;
  static constexpr int OFF_BAR = OFF_WORK + kItems * K_BYTES;
  static constexpr int BARS = 2 * (NQ + NO + NT + kItems) + 13;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkdv_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  using Ly = KvLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_wait();
  grid_release();  // the kernel of dQ, which needs nothing of this one, takes the SMs that come free
  const uint32_t failed = sb + Ly::OFF_MISC;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto QF = [&](int i) { return bar + 8 * i; };
  auto QE = [&](int i) { return bar + 8 * (Ly::NQ + i); };
  const uint32_t bo = bar + 16 * Ly::NQ, bt = bo + 16 * Ly::NO, bw = bt + 16 * Ly::NT, bx = bw + 16 * kItems;
  auto OF = [&](int i) { return bo + 8 * i; };
  auto OE = [&](int i) { return bo + 8 * (Ly::NO + i); };
  auto TF = [&](int i) { return bt + 8 * i; };
  auto TE = [&](int i) { return bt + 8 * (Ly::NT + i); };
  auto WF = [&](int i) { return bw + 8 * i; };  // an item is there, all have read it
  auto WE = [&](int i) { return bw + 8 * (kItems + i); };
  const uint32_t KF = bx, KE = bx + 8, SF = bx + 16, DF = bx + 24, PF = bx + 32, GF = bx + 40;  // K and V are there, done with; S, dP, P, dS are there
  const uint32_t DONE = bx + 48, AE = bx + 56, VR = bx + 64, VZ = bx + 72;  // dK and dV are whole, are read; a tile to clear is there, is clean
  const uint32_t DR = bx + 80, PH = bx + 88, NEAR = bx + 96;  // PH: half of P; NEAR: the item is about to end
  if (tid == 0) {
    for (int i = 0; i < Ly::NQ; ++i) { mbar_init(QF(i), 1); mbar_init(QE(i), 1); }
    for (int i = 0; i < Ly::NO; ++i) { mbar_init(OF(i), 1); mbar_init(OE(i), 1); }
    for (int i = 0; i < Ly::NT; ++i) { mbar_init(TF(i), 1); mbar_init(TE(i), 8); }
    for (int i = 0; i < kItems; ++i) { mbar_init(WF(i), 1); mbar_init(WE(i), 11); }
    for (uint32_t b : {KF, KE, SF, DF, DONE, VR, VZ, DR, NEAR}) mbar_init(b, 1);
    for (uint32_t b : {PF, PH, GF, AE}) mbar_init(b, 8);
    mbar_fence_init();
    sts_i(failed, 0);
  }
  if (warp == 9) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2;
  constexpr uint32_t kS = 0, kP = 128, kV = 256, kK = 256 + D;  // columns of S^T, dP^T, dV, dK
  auto item = [&](int it, uint32_t &w) {
    w = sb + Ly::OFF_WORK + it % kItems * K_BYTES;
    return wait_bar<kItemLimit>(WF(it % kItems), (it / kItems) & 1, failed, a.dev_status);
  };
  auto item_read = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(WE(it % kItems));
  };

  if (wg < 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");  // 3 x 168 = 2 x 208 + 88
    // -------------------------------------------------------------- P and dS
    const int half = wg * 64, r = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    if (lane == 0) mbar_arrive(AE);  // there are no sums yet
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      sts_i(failed, 1);
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    uint32_t n = 0, whole = 0;  // steps, items with some
    for (int it = 0;; ++it) {
      uint32_t work;
      ok = ok && item(it, work);
      if (!__all_sync(0xffffffffu, ok) || !lds_i(work + K_ON)) break;
      const int steps = lds_i(work + K_STEPS), k0 = lds_i(work + K_K0), past = lds_i(work + K_PAST), t0 = lds_i(work + K_T0), nt = lds_i(work + K_NT);
      const int key = k0 + r, hk = lds_i(work + K_HK), part_at = lds_i(work + K_PART);
      const bool on = key < lds_i(work + K_KEYS);
      const int64_t at = ((int64_t)(lds_i(work + K_K) + key) * a.HK + hk) * D + wg * (D / 2);
      int t = steps > 0 ? lds_i(work + K_S0) % nt : 0;
      item_read(it);
      for (int i = 0; i < steps; ++i, ++n) {
        const uint32_t numbers = sb + Ly::OFF_T + (n % Ly::NT) * (2 * kTile * 4) + half * 4;
        const int q0 = (t0 + t) * kTile + half;  // first of this thread's rows
        t = t + 1 == nt ? 0 : t + 1;
        const bool masked = a.causal && q0 + past < k0 + kTile - 1;
        const int from = key - past - q0;  // its first column that sees the key
        ok = wait_bar(TF(n % Ly::NT), (n / Ly::NT) & 1, failed, a.dev_status);
        float4 lse[16];  // read before the wait: the products read shared memory at its full rate
#pragma unroll
        for (int c = 0; c < 16; ++c) lse[c] = gdnkv::lds_f4(numbers + c * 16);
        ok = ok && wait_bar(SF, n & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        uint32_t p[64], b[64];
        load64(lanes + kS + half, p);
        wait64(p);
        // (one loop each for tiles with and without a mask, so that exponentials, sums and
        // roundings run side by side)
        auto weights = [&](auto mask, int part) {
#pragma unroll
          for (int c = part * 32; c < part * 32 + 32; c += 2) {
            const float4 m = lse[c / 4];
            float2 x = fma2v(pair(p, c / 2), a.scale_log2e, (c & 2) ? make_float2(m.z, m.w) : make_float2(m.x, m.y));
            x = make_float2(ex2f(x.x), ex2f(x.y));
            if (mask && c < from) x.x = 0.f;
            if (mask && c + 1 < from) x.y = 0.f;
            p[c] = __float_as_uint(x.x);
            p[c + 1] = __float_as_uint(x.y);
            b[c / 2] = pack_bf16(x.x, x.y);
          }
        };
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // the products with the first half of them begin meanwhile
          if (masked) weights(std::true_type{}, part);
          else weights(std::false_type{}, part);
          tmem_st16(lanes + kS + half + part * 16, b + part * 16);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(part ? PF : PH);
        }
        ok = wait_bar(DF, n & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        load64(lanes + kP + half, b);
        wait64(b);
        auto slopes = [&](auto mask) {
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 m = gdnkv::lds_f4(numbers + kTile * 4 + c * 4);
            float2 x = mul2(pair(p, c / 2), gdnkv::add2(pair(b, c / 2), make_float2(-m.x, -m.y)));
            float2 y = mul2(pair(p, c / 2 + 1), gdnkv::add2(pair(b, c / 2 + 1), make_float2(-m.z, -m.w)));
            if (mask) {  // a weight of 0 has no gradient, whatever a masked row's dP is
              if (c < from) x.x = 0.f;
              if (c + 1 < from) x.y = 0.f;
              if (c + 2 < from) y.x = 0.f;
              if (c + 3 < from) y.y = 0.f;
            }
            b[c / 2] = pack_bf16(x.x, x.y);
            b[c / 2 + 1] = pack_bf16(y.x, y.y);
          }
        };
        if (masked) slopes(std::true_type{});
        else slopes(std::false_type{});
        tmem_st32(lanes + kP + half, b);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(GF);
          mbar_arrive(TE(n % Ly::NT));
        }
      }
      // ------------------------------------------------------------- output
      if (ok && steps > 0) ok = wait_bar(DONE, whole++ & 1, failed, a.dev_status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float *part = a.part + ((int64_t)part_at * 2 * kTile + r) * D + wg * (D / 2);
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {  // dK, then dV: half a row each
        const bool second = i >= D / 2;
        const int c = second ? i - D / 2 : i;
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld32_issue(lanes + (second ? kV : kK) + wg * (D / 2) + c, o);
          tmem_ld_wait(o);
          if (i + 32 == D) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(AE);
          }
        }
        const float f = second ? 1.f : a.scale;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = steps > 0 ? __float_as_uint(__uint_as_float(o[e]) * f) : 0u;
        if (on && part_at < 0) {
          uint16_t *dst = (second ? a.dv : a.dk) + at + c;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4 *>(dst + e) = make_uint4(
                pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
        } else if (on) {
          float *dst = part + (second ? kTile * D : 0) + c;
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4 *>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ------------------------------------------------------------- copies
      if (elect_one()) {
        uint32_t q_in = 0, o_in = 0, t_in = 0, kv_in = 0;  // what has been asked for
        const int apart = rows_of(a).apart(kTile);
        bool ok = true;
        for (int it = 0; ok; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + K_ON)) break;
          const int steps = lds_i(work + K_STEPS), nt = lds_i(work + K_NT), t0 = lds_i(work + K_T0), s0 = lds_i(work + K_S0), hk = lds_i(work + K_HK);
          const int key = lds_i(work + K_K) + lds_i(work + K_K0), first = lds_i(work + K_Q), q_place = lds_i(work + K_QPLACE);
          mbar_arrive(WE(it % kItems));
          if (steps == 0) continue;
          if (kv_in > 0) ok = wait_bar(KE, (kv_in - 1) & 1, failed, a.dev_status);
          if (!ok) break;
          mbar_arrive_expect_tx(KF, 2 * Ly::TB);
          load_tile<D>(sb + Ly::OFF_K, &mk, KF, hk, key);
          load_tile<D>(sb + Ly::OFF_V, &mv, KF, hk, key);
          ++kv_in;
          int head = hk * a.G + s0 / nt, t = s0 % nt;
          for (int i = 0; i < steps; ++i) {
            const int row = first + (t0 + t) * kTile;
            const uint32_t iq = q_in % Ly::NQ, io = o_in % Ly::NO, is = t_in % Ly::NT;
            if (q_in >= Ly::NQ) ok = wait_bar(QE(iq), (q_in / Ly::NQ - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(QF(iq), Ly::TB);
            load_tile<D>(sb + Ly::OFF_Q + iq * Ly::TB, &mq, QF(iq), head, row);
            ++q_in;
            if (t_in >= Ly::NT) ok = wait_bar(TE(is), (t_in / Ly::NT - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(TF(is), 2 * kTile * 4);
            bulk_load(sb + Ly::OFF_T + is * (2 * kTile * 4), a.stats + ((int64_t)head * a.q_places + q_place + (t0 + t) * apart) * 2 * kTile, 2 * kTile * 4,
                      TF(is));
            ++t_in;
            if (o_in >= Ly::NO) ok = wait_bar(OE(io), (o_in / Ly::NO - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(OF(io), Ly::TB);
            load_tile<D>(sb + Ly::OFF_O + io * Ly::TB, &mo, OF(io), head, row);
            ++o_in;
            if (++t == nt) {
              t = 0;
              ++head;
            }
          }
        }
        if (lds_i(failed)) {  // copies in flight
          ok = kv_in == 0 || mbar_wait_bounded(KF, (kv_in - 1) & 1, gdnc::kWaitLimit);
          for (uint32_t i = 0; i < Ly::NQ && i < q_in; ++i) ok &= mbar_wait_bounded(QF(i), ((q_in - 1 - i) / Ly::NQ) & 1, gdnc::kWaitLimit);
          for (uint32_t i = 0; i < Ly::NT && i < t_in; ++i) ok &= mbar_wait_bounded(TF(i), ((t_in - 1 - i) / Ly::NT) & 1, gdnc::kWaitLimit);
          for (uint32_t i = 0; i < Ly::NO && i < o_in; ++i) ok &= mbar_wait_bounded(OF(i), ((o_in - 1 - i) / Ly::NO) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      if (elect_one()) {
        uint32_t n = 0, cleared = 0, items = 0;  // steps, tiles cleared, items with steps
        for (int it = 0;; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + K_ON)) break;
          const int steps = lds_i(work + K_STEPS), nt = lds_i(work + K_NT), tail = lds_i(work + K_ROWS) % kTile;
          int t = steps > 0 ? lds_i(work + K_S0) % nt : 0;
          mbar_arrive(WE(it % kItems));
          if (steps <= kNear) mbar_arrive(NEAR);
          if (steps == 0) continue;
          auto wait = [&](uint32_t b, uint32_t phase) { return wait_bar(b, phase & 1, failed, a.dev_status); };
          auto q_tile = [&](uint32_t m) { return sb + Ly::OFF_Q + m % Ly::NQ * Ly::TB; };
          auto o_tile = [&](uint32_t m) { return sb + Ly::OFF_O + m % Ly::NO * Ly::TB; };
          auto logits = [&](uint32_t m) {
            if (!wait(QF(m % Ly::NQ), m / Ly::NQ)) return false;
            if (tail != 0 && t + 1 == nt) {
              if (!wait(OF(m % Ly::NO), m / Ly::NO)) return false;
              mbar_arrive(VR);
              if (!wait(VZ, cleared++)) return false;
            }
            t = t + 1 == nt ? 0 : t + 1;
            tc_fence_after();
            mma_rows<D>(tmem + kS, sb + Ly::OFF_K, q_tile(m));
            umma_commit(SF);
            return true;
          };
          auto slopes = [&](uint32_t m, bool last) {
            if (!wait(OF(m % Ly::NO), m / Ly::NO)) return false;
            tc_fence_after();
            mma_rows<D>(tmem + kP, sb + Ly::OFF_V, o_tile(m));
            umma_commit(DF);
            if (last) umma_commit(KE);  // the last use of K and V
            return true;
          };
          bool ok = wait(KF, items) && logits(n) && slopes(n, steps == 1);
          for (int i = 0; ok && i < steps; ++i, ++n) {
            const bool more = i + 1 < steps;
            if (i > 0 && i == steps - kNear) mbar_arrive(NEAR);
            ok = wait(PH, n) && (i > 0 || wait(AE, items));
            if (!ok) break;
            tc_fence_after();
            mma_cols_half<D>(tmem + kV, tmem + kS, o_tile(n), 0, i > 0);
            ok = wait(PF, n);
            if (!ok) break;
            tc_fence_after();
            mma_cols_half<D>(tmem + kV, tmem + kS, o_tile(n), 1, true);
            umma_commit(OE(n % Ly::NO));
            if (more) ok = logits(n + 1);
            ok = ok && wait(GF, n);
            if (!ok) break;
            tc_fence_after();
            mma_cols<D>(tmem + kK, tmem + kP, q_tile(n), i > 0);
            umma_commit(QE(n % Ly::NQ));
            if (more) ok = slopes(n + 1, i + 2 == steps);
            else umma_commit(DONE);
          }
          if (!ok) break;
          ++items;
        }
        if (lds_i(failed)) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 10) {
      // Rows past the sequence in its last row tile: their P and dS are 0, but 0 times what
      // stands there need not be.
      uint32_t n = 0, turn = 0;
      bool there = true;
      for (int it = 0; there; ++it) {
        uint32_t work;
        if (!__all_sync(0xffffffffu, item(it, work)) || !lds_i(work + K_ON)) break;
        const int steps = lds_i(work + K_STEPS), nt = lds_i(work + K_NT), s0 = lds_i(work + K_S0), tail = lds_i(work + K_ROWS) % kTile;
        item_read(it);
        for (int i = 0; tail != 0 && i < steps; ++i) {
          if ((s0 + i) % nt != nt - 1) continue;
          // (no limit of its own: the products' warp gets there, or gives up and says so)
          while (there && !mbar_try_wait(VR, turn & 1)) there = !lds_i(failed);
          there = __all_sync(0xffffffffu, there);
          if (!there) break;
          ++turn;
          zero_rows<D>(sb + Ly::OFF_Q + (n + i) % Ly::NQ * Ly::TB, tail);
          zero_rows<D>(sb + Ly::OFF_O + (n + i) % Ly::NO * Ly::TB, tail);
          if (lane == 0) mbar_arrive(VZ);
        }
        n += steps;
      }
    } else {
      // -------------------------------------------------------------- items
      const int cut = a.shared->cut;
      const int64_t most = most_tokens(a.HQ, D);
      Walk w;
      walk_begin(a, w, kTile, true, most);
      for (int it = 0;; ++it) {
        Found f;
        // taken when the one before is about to end, which leaves time for its copies
        if (it > 0 && !__all_sync(0xffffffffu, wait_bar<kItemLimit>(NEAR, (it - 1) & 1, failed, a.dev_status))) break;
        const bool on = walk_to(a, w, kTile, true, true, most, take_item(&a.shared->next_kv), f, [&](int tile) {
          const int tn = tiles_in(w.rows.count, kTile);
          return a.HK * pieces_for(a, a.G * (tn - first_seen_by(a, tn, w.rows.count, w.keys.count, tile * kTile)), cut);
        });
        int t0 = 0, nt = 0, pieces = 1;
        if (on) {
          const int tn = tiles_in(f.rows.count, kTile);
          t0 = first_seen_by(a, tn, f.rows.count, f.keys.count, f.tile * kTile);
          nt = tn - t0;
          pieces = f.of / a.HK;
        }
        const int64_t all = (int64_t)a.G * nt;
        const int piece = f.in % pieces;
        if (it >= kItems && !__all_sync(0xffffffffu, wait_bar<kItemLimit>(WE(it % kItems), (it / kItems - 1) & 1, failed, a.dev_status))) break;
        if (lane == 0) {
          const uint32_t work = sb + Ly::OFF_WORK + it % kItems * K_BYTES;
          sts_i(work + K_ON, on);
          if (on) {
            const int s0 = (int)(all * piece / pieces), hk = f.in / pieces;
            const Side rows = rows_of(a), keys = keys_of(a);
            const int64_t place = keys.place(f.n, f.keys.first, kTile) + f.tile * keys.apart(kTile);
            sts_i(work + K_Q, f.rows.first);
            sts_i(work + K_ROWS, f.rows.count);
            sts_i(work + K_QPLACE, (int)rows.place(f.n, f.rows.first, kTile));
            sts_i(work + K_K, f.keys.first);
            sts_i(work + K_KEYS, f.keys.count);
            sts_i(work + K_K0, f.tile * kTile);
            sts_i(work + K_PAST, f.keys.count - f.rows.count);
            sts_i(work + K_T0, t0);
            sts_i(work + K_NT, nt);
            sts_i(work + K_S0, s0);
            sts_i(work + K_STEPS, (int)(all * (piece + 1) / pieces) - s0);
            sts_i(work + K_HK, hk);
            sts_i(work + K_PART, pieces == 1 ? -1 : (int)((piece * a.k_places + place) * a.HK + hk));
          }
          mbar_arrive(WF(it % kItems));
        }
        __syncwarp();
        if (!on) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Adds the pieces' sums of a (key tile, kv head) in order.
template <int D> __global__ void __launch_bounds__(256) attn_join_kernel(const BwdArgs a) {
  const int64_t place = blockIdx.x / a.HK;
  const int hk = blockIdx.x % a.HK;
  grid_wait();
  Tile t;
  if (!tile_of(a, place, kTile, true, t)) return;
  const int tn = tiles_in(t.rows.count, kTile);
  const int pieces = pieces_for(a, a.G * (tn - first_seen_by(a, tn, t.rows.count, t.keys.count, t.row0)), a.shared->cut);
  if (pieces == 1) return;
  const int rows = min(kTile, t.keys.count - t.row0);
  for (int i = blockIdx.y * 256 + threadIdx.x; i < 2 * rows * (D / 8); i += gridDim.y * 256) {
    const bool second = i >= rows * (D / 8);
    const int e = second ? i - rows * (D / 8) : i, r = e / (D / 8), c = e % (D / 8) * 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
      const float4 *src =
          reinterpret_cast<const float4 *>(a.part + ((((p * a.k_places + place) * a.HK + hk) * 2 + (second ? 1 : 0)) * kTile + r) * D + c);
      const float4 u = __ldcs(src), v = __ldcs(src + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    uint16_t *dst = (second ? a.dv : a.dk) + ((int64_t)(t.keys.first + t.row0 + r) * a.HK + hk) * D + c;
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
}

// --------------------------------------------------------------------- dQ
// An item, 32-bit words in shared memory: first row of q of the sequence, the item's first
// row in it, its rows; first key, keys, keys - rows; key tiles; the head; the place of the
// rows' numbers; whether it is one (0: there are no more).
enum QWord { Q_Q = 0, Q_ROW0 = 4, Q_COUNT = 8, Q_K = 12, Q_KEYS = 16, Q_PAST = 20, Q_TILES = 24, Q_HEAD = 28, Q_PLACE = 32, Q_ON = 36, Q_BYTES = 48 };
template <int D> struct QLay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NK = 3, NV = 2;
  static constexpr int OFF_Q = 0, OFF_O = TB, OFF_K = 2 * TB, OFF_V = OFF_K + NK * TB;
  static constexpr int OFF_WORK = OFF_V + NV * TB;
  static constexpr int OFF_BAR = OFF_WORK + kItems * Q_BYTES;
  static constexpr int BARS = 2 * (NK + NV + kItems) + 14;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};
// Half a row (D / 2 bf16) of a tile in shared memory to tensor memory.
template <int D> __device__ __forceinline__ void row_to_tmem(uint32_t taddr, uint32_t tile, int r, int half) {
#pragma unroll
  for (int i = 0; i < D / 16; i += 2) {
    const int c = half * (D / 16) + i;  // 16-byte chunks of the row
    const uint4 x = gdnkv::lds128(tile + (c / 8) * kTile * 128 + sw128(r, c % 8)), y = gdnkv::lds128(tile + (c / 8) * kTile * 128 + sw128(r, c % 8 + 1));
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    gdnkv::tmem_st8(taddr + c * 4, w);
  }
}
// D[128 x 128] = A B^T: A 128 x D bf16 in tensor memory, B 128 rows of D in shared memory.
template <int D> __device__ __forceinline__ void mma_rows_ta(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = umma_idesc_bf16(128, 128);
  const uint64_t db = umma_desc_sw128(b);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) umma_f16_ta(d, a + k * 8, db + (k / 4) * (kTile * 128 / 16) + (k % 4) * 2, id, k > 0);
}

// D[128 x D] (+)= A B: A 128 x 128 bf16 in tensor memory, in 64 columns one after another.
template <int D> __device__ __forceinline__ void mma_packed(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t id = umma_idesc_bf16(128, D, 0, 1);
  const uint64_t db = umma_desc_sw128_mn(b, kTile * 128);
#pragma unroll
  for (int k = 0; k < 8; ++k) umma_f16_ta(d, a + k * 8, db + k * 128, id, add || k > 0);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const BwdArgs a, int waits, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  using Ly = QLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // What the kernel of dK, dV has waited for is done when this one comes in; its end is waited
  // for at this one's, for the kernel after both.
  if (waits) grid_wait();
  const uint32_t failed = sb + Ly::OFF_MISC;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto KF = [&](int i) { return bar + 8 * i; };
  auto KE = [&](int i) { return bar + 8 * (Ly::NK + i); };
  const uint32_t bv = bar + 16 * Ly::NK, bw = bv + 16 * Ly::NV, bx = bw + 16 * kItems;
  auto VF = [&](int i) { return bv + 8 * i; };
  auto VE = [&](int i) { return bv + 8 * (Ly::NV + i); };
  auto WF = [&](int i) { return bw + 8 * i; };  // an item is there, all have read it
  auto WE = [&](int i) { return bw + 8 * (kItems + i); };
  const uint32_t QF = bx, QE = bx + 8, QT = bx + 16;                            // Q and dO are in shared memory, are read, are in tensor memory
  const uint32_t SF = bx + 24, SE = bx + 32, DF = bx + 40, GF = bx + 48;        // S is there, is read; dP, dS are there
  const uint32_t DONE = bx + 56, AE = bx + 64, VR = bx + 72, VZ = bx + 80;      // dQ is whole, is read; the last keys are there, are clean
  const uint32_t DR = bx + 88, PE = bx + 96, GE = bx + 104;  // PE: dP is read, GE: dS is done with
  if (tid == 0) {
    for (int i = 0; i < Ly::NK; ++i) { mbar_init(KF(i), 1); mbar_init(KE(i), 1); }
    for (int i = 0; i < Ly::NV; ++i) { mbar_init(VF(i), 1); mbar_init(VE(i), 1); }
    for (int i = 0; i < kItems; ++i) { mbar_init(WF(i), 1); mbar_init(WE(i), 11); }
    for (uint32_t b : {QF, SF, DF, DONE, VR, VZ, DR, GE}) mbar_init(b, 1);
    for (uint32_t b : {QT, SE, PE, GF, AE}) mbar_init(b, 8);
    mbar_init(QE, 1);
    mbar_fence_init();
    sts_i(failed, 0);
  }
  if (warp == 9) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2;
  constexpr uint32_t kS = 0, kP = 128, kA = 256, kO = 384, kG = 448;  // columns of S, dP, dQ, dO, dS
  auto item = [&](int it, uint32_t &w) {
    w = sb + Ly::OFF_WORK + it % kItems * Q_BYTES;
    return wait_bar<kItemLimit>(WF(it % kItems), (it / kItems) & 1, failed, a.dev_status);
  };
  auto item_read = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(WE(it % kItems));
  };

  if (wg < 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");  // 3 x 168 = 2 x 208 + 88
    // -------------------------------------------------------------------- dS
    const int half = wg * 64, r = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    if (lane == 0) mbar_arrive(AE);  // there is no dQ yet
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      sts_i(failed, 1);
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    uint32_t n = 0, with = 0, whole = 0;  // key tiles, items with some, of which dQ is out
    int64_t out = -1;                     // where the item before has its row; -1: it has none
    bool before = false, sums = false;    // there was an item before, with key tiles
    for (int it = 0;; ++it) {
      uint32_t work;
      ok = ok && item(it, work);
      if (!__all_sync(0xffffffffu, ok)) break;
      const bool on = lds_i(work + Q_ON);
      int tiles = 0, low = 0, limit = 0;
      int64_t at = -1;
      float n_lse = 0.f, n_delta = 0.f;
      if (on) {
        const int past = lds_i(work + Q_PAST), row0 = lds_i(work + Q_ROW0), keys = lds_i(work + Q_KEYS), head = lds_i(work + Q_HEAD);
        tiles = lds_i(work + Q_TILES);
        low = a.causal ? min(past + row0, keys - 1) : keys - 1;  // what the first row sees last
        limit = a.causal ? min(low + r, keys - 1) : low;
        if (r < lds_i(work + Q_COUNT)) at = ((int64_t)(lds_i(work + Q_Q) + row0 + r) * a.HQ + head) * D + wg * (D / 2);
        const float *stats = a.stats + ((int64_t)head * a.q_places + lds_i(work + Q_PLACE)) * 2 * kTile;
        n_lse = __ldcg(stats + r);
        n_delta = -__ldcg(stats + kTile + r);
        item_read(it);
        if (tiles > 0) {
          // dO goes to tensor memory, from where the products take it without a reading of
          // shared memory: those of the item before that read it are done
          ok = wait_bar(QF, with & 1, failed, a.dev_status);
          if (!__all_sync(0xffffffffu, ok)) break;
          row_to_tmem<D>(lanes + kO, sb + Ly::OFF_O, r, wg);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(QT);
          ++with;
        }
      }
      if (before) {
        // ----------------------------------------------------------- output
        if (sums) ok = wait_bar(DONE, whole++ & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < D / 2; i += 32) {
          uint32_t o[32];
          if (sums) {
            tmem_ld32_issue(lanes + kA + wg * (D / 2) + i, o);
            tmem_ld_wait(o);
            if (i + 32 == D / 2) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(AE);
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = sums ? __float_as_uint(__uint_as_float(o[e]) * a.scale) : 0u;
          if (out >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4 *>(a.dq + out + i + e) = make_uint4(
                  pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                  pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
          }
        }
      }
      if (!on) break;
      before = true;
      sums = tiles > 0;
      out = at;
      for (int j = 0; j < tiles; ++j, ++n) {
        ok = wait_bar(SF, n & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        uint32_t p[64], b[64];
        load64(lanes + kS + half, p);
        wait64(p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(SE);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 x = gdnkv::fma2(pair(p, c), a.scale_log2e, n_lse);
          p[2 * c] = __float_as_uint(ex2f(x.x));
          p[2 * c + 1] = __float_as_uint(ex2f(x.y));
        }
        ok = wait_bar(DF, n & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        load64(lanes + kP + half, b);
        wait64(b);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PE);
        const int k0 = j * kTile + half;
        // (one loop each for tiles with and without a mask)
        auto slopes = [&](auto mask) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float2 g = mul2(pair(p, c), gdnkv::add2(pair(b, c), make_float2(n_delta, n_delta)));
            if (mask) {  // what is masked has no gradient, whatever its S and dP are
              if (k0 + 2 * c > limit) g.x = 0.f;
              if (k0 + 2 * c + 1 > limit) g.y = 0.f;
            }
            b[c] = pack_bf16(g.x, g.y);
          }
        };
        if (k0 + 63 > low) slopes(std::true_type{});
        else slopes(std::false_type{});
        if (n > 0) ok = wait_bar(GE, (n - 1) & 1, failed, a.dev_status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        tmem_st32(lanes + kG + wg * 32, b);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(GF);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ------------------------------------------------------------- copies
      if (elect_one()) {
        uint32_t k_in = 0, v_in = 0, q_in = 0;  // what has been asked for
        bool ok = true;
        for (int it = 0; ok; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + Q_ON)) break;
          const int tiles = lds_i(work + Q_TILES), row = lds_i(work + Q_Q) + lds_i(work + Q_ROW0), key = lds_i(work + Q_K), head = lds_i(work + Q_HEAD);
          mbar_arrive(WE(it % kItems));
          if (tiles == 0) continue;
          if (q_in > 0) ok = wait_bar(QE, (q_in - 1) & 1, failed, a.dev_status);
          if (!ok) break;
          mbar_arrive_expect_tx(QF, 2 * Ly::TB);
          load_tile<D>(sb + Ly::OFF_Q, &mq, QF, head, row);
          load_tile<D>(sb + Ly::OFF_O, &mo, QF, head, row);
          ++q_in;
          for (int j = 0; j < tiles; ++j) {
            const uint32_t ik = k_in % Ly::NK, iv = v_in % Ly::NV;
            if (k_in >= Ly::NK) ok = wait_bar(KE(ik), (k_in / Ly::NK - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(KF(ik), Ly::TB);
            load_tile<D>(sb + Ly::OFF_K + ik * Ly::TB, &mk, KF(ik), head / a.G, key + j * kTile);
            ++k_in;
            if (v_in >= Ly::NV) ok = wait_bar(VE(iv), (v_in / Ly::NV - 1) & 1, failed, a.dev_status);
            if (!ok) break;
            mbar_arrive_expect_tx(VF(iv), Ly::TB);
            load_tile<D>(sb + Ly::OFF_V + iv * Ly::TB, &mv, VF(iv), head / a.G, key + j * kTile);
            ++v_in;
          }
        }
        if (lds_i(failed)) {  // copies in flight
          ok = q_in == 0 || mbar_wait_bounded(QF, (q_in - 1) & 1, gdnc::kWaitLimit);
          for (uint32_t i = 0; i < Ly::NK && i < k_in; ++i) ok &= mbar_wait_bounded(KF(i), ((k_in - 1 - i) / Ly::NK) & 1, gdnc::kWaitLimit);
          for (uint32_t i = 0; i < Ly::NV && i < v_in; ++i) ok &= mbar_wait_bounded(VF(i), ((v_in - 1 - i) / Ly::NV) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      if (elect_one()) {
        uint32_t n = 0, cleared = 0, items = 0;  // key tiles, last ones cleared, items with some
        for (int it = 0;; ++it) {
          uint32_t work;
          if (!item(it, work) || !lds_i(work + Q_ON)) break;
          const int tiles = lds_i(work + Q_TILES);
          const bool clear = tiles * kTile > lds_i(work + Q_KEYS);
          mbar_arrive(WE(it % kItems));
          if (tiles == 0) continue;
          auto wait = [&](uint32_t b, uint32_t phase) { return wait_bar(b, phase & 1, failed, a.dev_status); };
          auto k_tile = [&](uint32_t m) { return sb + Ly::OFF_K + m % Ly::NK * Ly::TB; };
          auto logits = [&](uint32_t m, bool last) {
            if (!wait(KF(m % Ly::NK), m / Ly::NK)) return false;
            if (clear && last) {
              mbar_arrive(VR);
              if (!wait(VZ, cleared++)) return false;
            }
            tc_fence_after();
            mma_rows<D>(tmem + kS, sb + Ly::OFF_Q, k_tile(m));
            umma_commit(SF);
            if (last) umma_commit(QE);
            return true;
          };
          auto slopes = [&](uint32_t m) {
            if (!wait(VF(m % Ly::NV), m / Ly::NV)) return false;
            tc_fence_after();
            mma_rows_ta<D>(tmem + kP, tmem + kO, sb + Ly::OFF_V + m % Ly::NV * Ly::TB);
            umma_commit(DF);
            umma_commit(VE(m % Ly::NV));
            return true;
          };
          bool ok = wait(QT, items) && logits(n, tiles == 1) && slopes(n);
          for (int j = 0; ok && j < tiles; ++j, ++n) {
            const bool more = j + 1 < tiles;
            if (more) ok = wait(SE, n) && logits(n + 1, j + 2 == tiles) && wait(PE, n) && slopes(n + 1);
            ok = ok && wait(GF, n) && (j > 0 || wait(AE, items));
            if (!ok) break;
            tc_fence_after();
            mma_packed<D>(tmem + kA, tmem + kG, k_tile(n), j > 0);
            umma_commit(GE);
            umma_commit(KE(n % Ly::NK));
            if (!more) umma_commit(DONE);
          }
          if (!ok) break;
          ++items;
        }
        if (lds_i(failed)) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 10) {
      // dS is 0 past the sequence's keys, but 0 times what stands there need not be.
      uint32_t n = 0, turn = 0;
      for (int it = 0;; ++it) {
        uint32_t work;
        if (!__all_sync(0xffffffffu, item(it, work)) || !lds_i(work + Q_ON)) break;
        const int tiles = lds_i(work + Q_TILES), keys = lds_i(work + Q_KEYS);
        item_read(it);
        n += tiles;
        if (tiles * kTile <= keys) continue;
        bool there = true;  // (no limit of its own: the products' warp gets there, or gives up and says so)
        while (there && !mbar_try_wait(VR, turn & 1)) there = !lds_i(failed);
        if (!__all_sync(0xffffffffu, there)) break;
        ++turn;
        zero_rows<D>(sb + Ly::OFF_K + (n - 1) % Ly::NK * Ly::TB, keys % kTile);
        if (lane == 0) mbar_arrive(VZ);
      }
    } else {
      // -------------------------------------------------------------- items
      const int64_t most = most_tokens(a.HK, D);
      Walk w;
      walk_begin(a, w, kTile, false, most);
      for (int it = 0;; ++it) {
        Found f;
        const bool on = walk_to(a, w, kTile, false, false, most, take_item(&a.shared->next_q), f, [&](int) { return a.HQ; });
        if (it >= kItems && !__all_sync(0xffffffffu, wait_bar<kItemLimit>(WE(it % kItems), (it / kItems - 1) & 1, failed, a.dev_status))) break;
        if (lane == 0) {
          const uint32_t work = sb + Ly::OFF_WORK + it % kItems * Q_BYTES;
          sts_i(work + Q_ON, on);
          if (on) {
            const Side rows = rows_of(a);
            const int row0 = f.tile * kTile, past = f.keys.count - f.rows.count, count = min(kTile, f.rows.count - row0);
            sts_i(work + Q_Q, f.rows.first);
            sts_i(work + Q_ROW0, row0);
            sts_i(work + Q_COUNT, count);
            sts_i(work + Q_K, f.keys.first);
            sts_i(work + Q_KEYS, f.keys.count);
            sts_i(work + Q_PAST, past);
            sts_i(work + Q_TILES, tiles_in(max(0, a.causal ? min(f.keys.count, past + row0 + count) : f.keys.count), kTile));
            sts_i(work + Q_HEAD, f.in);
            sts_i(work + Q_PLACE, (int)rows.place(f.n, f.rows.first, kTile) + f.tile * rows.apart(kTile));
          }
          mbar_arrive(WF(it % kItems));
        }
        __syncwarp();
        if (!on) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if (!waits) grid_wait();
}

// Most pieces of a (key tile, kv head)'s walk: enough for two items an SM.
int pieces_of(int64_t k_tiles, int HK) {
  const int64_t items = std::max<int64_t>(1, k_tiles * HK), want = (2 * kBlocks + items - 1) / items;
  return (int)std::min<int64_t>(want, 8);
}
// Pieces that this many (key tile, kv head)s, or fewer, have in all at most, so that the
// workspace of a call is large enough for every smaller one: x of them have 8 x or, as
// pieces_of rounds up, less than 2 kBlocks + x, and those from 2 kBlocks on are not cut.
int64_t most_pieces(int64_t k_tiles, int HK) {
  const int64_t items = k_tiles * HK, cut = std::min<int64_t>(items, 2 * kBlocks - 1);
  return std::min(8 * items, 2 * kBlocks - 1 + cut);
}

template <int D> cudaError_t launch(const BwdArgs &a, cudaStream_t s) {
  const int64_t q_blocks = std::max<int64_t>(1, a.q_places) * a.HQ, k_blocks = a.k_places * a.HK;  // (block 0 does more than its rows)
  const int64_t sms = gdn_host::sm_count();
  CUtensorMap mq, mk, mv, mo;
  // a side without rows is never loaded
  const bool rows = a.Tq > 0, keys = a.Tk > 0;
  const uint16_t *q = rows ? a.q : a.k, *dout = rows ? a.dout : a.k, *k = keys ? a.k : a.q, *v = keys ? a.v : a.q;
  const int hq = rows ? a.HQ : a.HK, hk = keys ? a.HK : a.HQ, tq = rows ? a.Tq : a.Tk, tk = keys ? a.Tk : a.Tq;
  if (!rows_map(&mq, q, D, hq, tq, rows ? a.ldq : a.ldk) || !rows_map(&mo, dout, D, hq, tq, rows ? (int64_t)a.HQ * D : a.ldk) ||
      !rows_map(&mk, k, D, hk, tk, keys ? a.ldk : a.ldq) || !rows_map(&mv, v, D, hk, tk, keys ? a.ldv : a.ldq))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done_kv{0}, done_q{0};
  cudaError_t e = gdn_host::allow_smem(attn_dkdv_kernel<D>, KvLay<D>::BYTES, done_kv);
  if (e == cudaSuccess) e = gdn_host::allow_smem(attn_dq_kernel<D>, QLay<D>::BYTES, done_q);
  static std::atomic<bool> known_kv{false}, known_q{false};
  if (e == cudaSuccess) e = check_registers(attn_dkdv_kernel<D>, 168, known_kv);
  if (e == cudaSuccess) e = check_registers(attn_dq_kernel<D>, 168, known_q);
  if (e != cudaSuccess) return e;
  e = gdn_host::launch_dependent(attn_stats_kernel<D>, dim3((unsigned)q_blocks), 256, 0, s, a);
  if (e == cudaSuccess && keys)
    e = gdn_host::launch_dependent(attn_dkdv_kernel<D>, dim3((unsigned)std::min(a.k_places * a.HK * a.pieces, sms)), kThreads,
                                   KvLay<D>::BYTES, s, a, mq, mk, mv, mo);
  if (e == cudaSuccess && rows)
    e = gdn_host::launch_dependent(attn_dq_kernel<D>, dim3((unsigned)std::min(a.q_places * a.HQ, sms)), kThreads, QLay<D>::BYTES,
                                   s, a, keys ? 0 : 1, mq, mk, mv, mo);
  if (e == cudaSuccess && keys && a.pieces > 1) e = gdn_host::launch_dependent(attn_join_kernel<D>, dim3((unsigned)k_blocks, 8), 256, 0, s, a);
  return e;
}

}  // namespace

namespace gdn_host {
static size_t stats_bytes(int N, int Tq, int HQ) { return (size_t)HQ * gdnat::most_tiles(Tq, N, gdnat::kTile) * 2 * gdnat::kTile * sizeof(float); }
bool attn_bwd_takes(int N, int Tq, int Tk, int HQ, int HK) {
  return gdnat::most_tiles(Tq, N, gdnat::kTile) * HQ <= INT_MAX && gdnat::most_tiles(Tk, N, gdnat::kTile) * HK <= INT_MAX;
}
size_t attn_bwd_workspace_bytes(int N, int Tq, int Tk, int HQ, int HK, int D) {
  return 16 + stats_bytes(N, Tq, HQ) +
         (size_t)most_pieces(gdnat::most_tiles(Tk, N, gdnat::kTile), HK) * 2 * gdnat::kTile * D * sizeof(float);
}
cudaError_t launch_attn_bwd(const TrainAttnArgs &c, cudaStream_t s) {
  BwdArgs a{};
  static_cast<TrainAttnArgs &>(a) = c;
  a.G = c.HQ / c.HK;
  a.scale_log2e = c.scale * gdnc::kLog2e;
  a.q_places = gdnat::most_tiles(c.Tq, c.N, gdnat::kTile);
  a.k_places = gdnat::most_tiles(c.Tk, c.N, gdnat::kTile);
  a.pieces = pieces_of(a.k_places, c.HK);
  a.shared = static_cast<BwdArgs::Shared *>(c.ws);
  a.stats = reinterpret_cast<float *>(static_cast<char *>(c.ws) + 16);
  a.part = a.stats + stats_bytes(c.N, c.Tq, c.HQ) / sizeof(float);
  return c.D == 128 ? launch<128>(a, s) : launch<64>(a, s);
}
}  // namespace gdn_host
