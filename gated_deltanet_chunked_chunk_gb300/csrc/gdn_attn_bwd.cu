// gdn_attn_bwd.cu -- attention of packed sequences, gradients, on tcgen05.
//
//   P = 2^(c S - lse log2 e),  S = q K^T,  c = scale log2 e      (formed again)
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  delta = sum dO o
//   dQ = scale dS K,  dK = scale dS^T Q
//
// Five products, 10 D operations a (row, key, head); bound: the tensor cores.
//
// Two kernels, one with the keys fixed (dK, dV) and one with the rows fixed (dQ), each
// of which forms S and dP itself: seven products instead of five.  In exchange every
// sum stays in one block's tensor memory from beginning to end: no sum of dQ passes
// through memory tile by tile in fp32, nothing is added by atomics, and two calls agree
// bit for bit.  A small kernel before them writes what both need of a row, -lse log2 e and
// delta, tile by tile (kTile numbers each, with rows past the sequence at -inf and 0:
// their P is 0).
//
// dK, dV: a block has 128 keys of one kv head and walks over (head of the group, 128
// rows).  S^T = K Q^T and dP^T = V dO^T have the keys as rows, so P^T and dS^T, written
// to tensor memory over what they came from, are the A operands of dV and dK as they
// stand and never pass through shared memory.  Tensor memory: S^T, dP^T, dV, dK, all
// 512 columns at D = 128.  The products' order is dV(i), S(i+1), dK(i), dP(i+1): P(i+1)
// is formed while dK(i) and dP(i+1) run, dS(i) while dV(i) and S(i+1) do.
// Where few (key tile, kv head) pairs exist a pair's walk is cut into pieces, whose sums
// a last kernel adds in order.
//
// dQ: a block has 128 rows of one head and walks over the keys.  Tensor memory: S twice
// (the next keys' is formed ahead), dP, dQ; dS goes over its S.
//
// P and dS enter the products in bf16 (8 significant bits), sums are fp32.
#include <limits.h>

#include <algorithm>

#include "gdn_attn.cuh"

namespace {

using namespace gdnat;

constexpr int kThreads = 384;  // warps 0-7 P and dS, 8 copies, 9 products, 10 clears rows past the end

struct BwdArgs : Args {
  float *stats;  // [HQ][q slots][2][kTile]: -lse log2 e, delta
  float *part;   // [piece][k slots][HK][2][kTile][D]: sums of dK and dV
  int64_t q_slots, k_slots;
  int pieces;
};

// ------------------------------------------------------------ of each row
template <int D> __global__ void __launch_bounds__(256) attn_stats_kernel(const BwdArgs a) {
  constexpr int L = D / 8, PER = 256 / L;  // lanes a row, rows at once
  const int64_t slot = blockIdx.x / a.HQ;
  const int head = blockIdx.x % a.HQ, l = threadIdx.x % L;
  grid_wait();
  if (blockIdx.x == 0) check_offsets(a);
  Tile t;
  if (!tile_of(a, slot, kTile, false, t)) return;
  float *out = a.stats + ((int64_t)head * a.q_slots + slot) * 2 * kTile;
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
template <int D> struct KvLay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NQ = 3, NO = 2, NT = 2;  // stages of Q, dO, the rows' numbers
  static constexpr int OFF_K = 0, OFF_V = TB, OFF_Q = 2 * TB, OFF_O = OFF_Q + NQ * TB;
  static constexpr int OFF_T = OFF_O + NO * TB;
  static constexpr int OFF_BAR = OFF_T + NT * 2 * kTile * 4;
  static constexpr int BARS = 2 * (NQ + NO + NT) + 9;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 80;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};
struct KvWork {
  int q_first, rows, k_first, keys;  // the sequence's
  int k0, past;                      // the block's first key; keys - rows
  int t0, nt;                        // first row tile that sees them, row tiles from there on
  int s0, steps;                     // the piece's steps: step s is head s / nt of the group, row tile t0 + s % nt
  int q_slot;                        // slot of the sequence's first row tile
  int on;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dkdv_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  using Ly = KvLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t slot = blockIdx.x / (a.HK * a.pieces);
  const int hk = blockIdx.x / a.pieces % a.HK, piece = blockIdx.x % a.pieces;
  grid_wait();
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  volatile KvWork *work = reinterpret_cast<volatile KvWork *>(smem + Ly::OFF_MISC + 16);
  static_assert(sizeof(KvWork) <= 64, "room for it");
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto QF = [&](int i) { return bar + 8 * i; };
  auto QE = [&](int i) { return bar + 8 * (Ly::NQ + i); };
  auto OF = [&](int i) { return bar + 8 * (2 * Ly::NQ + i); };
  auto OE = [&](int i) { return bar + 8 * (2 * Ly::NQ + Ly::NO + i); };
  auto TF = [&](int i) { return bar + 8 * (2 * Ly::NQ + 2 * Ly::NO + i); };
  auto TE = [&](int i) { return bar + 8 * (2 * Ly::NQ + 2 * Ly::NO + Ly::NT + i); };
  const uint32_t bx = bar + 16 * (Ly::NQ + Ly::NO + Ly::NT);
  const uint32_t KF = bx, SF = bx + 8, DF = bx + 16, PF = bx + 24, GF = bx + 32;  // K and V, S, dP, P, dS are there
  const uint32_t DONE = bx + 40, VR = bx + 48, VZ = bx + 56, DR = bx + 64;
  if (warp == 0) {
    Tile t;
    const bool on = tile_of(a, slot, kTile, true, t);
    if (lane == 0) {
      work->on = on;
      if (on) {
        const int past = t.keys.count - t.rows.count, tn = (t.rows.count + kTile - 1) / kTile;
        const int t0 = min(tn, a.causal ? max(0, t.row0 - past) / kTile : 0);
        const int64_t all = (int64_t)a.G * (tn - t0);
        work->q_first = t.rows.first;
        work->rows = t.rows.count;
        work->k_first = t.keys.first;
        work->keys = t.keys.count;
        work->q_slot = t.rows.first / kTile + t.n;
        work->k0 = t.row0;
        work->past = past;
        work->t0 = t0;
        work->nt = tn - t0;
        work->s0 = (int)(all * piece / a.pieces);
        work->steps = (int)(all * (piece + 1) / a.pieces) - work->s0;
      }
      for (int i = 0; i < Ly::NQ; ++i) { mbar_init(QF(i), 1); mbar_init(QE(i), 1); }
      for (int i = 0; i < Ly::NO; ++i) { mbar_init(OF(i), 1); mbar_init(OE(i), 1); }
      for (int i = 0; i < Ly::NT; ++i) { mbar_init(TF(i), 1); mbar_init(TE(i), 8); }
      mbar_init(KF, 1);
      mbar_init(SF, 1);
      mbar_init(DF, 1);
      mbar_init(PF, 8);
      mbar_init(GF, 8);
      mbar_init(DONE, 1);
      mbar_init(VR, 1);
      mbar_init(VZ, 1);
      mbar_init(DR, 1);
      mbar_fence_init();
      *failed = 0;
    }
  }
  __syncthreads();
  if (!work->on) return;
  if (warp == 9) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int steps = work->steps, s0 = work->s0, nt = work->nt, t0 = work->t0, rows = work->rows;
  const int wg = warp >> 2, r = tid & 127;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
  const uint32_t kS = 0, kP = 128, kV = 256, kK = 256 + D;  // columns of S^T, dP^T, dV, dK

  if (wg < 2) {
    // -------------------------------------------------------------- P and dS
    const int half = wg * 64, k0 = work->k0, past = work->past;
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      *failed = 1;
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    int t = nt > 0 ? s0 % nt : 0;
    for (int i = 0; i < steps; ++i) {
      const uint32_t numbers = sb + Ly::OFF_T + (i % Ly::NT) * (2 * kTile * 4) + half * 4;
      const int q0 = (t0 + t) * kTile + half;  // first of this thread's rows
      t = t + 1 == nt ? 0 : t + 1;
      const bool masked = a.causal && q0 + past < k0 + kTile - 1;
      const int from = k0 + r - past - q0;  // its first column that sees key r
      if (ok) ok = wait_bar(TF(i % Ly::NT), (i / Ly::NT) & 1, failed, a.dev_status) && wait_bar(SF, i & 1, failed, a.dev_status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t p[64], b[64];
      load64(tmem + lanes + kS + half, p);
      wait64(p);
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 n = gdnkv::lds_f4(numbers + c * 4);
        float2 x = fma2v(pair(p, c / 2), a.scale_log2e, make_float2(n.x, n.y)), y = fma2v(pair(p, c / 2 + 1), a.scale_log2e, make_float2(n.z, n.w));
        p[c] = __float_as_uint(ex2f(x.x));
        p[c + 1] = __float_as_uint(ex2f(x.y));
        p[c + 2] = __float_as_uint(ex2f(y.x));
        p[c + 3] = __float_as_uint(ex2f(y.y));
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < from) p[c] = 0;
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) b[c] = pack_bf16(__uint_as_float(p[2 * c]), __uint_as_float(p[2 * c + 1]));
      tmem_st32(tmem + lanes + kS + half, b);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(PF);
      ok = wait_bar(DF, i & 1, failed, a.dev_status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      load64(tmem + lanes + kP + half, b);
      wait64(b);
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 n = gdnkv::lds_f4(numbers + kTile * 4 + c * 4);
        const float2 x = mul2(pair(p, c / 2), gdnkv::add2(pair(b, c / 2), make_float2(-n.x, -n.y)));
        const float2 y = mul2(pair(p, c / 2 + 1), gdnkv::add2(pair(b, c / 2 + 1), make_float2(-n.z, -n.w)));
        // a weight of 0 has no gradient, whatever a masked row's dP is
        p[c / 2] = masked ? pack_bf16(c < from ? 0.f : x.x, c + 1 < from ? 0.f : x.y) : pack_bf16(x.x, x.y);
        p[c / 2 + 1] = masked ? pack_bf16(c + 2 < from ? 0.f : y.x, c + 3 < from ? 0.f : y.y) : pack_bf16(y.x, y.y);
      }
      tmem_st32(tmem + lanes + kP + half, p);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(GF);
        mbar_arrive(TE(i % Ly::NT));
      }
    }
    if (ok && !*failed && steps > 0) wait_bar(DONE, 0, failed, a.dev_status);
  } else {
    const int tail = rows % kTile, last = nt - 1;  // rows of a last row tile that is not full
    if (warp == 8) {
      // ----------------------------------------------------------- producer
      if (steps > 0 && elect_one()) {
        mbar_arrive_expect_tx(KF, 2 * Ly::TB);
        load_tile<D>(sb + Ly::OFF_K, &mk, KF, hk, work->k_first + work->k0);
        load_tile<D>(sb + Ly::OFF_V, &mv, KF, hk, work->k_first + work->k0);
        int g = s0 / nt, t = s0 % nt, q_in = 0, o_in = 0, t_in = 0;  // and what has been asked for
        for (int i = 0; i < steps; ++i) {
          const int head = hk * a.G + g, row = work->q_first + (t0 + t) * kTile;
          const int iq = i % Ly::NQ, io = i % Ly::NO, it = i % Ly::NT;
          if (i >= Ly::NQ && !wait_bar(QE(iq), (i / Ly::NQ - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(QF(iq), Ly::TB);
          load_tile<D>(sb + Ly::OFF_Q + iq * Ly::TB, &mq, QF(iq), head, row);
          q_in = i + 1;
          if (i >= Ly::NT && !wait_bar(TE(it), (i / Ly::NT - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(TF(it), 2 * kTile * 4);
          bulk_load(sb + Ly::OFF_T + it * (2 * kTile * 4), a.stats + ((int64_t)head * a.q_slots + work->q_slot + t0 + t) * 2 * kTile,
                    2 * kTile * 4, TF(it));
          t_in = i + 1;
          if (i >= Ly::NO && !wait_bar(OE(io), (i / Ly::NO - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(OF(io), Ly::TB);
          load_tile<D>(sb + Ly::OFF_O + io * Ly::TB, &mo, OF(io), head, row);
          o_in = i + 1;
          if (++t == nt) {
            t = 0;
            ++g;
          }
        }
        if (*failed) {  // copies in flight
          bool ok = mbar_wait_bounded(KF, 0, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NQ && i < q_in; ++i) ok &= mbar_wait_bounded(QF(i), ((q_in - 1 - i) / Ly::NQ) & 1, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NT && i < t_in; ++i) ok &= mbar_wait_bounded(TF(i), ((t_in - 1 - i) / Ly::NT) & 1, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NO && i < o_in; ++i) ok &= mbar_wait_bounded(OF(i), ((o_in - 1 - i) / Ly::NO) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 10) {
      // Rows past the sequence in its last row tile: their P and dS are 0, but 0 times
      // what stands there need not be.
      if (tail != 0) {
        int turn = 0;
        for (int i = 0; i < steps; ++i) {
          if ((s0 + i) % nt != last) continue;
          bool there = true;  // (no limit of its own: the products' warp gets there, or gives up and says so)
          while (there && !mbar_try_wait(VR, turn & 1)) there = !*failed;
          if (!__all_sync(0xffffffffu, there)) break;
          ++turn;
          zero_rows<D>(sb + Ly::OFF_Q + i % Ly::NQ * Ly::TB, tail);
          zero_rows<D>(sb + Ly::OFF_O + i % Ly::NO * Ly::TB, tail);
          if (lane == 0) mbar_arrive(VZ);
        }
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      if (steps > 0 && elect_one()) {
        int turn = 0;
        auto q_tile = [&](int i) { return sb + Ly::OFF_Q + i % Ly::NQ * Ly::TB; };
        auto o_tile = [&](int i) { return sb + Ly::OFF_O + i % Ly::NO * Ly::TB; };
        auto logits = [&](int i) {
          if (!wait_bar(QF(i % Ly::NQ), (i / Ly::NQ) & 1, failed, a.dev_status)) return false;
          if (tail != 0 && (s0 + i) % nt == last) {
            if (!wait_bar(OF(i % Ly::NO), (i / Ly::NO) & 1, failed, a.dev_status)) return false;
            mbar_arrive(VR);
            if (!wait_bar(VZ, turn++ & 1, failed, a.dev_status)) return false;
          }
          tc_fence_after();
          mma_rows<D>(tmem + kS, sb + Ly::OFF_K, q_tile(i));
          umma_commit(SF);
          return true;
        };
        auto slopes = [&](int i) {
          if (!wait_bar(OF(i % Ly::NO), (i / Ly::NO) & 1, failed, a.dev_status)) return false;
          tc_fence_after();
          mma_rows<D>(tmem + kP, sb + Ly::OFF_V, o_tile(i));
          umma_commit(DF);
          return true;
        };
        bool ok = wait_bar(KF, 0, failed, a.dev_status) && logits(0) && slopes(0);
        for (int i = 0; ok && i < steps; ++i) {
          ok = wait_bar(PF, i & 1, failed, a.dev_status);
          if (!ok) break;
          tc_fence_after();
          mma_cols<D>(tmem + kV, tmem + kS, o_tile(i), i > 0);
          umma_commit(OE(i % Ly::NO));
          if (i + 1 < steps) ok = logits(i + 1);
          ok = ok && wait_bar(GF, i & 1, failed, a.dev_status);
          if (!ok) break;
          tc_fence_after();
          mma_cols<D>(tmem + kK, tmem + kP, q_tile(i), i > 0);
          umma_commit(QE(i % Ly::NQ));
          if (i + 1 < steps) ok = slopes(i + 1);
          else umma_commit(DONE);
        }
        if (!ok) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (wg < 2 && !*failed) {
    // ---------------------------------------------------------------- output
    tc_fence_after();
    const int key = work->k0 + r;
    const bool on = key < work->keys, whole = a.pieces == 1;
    const int64_t at = ((int64_t)(work->k_first + key) * a.HK + hk) * D + wg * (D / 2);
    const int64_t part = (((piece * a.k_slots + slot) * a.HK + hk) * 2 * kTile + r) * D + wg * (D / 2);
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {  // dK, then dV: half a row each
      const bool second = i >= D / 2;
      const int c = second ? i - D / 2 : i;
      uint32_t o[32];
      if (steps > 0) {
        tmem_ld32_issue(tmem + lanes + (second ? kV : kK) + wg * (D / 2) + c, o);
        tmem_ld_wait(o);
      }
      const float f = second ? 1.f : a.scale;
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = steps > 0 ? __float_as_uint(__uint_as_float(o[e]) * f) : 0u;
      if (on && whole) {
        uint16_t *dst = (second ? a.dv : a.dk) + at + c;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4 *>(dst + e) =
              make_uint4(pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                         pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
      } else if (on) {
        float *dst = a.part + part + (second ? kTile * D : 0) + c;
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4 *>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Adds the pieces' sums of a (key tile, kv head) in order.
template <int D> __global__ void __launch_bounds__(256) attn_join_kernel(const BwdArgs a) {
  const int64_t slot = blockIdx.x / a.HK;
  const int hk = blockIdx.x % a.HK;
  grid_wait();
  Tile t;
  if (!tile_of(a, slot, kTile, true, t)) return;
  const int rows = min(kTile, t.keys.count - t.row0);
  for (int i = threadIdx.x; i < 2 * rows * (D / 8); i += 256) {
    const bool second = i >= rows * (D / 8);
    const int e = second ? i - rows * (D / 8) : i, r = e / (D / 8), c = e % (D / 8) * 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    for (int p = 0; p < a.pieces; ++p) {
      const float4 *src =
          reinterpret_cast<const float4 *>(a.part + ((((p * a.k_slots + slot) * a.HK + hk) * 2 + (second ? 1 : 0)) * kTile + r) * D + c);
      const float4 u = __ldcs(src), v = __ldcs(src + 1);
      x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
      y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    uint16_t *dst = (second ? a.dv : a.dk) + ((int64_t)(t.keys.first + t.row0 + r) * a.HK + hk) * D + c;
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
}

// --------------------------------------------------------------------- dQ
template <int D> struct QLay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NK = 3, NV = 2;
  static constexpr int OFF_Q = 0, OFF_O = TB, OFF_K = 2 * TB, OFF_V = OFF_K + NK * TB;
  static constexpr int OFF_BAR = OFF_V + NV * TB;
  static constexpr int BARS = 2 * (NK + NV) + 10;
  static constexpr int OFF_MISC = OFF_BAR + BARS * 8;
  static constexpr int BYTES = OFF_MISC + 64;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};
struct QWork {
  int q_first, row0, count;  // first row of the sequence, the block's first one in it, its rows
  int k_first, keys, past;
  int tiles;
  int on;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_dq_kernel(const BwdArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
  using Ly = QLay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the last rows, which see most keys, first
  const int64_t slot = a.q_slots - 1 - blockIdx.x / a.HQ;
  const int head = blockIdx.x % a.HQ;
  grid_wait();
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  volatile QWork *work = reinterpret_cast<volatile QWork *>(smem + Ly::OFF_MISC + 16);
  static_assert(sizeof(QWork) <= 48, "room for it");
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto KF = [&](int i) { return bar + 8 * i; };
  auto KE = [&](int i) { return bar + 8 * (Ly::NK + i); };
  auto VF = [&](int i) { return bar + 8 * (2 * Ly::NK + i); };
  auto VE = [&](int i) { return bar + 8 * (2 * Ly::NK + Ly::NV + i); };
  const uint32_t bx = bar + 16 * (Ly::NK + Ly::NV);
  auto SF = [&](int i) { return bx + 8 * i; };
  const uint32_t QF = bx + 16, DF = bx + 24, PR = bx + 32, GF = bx + 40;  // Q and dO, dP are there; dP is read; dS is there
  const uint32_t DONE = bx + 48, VR = bx + 56, VZ = bx + 64, DR = bx + 72;
  if (warp == 0) {
    Tile t;
    const bool on = tile_of(a, slot, kTile, false, t);
    if (lane == 0) {
      work->on = on;
      if (on) {
        const int past = t.keys.count - t.rows.count, count = min(kTile, t.rows.count - t.row0);
        const int seen = a.causal ? min(t.keys.count, past + t.row0 + count) : t.keys.count;
        work->q_first = t.rows.first;
        work->row0 = t.row0;
        work->count = count;
        work->k_first = t.keys.first;
        work->keys = t.keys.count;
        work->past = past;
        work->tiles = (max(0, seen) + kTile - 1) / kTile;
      }
      for (int i = 0; i < Ly::NK; ++i) { mbar_init(KF(i), 1); mbar_init(KE(i), 1); }
      for (int i = 0; i < Ly::NV; ++i) { mbar_init(VF(i), 1); mbar_init(VE(i), 1); }
      for (int i = 0; i < 2; ++i) mbar_init(SF(i), 1);
      mbar_init(QF, 1);
      mbar_init(DF, 1);
      mbar_init(PR, 8);
      mbar_init(GF, 8);
      mbar_init(DONE, 1);
      mbar_init(VR, 1);
      mbar_init(VZ, 1);
      mbar_init(DR, 1);
      mbar_fence_init();
      *failed = 0;
    }
  }
  __syncthreads();
  if (!work->on) return;
  if (warp == 9) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = work->tiles, keys = work->keys;
  const int wg = warp >> 2, r = tid & 127;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
  const uint32_t kP = 256, kQ = 384;  // columns of dP, dQ; S at 0 and 128

  if (wg < 2) {
    // -------------------------------------------------------------------- dS
    const int half = wg * 64, past = work->past, row0 = work->row0;
    const int low = a.causal ? past + row0 : keys - 1;
    const int limit = a.causal ? min(low + r, keys - 1) : low;
    const float *stats = a.stats + ((int64_t)head * a.q_slots + slot) * 2 * kTile;
    const float n_lse = stats[r], n_delta = -stats[kTile + r];
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      *failed = 1;
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    for (int j = 0; j < tiles; ++j) {
      const uint32_t S = tmem + lanes + (j & 1) * 128 + half;
      if (ok) ok = wait_bar(SF(j & 1), (j >> 1) & 1, failed, a.dev_status) && wait_bar(DF, j & 1, failed, a.dev_status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t s[64], b[64];
      load64(S, s);
      load64(tmem + lanes + kP + half, b);
      wait64(s);
      gdnkv::tie32(b);
      gdnkv::tie32(b + 32);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(PR);
      const int k0 = j * kTile + half;
      const bool masked = k0 + 63 > low || k0 + 63 >= keys;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float2 x = gdnkv::fma2(pair(s, c), a.scale_log2e, n_lse), d = gdnkv::add2(pair(b, c), make_float2(n_delta, n_delta));
        const float2 g = mul2(make_float2(ex2f(x.x), ex2f(x.y)), d);
        s[c] = masked ? pack_bf16(k0 + 2 * c > limit ? 0.f : g.x, k0 + 2 * c + 1 > limit ? 0.f : g.y) : pack_bf16(g.x, g.y);
      }
      tmem_st32(S, s);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(GF);
    }
    if (ok && !*failed && tiles > 0) wait_bar(DONE, 0, failed, a.dev_status);
  } else {
    const int tail = keys % kTile;  // keys of a last tile that is not full
    const bool clear = tail != 0 && tiles * kTile > keys;
    if (warp == 8) {
      // ----------------------------------------------------------- producer
      if (tiles > 0 && elect_one()) {
        const int row = work->q_first + work->row0, key = work->k_first, hk = head / a.G;
        mbar_arrive_expect_tx(QF, 2 * Ly::TB);
        load_tile<D>(sb + Ly::OFF_Q, &mq, QF, head, row);
        load_tile<D>(sb + Ly::OFF_O, &mo, QF, head, row);
        int k_in = 0, v_in = 0;
        for (int j = 0; j < tiles; ++j) {
          const int ik = j % Ly::NK, iv = j % Ly::NV;
          if (j >= Ly::NK && !wait_bar(KE(ik), (j / Ly::NK - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(KF(ik), Ly::TB);
          load_tile<D>(sb + Ly::OFF_K + ik * Ly::TB, &mk, KF(ik), hk, key + j * kTile);
          k_in = j + 1;
          if (j >= Ly::NV && !wait_bar(VE(iv), (j / Ly::NV - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(VF(iv), Ly::TB);
          load_tile<D>(sb + Ly::OFF_V + iv * Ly::TB, &mv, VF(iv), hk, key + j * kTile);
          v_in = j + 1;
        }
        if (*failed) {  // copies in flight
          bool ok = mbar_wait_bounded(QF, 0, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NK && i < k_in; ++i) ok &= mbar_wait_bounded(KF(i), ((k_in - 1 - i) / Ly::NK) & 1, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NV && i < v_in; ++i) ok &= mbar_wait_bounded(VF(i), ((v_in - 1 - i) / Ly::NV) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 10) {
      // dS is 0 past the sequence's keys, but 0 times what stands there need not be
      if (clear) {
        bool there = true;  // (no limit of its own: the products' warp gets there, or gives up and says so)
        while (there && !mbar_try_wait(VR, 0)) there = !*failed;
        if (__all_sync(0xffffffffu, there)) {
          zero_rows<D>(sb + Ly::OFF_K + (tiles - 1) % Ly::NK * Ly::TB, tail);
          if (lane == 0) mbar_arrive(VZ);
        }
      }
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      if (tiles > 0 && elect_one()) {
        auto k_tile = [&](int j) { return sb + Ly::OFF_K + j % Ly::NK * Ly::TB; };
        auto logits = [&](int j) {
          if (!wait_bar(KF(j % Ly::NK), (j / Ly::NK) & 1, failed, a.dev_status)) return false;
          if (clear && j == tiles - 1) {
            mbar_arrive(VR);
            if (!wait_bar(VZ, 0, failed, a.dev_status)) return false;
          }
          tc_fence_after();
          mma_rows<D>(tmem + (j & 1) * 128, sb + Ly::OFF_Q, k_tile(j));
          umma_commit(SF(j & 1));
          return true;
        };
        auto slopes = [&](int j) {
          if (!wait_bar(VF(j % Ly::NV), (j / Ly::NV) & 1, failed, a.dev_status)) return false;
          tc_fence_after();
          mma_rows<D>(tmem + kP, sb + Ly::OFF_O, sb + Ly::OFF_V + j % Ly::NV * Ly::TB);
          umma_commit(DF);
          umma_commit(VE(j % Ly::NV));
          return true;
        };
        bool ok = wait_bar(QF, 0, failed, a.dev_status) && logits(0) && slopes(0);
        if (ok && tiles > 1) ok = logits(1);
        for (int j = 0; ok && j < tiles; ++j) {
          if (j + 1 < tiles) ok = wait_bar(PR, j & 1, failed, a.dev_status) && slopes(j + 1);
          ok = ok && wait_bar(GF, j & 1, failed, a.dev_status);
          if (!ok) break;
          tc_fence_after();
          mma_cols<D>(tmem + kQ, tmem + (j & 1) * 128, k_tile(j), j > 0);
          umma_commit(KE(j % Ly::NK));
          if (j + 2 < tiles) ok = logits(j + 2);
          if (j + 1 == tiles) umma_commit(DONE);
        }
        if (!ok) {  // let the products in flight finish before the block leaves
          umma_commit(DR);
          if (!mbar_wait_bounded(DR, 0, gdnc::kWaitLimit)) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (wg < 2 && !*failed) {
    // ---------------------------------------------------------------- output
    tc_fence_after();
    const bool on = r < work->count;
    uint16_t *dst = a.dq + ((int64_t)(work->q_first + work->row0 + r) * a.HQ + head) * D + wg * (D / 2);
#pragma unroll 1
    for (int i = 0; i < D / 2; i += 32) {
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld32_issue(tmem + lanes + kQ + wg * (D / 2) + i, o);
        tmem_ld_wait(o);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = tiles > 0 ? __float_as_uint(__uint_as_float(o[e]) * a.scale) : 0u;
      if (on) {
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4 *>(dst + i + e) =
              make_uint4(pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                         pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Pieces that the walk of a (key tile, kv head) is cut into: where there are fewer than
// four for each SM, up to one for each head of the group, 8 at most.
int pieces_of(int64_t k_slots, int HQ, int HK) {
  const int64_t items = k_slots * HK, want = (4 * 152 + items - 1) / items;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 8), HQ / HK));
}

template <int D> cudaError_t launch(const BwdArgs &a, cudaStream_t s) {
  const int64_t q_blocks = a.q_slots * a.HQ, k_blocks = a.k_slots * a.HK;
  if (q_blocks > INT_MAX || k_blocks * a.pieces > INT_MAX) return cudaErrorInvalidConfiguration;
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
  if (e != cudaSuccess) return e;
  e = gdn_host::launch_dependent(attn_stats_kernel<D>, dim3((unsigned)q_blocks), 256, 0, s, a);
  if (e == cudaSuccess && keys)
    e = gdn_host::launch_dependent(attn_dkdv_kernel<D>, dim3((unsigned)(k_blocks * a.pieces)), kThreads, KvLay<D>::BYTES, s, a, mq, mk, mv, mo);
  if (e == cudaSuccess && rows) e = gdn_host::launch_dependent(attn_dq_kernel<D>, dim3((unsigned)q_blocks), kThreads, QLay<D>::BYTES, s, a, mq, mk, mv, mo);
  if (e == cudaSuccess && keys && a.pieces > 1) e = gdn_host::launch_dependent(attn_join_kernel<D>, dim3((unsigned)k_blocks), 256, 0, s, a);
  return e;
}

}  // namespace

namespace gdn_host {
static size_t stats_bytes(int N, int Tq, int HQ) { return (size_t)HQ * gdnat::slots_of(Tq, N, gdnat::kTile) * 2 * gdnat::kTile * sizeof(float); }
size_t attn_bwd_workspace_bytes(int N, int Tq, int Tk, int HQ, int HK, int D) {
  const int64_t k_slots = gdnat::slots_of(Tk, N, gdnat::kTile);
  const int pieces = pieces_of(k_slots, HQ, HK);
  return stats_bytes(N, Tq, HQ) + (pieces > 1 ? (size_t)pieces * k_slots * HK * 2 * gdnat::kTile * D * sizeof(float) : 0);
}
cudaError_t launch_attn_bwd(const TrainAttnArgs &c, cudaStream_t s) {
  BwdArgs a{};
  static_cast<TrainAttnArgs &>(a) = c;
  a.G = c.HQ / c.HK;
  a.scale_log2e = c.scale * gdnc::kLog2e;
  a.q_slots = gdnat::slots_of(c.Tq, c.N, gdnat::kTile);
  a.k_slots = gdnat::slots_of(c.Tk, c.N, gdnat::kTile);
  a.pieces = pieces_of(a.k_slots, c.HQ, c.HK);
  a.stats = static_cast<float *>(c.ws);
  a.part = a.stats + stats_bytes(c.N, c.Tq, c.HQ) / sizeof(float);
  return c.D == 128 ? launch<128>(a, s) : launch<64>(a, s);
}
}  // namespace gdn_host
