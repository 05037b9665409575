// gdn_attn_fwd.cu -- attention of packed sequences, forward, on tcgen05.
//
//   S = q K^T,  p_j = 2^(c S_j - m),  l = sum p_j,  o = sum p_j v_j / l,
//   lse = (m + log2 l) ln 2,  c = scale log2 e
//
// with m the running maximum of c S.  Bound: the tensor cores, 4 D operations a (row,
// key, head).
//
// A block works on two tiles of 128 rows of one head, which share the keys and values
// that TMA brings, and whose softmaxes take turns on the tensor cores (one tile, where
// fewer blocks than SMs would come out).  Warps 0-7 and 8-15 are the softmax of the two
// tiles: a thread holds half a row, 64 logits; 16 brings the tiles, 17 issues the
// products, 18 clears what the last tile of values holds past the sequence.
//
// Tensor memory (512 columns): S of both tiles, P in bf16 over its S (each half over
// the half that its threads read), O of both tiles.  Products of one thread execute in
// order, so an S of the next keys, issued after the P V that reads the same columns, is
// safe, and "S is there" also says that O may be touched.
//
// m grows only where an exponent is more than kMost above it: both threads of a row
// agree on that in one barrier that also joins their votes, and O is then rescaled.
// P has 8 significant bits (bf16 keeps fp32's range, so any m near the maximum is as
// good), l is the sum before that rounding, whose errors (2^-8 of a weight at most, either
// way) mostly cancel in o.
#include <limits.h>

#include "gdn_attn.cuh"

namespace {

using namespace gdnat;

constexpr int kThreads = 640;
constexpr float kMost = 8.f;

template <int D> struct Lay {
  static constexpr int TB = tile_bytes<D>();
  static constexpr int NS = D == 128 ? 4 : 8;  // stages of the line K0 V0 K1 V1 ..
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TB;
  static constexpr int OFF_X = OFF_KV + NS * TB;  // float [tile][half][row]: what a row's threads tell each other
  static constexpr int OFF_BAR = OFF_X + 2 * 2 * 128 * 4;
  static constexpr int OFF_MISC = OFF_BAR + (2 * NS + 10) * 8;
  static constexpr int BYTES = OFF_MISC + 64;
  static_assert(BYTES <= 227 * 1024, "one block an SM");
};

// What the block works on, in shared memory.
struct Work {
  int q_first, k_first, keys;  // first row of q and of k of the sequence, its keys
  int row0, past;              // the block's first row in the sequence; keys - rows
  int count[2], tiles[2];      // rows and key tiles of both row tiles
  int on;
};

__device__ __forceinline__ bool vote_any(int id, bool mine) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.pred q, %1, 256, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"(id), "r"((uint32_t)mine)
               : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const Args a, int tiles_a_block, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv) {
  using Ly = Lay<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a head's blocks from the last rows on: those that see most keys come first
  const int head = blockIdx.x % a.HQ;
  grid_wait();
  volatile Work *work = reinterpret_cast<volatile Work *>(smem + Ly::OFF_MISC + 16);
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_MISC);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + Ly::OFF_MISC + 8);
  static_assert(sizeof(Work) <= 48, "room for it");
  const uint32_t bar = sb + Ly::OFF_BAR;
  auto FULL = [&](int i) { return bar + 8 * i; };
  auto EMPTY = [&](int i) { return bar + 8 * (Ly::NS + i); };
  const uint32_t bx = bar + 16 * Ly::NS;
  auto SF = [&](int w) { return bx + 8 * w; };       // S is there
  auto PF = [&](int w) { return bx + 16 + 8 * w; };  // P is there
  auto OD = [&](int w) { return bx + 32 + 8 * w; };  // O is whole
  const uint32_t QF = bx + 48, VR = bx + 56, VZ = bx + 64;  // VR: the last values are there, VZ: and clean behind the keys
  const uint32_t DR = bx + 72;                              // also what the test's wait finds never done
  if (warp == 0) {
    const int R = tiles_a_block * kTile;
    const int64_t slot = slots_of(a.Tq, a.N, R) - 1 - blockIdx.x / a.HQ;
    Tile t;
    const bool on = tile_of(a, slot, R, false, t);
    if (lane == 0) {
      work->on = on;
      if (on) {
        work->q_first = t.rows.first;
        work->k_first = t.keys.first;
        work->keys = t.keys.count;
        work->row0 = t.row0;
        work->past = t.keys.count - t.rows.count;
        for (int w = 0; w < 2; ++w) {
          const int left = t.rows.count - t.row0 - w * kTile, count = w < tiles_a_block ? max(0, min(kTile, left)) : 0;
          const int seen = a.causal ? min(t.keys.count, t.keys.count - t.rows.count + t.row0 + w * kTile + count) : t.keys.count;
          work->count[w] = count;
          work->tiles[w] = count > 0 ? (max(0, seen) + kTile - 1) / kTile : 0;
        }
      }
      for (int i = 0; i < Ly::NS; ++i) { mbar_init(FULL(i), 1); mbar_init(EMPTY(i), 1); }
      for (int w = 0; w < 2; ++w) { mbar_init(SF(w), 1); mbar_init(PF(w), 8); mbar_init(OD(w), 1); }
      mbar_init(QF, 1);
      mbar_init(VR, 1);
      mbar_init(VZ, 1);
      mbar_init(DR, 1);
      mbar_fence_init();
      *failed = 0;
    }
  }
  if (blockIdx.x == 0) check_offsets(a);
  __syncthreads();
  if (!work->on) return;
  if (warp == 17) tmem_alloc(sb + Ly::OFF_MISC + 8, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int wg = warp >> 2, w = wg >> 1, half = wg & 1, r = tid & 127;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
  const uint32_t S_col = tmem + lanes + w * 128 + half * 64, O_col = tmem + lanes + 256 + w * D + half * (D / 2);
  float m_ref = -INFINITY, l_sum = 0.f;
  int issued = 0;  // stages that the producer has filled
  bool q_issued = false;

  // 640 threads x 96 registers at the start: 512 x 104 + 128 x 64
  if (wg < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // -------------------------------------------------------------- softmax
    const int tiles = work->tiles[w], keys = work->keys, row0 = work->row0 + w * kTile;
    const int low = a.causal ? work->past + row0 : keys - 1;  // what the tile's first row sees last
    const int limit = a.causal ? min(low + r, keys - 1) : low;
    volatile float *told = reinterpret_cast<volatile float *>(smem + Ly::OFF_X) + w * 256 + r;
    bool ok = true;
    if (a.force_expiry && !mbar_wait_bounded(DR, 0, gdnc::kTestWaitLimit)) {
      *failed = 1;
      set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
      ok = false;
    }
    for (int j = 0; j < tiles; ++j) {
      if (ok) ok = wait_bar(SF(w), j & 1, failed, a.dev_status);
      tc_fence_after();
      uint32_t s[64];
      load64(S_col, s);
      wait64(s);
      const int k0 = j * kTile + half * 64;
      if (k0 + 63 > low || k0 + 63 >= keys) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (k0 + i > limit) s[i] = __float_as_uint(-INFINITY);
      }
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(s[16 * i]);
#pragma unroll
        for (int e = 1; e < 15; e += 2) x[i] = gdnkv::max3(x[i], __uint_as_float(s[16 * i + e]), __uint_as_float(s[16 * i + e + 1]));
        x[i] = fmaxf(x[i], __uint_as_float(s[16 * i + 15]));
      }
      float top = fmaxf(gdnkv::max3(x[0], x[1], x[2]), x[3]) * a.scale_log2e;
      // (of -inf both, NaN: no.  A wait that gave up votes too, so that all leave together.)
      if (vote_any(1 + w, top - m_ref > kMost || !ok)) {
        told[half * 128] = top;
        if (vote_any(1 + w, !ok)) break;
        top = fmaxf(top, told[(half ^ 1) * 128]);
        float grow = 1.f;
        if (top - m_ref > kMost) {
          grow = ex2f(m_ref - top);
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
      const float ref = m_ref == -INFINITY ? 0.f : m_ref;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float2 t = gdnkv::fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), a.scale_log2e, -ref);
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
    if (ok && !*failed && tiles > 0) wait_bar(OD(w), 0, failed, a.dev_status);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int tiles0 = work->tiles[0], tiles1 = work->tiles[1], tiles = max(tiles0, tiles1), keys = work->keys;
    const int tail = keys % kTile;  // keys of a last tile that is not full
    const bool clear = tail != 0 && tiles * kTile > keys;
    if (warp == 16) {
      // ----------------------------------------------------------- producer
      if (tiles > 0 && elect_one()) {
        const int row = work->q_first + work->row0, key = work->k_first, hk = head / a.G;
        q_issued = true;
        mbar_arrive_expect_tx(QF, (tiles0 > 0 && tiles1 > 0 ? 2 : 1) * Ly::TB);
        if (tiles0 > 0) load_tile<D>(sb + Ly::OFF_Q, &mq, QF, head, row);
        if (tiles1 > 0) load_tile<D>(sb + Ly::OFF_Q + Ly::TB, &mq, QF, head, row + kTile);
        for (int i = 0; i < 2 * tiles; ++i) {
          const int st = i % Ly::NS;
          if (i >= Ly::NS && !wait_bar(EMPTY(st), (i / Ly::NS - 1) & 1, failed, a.dev_status)) break;
          mbar_arrive_expect_tx(FULL(st), Ly::TB);
          load_tile<D>(sb + Ly::OFF_KV + st * Ly::TB, (i & 1) ? &mv : &mk, FULL(st), hk, key + (i >> 1) * kTile);
          issued = i + 1;
        }
        if (*failed) {  // copies in flight
          bool ok = mbar_wait_bounded(QF, 0, gdnc::kWaitLimit);
          for (int i = 0; i < Ly::NS && i < issued; ++i)
            ok &= mbar_wait_bounded(FULL(i), ((issued - 1 - i) / Ly::NS) & 1, gdnc::kWaitLimit);
          if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
        }
      }
    } else if (warp == 18) {
      // P is 0 past the sequence's keys, but 0 times what stands there need not be
      if (clear) {
        // (no limit of its own: the products' warp gets there, or gives up and says so)
        bool there = true;
        while (there && !mbar_try_wait(VR, 0)) there = !*failed;
        if (__all_sync(0xffffffffu, there)) {
          zero_rows<D>(sb + Ly::OFF_KV + (2 * tiles - 1) % Ly::NS * Ly::TB, tail);
          if (lane == 0) mbar_arrive(VZ);
        }
      }
    } else if (warp == 17) {
      // ----------------------------------------------------------- products
      if (tiles > 0 && elect_one()) {
        auto stage = [&](int i) { return sb + Ly::OFF_KV + (i % Ly::NS) * Ly::TB; };
        auto here = [&](int i) { return wait_bar(FULL(i % Ly::NS), (i / Ly::NS) & 1, failed, a.dev_status); };
        // the row tiles that take part in key tile j: the first, the last
        auto first = [&](int j) { return j < tiles0 ? 0 : 1; };
        auto last = [&](int j) { return j < tiles1 ? 1 : 0; };
        auto logits = [&](int x, int j) {
          if (x == first(j)) {
            if (!here(2 * j)) return false;
            tc_fence_after();
          }
          mma_rows<D>(tmem + x * 128, sb + Ly::OFF_Q + x * Ly::TB, stage(2 * j));
          umma_commit(SF(x));
          if (x == last(j)) umma_commit(EMPTY(2 * j % Ly::NS));
          return true;
        };
        bool ok = wait_bar(QF, 0, failed, a.dev_status);
        for (int x = 0; x < 2; ++x)
          if (ok && work->tiles[x] > 0) ok = logits(x, 0);
        for (int j = 0; ok && j < tiles; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int mine = x ? tiles1 : tiles0;
            if (!ok || j >= mine) continue;
            ok = wait_bar(PF(x), j & 1, failed, a.dev_status);
            if (ok && x == first(j)) {
              ok = here(2 * j + 1);
              if (ok && clear && j == tiles - 1) {
                mbar_arrive(VR);
                ok = wait_bar(VZ, 0, failed, a.dev_status);
              }
            }
            if (!ok) break;
            tc_fence_after();
            mma_cols<D>(tmem + 256 + x * D, tmem + x * 128, stage(2 * j + 1), j > 0);
            if (x == last(j)) umma_commit(EMPTY((2 * j + 1) % Ly::NS));
            if (j + 1 < mine) ok = logits(x, j + 1);
            else umma_commit(OD(x));
          }
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
  if (wg < 4 && !*failed) {
    // ---------------------------------------------------------------- output
    tc_fence_after();
    const int count = work->count[w], tiles = work->tiles[w];
    volatile float *told = reinterpret_cast<volatile float *>(smem + Ly::OFF_X) + w * 256 + r;
    told[half * 128] = l_sum;
    named_bar_sync(1 + w, 256);
    const float l = told[0] + told[128], inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = (int64_t)(work->q_first + work->row0 + w * kTile + r) * a.HQ + head;
#pragma unroll 1
    for (int i = 0; i < D / 2; i += 32) {
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld32_issue(O_col + i, o);
        tmem_ld_wait(o);
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = tiles > 0 && l != 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
      if (r < count) {
        uint16_t *dst = a.o + at * D + half * (D / 2) + i;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4 *>(dst + e) =
              make_uint4(pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                         pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])), pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
      }
    }
    if (r < count && half == 0) a.lse[at] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
    tc_fence_before();
  }
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
  const cudaError_t e = gdn_host::allow_smem(attn_fwd_kernel<D>, Lay<D>::BYTES, done);
  if (e != cudaSuccess) return e;
  // the warps' shares of the registers are those of a launch with 96 a thread
  static const bool shares = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, attn_fwd_kernel<D>) == cudaSuccess && f.numRegs == 96;
  }();
  if (!shares) return cudaErrorInvalidConfiguration;
  const int each = slots_of(a.Tq, a.N, 2 * kTile) * a.HQ >= gdn_host::sm_count() ? 2 : 1;
  const int64_t blocks = slots_of(a.Tq, a.N, each * kTile) * a.HQ;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
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
