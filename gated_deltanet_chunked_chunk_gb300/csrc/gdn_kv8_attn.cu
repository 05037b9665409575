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
// with m_i the running maximum of t less 13.  So p' is at most 2^13 whatever the
// scales are, codes enter the products as they are (e4m3 is exact in f16), and o =
// O / l, logsumexp = (m + log2 l) ln 2.  Maxima, sums and accumulators are fp32.
// p' rounds to f16: 11 bits down to 2^-27 of the row's largest weight, steps of
// 2^-37 of it below that (p' of at most 1 would lose all weights under 2^-25).  q,
// brought to a largest magnitude of 1 to 2 by a power of two for each row, loses
// nothing there (bf16 has 8 bits) but elements under 2^-24 of the row's largest.
//
// Bound: HBM, 2 D bytes for each (token, kv head), read once for all the query
// rows of the head's group.
//
// Work.  The contexts of all (request, kv head) pairs, cut into stages of 64
// keys, form one line of stages; a team, one warp (rows are (token, head of
// the group) pairs, 8 NT of them), takes a stretch of it, all teams stretches of
// the same length, so ragged contexts balance by themselves.  A team that meets
// a whole pair writes its output; of a pair that several teams share each writes
// a partial result (two a team at most), and a second kernel joins them in
// order.  A team finds its place by a prefix sum over the requests.
// Every team has K and V tiles of its own in shared memory, 100 to 200 KB on a
// SM: the next K tile is called (TMA, swizzled) as soon as the products with
// the present one are done, the next V tile likewise, and other warps compute
// meanwhile.
//
// Fragments (mma.sync m16n8k16, f16).  The products are taken transposed, S^T =
// K Q^T and O^T = V^T P^T, so that keys and columns fill the 16 rows of a tile
// and 8 query rows its 8 columns: a group of 8 heads wastes nothing, and the
// widening of a code, which is what most instructions do, serves all of a
// warp's rows.  (With the rows as the 16 of a tile: 1140 instructions a stage,
// 202 us for 256 ragged contexts; an e4m3 mma.sync is taken apart into
// conversions and f16 products on this GPU: 1630, 246 us.)  Thread (g, t) =
// (lane / 4, lane % 4) holds for keys g and g + 8 of a tile the 16-byte chunks
// t, t + 4, .. of their rows; the order of d inside a product is free as long as
// Q has the same, so no byte moves.  Keys of 8 are taken in the order 0 4 1 5 2
// 6 3 7: then the 8 lanes that read shared memory together hit 8 different
// 16-byte places.  P's 8 x 8 blocks are transposed by movmatrix; for V^T a byte
// permutation pairs the two keys of a thread for each d.
// mma.sync rather than tcgen05: up to 16 rows the products take less time than
// their bytes do.  17 to 32 rows, where they do not, are gdn_kv8_rows.cu's, more are
// gdn_kv8_prefill.cu's (40 rows: two warps a team took 270 us
// where that takes 209 for 4 requests of 131072 keys, and 22 against 27 for one of 4096).
#include "gdn_kv8_attn.cuh"

namespace {

using namespace gdn;
using namespace gdnkv;

constexpr int kKeys = 64;         // keys a stage
constexpr float kLift = 13.f;     // exponent of a row's largest weight

// D: head size; NT: tiles of 8 rows a team.
template <int D, int NT>
struct DecodeLay {
  static constexpr int TILE = kKeys * D;                // bytes of a K or V tile
  static constexpr int R = D == 128 ? 1 : 2;            // tiles of K, and of V, that a team holds
  static constexpr int PER_SM = 12;                     // teams on a SM (168 registers a thread)
  static constexpr int TEAMS = PER_SM * kSMs;
  static constexpr int ROWS = 8 * NT;                   // rows a team
  static constexpr int KP = NT == 1 ? 64 : 32;          // keys a pass
  static constexpr int OFF_K = 0, OFF_V = R * TILE;
  static constexpr int OFF_PAR = 2 * R * TILE;          // float4 {k scale, lv, 2^-lv, 0} x 4 pages, R + 1 slots
  static constexpr int OFF_BAR = OFF_PAR + (R + 1) * 64;
  static constexpr int OFF_AHEAD = OFF_BAR + (2 * R + 1) * 8 + 8;
  static constexpr int BYTES = OFF_AHEAD + 48;
  static_assert((BYTES + 1024) * PER_SM <= 228 * 1024, "all teams of a SM fit");
};
// Partial rows of all teams, two results a team, of the largest variant.
constexpr int64_t kPartRows = (int64_t)kSMs * 2 * 12 * 16;

__device__ __forceinline__ void mma_f16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8 x 8 block of f16 that the warp holds (row lane / 4, columns 2 (lane % 4),
// + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
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
// Over the lanes of one t (the keys of a query row).
__device__ __forceinline__ float keys_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float keys_add(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows as TMA
// leaves it (128-byte swizzle for D = 128, 64-byte swizzle for D = 64).
template <int D> __device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t c) {
  return D == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <int D, int NT>
__global__ void __launch_bounds__(32, DecodeLay<D, NT>::PER_SM)
    kv8_decode_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Ly = DecodeLay<D, NT>;
  constexpr int R = Ly::R;
  constexpr int NCH = D / 64;       // 16-byte chunks of a key row that a thread holds
  constexpr int NA = D / 16;        // tiles of 16 columns of O
  constexpr int NK = Ly::KP / 16;   // tiles of 16 keys a pass
  constexpr int WPK = D / 32;       // words of a value row that a thread holds
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const int lane = threadIdx.x, team = blockIdx.x;

  const uint32_t bar = sb + Ly::OFF_BAR, never = bar + 16 * R;
  volatile int *failed = reinterpret_cast<volatile int *>(smem + Ly::OFF_BAR + (2 * R + 1) * 8);
  auto KF = [&](int i) { return bar + 8 * i; };
  auto VF = [&](int i) { return bar + 8 * (R + i); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * R + 1; ++i) mbar_init(bar + 8 * i, 1);
    mbar_fence_init();
    *failed = 0;
  }
  __syncwarp();
  grid_wait();
  // Only now: the joining kernel reads lengths and offsets before its own wait.
  grid_release();

  Place at{};
  const int left_all = find_place(a, team, Ly::TEAMS, true, at);
  if (left_all == 0) return;
  int left = left_all;  // stages of this team still to do

  // -------------------------------------------------------------- calling
  // Warp 0 runs R stages ahead of the products: `ahead` is its place, `to_call`
  // the stages it has still to call.  Table entries and scales are read 32
  // pages at a time, a page a lane.  A page that is not there counts as keys
  // that nothing sees (logits of -inf) and reads zeros.
  // The place is kept in shared memory: the products need the registers.
  // The first pair's queries are read meanwhile.
  const int g = lane >> 2, t = lane & 3;
  uint4 qraw[NT][2 * NCH];
  auto read_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g;
      const uint16_t *src = a.q + (int64_t)(at.s.t0 + row / a.G) * a.ldq + (int64_t)(at.h * a.G + row % a.G) * D;
#pragma unroll
      for (int i = 0; i < 2 * NCH; ++i)
        qraw[nt][i] = row < at.s.m * a.G ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * (t + 4 * (i >> 1))) + (i & 1))
                                         : make_uint4(0, 0, 0, 0);
    }
  };
  if (NT == 1) read_q();
  Place &ahead = *reinterpret_cast<Place *>(smem + Ly::OFF_AHEAD);
  static_assert(sizeof(Place) <= 48, "room for the place");
  int to_call = left;
  int called = 0, called_k = 0;  // stages called so far; their K tiles
  int batch = -1, page = -1;
  float ks = 0.f, lv = 0.f, iv = 1.f;
  int zc = 0, yc = 0;  // the called stage's coordinates
  const int ppt = a.bs >= kKeys ? 1 : kKeys / a.bs;  // copies a tile
  const int box = kKeys / ppt;                       // keys a copy
  const int page_bits = 31 - __clz(a.bs);
  auto call_k = [&]() {
    if (to_call == 0 || *failed) return;
    const int stage = ahead.stage, head = ahead.h;
    const int first = (stage * kKeys) >> page_bits;
    const bool fresh = first / 32 != batch;
    float vs = 0.f;
    if (fresh) {
      batch = first / 32;
      const int pi = batch * 32 + lane;
      page = -1;
      if (((int64_t)pi << page_bits) < ahead.s.keys) {
        page = a.table[(int64_t)ahead.n * a.width + pi];
        if (page < 0 || page >= a.P) {
          set_status(a.dev_status, GDN_DEV_BAD_SLOT);
          page = -1;
        }
      }
      ks = 0.f;
      if (page >= 0) {
        const int64_t i = (int64_t)page * a.HK + head;
        ks = a.ks[i];
        vs = a.vs[i];
      }
    }
    const int src = (first - batch * 32 + (lane & (ppt - 1))) & 31;
    const int pg = __shfl_sync(0xffffffffu, page, src);
    zc = pg >= 0 ? pg * a.HK + head : a.P * a.HK;  // outside the tensor: TMA fills in zeros
    yc = (stage * kKeys) & (a.bs - 1);
    // The tile is called before the scales are looked at, whose reads are on
    // their way too; the arrival, which makes the constants visible, comes last.
    const int slot = called % R;
    if (lane == 0) mbar_expect_tx(KF(slot), Ly::TILE);
    __syncwarp();
    if (lane < ppt) tma_load_3d(sb + Ly::OFF_K + slot * Ly::TILE + lane * box * D, &mk, KF(slot), 0, yc, zc);
    ++called_k;
    if (fresh) {  // a page that is not there: -inf
      lv = log2f(vs);
      iv = vs > 0.f ? 1.f / vs : 1.f;
    }
    const float4 par = make_float4(__shfl_sync(0xffffffffu, ks, src), __shfl_sync(0xffffffffu, lv, src),
                                   __shfl_sync(0xffffffffu, iv, src), 0.f);
    if (lane < ppt) *reinterpret_cast<float4 *>(smem + Ly::OFF_PAR + (called % (R + 1)) * 64 + lane * 16) = par;
    __syncwarp();
    if (lane == 0) mbar_arrive(KF(slot));
    // on to the next stage
    if (stage + 1 < ahead.of) {
      __syncwarp();
      if (lane == 0) ahead.stage = stage + 1;
    } else {
      Place p = ahead;
      p.stage = 0;
      batch = -1;
      if (++p.h == a.HK && to_call > 1) next_request(a, p);
      __syncwarp();
      if (lane == 0) ahead = p;
    }
    __syncwarp();
  };
  auto call_v = [&]() {  // the V tile of the stage that call_k has just called
    if (to_call == 0 || *failed) return;
    const int slot = called % R;
    if (lane == 0) mbar_arrive_expect_tx(VF(slot), Ly::TILE);
    __syncwarp();
    if (lane < ppt) tma_load_3d(sb + Ly::OFF_V + slot * Ly::TILE + lane * box * D, &mv, VF(slot), 0, yc, zc);
    ++called;
    --to_call;
  };
  if (lane == 0) ahead = at;
  __syncwarp();
  for (int i = 0; i < R; ++i) {
    call_k();
    call_v();
  }

  const int kperm = (g >> 1) | ((g & 1) << 2);  // row of key g of 8
  const uint32_t sel0 = (g & 1) ? 0x1504u : 0x5140u, sel1 = (g & 1) ? 0x3726u : 0x7362u;
  const int va = t + 4 * (g & 1), vb = t + 4 * ((g & 1) ^ 1);
  int done = 0;  // stages that the products have used

  while (left > 0) {
    // ---------------------------------------------- one pair's stretch
    const Span s = at.s;
    const int h = at.h, L = s.L, m = s.m;
    const bool from_start = at.stage == 0, to_end = left >= at.of - at.stage;
    const int count = to_end ? at.of - at.stage : left;
    // Queries: row 8 nt + g; thread t holds d = 16 (t + 4 i) + 0..15,
    // k-step 4 i + w taking 4 w + {0, 1 | 2, 3} of them.
    uint32_t qf[4 * NCH][NT][2];
    float krow[NT][2];  // of rows 8 nt + 2 t + e
    if (NT > 1 || done > 0) read_q();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 *u = qraw[nt];
      float top = 0.f, bad = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * NCH; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = bf16lo_f(w[e]), y = bf16hi_f(w[e]);
          top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
          bad = fmaf(x, 0.f, fmaf(y, 0.f, bad));  // NaN once an element is not finite
        }
      }
      top = quad_max(top);
      bad = quad_add(bad);
      int e2 = (int)(__float_as_uint(top) >> 23) - 127;
      e2 = e2 < -100 ? -100 : e2 > 120 ? 120 : e2;
      const float down = pow2(-e2), kr = pow2(e2) * a.scale_log2e + bad;
      krow[nt][0] = __shfl_sync(0xffffffffu, kr, 8 * t);
      krow[nt][1] = __shfl_sync(0xffffffffu, kr, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < 2 * NCH; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = pack_f16(bf16lo_f(w[e]) * down, bf16hi_f(w[e]) * down);
        qf[2 * i][nt][0] = f[0];
        qf[2 * i][nt][1] = f[1];
        qf[2 * i + 1][nt][0] = f[2];
        qf[2 * i + 1][nt][1] = f[3];
      }
    }
    const int low = L - m;  // what the first row sees last
    // O^T: tile x, row tile nt: columns 2 NA.. of this thread g are d = NA g .. ;
    // o[x][nt][e + 2 f] is d = 2 NA g + 2 x + f (NA = D / 16) of row 2 t + e.
    float o[NA][NT][4];
    float mx[NT][2], ls[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt][0] = mx[nt][1] = -INFINITY;
      ls[nt][0] = ls[nt][1] = 0.f;
#pragma unroll
      for (int x = 0; x < NA; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][nt][e] = 0.f;
    }

    for (int it = 0; it < count; ++it, ++done) {
      const int slot = done % R, phase = (done / R) & 1;
      const int k0 = (at.stage + it) * kKeys;
      if (!*failed) {
        bool ok = true;
        if (a.force_expiry) ok = mbar_wait_bounded(never, 0, gdnc::kTestWaitLimit);
        if (ok) ok = mbar_wait_bounded(KF(slot), phase, gdnc::kWaitLimit);
        if (!ok) {
          set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
          *failed = 1;
        }
      }
      const uint32_t kt = sb + Ly::OFF_K + slot * Ly::TILE, vt = sb + Ly::OFF_V + slot * Ly::TILE;
      const uint32_t par = sb + Ly::OFF_PAR + (done % (R + 1)) * 64;
      const bool masked = k0 + kKeys - 1 > low;
      uint32_t nan_seen = 0;
#pragma unroll 1
      for (int pass = 0; pass < kKeys / Ly::KP; ++pass) {
        const int kp = pass * Ly::KP;
        float p[NK][NT][4];
#pragma unroll
        for (int x = 0; x < NK; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) p[x][nt][0] = p[x][nt][1] = p[x][nt][2] = p[x][nt][3] = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          uint32_t kw[NK][2][4];
#pragma unroll
          for (int x = 0; x < NK; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4 u = lds128(kt + tile_at<D>(kp + 16 * x + 8 * r + kperm, t + 4 * i));
              kw[x][r][0] = u.x; kw[x][r][1] = u.y; kw[x][r][2] = u.z; kw[x][r][3] = u.w;
            }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int x = 0; x < NK; ++x) {
              uint32_t f[4];
              e4m3x4_f16x2(kw[x][0][w], f[0], f[2]);
              e4m3x4_f16x2(kw[x][1][w], f[1], f[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(p[x][nt], f, qf[4 * i + w][nt][0], qf[4 * i + w][nt][1]);
            }
          }
        }
        if (pass == kKeys / Ly::KP - 1) {
          __syncwarp();  // the K tile is free
          call_k();
        }

        float top[NT][2], iv_of[NK];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
        for (int x = 0; x < NK; ++x) {  // a page holds 16 keys at least
          const float4 f = lds_f4(par + ((a.bs >= kKeys ? 0 : kp + 16 * x) >> page_bits) * 16);
          iv_of[x] = f.z;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float c = krow[nt][e] * f.x;
              p[x][nt][e] = fmaf(p[x][nt][e], c, f.y);
              p[x][nt][2 + e] = fmaf(p[x][nt][2 + e], c, f.y);
            }
        }
        if (masked) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = 8 * nt + 2 * t + e;
              const int limit = row < m * a.G ? L - m + row / a.G : -1;
#pragma unroll
              for (int x = 0; x < NK; ++x) {
                if (k0 + kp + 16 * x + kperm > limit) p[x][nt][e] = -INFINITY;
                if (k0 + kp + 16 * x + 8 + kperm > limit) p[x][nt][2 + e] = -INFINITY;
              }
            }
        }
        float base[NT][2], down[NT][2];
        bool moved = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x0 = -INFINITY;
#pragma unroll
            for (int x = 0; x < NK; ++x) x0 = fmaxf(x0, fmaxf(p[x][nt][e], p[x][nt][2 + e]));
            const float now = fmaxf(mx[nt][e], reference_of(keys_max(x0), kLift));
            base[nt][e] = now == -INFINITY ? 0.f : now;
            down[nt][e] = ex2f(mx[nt][e] - base[nt][e]);
            moved |= now != mx[nt][e];
            mx[nt][e] = now;
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            ls[nt][0] *= down[nt][0];
            ls[nt][1] *= down[nt][1];
#pragma unroll
            for (int x = 0; x < NA; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[x][nt][e] *= down[nt][e & 1];
          }
        }
        uint32_t pb[NK][NT][2];
#pragma unroll
        for (int x = 0; x < NK; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[x][nt][e] = ex2f(p[x][nt][e] - base[nt][e & 1]);
            ls[nt][0] = fmaf(p[x][nt][0] + p[x][nt][2], iv_of[x], ls[nt][0]);
            ls[nt][1] = fmaf(p[x][nt][1] + p[x][nt][3], iv_of[x], ls[nt][1]);
            pb[x][nt][0] = transpose8(pack_f16(p[x][nt][0], p[x][nt][1]));
            pb[x][nt][1] = transpose8(pack_f16(p[x][nt][2], p[x][nt][3]));
          }

        if (pass == 0 && !*failed && !mbar_wait_bounded(VF(slot), phase, gdnc::kWaitLimit)) {
          set_status(a.dev_status, GDN_DEV_WAIT_TIMEOUT);
          *failed = 1;
        }
#pragma unroll
        for (int x = 0; x < NK; ++x) {
          uint32_t wa[2][WPK], wb[2][WPK];  // keys of 8: this thread's two, WPK words of each
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = kp + 16 * x + 8 * r;
            if (D == 128) {
              const uint4 u = lds128(vt + tile_at<D>(j + va, g)), w = lds128(vt + tile_at<D>(j + vb, g));
              wa[r][0] = u.x; wa[r][1] = u.y; wa[r][WPK / 2] = u.z; wa[r][WPK - 1] = u.w;
              wb[r][0] = w.x; wb[r][1] = w.y; wb[r][WPK / 2] = w.z; wb[r][WPK - 1] = w.w;
            } else {
              const uint2 u = lds64(vt + tile_at<D>(j + va, g >> 1) + 8 * (g & 1));
              const uint2 w = lds64(vt + tile_at<D>(j + vb, g >> 1) + 8 * (g & 1));
              wa[r][0] = u.x; wa[r][1] = u.y;
              wb[r][0] = w.x; wb[r][1] = w.y;
            }
          }
          if (masked) {
            // Keys past the context hold whatever the page held before, and a
            // key that only later rows see may be NaN: p' is 0 there, but
            // 0 x NaN is not.  Such codes become 0; NaN that a row does see is
            // put back below.
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int j = k0 + kp + 16 * x + 8 * r;
#pragma unroll
              for (int y = 0; y < WPK; ++y) {
                if (j + va >= L) wa[r][y] = 0;
                if (j + vb >= L) wb[r][y] = 0;
                nan_seen |= any_nan(wa[r][y]) | any_nan(wb[r][y]);
                wa[r][y] = drop_nan(wa[r][y]);
                wb[r][y] = drop_nan(wb[r][y]);
              }
            }
          }
#pragma unroll
          for (int y = 0; y < WPK; ++y) {
            uint32_t f[4];
            e4m3x4_f16x2(__byte_perm(wa[0][y], wb[0][y], sel0), f[0], f[1]);
            e4m3x4_f16x2(__byte_perm(wa[1][y], wb[1][y], sel0), f[2], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * y][nt], f, pb[x][nt][0], pb[x][nt][1]);
            e4m3x4_f16x2(__byte_perm(wa[0][y], wb[0][y], sel1), f[0], f[1]);
            e4m3x4_f16x2(__byte_perm(wa[1][y], wb[1][y], sel1), f[2], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * y + 1][nt], f, pb[x][nt][0], pb[x][nt][1]);
          }
        }
      }
      if (masked && __any_sync(0xffffffffu, nan_seen != 0)) {
        const unsigned char *v = smem + Ly::OFF_V + slot * Ly::TILE;
#pragma unroll 1
        for (int key = 0; key < kKeys && k0 + key < L; ++key)
#pragma unroll
          for (int x = 0; x < 2 * NA; ++x) {
            const int d = 2 * NA * g + x;
            if ((v[tile_at<D>(key, d >> 4) + (d & 15)] & 0x7f) != 0x7f) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (k0 + key <= L - m + (8 * nt + 2 * t + e) / a.G) o[x >> 1][nt][e + 2 * (x & 1)] = NAN;
          }
      }
      __syncwarp();  // the V tile is free
      call_v();
    }

    // ------------------------------------------------ the stretch's result
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float l = keys_add(ls[nt][e]);
        const int row = 8 * nt + 2 * t + e;
        if (row >= m * a.G || *failed) continue;
        if (from_start && to_end) {
          const int64_t out = (int64_t)(s.t0 + row / a.G) * a.HQ + h * a.G + row % a.G;
          const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing is 0
#pragma unroll
          for (int x = 0; x < NA; x += 4)
            *reinterpret_cast<uint4 *>(a.o + out * D + 2 * NA * g + 2 * x) =
                make_uint4(pack_bf16(o[x][nt][e] * inv, o[x][nt][e + 2] * inv), pack_bf16(o[x + 1][nt][e] * inv, o[x + 1][nt][e + 2] * inv),
                           pack_bf16(o[x + 2][nt][e] * inv, o[x + 2][nt][e + 2] * inv),
                           pack_bf16(o[x + 3][nt][e] * inv, o[x + 3][nt][e + 2] * inv));
          if (a.lse && g == 0) a.lse[out] = l == 0.f ? -INFINITY : (mx[nt][e] + log2f(l)) * kLn2;
        } else {
          // the pair began before this team's stretch: slot 0, else slot 1
          const int64_t part = ((int64_t)team * 2 + (from_start ? 1 : 0)) * a.row_cap + row;
#pragma unroll
          for (int x = 0; x < NA; x += 2)
            *reinterpret_cast<float4 *>(a.part_o + part * D + 2 * NA * g + 2 * x) =
                make_float4(o[x][nt][e], o[x][nt][e + 2], o[x + 1][nt][e], o[x + 1][nt][e + 2]);
          if (g == 0) a.part_ml[part] = make_float2(mx[nt][e], l);
        }
      }
    left -= count;
    at.stage = 0;
    if (left > 0 && ++at.h == a.HK) next_request(a, at);
  }

  if (*failed && lane == 0) {
    // A wait ran out, nothing was written since; stay until the copies are in.
    bool ok = true;
    for (int i = 0; i < R && i < called_k; ++i) ok &= mbar_wait_bounded(KF(i), ((called_k - 1 - i) / R) & 1, gdnc::kWaitLimit);
    for (int i = 0; i < R && i < called; ++i) ok &= mbar_wait_bounded(VF(i), ((called - 1 - i) / R) & 1, gdnc::kWaitLimit);
    if (!ok) set_status(a.dev_status, GDN_DEV_DRAIN_TIMEOUT);
  }
}

// Joins the partial results of a pair's rows, in order.  W > 1: block x of a pair
// takes row x, each of its W warps a share of the pieces (calls with few
// pairs, which are cut into many pieces each); else rows 4 x .. 4 x + 3, a warp
// each.  A lane reads the maximum and sum of one piece, 32 at a time; D / 4
// lanes hold four columns each.  Latency counts here: three dependent reads.
template <int D, int W>
__global__ void __launch_bounds__(W > 1 ? 32 * W : 128) kv8_join_kernel(const AttnArgs a, int teams) {
  constexpr int LANES = D / 4;
  constexpr bool WIDE = W > 1;
  __shared__ float4 so[W][LANES];
  __shared__ float2 sml[W];
  const int n = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = WIDE ? blockIdx.x : 4 * blockIdx.x + warp;
  // A dependent launch that the decode kernel, which has waited for what came
  // before, lets in: lengths and offsets may be read before the wait.
  grid_release();
  Span s;
  const int of = stages_of(a, n, s);
  // The request's place on the line: from the decode kernel, or, where the
  // requests are few, formed here while that kernel still runs.
  int64_t total = 0, place = 0;
  if (a.N <= 32) {
    Span other;
    for (int i = lane; i < a.N; i += 32) {
      const int64_t c = (int64_t)stages_of(a, i, other) * a.HK;
      total += c;
      if (i < n) place += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      place += __shfl_xor_sync(0xffffffffu, place, o);
    }
  }
  grid_wait();
  if (of == 0 || row >= s.m * a.G) return;
  if (a.N > 32) {
    total = a.place[a.N];
    place = a.place[n];
  }
  const int64_t per = stretch_of(total, teams);
  const int64_t from = place + (int64_t)h * of, first = from / per, last = (from + of - 1) / per;
  const int pieces = (int)(last - first) + 1;
  if (pieces == 1) return;
  const int share = (pieces + W - 1) / W;
  const int i0 = WIDE ? warp * share : 0, i1 = min(pieces, i0 + share);
  const int c = lane % LANES;
  // piece 0 is its team's slot 1, the others their teams' slot 0
  auto at = [&](int i) { return ((first + i) * 2 + (i == 0 ? 1 : 0)) * a.row_cap + row; };
  float top = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b = i0; b < i1; b += 32) {
    const int cnt = min(32, i1 - b);
    const float2 ml = lane < cnt ? a.part_ml[at(b + lane)] : make_float2(-INFINITY, 0.f);
    float now = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
    now = fmaxf(now, top);
    const float base = now == -INFINITY ? 0.f : now;
    const float w = ex2f(ml.x - base), old = ex2f(top - base);
    top = now;
    l = fmaf(l, old, warp_sum(w * ml.y));
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll 8
    for (int i = 0; i < cnt; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(a.part_o + at(b + i) * D + 4 * c);
      const float wi = __shfl_sync(0xffffffffu, w, i);
      acc.x = fmaf(wi, v.x, acc.x);
      acc.y = fmaf(wi, v.y, acc.y);
      acc.z = fmaf(wi, v.z, acc.z);
      acc.w = fmaf(wi, v.w, acc.w);
    }
  }
  if (WIDE) {
    if (lane < LANES) so[warp][c] = acc;
    if (lane == 0) sml[warp] = make_float2(top, l);
    __syncthreads();
    if (warp != 0) return;
    top = -INFINITY;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, sml[i].x);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float w = ex2f(sml[i].x - base);
      const float4 v = so[i][c];
      l = fmaf(w, sml[i].y, l);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  if (lane < LANES) store_row4(a, s.t0 + row / a.G, h * a.G + row % a.G, D, 4 * c, acc, top, l);
}

// ---------------------------------------------------------------- host side
// How a call's requests are worked on, from its host bounds.  Requests of up to
// row_most rows (tokens x heads of a group) go to kv8_decode_kernel, with 8 or 16
// rows a team, or, where 17 to 32 is the most, to kv8_rows_kernel (stages of 128
// keys there), the others to kv8_prefill_kernel.  A call whose bounds allow more
// than 32 rows may mix long and short requests (a serving step that prefills some
// and decodes others): then those of at most 16 rows (32 where the group itself
// is larger than 16) stay with the first kernels, where a long context of few rows
// is split over many teams.
struct DecodePlan {
  int row_cap, row_most;
};
DecodePlan plan_decode(int N, int T, int G, int max_q) {
  DecodePlan p{};
  const int64_t rows = (int64_t)max_q * G;
  if (rows <= 32) p.row_most = (int)rows;
  else if (N == 1 || G > 32) p.row_most = 0;
  else p.row_most = G <= 16 ? 16 : 32;
  // T tokens of N requests, none with more than max_q: where even the shortest
  // possible one has more rows than that, the first kernel is not launched.
  if (rows > 32 && (T - (N - 1) * (int64_t)max_q) * G > p.row_most) p.row_most = 0;
  p.row_cap = p.row_most <= 8 ? 8 : p.row_most <= 16 ? 16 : 32;
  return p;
}

template <int D>
cudaError_t launch_join(const AttnArgs &a, int teams, cudaStream_t s) {
  // Eight pieces a pair, or more; 64 or more take 16 warps (one context of 131072
  // keys, 456 pieces: 36 us against 55; with 28 pieces 59 against 51).
  const int64_t pairs = (int64_t)a.N * a.HK;
  const bool wide = pairs * 8 < teams;
  const dim3 grid(wide ? a.row_most : (a.row_most + 3) / 4, a.HK, a.N);
  if (pairs * 64 < teams) return gdn_host::launch_dependent(kv8_join_kernel<D, 16>, grid, 512, 0, s, a, teams);
  if (wide) return gdn_host::launch_dependent(kv8_join_kernel<D, 4>, grid, 128, 0, s, a, teams);
  return gdn_host::launch_dependent(kv8_join_kernel<D, 1>, grid, 128, 0, s, a, teams);
}
template <int D, int NT>
cudaError_t launch_decode(const AttnArgs &a, cudaStream_t s) {
  using Ly = DecodeLay<D, NT>;
  static_assert((int64_t)Ly::TEAMS * 2 * Ly::ROWS <= kPartRows, "partial results");
  CUtensorMap mk, mv;
  const int keys = a.bs < kKeys ? a.bs : kKeys;
  if (!cache_map(&mk, a.kc, D, a.bs, (int64_t)a.P * a.HK, keys, true) ||
      !cache_map(&mv, a.vc, D, a.bs, (int64_t)a.P * a.HK, keys, true))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = gdn_host::allow_smem(kv8_decode_kernel<D, NT>, Ly::BYTES, done);
  if (e != cudaSuccess) return e;
  if ((e = gdn_host::launch_dependent(kv8_decode_kernel<D, NT>, dim3(Ly::TEAMS), 32, Ly::BYTES, s, a, mk, mv)) != cudaSuccess)
    return e;
  return launch_join<D>(a, Ly::TEAMS, s);
}
template <int D> cudaError_t launch_rows(const AttnArgs &a, cudaStream_t s) {
  if (a.row_cap == 8) return launch_decode<D, 1>(a, s);
  if (a.row_cap == 16) return launch_decode<D, 2>(a, s);
  const cudaError_t e = launch_kv8_rows(a, s);
  return e != cudaSuccess ? e : launch_join<D>(a, kSMs, s);
}

}  // namespace

namespace gdn_host {

namespace {
// Bytes of the decode kernel's part of the workspace, a multiple of 16.
size_t decode_workspace(int N, int D) {
  const size_t bytes = (size_t)kPartRows * (size_t)(D + 2) * sizeof(float) + ((size_t)N + 1) * sizeof(int64_t);
  return (bytes + 15) / 16 * 16;
}
}  // namespace

size_t kv8_attn_workspace_bytes(int N, int T, int G, int D, int max_q) {
  if (N <= 0 || max_q <= 0) return 0;
  const int most = plan_decode(N, T, G, max_q).row_most;
  return (most > 0 ? decode_workspace(N, D) : 0) + ((int64_t)max_q * G > most ? gdnkv::prefill_workspace(D) : 0);
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs &c, cudaStream_t s) {
  AttnArgs a{};
  static_cast<Kv8AttnArgs &>(a) = c;
  a.G = c.HQ / c.HK;
  const DecodePlan p = plan_decode(c.N, c.T, a.G, c.max_q);
  a.scale_log2e = c.scale * gdnc::kLog2e;
  a.row_cap = p.row_cap;
  a.row_most = p.row_most;
  a.stage_bits = p.row_cap == 32 ? 7 : 6;
  unsigned char *ws = static_cast<unsigned char *>(c.ws);
  if (p.row_most > 0) {
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + kPartRows * c.D);
    a.place = reinterpret_cast<int64_t *>(a.part_ml + kPartRows);
    ws += decode_workspace(c.N, c.D);
  }
  if ((int64_t)c.max_q * a.G > p.row_most) {
    gdnkv::prefill_place(a, ws);
    const cudaError_t e = gdnkv::launch_prefill(a, p.row_most + 1, s);
    if (e != cudaSuccess || p.row_most == 0) return e;
  }
  return c.D == 128 ? launch_rows<128>(a, s) : launch_rows<64>(a, s);
}

}  // namespace gdn_host
