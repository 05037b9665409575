// gdn_paged.cu -- the paged 8-bit cache of the attention layers: block tables,
// slot maps and positions from request lengths (plan), and the write of new
// keys and values (append).
#include "gdn_common.cuh"
#include "gdn_kv8.cuh"

namespace {

using gdn::set_status;

// ------------------------------------------------------------------- plan
// Request n holds cached[n] tokens and gets new[n] = cu[n + 1] - cu[n] more.
// It needs ceil((cached + new) / bs) - ceil(cached / bs) further pages; the
// requests take theirs in order from the end of the free list, so page j of
// request n is free[left - 1 - (pages of the requests before n) - j].
//
// The work is a prefix sum over the requests and 8 bytes a token: a few
// microseconds of latency, so it is one launch.  Every block owns 1024 tokens
// (a thread each) and walks over all requests, 1024 at a time: it forms their
// prefix sums in shared memory, and the threads whose token belongs to one of
// them find it there by binary search.  That repeats the scan in each block,
// which costs a block N / 1024 short steps, against a second launch and a
// round trip through memory.  The token that opens a page writes its table
// entry; block 0 writes the lengths.
constexpr int kPlan = 1024;

__global__ void __launch_bounds__(kPlan) paged_plan_kernel(
    const int32_t *__restrict__ cached, const int32_t *__restrict__ cu, int N, int32_t T, int32_t *table, int width,
    const int32_t *__restrict__ free_pages, int F, const int32_t *__restrict__ num_free, int bs, int page_bits,
    int32_t *seq_lens, int32_t *slots, int32_t *positions, int32_t *num_free_out, int32_t *dev_status) {
  __shared__ int32_t s_start[kPlan], s_cached[kPlan], s_before[kPlan], s_end[kPlan];
  __shared__ int32_t s_warp[32];
  gdn::grid_release();
  gdn::grid_wait();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  auto pages_of = [&](uint32_t tokens) {  // below 2^31 tokens
    const uint32_t x = tokens + (uint32_t)bs - 1;
    return page_bits >= 0 ? x >> page_bits : x / (uint32_t)bs;
  };
  const int32_t tok = (int32_t)min((int64_t)blockIdx.x * kPlan + tid, (int64_t)T);
  int left = *num_free;
  left = left < 0 ? 0 : left > F ? F : left;
  int32_t slot = -1, pos = 0, base = 0;
  int bits = 0;
  bool found = false;
  for (int n0 = 0; n0 < N; n0 += kPlan) {
    const int n = n0 + tid, cnt = min(kPlan, N - n0);
    int32_t a = 0, b = 0, c = 0, want = 0;
    bool broken = false;
    if (n < N) {
      a = cu[n];
      b = cu[n + 1];
      c = cached[n];
      broken = a < 0 || b < a || b > T || (n == 0 && a != 0);
      if (broken) a = b = 0;
      if (broken || c < 0 || (int64_t)c + b - a > 2147483647LL) {
        bits |= GDN_DEV_BAD_CU_SEQLENS;
        b = a;
        c = c < 0 ? 0 : c;
      }
      const uint32_t total = (uint32_t)c + (uint32_t)(b - a);  // below 2^31, as checked
      const uint32_t have = pages_of(c);
      uint32_t need = pages_of(total);
      if (need > (uint32_t)width) {
        bits |= GDN_DEV_NO_PAGE;
        need = (uint32_t)width;
      }
      want = need > have ? (int32_t)(need - have) : 0;
      if (blockIdx.x == 0) seq_lens[n] = (int32_t)total;
    }
    // inclusive scan of want over the block
    int32_t x = want;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    s_start[tid] = a;
    s_end[tid] = b;
    s_cached[tid] = c;
    const bool ordered = !__syncthreads_or(broken);
    int32_t sums = s_warp[lane];  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, sums, o);
      if (lane >= o) sums += y;
    }
    const int32_t all = __shfl_sync(0xffffffffu, sums, 31);
    const int32_t add = w == 0 ? 0 : __shfl_sync(0xffffffffu, sums, (w + 31) & 31);
    s_before[tid] = base + add + x - want;
    __syncthreads();
    if (tok < T && !found) {
      // the last request of these that starts at or before the token and is not empty
      int lo = 0, hi = cnt - 1;
      if (ordered) {
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_start[mid] <= tok) lo = mid; else hi = mid - 1;
        }
      } else {
        for (lo = hi; lo > 0 && !(s_start[lo] <= tok && tok < s_end[lo]);) --lo;
      }
      if (s_start[lo] <= tok && tok < s_end[lo]) {
        found = true;
        pos = s_cached[lo] + (tok - s_start[lo]);
        const int pg = (int)(page_bits >= 0 ? (uint32_t)pos >> page_bits : (uint32_t)pos / (uint32_t)bs), off = pos - pg * bs;
        const int have = (int)pages_of(s_cached[lo]);
        int32_t page = -1;
        if (pg < width) {
          int32_t *entry = table + (int64_t)(n0 + lo) * width + pg;
          if (pg < have) {
            page = *entry;
          } else {
            const int32_t at = left - 1 - (s_before[lo] + pg - have);
            if (at >= 0) page = max(free_pages[at], -1);
            if (off == 0) *entry = page;
          }
        }
        if (page >= 0) slot = page * bs + off;
        else bits |= GDN_DEV_NO_PAGE;
      }
    }
    base += all;
    __syncthreads();
  }
  if (tok < T) {
    slots[tok] = slot;
    positions[tok] = pos;
  }
  if (blockIdx.x == 0 && tid == 0) *num_free_out = left - min(base, left);
  if (bits) set_status(dev_status, bits);
}

// ----------------------------------------------------------------- append
// A run is a stretch of consecutive new tokens that go to consecutive places
// of one page.  For a run of one head of K or V: the largest magnitude, the
// exponent e of the page's new scale 2^e, the codes that were there before moved
// to that scale, the new ones written.
//
// The scale is a power of two because then x 2^-e is exact, the only rounding
// is the one to the 8-bit format, and a page whose scale grows keeps its older
// codes' bits as long as they stay normal numbers of the format.
//
// Bound: HBM for a prefill (2 bytes read, 1 written an element), latency for a
// decode step.  Runs are found with ballots over 32 slots.  Where tokens are
// many (windows of a page's length), a block of four warps takes the runs that
// begin in a window and keeps a run's values in registers between the maximum
// and the rounding (reading them twice: 104 us for 65536 tokens of 4 heads,
// against 38, 5.2 TB/s).  Where they are few, a warp takes the run, if any, that
// begins with its token, and reads the values twice.
struct AppendArgs {
  const uint16_t *k, *v;
  int64_t ldk, ldv;
  uint8_t *kc, *vc;
  float *ks, *vs;
  const int32_t *slots;
  int64_t T;
  int P, HK, D, bs, window;
  int page_bits;  // log2(bs), or -1
  int32_t *dev_status;
};
__device__ __forceinline__ int page_of(const AppendArgs &a, int32_t slot) { return a.page_bits >= 0 ? slot >> a.page_bits : slot / a.bs; }
__device__ __forceinline__ int place_of(const AppendArgs &a, int32_t slot) {
  return a.page_bits >= 0 ? slot & (a.bs - 1) : slot % a.bs;
}

// Place of token t, or -1 (PAD, a slot outside the cache, no token).
__device__ __forceinline__ int32_t slot_of(const AppendArgs &a, int64_t t, int &bits) {
  if (t < 0 || t >= a.T) return -1;
  const int32_t s = a.slots[t];
  if (s >= 0 && page_of(a, s) < a.P) return s;
  if (s != -1) bits |= GDN_DEV_BAD_SLOT;
  return -1;
}
// For every lane's token t, whose place is s: the place of the last token before it
// that has one, of those up to 32 before the warp's first; -1: none has.
__device__ __forceinline__ int32_t last_before(const AppendArgs &a, int64_t t, int32_t s) {
  const int lane = threadIdx.x & 31;
  int ignore = 0;
  const int32_t behind = slot_of(a, t - 32, ignore);
  const uint32_t here = __ballot_sync(0xffffffffu, s >= 0) & ((1u << lane) - 1), there = __ballot_sync(0xffffffffu, behind >= 0);
  const int32_t near = __shfl_sync(0xffffffffu, s, here ? 31 - __clz((int)here) : 0);
  const int32_t far = __shfl_sync(0xffffffffu, behind, there ? 31 - __clz((int)there) : 0);
  return here ? near : far;
}
__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x <= 3.402823466e38f ? x : 0.f;  // infinities and NaN do not set a scale
}
// Largest finite magnitude of two bf16, given their bits.
__device__ __forceinline__ float amax2(uint32_t u) {
  return fmaxf(finite_abs(__uint_as_float(u << 16)), finite_abs(__uint_as_float(u & 0xffff0000u)));
}
__device__ __forceinline__ uint32_t codes2(uint32_t u, float inv) {
  const float2 x = gdn::f2_get(gdn::f2_mul(gdn::f2_bf16(u), gdn::f2_both(inv)));
  return gdnkv::cvt_e4m3x2(x.x, x.y);
}

// WARPS warps write a run of n tokens from t0 to places from `slot` on.  NV > 0:
// a thread holds up to NV units of 16 elements (NV * 32 * WARPS units hold a
// page; D / 16 divides 32 WARPS); NV = 0: values read twice, in units of 16 with
// VEC, else element by element (any D and alignment).
template <int WARPS, int NV, bool VEC>
__device__ __forceinline__ void write_run(const AppendArgs &a, int kv, int h, int64_t t0, int n, int32_t slot, float *sh) {
  constexpr int TH = 32 * WARPS;
  const int tid = WARPS > 1 ? (int)threadIdx.x : (int)(threadIdx.x & 31);
  const int page = page_of(a, slot), off = place_of(a, slot);
  const int64_t ld = kv ? a.ldv : a.ldk;
  const uint16_t *x = (kv ? a.v : a.k) + t0 * ld + (int64_t)h * a.D;
  uint8_t *codes = (kv ? a.vc : a.kc) + ((int64_t)page * a.HK + h) * (int64_t)a.bs * a.D;
  float *scale = (kv ? a.vs : a.ks) + (int64_t)page * a.HK + h;
  const float before = off > 0 ? *scale : 0.f;
  uint8_t *dst = codes + (int64_t)off * a.D;
  float amax = 0.f;
  uint4 v[NV > 0 ? NV : 1][2];
  const int upr = a.D / 16;  // units a row
  const int units = n * upr;
  if (NV > 0) {
    const int r0 = tid / upr, c = (tid - r0 * upr) * 16, dr = TH / upr;
    const uint16_t *src = x + (int64_t)r0 * ld + c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool on = tid + j * TH < units;
      const uint4 *p = reinterpret_cast<const uint4 *>(src + (int64_t)j * dr * ld);
      v[j][0] = on ? __ldcs(p) : make_uint4(0, 0, 0, 0);
      v[j][1] = on ? __ldcs(p + 1) : make_uint4(0, 0, 0, 0);
    }
    // maxima of the magnitudes' bits, two at a time
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top = __vmaxu2(top, __vmaxu2(v[j][k].x & 0x7fff7fffu, v[j][k].y & 0x7fff7fffu));
        top = __vmaxu2(top, __vmaxu2(v[j][k].z & 0x7fff7fffu, v[j][k].w & 0x7fff7fffu));
      }
    if ((top & 0xffffu) < 0x7f80u && (top >> 16) < 0x7f80u) {
      amax = amax2(top);
    } else {  // an infinity or NaN among them
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          amax = fmaxf(amax, fmaxf(fmaxf(amax2(v[j][k].x), amax2(v[j][k].y)), fmaxf(amax2(v[j][k].z), amax2(v[j][k].w))));
    }
  } else if (VEC) {
    for (int e = tid; e < units; e += TH) {
      const int r = e / upr, c = (e - r * upr) * 16;
      const uint4 *p = reinterpret_cast<const uint4 *>(x + (int64_t)r * ld + c);
      const uint4 u = p[0], w = p[1];
      amax = fmaxf(amax, fmaxf(fmaxf(amax2(u.x), amax2(u.y)), fmaxf(amax2(u.z), amax2(u.w))));
      amax = fmaxf(amax, fmaxf(fmaxf(amax2(w.x), amax2(w.y)), fmaxf(amax2(w.z), amax2(w.w))));
    }
  } else {
    for (int e = tid; e < n * a.D; e += TH) {
      const int r = e / a.D, c = e - r * a.D;
      amax = fmaxf(amax, finite_abs(gdn::bf2f(x[(int64_t)r * ld + c])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (WARPS > 1) {
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) amax = fmaxf(amax, sh[i]);
    __syncthreads();
  }
  int e = gdnkv::scale_exponent(amax);
  if (off > 0) {
    // The page's scale does not fall.  Older codes move to the new one, rounded to
    // the format again, where it is another: a larger power of two, or the page came
    // with a scale that is none.
    e = max(e, gdnkv::exponent_over(before));
    const float f = before * gdnkv::pow2(-e);  // in [0, 1]; up to 4 where 2^126 is the most that e can be
    if (f != 1.f) {
      if (a.D % 4 == 0 && (reinterpret_cast<uintptr_t>(codes) & 3) == 0) {  // four at once where their address allows
        uint32_t *p = reinterpret_cast<uint32_t *>(codes);
        for (int i = tid; i < off * a.D / 4; i += TH) p[i] = gdnkv::rescale4(p[i], f);
      } else {
        for (int i = tid; i < off * a.D; i += TH) codes[i] = (uint8_t)gdnkv::rescale4(codes[i], f);
      }
    }
  }
  const float inv = gdnkv::pow2(-e);
  if (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (tid + j * TH >= units) break;
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        o[2 * k] = codes2(v[j][k].x, inv) | (codes2(v[j][k].y, inv) << 16);
        o[2 * k + 1] = codes2(v[j][k].z, inv) | (codes2(v[j][k].w, inv) << 16);
      }
      *reinterpret_cast<uint4 *>(dst + (int64_t)(tid + j * TH) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else if (VEC) {
    for (int e = tid; e < units; e += TH) {
      const int r = e / upr, c = (e - r * upr) * 16;
      const uint4 *p = reinterpret_cast<const uint4 *>(x + (int64_t)r * ld + c);
      const uint4 u = p[0], w = p[1];
      *reinterpret_cast<uint4 *>(dst + (int64_t)e * 16) =
          make_uint4(codes2(u.x, inv) | (codes2(u.y, inv) << 16), codes2(u.z, inv) | (codes2(u.w, inv) << 16),
                     codes2(w.x, inv) | (codes2(w.y, inv) << 16), codes2(w.z, inv) | (codes2(w.w, inv) << 16));
    }
  } else {
    for (int i = tid; i < n * a.D; i += TH) {
      const int r = i / a.D, c = i - r * a.D;
      dst[i] = (uint8_t)gdnkv::cvt_e4m3x2(gdn::bf2f(x[(int64_t)r * ld + c]) * inv, 0.f);
    }
  }
  if (tid == 0) *scale = gdnkv::pow2(e);
}

// One head of K or V and one window of tokens a group of WARPS warps; a warp of
// a wider group finds the runs for itself, all alike.  Short runs (a large
// decode step's) go to the warps in turn, long ones to all of them.
template <int WARPS, int NV, bool VEC>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : 32 * WARPS, NV == 8 ? 5 : 0) kv8_append_kernel(const AppendArgs a) {
  __shared__ float sh[WARPS];
  gdn::grid_release();
  gdn::grid_wait();
  const int64_t unit = WARPS == 1 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int64_t t0 = unit * a.window, t1 = min(t0 + a.window, a.T);
  if (t0 >= a.T) return;
  const int kv = blockIdx.y & 1, h = blockIdx.y >> 1;
  int bits = 0, ignore = 0, short_runs = 0;
  for (int64_t base = t0; base < t1; base += 32) {
    const int64_t t = base + lane;
    const int32_t s = slot_of(a, t, t < t1 ? bits : ignore);
    int32_t prev = __shfl_up_sync(0xffffffffu, s, 1);
    if (lane == 0) prev = slot_of(a, t - 1, ignore);
    const bool same = s >= 0 && prev >= 0 && page_of(a, prev) == page_of(a, s), follows = same && s == prev + 1;
    const uint32_t cont = __ballot_sync(0xffffffffu, follows);
    bool begins = t < t1 && s >= 0 && !follows;
    // A second run of a page would race with the first for its scale: where the last
    // token with a place is that page's, it is left out and reported.  That token is
    // mostly the one before; behind skipped ones it is looked for, 32 places back.
    if (__any_sync(0xffffffffu, begins && (same || (prev < 0 && t > 0)))) {
      const int32_t last = last_before(a, t, s);
      if (begins && last >= 0 && page_of(a, last) == page_of(a, s)) {
        begins = false;
        bits |= GDN_DEV_BAD_SLOT;
      }
    }
    uint32_t lead = __ballot_sync(0xffffffffu, begins);
    while (lead) {
      const int p = __ffs((int)lead) - 1;
      lead &= lead - 1;
      const int32_t slot = __shfl_sync(0xffffffffu, s, p);
      // tokens p + 1 .. that follow; a run that reaches the last of the 32 may go on
      const uint32_t stop = ~(p == 31 ? 0u : cont >> (p + 1)) ;
      int n = 1 + min(31 - p, __ffs((int)stop) - 1);
      if (p + n == 32) {
        for (;;) {
          const int32_t more = slot_of(a, base + p + n + lane, ignore);
          const bool ok = more == slot + n + lane && place_of(a, slot) + n + lane < a.bs;
          const uint32_t m = ~__ballot_sync(0xffffffffu, ok);
          n += m ? __ffs((int)m) - 1 : 32;
          if (m) break;
        }
      }
      if (WARPS > 1 && n * a.D <= 512) {
        if (short_runs++ % WARPS == (int)(threadIdx.x >> 5)) write_run<1, 0, VEC>(a, kv, h, base + p, n, slot, sh);
      } else {
        write_run<WARPS, NV, VEC>(a, kv, h, base + p, n, slot, sh);
      }
    }
  }
  if (bits && (WARPS == 1 || threadIdx.x < 32)) set_status(a.dev_status, bits);
}

template <int WARPS, int NV, bool VEC> cudaError_t launch_append(const AppendArgs &a, int64_t blocks, cudaStream_t s) {
  return gdn_host::launch_dependent(kv8_append_kernel<WARPS, NV, VEC>, dim3((unsigned)blocks, 2 * a.HK), WARPS == 1 ? 256 : 32 * WARPS, 0,
                                    s, a);
}

// log2(x) where x is a power of two, else -1.
int bits_of(int x) {
  for (int i = 0; i < 31; ++i)
    if (x == 1 << i) return i;
  return -1;
}

}  // namespace

namespace gdn_host {

cudaError_t launch_paged_plan(const int32_t *cached, const int32_t *cu, int N, int T, int32_t *table, int width,
                              const int32_t *free_pages, int F, const int32_t *num_free, int bs, int32_t *seq_lens,
                              int32_t *slots, int32_t *positions, int32_t *num_free_out, int32_t *dev_status,
                              cudaStream_t s) {
  const int blocks = T > 0 ? (T + kPlan - 1) / kPlan : 1;
  return launch_dependent(paged_plan_kernel, dim3(blocks), kPlan, 0, s, cached, cu, N, T, table, width, free_pages, F, num_free, bs,
                          bits_of(bs), seq_lens, slots, positions, num_free_out, dev_status);
}

cudaError_t launch_kv8_append(const uint16_t *k, const uint16_t *v, int64_t ldk, int64_t ldv, uint8_t *kc, uint8_t *vc,
                              float *ks, float *vs, const int32_t *slots, int64_t T, int P, int HK, int D, int bs,
                              int32_t *dev_status, cudaStream_t s) {
  const int sms = sm_count();
  AppendArgs a{k, v, ldk, ldv, kc, vc, ks, vs, slots, T, P, HK, D, bs, 1, bits_of(bs), dev_status};
  const uintptr_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(kc) |
                         reinterpret_cast<uintptr_t>(vc);
  // 16-byte accesses, and threads that keep their column from row to row
  const bool vec = !(bits & 15) && (D == 16 || D == 32 || D == 64 || D == 128 || D == 256 || D == 512) && ldk % 8 == 0 && ldv % 8 == 0;
  // Windows of a page's length once the tokens would fill every SM with blocks
  // four times over and a thread can hold its share of a page; else a token each.
  const int held = (bs * (D / 16) + 127) / 128;  // units a thread
  const bool wide = vec && held <= 8 && bs >= 8 && (T + bs - 1) / bs * 2 * HK >= 4 * (int64_t)sms;
  if (wide) a.window = bs;
  const int64_t units = (T + a.window - 1) / a.window, blocks = wide ? units : (units + 7) / 8;
  if (blocks > 2147483647LL) return cudaErrorInvalidValue;
  if (!wide) return vec ? launch_append<1, 0, true>(a, blocks, s) : launch_append<1, 0, false>(a, blocks, s);
  if (held <= 1) return launch_append<4, 1, true>(a, blocks, s);
  if (held <= 2) return launch_append<4, 2, true>(a, blocks, s);
  if (held <= 4) return launch_append<4, 4, true>(a, blocks, s);
  return launch_append<4, 8, true>(a, blocks, s);
}

}  // namespace gdn_host
