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
    const int32_t *__restrict__ free_pages, int F, const int32_t *__restrict__ num_free, int bs, int32_t *seq_lens,
    int32_t *slots, int32_t *positions, int32_t *num_free_out, int32_t *dev_status) {
  __shared__ int32_t s_start[kPlan], s_cached[kPlan], s_before[kPlan], s_end[kPlan];
  __shared__ int32_t s_warp[32];
  __shared__ int32_t s_lo, s_hi;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int32_t tok = (int32_t)min((int64_t)blockIdx.x * kPlan + tid, (int64_t)T);
  int left = *num_free;
  left = left < 0 ? 0 : left > F ? F : left;
  int32_t slot = -1, pos = 0, base = 0;
  int bits = 0;
  for (int n0 = 0; n0 < N; n0 += kPlan) {
    const int n = n0 + tid, cnt = min(kPlan, N - n0);
    int32_t a = 0, b = 0, c = 0, want = 0;
    if (n < N) {
      a = cu[n];
      b = cu[n + 1];
      c = cached[n];
      if (a < 0 || b < a || b > T || c < 0 || (n == 0 && a != 0) || (int64_t)c + b - a > 2147483647LL) {
        bits |= GDN_DEV_BAD_CU_SEQLENS;
        a = b = 0;
        c = c < 0 ? 0 : c;
      }
      const int64_t total = (int64_t)c + b - a;
      int64_t have = ((int64_t)c + bs - 1) / bs, need = (total + bs - 1) / bs;
      if (need > width) {
        bits |= GDN_DEV_NO_PAGE;
        need = width;
      }
      want = (int32_t)(need > have ? need - have : 0);
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
    __syncthreads();
    int32_t add = 0, all = 0;
    for (int i = 0; i < 32; ++i) {
      const int32_t v = s_warp[i];
      if (i < w) add += v;
      all += v;
    }
    s_before[tid] = base + add + x - want;
    __syncthreads();
    if (tok < T && tok >= s_start[0] && slot < 0) {
      // the last request of these that starts at or before the token and is not empty
      int lo = 0, hi = cnt - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= tok) lo = mid; else hi = mid - 1;
      }
      if (s_start[lo] <= tok && tok < s_end[lo]) {
        pos = s_cached[lo] + (tok - s_start[lo]);
        const int pg = pos / bs, off = pos - pg * bs;
        const int have = (int)(((int64_t)s_cached[lo] + bs - 1) / bs);
        int32_t page = -1;
        if (pg < width) {
          int32_t *entry = table + (int64_t)(n0 + lo) * width + pg;
          if (pg < have) {
            page = *entry;
          } else {
            const int32_t at = left - 1 - (s_before[lo] + pg - have);
            if (at >= 0) page = free_pages[at];
            else bits |= GDN_DEV_NO_PAGE;
            if (off == 0) *entry = page;
          }
        }
        if (page >= 0) slot = page * bs + off;
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
// of one page.  One warp writes a run of one head of K or V: it forms the
// largest magnitude, the exponent e of the page's new scale 2^e, moves the
// codes that were there before to that scale, and writes the new ones.
//
// The scale is a power of two because then x 2^-e is exact, the only rounding
// is the one to the 8-bit format, and a page whose scale grows keeps its older
// codes' bits as long as they stay normal numbers of the format.
//
// Bound: HBM for a prefill (2 bytes read, 1 written an element), latency for a
// decode step.  A warp takes the runs that begin in a window of `window`
// tokens: one token where there are few, a page's worth where there are many,
// so that a long prefill has one run a warp.
struct AppendArgs {
  const uint16_t *x[2];
  int64_t ld[2];
  uint8_t *cache[2];
  float *scale[2];
  const int32_t *slots;
  int64_t T;
  int P, HK, D, bs, window;
  int32_t *dev_status;
};

// Place of token t, or -1 (PAD, or a slot outside the cache).
__device__ __forceinline__ int32_t slot_of(const AppendArgs &a, int64_t t, int &bits) {
  const int32_t s = a.slots[t];
  if (s >= 0 && s / a.bs < a.P) return s;
  if (s != -1) bits |= GDN_DEV_BAD_SLOT;
  return -1;
}
__device__ __forceinline__ bool follows(const AppendArgs &a, int32_t prev, int32_t s) {
  return prev >= 0 && s == prev + 1 && s % a.bs != 0;
}
__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x <= 3.402823466e38f ? x : 0.f;  // infinities and NaN do not set a scale
}

template <bool VEC>
__device__ void write_run(const AppendArgs &a, int kv, int h, int64_t t0, int n, int32_t slot) {
  const int lane = threadIdx.x & 31;
  const int page = slot / a.bs, off = slot - page * a.bs;
  const uint16_t *x = a.x[kv] + t0 * a.ld[kv] + (int64_t)h * a.D;
  uint8_t *codes = a.cache[kv] + ((int64_t)page * a.HK + h) * (int64_t)a.bs * a.D;
  float *scale = a.scale[kv] + (int64_t)page * a.HK + h;
  const int vpr = a.D / 8;
  float amax = 0.f;
  if (VEC) {
    for (int e = lane; e < n * vpr; e += 32) {
      const int r = e / vpr, c = e - r * vpr;
      const uint4 v = *reinterpret_cast<const uint4 *>(x + (int64_t)r * a.ld[kv] + c * 8);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        amax = fmaxf(amax, finite_abs(__uint_as_float(u[j] << 16)));
        amax = fmaxf(amax, finite_abs(__uint_as_float(u[j] & 0xffff0000u)));
      }
    }
  } else {
    for (int e = lane; e < n * a.D; e += 32) {
      const int r = e / a.D, c = e - r * a.D;
      amax = fmaxf(amax, finite_abs(gdn::bf2f(x[(int64_t)r * a.ld[kv] + c])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  int e = gdnkv::scale_exponent(amax);
  if (off > 0) {
    const int old = gdnkv::exponent_of(*scale);
    if (old >= e) {
      e = old;
    } else {
      // older codes move to the larger scale, rounded to the format again
      const float f = gdnkv::pow2(max(old - e, -126));
      const int words = off * a.D / 4;
      if (a.D % 4 == 0) {
        uint32_t *p = reinterpret_cast<uint32_t *>(codes);
        for (int i = lane; i < words; i += 32) p[i] = gdnkv::rescale4(p[i], f);
      } else {
        for (int i = lane; i < off * a.D; i += 32) codes[i] = (uint8_t)gdnkv::rescale4(codes[i], f);
      }
    }
  }
  const float inv = gdnkv::pow2(-e);
  uint8_t *dst = codes + (int64_t)off * a.D;
  if (VEC) {
    for (int i = lane; i < n * vpr; i += 32) {
      const int r = i / vpr, c = i - r * vpr;
      const uint4 v = *reinterpret_cast<const uint4 *>(x + (int64_t)r * a.ld[kv] + c * 8);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t lo = gdnkv::cvt_e4m3x2(__uint_as_float(u[2 * j] << 16) * inv, __uint_as_float(u[2 * j] & 0xffff0000u) * inv);
        const uint32_t hi =
            gdnkv::cvt_e4m3x2(__uint_as_float(u[2 * j + 1] << 16) * inv, __uint_as_float(u[2 * j + 1] & 0xffff0000u) * inv);
        o[j] = lo | (hi << 16);
      }
      *reinterpret_cast<uint2 *>(dst + (int64_t)i * 8) = make_uint2(o[0], o[1]);
    }
  } else {
    for (int i = lane; i < n * a.D; i += 32) {
      const int r = i / a.D, c = i - r * a.D;
      dst[i] = (uint8_t)gdnkv::cvt_e4m3x2(gdn::bf2f(x[(int64_t)r * a.ld[kv] + c]) * inv, 0.f);
    }
  }
  __syncwarp();
  if (lane == 0) *scale = gdnkv::pow2(e);
}

template <bool VEC>
__global__ void __launch_bounds__(256) kv8_append_kernel(const AppendArgs a) {
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int per = 2 * a.HK;
  const int64_t win = unit / per;
  const int64_t t0 = win * a.window;
  if (t0 >= a.T) return;
  const int kv = (int)(unit % per) & 1, h = (int)(unit % per) >> 1;
  const int64_t t1 = min(t0 + a.window, a.T);
  int bits = 0;
  for (int64_t t = t0; t < t1;) {
    const int32_t s = slot_of(a, t, bits);
    if (s < 0) {
      ++t;
      continue;
    }
    if (t > 0) {
      int ignore = 0;
      if (follows(a, slot_of(a, t - 1, ignore), s)) {  // an earlier token leads this run
        ++t;
        continue;
      }
    }
    // the run's length: 32 tokens at a time
    int n = 1;
    const int most = a.bs - s % a.bs;
    while (n < most) {
      int ignore = 0;
      const int64_t tt = t + n + lane;
      const bool ok = n + lane < most && tt < a.T && slot_of(a, tt, ignore) == s + n + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, ok);
      const int k = m == 0xffffffffu ? 32 : __ffs((int)~m) - 1;
      n += k;
      if (k < 32) break;
    }
    write_run<VEC>(a, kv, h, t, n, s);
    t += n;
  }
  if (bits && lane == 0) set_status(a.dev_status, bits);
}

}  // namespace

namespace gdn_host {

cudaError_t launch_paged_plan(const int32_t *cached, const int32_t *cu, int N, int T, int32_t *table, int width,
                              const int32_t *free_pages, int F, const int32_t *num_free, int bs, int32_t *seq_lens,
                              int32_t *slots, int32_t *positions, int32_t *num_free_out, int32_t *dev_status,
                              cudaStream_t s) {
  const int blocks = T > 0 ? (T + kPlan - 1) / kPlan : 1;
  paged_plan_kernel<<<blocks, kPlan, 0, s>>>(cached, cu, N, T, table, width, free_pages, F, num_free, bs, seq_lens, slots,
                                             positions, num_free_out, dev_status);
  return cudaGetLastError();
}

cudaError_t launch_kv8_append(const uint16_t *k, const uint16_t *v, int64_t ldk, int64_t ldv, uint8_t *kc, uint8_t *vc,
                              float *ks, float *vs, const int32_t *slots, int64_t T, int P, int HK, int D, int bs,
                              int32_t *dev_status, cudaStream_t s) {
  const int sms = sm_count();
  AppendArgs a{{k, v}, {ldk, ldv}, {kc, vc}, {ks, vs}, slots, T, P, HK, D, bs, 1, dev_status};
  int64_t window = T * 2 * HK / ((int64_t)sms * 48);  // about 48 warps an SM
  a.window = (int)(window < 1 ? 1 : window > bs ? bs : window);
  const int64_t units = (T + a.window - 1) / a.window * 2 * HK;
  const int64_t blocks = (units + 7) / 8;
  if (blocks > 2147483647LL) return cudaErrorInvalidValue;
  const uintptr_t in = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  const uintptr_t out = reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc);
  if (!(in & 15) && !(out & 7) && D % 8 == 0 && ldk % 8 == 0 && ldv % 8 == 0)
    kv8_append_kernel<true><<<(int)blocks, 256, 0, s>>>(a);
  else
    kv8_append_kernel<false><<<(int)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn_host
