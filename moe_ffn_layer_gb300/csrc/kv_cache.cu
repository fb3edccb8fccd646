// Writing into and evicting from the 8-bit paged KV cache.
//
// Append: of each page that new tokens reach, one CTA per (page, head, K or V)
// takes the largest magnitude of the page's new rows, grows the page's scale
// where they need it (requantising the page's older rows), and stores the new
// rows' codes.
//
// Evict: one CTA per (sequence, head) finds the tokens to keep by their
// accumulated attention weight; then one CTA per destination (page, head)
// gathers the kept rows.
#include <limits.h>

#include "kv_cache.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- append
constexpr int kAppendThreads = 128;

// A sequence's touched pages are numbered from floor(cu[b] / page) + 2 b on: a
// run of n > 0 tokens touches at most floor((n - 1) / page) + 2 pages, and the
// next sequence's first number lies at least floor(n / page) + 2 further, so
// the numbers never meet and need no prefix sum.
__device__ __forceinline__ long long first_item(const int32_t* cu, int b, int shift) {
  return (cu[b] >> shift) + 2ll * b;
}

__device__ __forceinline__ uint32_t absmax_bits(const uint4& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(v.x & m, v.y & m), b = __vmaxu2(v.z & m, v.w & m), c = __vmaxu2(a, b);
  return max(c & 0xFFFFu, c >> 16);
}

// The largest finite magnitude of eight bf16 (their bits), for a vector that holds a NaN or an infinity.
__device__ __forceinline__ uint32_t absmax_finite_bits(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
  }
  return m;
}

// x / s rounded once, a NaN as 0.  inv is 1 / s where that product is exact.
__device__ __forceinline__ float quotient(float x, float s, float inv, bool exact) {
  const float y = exact ? x * inv : __fdiv_rn(x, s);
  return y == y ? y : 0.f;
}

// Bound: the bf16 rows read once and their codes written once (3 bytes a
// value): 13.9k tokens of 8 heads of 128 in 18 us, 4.7 TB/s; a decode step's single
// rows are launch latency, 4.5 us.  The rows stay in
// registers between the maximum and the rounding: kVecs vectors a thread, as
// many as a page has (4 to 16), so that small pages leave room for more CTAs
// and their loads: 12000 tokens in pages of 16, 32 and 64 (D = 128)
// 22, 17 and 17 us, with 16 for all 37, 24 and 19.
template <int kVecs>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(KvDims d, KvPool pool, KvSeqs s,
                                                                   const __nv_bfloat16* __restrict__ kn,
                                                                   const __nv_bfloat16* __restrict__ vn,
                                                                   long long kv_stride, const int32_t* __restrict__ cu,
                                                                   int T, int* status) {
  chain_wait();
  ChainReleaseAtExit release;
  // heads, K and V of a page lie side by side: its tokens' rows are read whole
  const int parts = 2 * d.Hkv, part = blockIdx.x % parts, h = part >> 1;
  const long long item = blockIdx.x / parts;
  const bool is_v = part & 1;
  // the sequence whose numbers hold this item: each round of loads leaves one in 32
  int b = 0;
  for (int left = s.B; left > 1;) {
    const int step = (left + 31) / 32, i = (threadIdx.x & 31) * step;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, i < left && first_item(cu, b + min(i, left - 1), d.shift) <= item);
    const int k = below ? 31 - __clz(below) : 0;
    b += k * step;
    left = min(step, left - k * step);
  }
  int first, n, len;
  if (!kv_sequence(s, cu, T, b, d, status, &first, &n, &len)) return;
  const int start = len - n;
  if (start < 0) {
    set_status(status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  const long long p = (start >> d.shift) + (item - first_item(cu, b, d.shift));   // page of the sequence
  if (n == 0 || item < first_item(cu, b, d.shift) || p * d.page >= len) return;
  const int page_id = s.table[static_cast<size_t>(b) * s.width + p];
  if (page_id < 0 || page_id >= pool.num_pages) {
    set_status(status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  const int t0 = static_cast<int>(p) * d.page;
  const int s0 = max(start - t0, 0), s1 = min(len - t0, d.page);   // slots of the new rows
  const __nv_bfloat16* src = (is_v ? vn : kn) + static_cast<long long>(first + t0 + s0 - start) * kv_stride +
                             static_cast<long long>(h) * d.D;
  uint8_t* codes = (is_v ? pool.v : pool.k) + kv_row(page_id, d.Hkv, h, d.page, 0, d.D);
  float* scale = (is_v ? pool.v_scale : pool.k_scale) + static_cast<size_t>(page_id) * d.Hkv + h;
  const int row_shift = d.D == 128 ? 4 : 3, vecs = (s1 - s0) << row_shift;   // vectors of a row: 16 or 8
  uint4 x[kVecs];
  uint32_t m = 0;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = threadIdx.x + i * kAppendThreads;
    if (j >= vecs) break;
    x[i] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(j >> row_shift) * kv_stride + (j & ((1 << row_shift) - 1)) * 8);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (threadIdx.x + i * kAppendThreads >= vecs) break;
    uint32_t a = absmax_bits(x[i]);
    if (a >= 0x7F80u) {
      odd = true;
      a = absmax_finite_bits(x[i]);
    }
    m = max(m, a);
  }
  if (odd) set_status(status, MOE_ERR_DEVICE_CHECK);
  __shared__ uint32_t warp_max[kAppendThreads / 32];
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  const float before = *scale;
  __syncthreads();   // (also: every thread has read the scale before it is written)
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) m = max(m, warp_max[i]);
  const float need = kv_pow2_scale(__uint_as_float(m << 16));
  const float now = s0 > 0 ? fmaxf(before, need) : need;
  if (threadIdx.x == 0) *scale = now;
  if (s0 > 0 && now != before) {
    const float ratio = __fdiv_rn(before, now);
    for (int j = threadIdx.x; j < s0 * d.D / 16; j += kAppendThreads) {
      uint4* at = reinterpret_cast<uint4*>(codes) + j;
      *at = e4m3x16_scaled(*at, ratio);
    }
  }
  const bool exact = (__float_as_uint(now) & 0x7FFFFFu) == 0;
  const float inv = __fdiv_rn(1.f, now);
  uint8_t* to = codes + static_cast<size_t>(s0) * d.D;
  if (exact && !odd) {   // a power of two and finite values: one multiplication each
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int j = threadIdx.x + i * kAppendThreads;
      if (j >= vecs) break;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = e4m3x2_of(bf16_lo(w[e]) * inv, bf16_hi(w[e]) * inv);
      *reinterpret_cast<uint2*>(to + j * 8) = make_uint2(prmt(c[0], c[1], 0x5410u), prmt(c[2], c[3], 0x5410u));
    }
    return;
  }
#pragma unroll 1
  for (int j = threadIdx.x; j < vecs; j += kAppendThreads) {   // (read again: seldom taken)
    const uint4 v = *reinterpret_cast<const uint4*>(src + static_cast<long long>(j >> row_shift) * kv_stride + (j & ((1 << row_shift) - 1)) * 8);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c[e] = e4m3x2_of(quotient(bf16_lo(w[e]), now, inv, exact), quotient(bf16_hi(w[e]), now, inv, exact));
    *reinterpret_cast<uint2*>(to + j * 8) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
}

// ---------------------------------------------------------------- evict
constexpr int kSelectThreads = 1024;

// Order-preserving integer of a weight: larger weight, larger key; -0 as +0,
// a NaN above everything (a token whose weight is not a number stays).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Which tokens of (sequence b, head h) stay: all of a sequence within the
// budget; else the first `sink`, the last `recent`, and of those between the
// budget - sink - recent heaviest, the lower index first among equal ones.
// Radix selection of the threshold key (11, 11 and 10 bits), then one pass in
// index order writes the kept indices, so the result does not depend on
// scheduling.  The weights are read five times; where the longest sequence's fit
// (kStaged), the first pass leaves them in shared memory.  Latency of its passes:
// 31 us for 256 (sequence, head) pairs of up to 16384.  With and without staging,
// selection and gathering, us: 32 sequences of 16384 120 and 126, of 32768 (one CTA
// an SM) 151 and 154, of 49152 179 and 181; one of 16384 21 and 23, of 32768 32 and
// 34, of 49152 43 and 47.
constexpr int kMostStaged = 49152;   // 192 KB
template <bool kStaged>
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(KvDims d, KvSeqs s, KvEvict e, int* status) {
  extern __shared__ float staged[];
  chain_wait();
  ChainReleaseAtExit release;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int len = s.seq_lens[b];
  if (!kv_length_is(s, d, len)) {
    if (tid == 0) set_status(status, MOE_ERR_DEVICE_CHECK);
    len = 0;   // skipped: nothing is kept
  }
  const float* w = e.weights + (static_cast<long long>(b) * d.Hkv + h) * e.w_stride;
  const size_t row = (static_cast<size_t>(b) * d.Hkv + h) * static_cast<size_t>(e.budget);
  int32_t* kept = e.kept + row;
  float* wout = e.dst_weights + row;
  const int keep = min(len, e.budget);
  if (h == 0 && tid == 0) e.dst_lens[b] = keep;
  for (int j = keep + tid; j < e.budget; j += kSelectThreads) {
    kept[j] = -1;
    wout[j] = 0.f;
  }
  if (len <= e.budget) {
    for (int j = tid; j < keep; j += kSelectThreads) {
      kept[j] = j;
      wout[j] = w[j];
    }
    return;
  }
  __shared__ int hist[2048];
  __shared__ int scan[64];
  __shared__ int pick[2];
  const int m0 = e.sink, m1 = len - e.recent;
  int want = e.budget - e.sink - e.recent;   // heaviest of [m0, m1) still to place
  uint32_t prefix = 0;
  int bits_done = 0;
  const int widths[3] = {11, 11, 10};
  if (kStaged) {
#pragma unroll 8
    for (int t = tid; t < len; t += kSelectThreads) staged[t] = w[t];
    __syncthreads();
    w = staged;
  }
  if (want > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int width = widths[pass], shift = 32 - bits_done - width, bins = 1 << width;
      for (int i = tid; i < bins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int t = m0 + tid; t < m1; t += kSelectThreads) {
        const uint32_t key = weight_key(w[t]);
        if (bits_done == 0 || key >> (32 - bits_done) == prefix) atomicAdd(&hist[key >> shift & (bins - 1)], 1);
      }
      __syncthreads();
      // from the top bin down: the bin in which the want-th largest key lies
      const int per = bins / kSelectThreads;   // 2 or 1
      const int top = bins - 1 - tid * per;
      int mine = 0;
      for (int i = 0; i < per; ++i) mine += hist[top - i];
      int before = mine;   // inclusive sum over threads 0..tid
      const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += up;
      }
      if (lane == 31) scan[warp] = before;
      __syncthreads();
      before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[lane] : 0) - mine;
      if (before < want && before + mine >= want) {
        int i = 0, above = before;
        while (above + hist[top - i] < want) above += hist[top - i++];
        pick[0] = top - i;
        pick[1] = want - above;
      }
      __syncthreads();
      prefix = prefix << width | static_cast<uint32_t>(pick[0]);
      want = pick[1];
      bits_done += width;
      __syncthreads();
    }
  }
  // `prefix` is the smallest key kept, `want` how many of the equal ones.  Each
  // warp has a run of tokens of its own: it counts those that stay for sure and
  // the equal ones; the sums over the warps before then say where its own go.
  const bool any = e.budget - e.sink - e.recent > 0;
  const int lane = tid & 31, warp = tid >> 5, run = (len + kSelectThreads - 1) / kSelectThreads * 32;
  const int r0 = min(warp * run, len), r1 = min(r0 + run, len);
  const auto sort_of = [&](int t, float x, bool* equal) {   // stays for sure; equal: perhaps
    const bool ends = t < m0 || t >= m1;
    const uint32_t key = weight_key(x);
    *equal = t < r1 && !ends && any && key == prefix;
    return t < r1 && (ends || (any && key > prefix));
  };
  int sure = 0, equal = 0;
#pragma unroll 4
  for (int t = r0 + lane; t < r0 + run && t - lane < r1; t += 32) {
    bool eq;
    const bool stays = sort_of(t, t < r1 ? w[t] : 0.f, &eq);
    sure += __popc(__ballot_sync(0xFFFFFFFFu, stays));
    equal += __popc(__ballot_sync(0xFFFFFFFFu, eq));
  }
  __syncthreads();   // (scan was read)
  if (lane == 0) {
    scan[warp] = sure;
    scan[32 + warp] = equal;
  }
  __syncthreads();
  const int sure_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[lane] : 0);
  int equal_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[32 + lane] : 0);
  int at = sure_before + min(equal_before, want);
#pragma unroll 4
  for (int t = r0 + lane; t < r0 + run && t - lane < r1; t += 32) {
    bool eq;
    const float x = t < r1 ? w[t] : 0.f;
    bool stays = sort_of(t, x, &eq);
    const uint32_t eqs = __ballot_sync(0xFFFFFFFFu, eq), below = (1u << lane) - 1;
    stays |= eq && equal_before + __popc(eqs & below) < want;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, stays);
    if (stays) {
      const int to = at + __popc(all & below);
      kept[to] = t;
      wout[to] = x;
    }
    at += __popc(all);
    equal_before += __popc(eqs);
  }
}

constexpr int kGatherThreads = 128;

// One destination (page, head): its kept rows, K then V.  The page's scale is
// the largest of its rows' scales; a row from a page of another scale has its
// codes rescaled (exact for powers of two, except into the subnormals).
// Bound: the kept codes read and written once: 32 sequences of 3000 to 16384
// tokens back to 4096 in 86 us, 5.6 TB/s of DRAM traffic.
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(KvDims d, KvPool src, KvSeqs s, KvPool dst,
                                                                   KvEvict e, int* status) {
  chain_wait();
  ChainReleaseAtExit release;
  const int p = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = min(e.dst_lens[b] - p * d.page, d.page);   // rows of this page
  if (n <= 0) return;
  const int to_id = e.dst_table[static_cast<size_t>(b) * e.dst_width + p];
  if (to_id < 0 || to_id >= dst.num_pages) {
    if (tid == 0) set_status(status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  const int32_t* kept = e.kept + (static_cast<size_t>(b) * d.Hkv + h) * static_cast<size_t>(e.budget) +
                        static_cast<size_t>(p) * d.page;
  __shared__ size_t from[128];        // byte offset of each row in the source pools
  __shared__ float scale[2][128];
  __shared__ uint32_t top[2];
  if (tid < 2) top[tid] = 0;
  __syncthreads();
  if (tid < n) {
    const int t = kept[tid];
    const int q = t >> d.shift;
    int id = q < s.width ? s.table[static_cast<size_t>(b) * s.width + q] : -1;
    if (id < 0 || id >= src.num_pages) {
      set_status(status, MOE_ERR_DEVICE_CHECK);
      from[tid] = ~static_cast<size_t>(0);
      scale[0][tid] = scale[1][tid] = 0.f;
    } else {
      from[tid] = kv_row(id, d.Hkv, h, d.page, t & (d.page - 1), d.D);
      const float a = src.k_scale[static_cast<size_t>(id) * d.Hkv + h], c = src.v_scale[static_cast<size_t>(id) * d.Hkv + h];
      scale[0][tid] = a;
      scale[1][tid] = c;
      // scales are not negative: their bits order as they do
      atomicMax(&top[0], __float_as_uint(a));
      atomicMax(&top[1], __float_as_uint(c));
    }
  }
  __syncthreads();
  const int row_shift = d.D == 128 ? 3 : 2, chunks = n << row_shift;   // 16-byte chunks of a row: 8 or 4
  const float big[2] = {__uint_as_float(top[0]), __uint_as_float(top[1])};
  const size_t to = kv_row(to_id, d.Hkv, h, d.page, 0, d.D);
  if (tid < 2) (tid ? dst.v_scale : dst.k_scale)[static_cast<size_t>(to_id) * d.Hkv + h] = big[tid];
  // four chunks of K and of V a thread are on their way at once
  for (int j0 = tid; j0 < chunks; j0 += 4 * kGatherThreads) {
    uint4 c[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i * kGatherThreads, r = j >> row_shift;
      const bool in = j < chunks && from[min(r, n - 1)] != ~static_cast<size_t>(0);
      const size_t at = in ? from[r] + (j & ((1 << row_shift) - 1)) * 16 : 0;
      c[0][i] = in ? __ldg(reinterpret_cast<const uint4*>(src.k + at)) : make_uint4(0, 0, 0, 0);
      c[1][i] = in ? __ldg(reinterpret_cast<const uint4*>(src.v + at)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i * kGatherThreads;
      if (j >= chunks) break;
      const int r = j >> row_shift;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (scale[kv][r] != big[kv]) c[kv][i] = e4m3x16_scaled(c[kv][i], __fdiv_rn(scale[kv][r], big[kv]));
        *reinterpret_cast<uint4*>((kv ? dst.v : dst.k) + to + static_cast<size_t>(j) * 16) = c[kv][i];
      }
    }
  }
}

}  // namespace

int kv_append_launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, const void* k, const void* v,
                     long long kv_stride, const int32_t* cu_new, int T_new, int* status, cudaStream_t stream,
                     int* launches) {
  const long long grid = (T_new / d.page + 2ll * s.B) * 2 * d.Hkv;
  if (grid > INT_MAX) return MOE_ERR_UNSUPPORTED;
  const int vecs = d.page * d.D / 8 / kAppendThreads;   // of a page, per thread: 1 to 16
  const auto kernel = vecs <= 4 ? kv_append_kernel<4> : vecs <= 8 ? kv_append_kernel<8> : kv_append_kernel<16>;
  if (launch_chained(kernel, dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0, stream, d, pool, s,
                     static_cast<const __nv_bfloat16*>(k),
                     static_cast<const __nv_bfloat16*>(v), kv_stride, cu_new, T_new, status) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

int kv_evict_launch(const KvDims& d, const KvPool& src, const KvSeqs& s, const KvPool& dst, const KvEvict& e,
                    int* status, cudaStream_t stream, int* launches) {
  const bool staged = s.max_len <= kMostStaged;
  const size_t smem = staged ? s.max_len * sizeof(float) : 0;
  if (staged && kv_allow_smem<kv_select_kernel<true>>(kMostStaged * sizeof(float)) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_chained(staged ? kv_select_kernel<true> : kv_select_kernel<false>, dim3(d.Hkv, s.B), dim3(kSelectThreads),
                     smem, stream, d, s, e, status) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  const int most = s.max_len < e.budget ? s.max_len : e.budget;
  const int pages = (most + d.page - 1) / d.page;
  if (pages == 0) return MOE_OK;
  if (launch_chained(kv_gather_kernel, dim3(pages, d.Hkv, s.B), dim3(kGatherThreads), 0, stream, d, src, s, dst, e,
                     status) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

}  // namespace moe
