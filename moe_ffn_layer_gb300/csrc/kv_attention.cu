// Attention over the 8-bit paged KV cache.
//
// For query row i of sequence b (position len - n + i) and head h of kv head
// h / g:  s_t = scale * ks * (q . kc_t) over the tokens t <= position,
// p = softmax(s), out = sum_t p_t * vs * vc_t, lse = ln sum_t exp(s_t); a row
// that sees nothing has out = 0 and lse = -inf.
//
// The g heads of a kv head share its keys, so a tile's rows are (query, head)
// pairs: row r is query r / g, head h * g + r % g.
//
// Both products run on the tensor cores with fp32 accumulation, their operands
// exact or kept to 16 bits at least:
//  - scores: f16, which holds a K code exactly.  A query row is scaled by a
//    power of two to a largest magnitude in [2^7, 2^8), which keeps all of a
//    bf16's bits down to 2^-21 of it.  (An e4m3 MMA takes the codes as they
//    are, but this GPU runs it as conversions and f16 MMAs: 5.8 clocks an SM
//    for 16x8x32 when its operands change, against 4.9 for two f16 ones.)
//  - output: bf16, which has fp32's range.  A V code becomes bf16 exactly; a
//    weight p * vs enters as two bf16 terms, so that it keeps 16 bits however
//    far it lies below the row's largest (a long sequence's many small weights
//    count as they should, whatever the pages' scales).  Below 2^-117, and so
//    with V scales near fp32's least, bf16's own floor of 2^-133 takes bits.
// What lies beyond a sequence's end is loaded as zeros, scores are masked by
// being replaced, and V's conversion reads any code byte as a finite value: no
// slot that a row does not see turns its result into a NaN.
#include <limits.h>

#include <algorithm>

#include "kv_cache.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTok = 32;          // tokens of a warp's step
constexpr int kWarps = 4;
constexpr int kSpan = kWarps * kTok;   // tokens of a CTA's step: one step of each warp
constexpr int kDecodeRows = 64;        // query rows of a kv head up to which the decode kernel is taken (on_prefill)
constexpr int kBesideRows = 32;        // the same beside the prefill kernel (beside_prefill)
constexpr float kSlack = 8.f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The bytes of v that sel picks (two code bytes, each followed by its sign
// copy) as two bf16 of the codes' values.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t v) {
  return bf16x2_mul((prmt(v, 0u, kSel) << 4) & 0x87F087F0u, 0x7B807B80u);   // times 2^120: e4m3's bias for bf16's
}
constexpr uint32_t kBytes02 = 0xA280u, kBytes13 = 0xB391u;

// Two floats as bf16 pairs hi + lo: hi the upper halves as they are, lo what
// is left, rounded (16 bits in all).
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t* hi, uint32_t* lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  *hi = prmt(ua, ub, 0x7632u);
  *lo = pack_bf16x2(a - __uint_as_float(ua & 0xFFFF0000u), b - __uint_as_float(ub & 0xFFFF0000u));
}

// d += a (16x16, row) * b (16x8, col), f16 inputs, fp32 accumulator
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d += a (16x16, row) * b (16x8, col), bf16 inputs, fp32 accumulator
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 bytes global -> shared, zeros where !ok (the address is then not read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows, chunks
// permuted so that neither the rows read by a quarter warp (K) nor eight rows
// of one chunk (V, ldmatrix) meet in a bank.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// A tile's 8 R query rows as MMA operands, R = 1 or 2 of them per lane: lane/4
// and lane/4 + 8 (zeros for R = 1).  The MMA's K index may stand for any order
// of the head dimension as long as both operands agree: lane (n, c) of a K
// operand holds 16-byte chunk 2c + h of token n's row (chunk c for D = 64), four
// codes per K step, so the query operand of step 4h + r holds
// d = 16 (2c + h) + 4r + {0, 1} and + {2, 3}.
template <int D, int R>
struct QueryTile {
  uint32_t a[D / 16][4];
  float unscale[R];   // scale * log2(e) / (the row's power of two)

  __device__ __forceinline__ void load(const KvAttention& at, int first, int h, int g, int row0, int rows, int lane) {
    const int c = lane & 3;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) a[k][1] = a[k][3] = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = row0 + (lane >> 2) + 8 * i;
      const bool real = r < rows;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(at.q) +
                               static_cast<long long>(first + (real ? r / g : 0)) * at.q_stride +
                               (static_cast<long long>(h) * g + (real ? r % g : 0)) * D;
      uint4 raw[D / 32];
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const int d0 = (D == 128 ? 16 * (2 * c + (k >> 1)) : 16 * c) + 8 * (k & 1);
        raw[k] = real ? __ldg(reinterpret_cast<const uint4*>(q + d0)) : make_uint4(0, 0, 0, 0);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(raw[k].x & 0x7FFF7FFFu, raw[k].y & 0x7FFF7FFFu),
                                 __vmaxu2(raw[k].z & 0x7FFF7FFFu, raw[k].w & 0x7FFF7FFFu)));
      }
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      // 2^(7 - floor(log2 max)), kept normal on both sides; a NaN or an
      // infinity in the row makes its scores NaN
      const uint32_t e = max(m >> 7, 8u);   // biased exponent of the largest
      const float up = __uint_as_float((261 - e) << 23), down = __uint_as_float((e - 7) << 23);
      unscale[i] = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : at.scale * kLog2e * down;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        a[2 * k][i] = pack_f16x2(bf16_lo(raw[k].x) * up, bf16_hi(raw[k].x) * up);
        a[2 * k][2 + i] = pack_f16x2(bf16_lo(raw[k].y) * up, bf16_hi(raw[k].y) * up);
        a[2 * k + 1][i] = pack_f16x2(bf16_lo(raw[k].z) * up, bf16_hi(raw[k].z) * up);
        a[2 * k + 1][2 + i] = pack_f16x2(bf16_lo(raw[k].w) * up, bf16_hi(raw[k].w) * up);
      }
    }
  }
};

// s[nt] = raw scores of the lane's rows and two tokens of each eight (in units
// that QueryTile::unscale and the page's scale undo)
template <int D, int R>
__device__ __forceinline__ void scores(float (&s)[kTok / 8][2 * R], const QueryTile<D, R>& q, uint32_t k_tile,
                                       int lane) {
  const int n = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < kTok / 8; ++nt) {
    float x[4] = {};
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      const uint4 v = lds_u4(k_tile + swz<D>(nt * 8 + n, D == 128 ? 2 * c + half : c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint2 b = e4m3x4_to_f16x4(w[r]);
        mma_f16(x, q.a[4 * half + r], b.x, b.y);
      }
    }
#pragma unroll
    for (int e = 0; e < 2 * R; ++e) s[nt][e] = x[e];
  }
}

// Where a call's work lies: the row tile's sequence, its rows and what they see.
struct Tile {
  int first, n, len, rows, row0, seen;   // seen: tokens that the tile's last real row sees
  __device__ __forceinline__ bool find(const KvSeqs& s, const KvAttention& at, int b, int g, int mt, int tile_rows,
                                       const KvDims& d, int* status) {
    if (!kv_sequence(s, at.cu_q, at.T_q, b, d, status, &first, &n, &len)) return false;
    if (n > at.max_q) {
      set_status(status, MOE_ERR_DEVICE_CHECK);
      return false;
    }
    rows = n * g;
    row0 = mt * tile_rows;
    if (row0 >= rows) return false;
    const int last = min(row0 + tile_rows, rows) - 1;
    seen = max(len - n + last / g + 1, 0);
    return true;
  }
};

// One warp's ring of 32-token steps in shared memory.  A step is two halves of
// 16 tokens (a page holds whole halves).
template <int D>
struct Ring {
  static constexpr int kStageBytes = 2 * kTok * D;
  uint32_t base;         // stages x (K rows, V rows)
  float* scales;         // stages x {ks, ks, vs, vs} of the halves
  // The page ids of a step, asked for a step before copy() needs them.
  __device__ __forceinline__ void look(int (&id)[2], const KvDims& d, const KvSeqs& s, int b, int t0, int end) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 16 * i;
      id[i] = t < end ? __ldg(s.table + static_cast<size_t>(b) * s.width + (t >> d.shift)) : -1;
    }
  }
  // Starts the copies of tokens [t0, t0 + 32); rows at or beyond `end` are zeros.
  __device__ __forceinline__ void copy(int stage, const int (&id)[2], const KvDims& d, const KvPool& pool, int h,
                                       int t0, int end, int lane, int* status) const {
    constexpr int kChunks = D / 16, kRowsAtOnce = 32 / kChunks;
    const uint32_t k = base + stage * kStageBytes, v = k + kTok * D;
    const int row = lane / kChunks, c = lane % kChunks;
    const uint32_t pages = pool.num_pages;
    if (t0 + kTok <= end && static_cast<uint32_t>(id[0]) < pages && static_cast<uint32_t>(id[1]) < pages) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t at = kv_row(id[i], d.Hkv, h, d.page, ((t0 + 16 * i) & (d.page - 1)) + row, D) + c * 16;
        const uint8_t *ks = pool.k + at, *vs = pool.v + at;
#pragma unroll
        for (int j = 0; j < 16; j += kRowsAtOnce) {
          const uint32_t to = swz<D>(16 * i + j + row, c);
          cp_async16(k + to, ks + j * D);
          cp_async16(v + to, vs + j * D);
        }
      }
      if (lane < 4)
        cp_async4(smem_u32(scales + stage * 4 + lane), (lane < 2 ? pool.k_scale : pool.v_scale) +
                                                           static_cast<size_t>(lane & 1 ? id[1] : id[0]) * d.Hkv + h);
      return;
    }
    // the sequence ends here, or a page is not there
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 16 * i;
      const bool ok = static_cast<uint32_t>(id[i]) < pages;
      if (t < end && !ok) set_status(status, MOE_ERR_DEVICE_CHECK);
      const size_t at = ok ? kv_row(id[i], d.Hkv, h, d.page, (t & (d.page - 1)) + row, D) + c * 16 : 0;
#pragma unroll
      for (int j = 0; j < 16; j += kRowsAtOnce) {
        const bool in = ok && t + j + row < end;
        const uint32_t to = swz<D>(16 * i + j + row, c);
        cp_async16(k + to, pool.k + at + (in ? j * D : 0), in);
        cp_async16(v + to, pool.v + at + (in ? j * D : 0), in);
      }
      if ((lane & 1) == i && lane < 4) {
        float* to = scales + stage * 4 + lane;
        const size_t of = static_cast<size_t>(ok ? id[i] : 0) * d.Hkv + h;
        if (ok)
          cp_async4(smem_u32(to), (lane < 2 ? pool.k_scale : pool.v_scale) + of);
        else   // a page that is not there: a NaN of its own, taken as masked
          *to = lane < 2 ? __uint_as_float(0x7FFFFFFFu) : 0.f;
      }
    }
  }
};

__device__ __forceinline__ bool no_page(float k_scale) { return __float_as_uint(k_scale) == 0x7FFFFFFFu; }

__device__ __forceinline__ float exp2_diff(float a, float b) { return a == -INFINITY ? 0.f : exp2_approx(a - b); }

// Running softmax and output of a warp's rows.  For R = 1 the MMA's upper
// eight rows take the weights' low terms, so o[..][2..3] adds to o[..][0..1].
template <int D, int R>
struct State {
  float m[R], l[R];   // l is this lane's share of the row's sum
  float o[D / 16][2][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][p][i] = 0.f;
  }

  // One step: the ring stage's 32 tokens from t0 on; row i sees those below
  // sees[i].  keep (R = 1, nullable): where the lane's row keeps its scores.
  __device__ __forceinline__ void add(const QueryTile<D, R>& q, const Ring<D>& ring, int stage, int t0,
                                      const int (&sees)[R], int sees_least, float* keep, int lane) {
    const uint32_t k_tile = ring.base + stage * Ring<D>::kStageBytes, v_tile = k_tile + kTok * D;
    const float4 page = *reinterpret_cast<const float4*>(ring.scales + stage * 4);
    const float ks0 = page.x, ks1 = page.y, vs0 = page.z, vs1 = page.w;
    float sc[kTok / 8][2 * R];
    scores<D, R>(sc, q, k_tile, lane);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float f0 = ks0 * q.unscale[i], f1 = ks1 * q.unscale[i];
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) {
        sc[nt][2 * i] *= nt < 2 ? f0 : f1;
        sc[nt][2 * i + 1] *= nt < 2 ? f0 : f1;
      }
    }
    if (t0 + kTok > sees_least || no_page(ks0) || no_page(ks1)) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (t0 + nt * 8 + 2 * (lane & 3) + e >= sees[i] || no_page(nt < 2 ? ks0 : ks1)) sc[nt][2 * i + e] = -INFINITY;
    }
    if (R == 1 && keep) {
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt)
        *reinterpret_cast<float2*>(keep + t0 + nt * 8 + 2 * (lane & 3)) = make_float2(sc[nt][0], sc[nt][1]);
    }
    // The maximum that the exponents are taken against follows the scores only
    // where they pass it by more than 2^kSlack: the weights then stay below
    // 2^kSlack, which costs no accuracy, and o is seldom rescaled.
    float top[R];
    bool grew = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      top[i] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) top[i] = fmaxf(top[i], fmaxf(sc[nt][2 * i], sc[nt][2 * i + 1]));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
      grew |= top[i] > m[i] + kSlack;
    }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        top[i] = fmaxf(top[i], m[i]);
        const float f = exp2_diff(m[i], top[i]);
        m[i] = top[i];
        l[i] *= f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 2 * i; e < (R == 1 ? 4 : 2 * i + 2); ++e) o[j][p][e] *= f;
      }
    }
    uint32_t hi[kTok / 16][4], lo[kTok / 16][4];   // R = 1: both terms in hi
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float base = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) {
        const float vs = nt < 2 ? vs0 : vs1;
        const float p0 = exp2_approx(sc[nt][2 * i] - base), p1 = exp2_approx(sc[nt][2 * i + 1] - base);
        l[i] += p0 + p1;
        uint32_t* a = hi[nt >> 1] + 2 * (nt & 1);
        split_bf16x2(p0 * vs, p1 * vs, a + i, R == 1 ? a + 1 : lo[nt >> 1] + 2 * (nt & 1) + i);
      }
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t v[4];
      ldmatrix_x4_trans(v, v_tile + swz<D>(lane, j));
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k) {
        const uint32_t even0 = codes_to_bf16x2<kBytes02>(v[2 * k]), even1 = codes_to_bf16x2<kBytes02>(v[2 * k + 1]);
        const uint32_t odd0 = codes_to_bf16x2<kBytes13>(v[2 * k]), odd1 = codes_to_bf16x2<kBytes13>(v[2 * k + 1]);
        mma_bf16(o[j][0], hi[k], even0, even1);
        mma_bf16(o[j][1], hi[k], odd0, odd1);
        if (R == 2) {
          mma_bf16(o[j][0], lo[k], even0, even1);
          mma_bf16(o[j][1], lo[k], odd0, odd1);
        }
      }
    }
  }

  // Columns 16 j + 4 (lane % 4) .. + 3 of the lane's row i: even and odd
  // columns of the V bytes interleave.
  __device__ __forceinline__ float4 out(int j, int i) const {
    if (R == 1) return make_float4(o[j][0][0] + o[j][0][2], o[j][1][0] + o[j][1][2], o[j][0][1] + o[j][0][3], o[j][1][1] + o[j][1][3]);
    return make_float4(o[j][0][2 * i], o[j][1][2 * i], o[j][0][2 * i + 1], o[j][1][2 * i + 1]);
  }
  __device__ __forceinline__ void give(float* to, int lane) const {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float4*>(to + ((lane >> 2) + 8 * i) * (D + 4) + 16 * j + 4 * (lane & 3)) = out(j, i);
  }
  // this state times own plus the given one times other (by row)
  __device__ __forceinline__ void take(const float* from, const float (&own)[R], const float (&other)[R], int lane) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(from + ((lane >> 2) + 8 * i) * (D + 4) + 16 * j + 4 * (lane & 3));
        const float4 x = out(j, i);
        o[j][0][2 * i] = x.x * own[i] + v.x * other[i];
        o[j][1][2 * i] = x.y * own[i] + v.y * other[i];
        o[j][0][2 * i + 1] = x.z * own[i] + v.z * other[i];
        o[j][1][2 * i + 1] = x.w * own[i] + v.w * other[i];
        if (R == 1) o[j][0][2] = o[j][0][3] = o[j][1][2] = o[j][1][3] = 0.f;
      }
  }
};

// The work of a call: units (sequence, kv head, row tile), each of as many
// steps as its sequence has spans of 128 tokens, one after another in that
// order.  CTA c of n takes steps [c q + min(c, r), ...) of the total n q + r,
// so all end together whatever the lengths; a unit cut between CTAs is joined
// by the CTA that finishes last.
struct Cursor {
  int b, h, mt, step;              // where
  int first, n, len, tiles, steps;   // of sequence b: queries, length; its row tiles and its spans
  int seen;                          // tokens that the last real row of tile mt sees
  // sequence b's sizes; no units where it has no rows or fails its checks
  __device__ __forceinline__ void sequence(const KvDims& d, const KvSeqs& s, const KvAttention& at, int tile_rows,
                                           int* status) {
    tiles = 0;
    steps = 1;
    if (!kv_sequence(s, at.cu_q, at.T_q, b, d, status, &first, &n, &len)) return;
    if (n > at.max_q) {
      set_status(status, MOE_ERR_DEVICE_CHECK);
      return;
    }
    if (at.few && n * (at.Hq / d.Hkv) > at.few) return;   // the other kernel's
    tiles = (n * (at.Hq / d.Hkv) + tile_rows - 1) / tile_rows;
    steps = max((len + kSpan - 1) / kSpan, 1);
  }
  __device__ __forceinline__ void look(int g, int tile_rows) {
    seen = max(len - n + (min((mt + 1) * tile_rows, n * g) - 1) / g + 1, 0);
  }
  __device__ __forceinline__ void next(const KvDims& d, const KvSeqs& s, const KvAttention& at, int tile_rows,
                                       int* status) {
    if (++step < steps) return;
    step = 0;
    if (++mt == tiles) {
      mt = 0;
      if (++h == d.Hkv) {
        h = 0;
        do {
          if (++b >= s.B) return;
          sequence(d, s, at, tile_rows, status);
        } while (tiles == 0);
      }
    }
    if (tiles > 1 || h == 0) look(at.Hq / d.Hkv, tile_rows);
  }
};

// Steps of sequence b.
__device__ __forceinline__ uint32_t steps_of(Cursor& c, int b, const KvDims& d, const KvSeqs& s,
                                              const KvAttention& at, int tile_rows, int* status) {
  if (b >= s.B) return 0;
  c.b = b;
  c.sequence(d, s, at, tile_rows, status);
  return static_cast<uint32_t>(c.tiles) * c.steps * d.Hkv;
}

// Workspace of a call: tickets (zero between calls), and two slots of partial
// results per CTA: slot 0 for the unit that an earlier CTA began, slot 1 for
// the one that it began itself.
constexpr int kMostCtas = 512;
struct Parts {
  int* ticket;   // by the CTA that began the unit
  float* o;      // [CTA][2][rows][D], relative to the row's maximum
  float2* ml;    // [CTA][2][rows]: maximum (base 2) and sum
  float* scores;   // 8-row tiles, nullable: [T_q * Hq][pitch], every row's scores in units of the base-2 exponent
  int pitch;
};

// The n parts of a unit, in order: a warp takes every kWarps-th row, a lane D / 32 columns.
template <int D, int R>
__device__ __forceinline__ void join_parts(const Parts& parts, int c0, int n, const KvAttention& at, int first, int h,
                                           int g, int row0, int rows, int warp, int lane) {
  constexpr int kRows = 8 * R, kPer = D / 32;
  for (int r = warp; r < kRows && row0 + r < rows; r += kWarps) {
    const auto slot = [&](int p) { return (static_cast<size_t>(c0 + p) * 2 + (p == 0)) * kRows + r; };
    float m = -INFINITY;
    for (int p = lane; p < n; p += 32) m = fmaxf(m, __ldcg(parts.ml + slot(p)).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float acc[kPer] = {}, l = 0.f;
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
      const float2 ml = __ldcg(parts.ml + slot(p));
      const float f = exp2_diff(ml.x, m);
      l += ml.y != ml.y ? ml.y : f * ml.y;
      const float* o = parts.o + slot(p) * D + lane * kPer;
      if (kPer == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(o));
        acc[0] += f * v.x;
        acc[1] += f * v.y;
        acc[kPer - 2] += f * v.z;
        acc[kPer - 1] += f * v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
        acc[0] += f * v.x;
        acc[1] += f * v.y;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = row0 + r;
    const size_t at_row = static_cast<size_t>(first + row / g) * at.Hq + h * g + row % g;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(at.out) + at_row * D + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && at.lse) at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// CTAs an SM holds, and stages of a warp's ring.  Tiles of 8 rows, D = 128: two
// CTAs of three stages (64 sequences of 513 to 16384 tokens: 206 us) against
// three of two (227 us: 168 registers, spilled); D = 64 fits three of three.
// Tiles of 16 rows have 8 KB more to meet in, so two of two stages (57 us on 4
// queries each of 16 sequences, 83 us at one CTA of three).
template <int D, int R>
constexpr int ctas_per_sm() { return D == 64 && R == 1 ? 3 : 2; }
template <int R>
constexpr int ring_stages() { return R == 1 ? 3 : 2; }

// Bound: HBM (2 D bytes per token and kv head, read once), behind it instruction
// issue (727 instructions a warp for 32 tokens, 256 of them V's codes to bf16, 64
// pairs of four): 64 sequences of 513 to 16384 tokens, 8 kv heads of 128: 207 us, 5.4 TB/s;
// one of 131071: 60 us, 4.5 TB/s.  16-row tiles (drafted tokens, two tiles of 16
// sequences) are bound by issue, 56 us for 68 MB.  Each of a CTA's
// four warps takes a quarter of every 128-token span, with a ring of
// asynchronous copies and a running softmax of its own; the ring runs on
// across units.  At a unit's end the warps' states meet in shared memory.
template <int D, int R>
__global__ void __launch_bounds__(kWarps * 32, ctas_per_sm<D, R>()) kv_decode_kernel(KvDims d, KvPool pool, KvSeqs s,
                                                                                 KvAttention at, Parts parts,
                                                                                 int* status) {
  constexpr int kRows = 8 * R, kPitch = D + 4, kStages = ring_stages<R>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 all_ml[kWarps * kRows];
  __shared__ int last;
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = at.Hq / d.Hkv;
  Cursor cur;
  uint32_t total = 0;   // (below 2^31: checked on the host for the largest lengths)
  for (int base = 0; base < s.B; base += 32)
    total += __reduce_add_sync(0xFFFFFFFFu, steps_of(cur, base + lane, d, s, at, kRows, status));
  const uint32_t ctas = min(total, gridDim.x), cta = blockIdx.x;
  if (cta >= ctas) return;
  const uint32_t q = total / ctas, r = total - q * ctas;
  const uint32_t start = cta * q + min(cta, r);
  const int count = static_cast<int>(q + (cta < r));
  uint32_t before = 0;   // the sequence, unit and step at `start`
  for (int base = 0;; base += 32) {
    const uint32_t w = steps_of(cur, base + lane, d, s, at, kRows, status);
    uint32_t upto = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += up;
    }
    const uint32_t beyond = __ballot_sync(0xFFFFFFFFu, before + upto > start);
    if (beyond) {
      const int l = __ffs(beyond) - 1;
      const uint32_t in = start - before - __shfl_sync(0xFFFFFFFFu, upto - w, l);
      cur.b = base + l;
      cur.sequence(d, s, at, kRows, status);
      const uint32_t unit = in / cur.steps;
      cur.step = static_cast<int>(in - unit * cur.steps);
      cur.h = static_cast<int>(unit / cur.tiles);
      cur.mt = static_cast<int>(unit - cur.h * cur.tiles);
      cur.look(g, kRows);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  Ring<D> ring{smem_u32(smem) + warp * kStages * Ring<D>::kStageBytes,
               reinterpret_cast<float*>(smem + kWarps * kStages * Ring<D>::kStageBytes) + warp * kStages * 4};
  float* meet = reinterpret_cast<float*>(smem + kWarps * kStages * (Ring<D>::kStageBytes + 16));
  Cursor ahead = cur;   // the step that is copied next
  int id[2];
  ring.look(id, d, s, ahead.b, ahead.step * kSpan + warp * kTok, ahead.seen);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < count) {
      ring.copy(i, id, d, pool, ahead.h, ahead.step * kSpan + warp * kTok, ahead.seen, lane, status);
      if (i + 1 < count) {
        ahead.next(d, s, at, kRows, status);
        ring.look(id, d, s, ahead.b, ahead.step * kSpan + warp * kTok, ahead.seen);
      }
    }
    cp_async_commit();
  }
  QueryTile<D, R> query;
  State<D, R> x;
  int sees[R], sees_least = 0, row0 = 0, rows = 0;
  float* keep = nullptr;
  int stage = 0;
  bool fresh = true;   // the unit that cur is in begins, for this CTA
  int from = cur.step;
  for (int i = 0; i < count; ++i) {
    __syncwarp();   // every lane is done with the stage that is filled now
    if (i + kStages - 1 < count) {
      ring.copy((stage + kStages - 1) % kStages, id, d, pool, ahead.h, ahead.step * kSpan + warp * kTok, ahead.seen,
                lane, status);
      if (i + kStages < count) {
        ahead.next(d, s, at, kRows, status);
        ring.look(id, d, s, ahead.b, ahead.step * kSpan + warp * kTok, ahead.seen);
      }
    }
    cp_async_commit();
    if (fresh) {
      fresh = false;
      from = cur.step;
      row0 = cur.mt * kRows;
      rows = cur.n * g;
      query.load(at, cur.first, cur.h, g, row0, rows, lane);
      x.clear();
#pragma unroll
      for (int j = 0; j < R; ++j)   // (rows beyond the last real one see what it sees)
        sees[j] = max(cur.len - cur.n + min(row0 + (lane >> 2) + 8 * j, rows - 1) / g + 1, 0);
      sees_least = max(cur.len - cur.n + row0 / g + 1, 0);
      if (R == 1 && parts.scores) {
        const int row = row0 + (lane >> 2);
        keep = row >= rows ? nullptr
                           : parts.scores + (static_cast<size_t>(cur.first + row / g) * at.Hq + cur.h * g + row % g) * parts.pitch;
      }
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const int t0 = cur.step * kSpan + warp * kTok;
    if (t0 < cur.seen) x.add(query, ring, stage, t0, sees, sees_least, keep, lane);
    stage = (stage + 1) % kStages;
    const bool whole = cur.step + 1 == cur.steps;
    if (whole || i + 1 == count) {
      // the warps' states meet: 2 and 3 hand theirs to 0 and 1, then 1 to 0
#pragma unroll
      for (int j = 0; j < R; ++j) {
        float l = x.l[j];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if ((lane & 3) == 0) all_ml[warp * kRows + (lane >> 2) + 8 * j] = make_float2(x.m[j], l);
      }
      if (warp >= 2) x.give(meet + (warp - 2) * kRows * kPitch, lane);
      __syncthreads();
      float m[R], l[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float2* ml = all_ml + (lane >> 2) + 8 * j;
        m[j] = fmaxf(fmaxf(ml[0].x, ml[kRows].x), fmaxf(ml[2 * kRows].x, ml[3 * kRows].x));
        l[j] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = ml[w * kRows];   // (a NaN sum belongs to a row of NaN scores, whose maximum is -inf)
          l[j] += v.y != v.y ? v.y : exp2_diff(v.x, m[j]) * v.y;
        }
      }
      if (warp < 2) {
        float own[R], other[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          own[j] = exp2_diff(x.m[j], m[j]);
          other[j] = exp2_diff(all_ml[(warp + 2) * kRows + (lane >> 2) + 8 * j].x, m[j]);
        }
        x.take(meet + warp * kRows * kPitch, own, other, lane);
      }
      __syncthreads();
      if (warp == 1) x.give(meet, lane);
      __syncthreads();
      const bool begun = from == 0;
      if (warp == 0) {
        float one[R];
#pragma unroll
        for (int j = 0; j < R; ++j) one[j] = 1.f;
        x.take(meet, one, one, lane);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int row = row0 + (lane >> 2) + 8 * j;
          if (row < rows) {
            const size_t at_row = static_cast<size_t>(cur.first + row / g) * at.Hq + cur.h * g + row % g;
            const size_t slot = (static_cast<size_t>(cta) * 2 + begun) * kRows + (lane >> 2) + 8 * j;
            const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const float4 o = x.out(c, j);
              const int col = 16 * c + 4 * (lane & 3);
              if (begun && whole)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(at.out) + at_row * D + col) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
              else
                *reinterpret_cast<float4*>(parts.o + slot * D + col) = o;
            }
            if ((lane & 3) == 0) {
              if (!(begun && whole))
                parts.ml[slot] = make_float2(m[j], l[j]);
              else if (at.lse)
                at.lse[at_row] = l[j] == 0.f ? -INFINITY : (m[j] + log2f(l[j])) * kLn2;
            }
          }
        }
      }
      if (!(begun && whole)) {
        // the CTAs of this unit's first and last step; the last to arrive joins their parts in order
        const uint32_t u0 = start + i - cur.step, u1 = u0 + cur.steps - 1;
        const auto owner = [&](uint32_t t) {
          const uint32_t longer = r * (q + 1);
          return static_cast<int>(t < longer ? t / (q + 1) : r + (t - longer) / q);
        };
        const int c0 = owner(u0), n_parts = owner(u1) - c0 + 1;
        __syncthreads();
        if (threadIdx.x == 0) {
          __threadfence();
          last = atomicAdd(parts.ticket + c0, 1) == n_parts - 1;
          __threadfence();
        }
        __syncthreads();
        if (last) {
          if (threadIdx.x == 0) parts.ticket[c0] = 0;
          join_parts<D, R>(parts, c0, n_parts, at, cur.first, cur.h, g, row0, rows, warp, lane);
        }
      }
      __syncthreads();   // `meet` is free again
      fresh = true;
    }
    if (i + 1 < count) cur.next(d, s, at, kRows, status);
  }
  cp_async_wait<0>();
}

// weights[b][h][t] += sum over the rows of (b, h) of exp(s_t - lse), the rows
// in order, so that the sums do not depend on scheduling.

// From the scores that the decode kernel kept (8-row tiles): four tokens a thread.
// Writing and reading 4 bytes per row and token beats reading K again (D bytes)
// up to these 8 rows.  Bound: HBM and L2, 4 rows + 8 bytes per token.
constexpr int kGainThreads = 128, kGainTokens = 4 * kGainThreads;
__global__ void __launch_bounds__(kGainThreads) kv_gain_kept_kernel(KvDims d, KvSeqs s, KvAttention at,
                                                                    const float* __restrict__ scores, int pitch,
                                                                    int* status) {
  chain_wait();
  ChainReleaseAtExit release;
  const int h = blockIdx.y, b = blockIdx.z, g = at.Hq / d.Hkv, t = (blockIdx.x * kGainThreads + threadIdx.x) * 4;
  Tile tile;
  if (!tile.find(s, at, b, g, 0, 8, d, status) || t >= tile.len) return;
  float sum[4] = {};
  for (int i = 0; i < tile.n; ++i) {
    const int sees = tile.len - tile.n + i + 1;   // tokens that query i sees
    if (t >= sees) continue;
    const size_t row0 = static_cast<size_t>(tile.first + i) * at.Hq + h * g;
#pragma unroll 4
    for (int r = 0; r < g; ++r) {
      float lse = at.lse[row0 + r] * kLog2e;
      if (lse == -INFINITY) lse = INFINITY;   // every page of the row's is missing: it adds nothing
      const float4 v = *reinterpret_cast<const float4*>(scores + (row0 + r) * pitch + t);   // (pitch holds whole steps)
      sum[0] += exp2_approx(v.x - lse);
      sum[1] += t + 1 < sees ? exp2_approx(v.y - lse) : 0.f;
      sum[2] += t + 2 < sees ? exp2_approx(v.z - lse) : 0.f;
      sum[3] += t + 3 < sees ? exp2_approx(v.w - lse) : 0.f;
    }
  }
  float* w = at.weights + (static_cast<long long>(b) * d.Hkv + h) * at.w_stride + t;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (t + e < tile.len) w[e] += sum[e];
}

// More rows: the scores again, from K and the queries as MMA operands, which a
// launch of their own lays out once in the order that lanes load them.
struct Laid {
  uint4* a;       // [tile][D / 16][32 lanes]
  float2* info;   // [tile][16]: what QueryTile::unscale is, and the row's lse in base 2 (+inf: adds nothing)
};
// The 16-row tiles of (sequence b, head h) lie at (floor(cu[b] g / 16) + b + tile) Hkv + h: a sequence of n
// rows has at most floor(n / 16) + 1 beyond the next one's start, so none meet and no prefix sum is needed.
__device__ __forceinline__ size_t laid_tile(const KvAttention& at, int first, int b, int g, int mt, int Hkv, int h) {
  return (static_cast<size_t>(first) * g / 16 + b + mt) * Hkv + h;
}
size_t laid_tiles(int Hq, int Hkv, int B, int T_q) {
  return (static_cast<size_t>(T_q) * (Hq / Hkv) / 16 + B) * Hkv;
}

template <int D>
__global__ void __launch_bounds__(128) kv_lay_kernel(KvDims d, KvSeqs s, KvAttention at, Laid laid, int* status) {
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, mt = blockIdx.x * 4 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  const int g = at.Hq / d.Hkv;
  Tile tile;
  if (!tile.find(s, at, b, g, mt, 16, d, status)) return;
  QueryTile<D, 2> q;
  q.load(at, tile.first, h, g, tile.row0, tile.rows, lane);
  const size_t slot = laid_tile(at, tile.first, b, g, mt, d.Hkv, h);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    laid.a[(slot * (D / 16) + k) * 32 + lane] = make_uint4(q.a[k][0], q.a[k][1], q.a[k][2], q.a[k][3]);
  if ((lane & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = tile.row0 + (lane >> 2) + 8 * i;
      float lse = r < tile.rows ? at.lse[static_cast<size_t>(tile.first + r / g) * at.Hq + h * g + r % g] : -INFINITY;
      if (lse == -INFINITY) lse = INFINITY;
      laid.info[slot * 16 + (lane >> 2) + 8 * i] = make_float2(r < tile.rows ? q.unscale[i] : 0.f, lse * kLog2e);
    }
  }
}

// A CTA per 256 tokens of a (sequence, kv head): each of eight warps holds 32
// tokens' codes in registers and runs over the row tiles that see them, the
// even ones in warps 0 to 7, the odd ones in 8 to 15; the two sums are added at
// the end.  The tiles come through a ring in shared memory that all warps read.
// With few such CTAs `parts` of them share the row tiles of the same tokens (a
// prompt of 4096 with weights: 650 us without, 477 with), and the last to end adds
// their sums in order.  Measured: 206 us for 247 M pairs of row and
// token (D = 128), the tensor pipe active 51% of the time.
// A stage is four pairs: with a barrier at each pair the warps' MMAs and
// exponentials fell into step.
constexpr int kGainWarps = 16, kGainStages = 3, kGainPairs = 4, kGainBlock = 256, kGainTickets = 4096;
struct GainParts {
  int parts;       // 1: no tickets
  int* ticket;     // [B][Hkv][blocks], zero between calls
  float* sums;     // [B][Hkv][blocks][parts][kGainBlock]
};
template <int D>
struct GainStage {
  uint4 a[kGainPairs][2][D / 16][32];
  float2 info[kGainPairs][2][16];
};
template <int D>
__global__ void __launch_bounds__(kGainWarps * 32) kv_gain_kernel(KvDims d, KvPool pool, KvSeqs s, KvAttention at,
                                                                  Laid laid, GainParts gp, int* status) {
  __shared__ int last;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float half[8][32];
  GainStage<D>* ring = reinterpret_cast<GainStage<D>*>(smem);
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y, b = blockIdx.z, g = at.Hq / d.Hkv;
  const int block = blockIdx.x / gp.parts, row_part = blockIdx.x % gp.parts;
  const int first = block * kGainBlock, t0 = first + (warp & 7) * kTok, part = warp >> 3, n = lane >> 2, c = lane & 3;
  Tile tile;
  if (!tile.find(s, at, b, g, 0, 16, d, status) || first >= tile.len) return;
  uint2 k[kTok / 8][D / 16];
  float ks[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + 16 * i;
    const int id = t < tile.len ? __ldg(s.table + static_cast<size_t>(b) * s.width + (t >> d.shift)) : -1;
    const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(pool.num_pages);
    if (t < tile.len && !ok) set_status(status, MOE_ERR_DEVICE_CHECK);
    ks[i] = ok ? __ldg(pool.k_scale + static_cast<size_t>(id) * d.Hkv + h) : __uint_as_float(0x7FFFFFFFu);
#pragma unroll
    for (int nt = 2 * i; nt < 2 * i + 2; ++nt) {
      const bool in = ok && t0 + nt * 8 + n < tile.len;
      const uint8_t* row = pool.k + (in ? kv_row(id, d.Hkv, h, d.page, (t0 + nt * 8 + n) & (d.page - 1), D) : 0);
#pragma unroll
      for (int f = 0; f < D / 64; ++f) {
        const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(row) + (D == 128 ? 2 * c + f : c)) : make_uint4(0, 0, 0, 0);
        k[nt][4 * f] = e4m3x4_to_f16x4(v.x);
        k[nt][4 * f + 1] = e4m3x4_to_f16x4(v.y);
        k[nt][4 * f + 2] = e4m3x4_to_f16x4(v.z);
        k[nt][4 * f + 3] = e4m3x4_to_f16x4(v.w);
      }
    }
  }
  // Row r sees token t where r >= (t - (len - n)) g.  Pairs of row tiles, from
  // the first that sees the CTA's first token.
  const int base = tile.len - tile.n, tiles = (tile.rows + 15) / 16, pairs = (tiles + 1) / 2;
  const int pair0 = (first > base ? (first - base) * g / 32 : 0) + row_part * kGainPairs;
  const int stride = gp.parts * kGainPairs;   // the parts take stages in turn
  const int need_any = t0 < tile.len ? max(t0 - base, 0) * g : INT_MAX;
  const int need_all = max(min(t0 + kTok, tile.len) - 1 - base, 0) * g;
  const bool gone = no_page(ks[0]) || no_page(ks[1]);
  const auto fetch = [&](int pair, int stage) {   // kGainPairs pairs from `pair` on
    GainStage<D>& st = ring[stage];
    constexpr int kVecs = D / 16 * 32;   // of a tile
    const int left = min(2 * kGainPairs, tiles - 2 * pair);
    for (int i = threadIdx.x; i < left * kVecs; i += kGainWarps * 32)
      cp_async16(smem_u32(&st.a[0][0][0][0] + i),
                 laid.a + laid_tile(at, tile.first, b, g, 2 * pair + i / kVecs, d.Hkv, h) * kVecs + i % kVecs);
    for (int i = threadIdx.x; i < left * 8; i += kGainWarps * 32)
      cp_async16(smem_u32(&st.info[0][0][0] + 2 * i),
                 laid.info + laid_tile(at, tile.first, b, g, 2 * pair + i / 8, d.Hkv, h) * 16 + i % 8 * 2);
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kGainStages - 1; ++i) fetch(pair0 + i * stride, i);
  float sum[kTok / 8][2] = {};
  int stage = 0;
  for (int pair = pair0; pair < pairs; pair += stride) {
    cp_async_wait<kGainStages - 2>();
    __syncthreads();   // everybody's copies of this stage are there; everybody is done with the one before
    fetch(pair + (kGainStages - 1) * stride, stage == 0 ? kGainStages - 1 : stage - 1);
    const GainStage<D>& st = ring[stage];
    stage = stage + 1 == kGainStages ? 0 : stage + 1;
#pragma unroll 1
    for (int q = 0; q < kGainPairs; ++q) {
      const int mt = 2 * (pair + q) + part;
      if (mt >= tiles || mt * 16 + 15 < need_any) continue;
      float x[kTok / 8][4] = {};
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        uint32_t a[4];
        *reinterpret_cast<uint4*>(a) = lds_u4(smem_u32(&st.a[q][part][f][lane]));
#pragma unroll
        for (int nt = 0; nt < kTok / 8; ++nt) mma_f16(x[nt], a, k[nt][f].x, k[nt][f].y);
      }
      const float2 r0 = st.info[q][part][n], r1 = st.info[q][part][8 + n];
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) {
        const float f0 = ks[nt >> 1] * r0.x, f1 = ks[nt >> 1] * r1.x;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[nt][e] = exp2_approx(fmaf(x[nt][e], f0, -r0.y));
          x[nt][2 + e] = exp2_approx(fmaf(x[nt][2 + e], f1, -r1.y));
        }
      }
      if (mt * 16 < need_all || gone) {
#pragma unroll
        for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int need = max(t0 + nt * 8 + 2 * c + e - base, 0) * g;   // (far below `base` the product would not fit)
            if (mt * 16 + n < need || no_page(ks[nt >> 1])) x[nt][e] = 0.f;
            if (mt * 16 + 8 + n < need || no_page(ks[nt >> 1])) x[nt][2 + e] = 0.f;
          }
      }
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) sum[nt][e] += x[nt][e] + x[nt][2 + e];
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][e], o);
      if (part == 1 && n == 0) half[warp & 7][nt * 8 + 2 * c + e] = sum[nt][e];
    }
  __syncthreads();
  float* w = at.weights + (static_cast<long long>(b) * d.Hkv + h) * at.w_stride + first;
  if (gp.parts == 1) {
    if (part == 0 && n == 0) {
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = nt * 8 + 2 * c + e;
          if (t0 + i < tile.len) w[t0 - first + i] += sum[nt][e] + half[warp][i];
        }
    }
    return;
  }
  const size_t slot = (static_cast<size_t>(b) * d.Hkv + h) * (gridDim.x / gp.parts) + block;
  float* sums = gp.sums + slot * gp.parts * kGainBlock;
  if (part == 0 && n == 0) {
#pragma unroll
    for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = nt * 8 + 2 * c + e;
        sums[row_part * kGainBlock + t0 - first + i] = sum[nt][e] + half[warp][i];
      }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(gp.ticket + slot, 1) == gp.parts - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) gp.ticket[slot] = 0;
  if (threadIdx.x < kGainBlock && first + static_cast<int>(threadIdx.x) < tile.len) {
    float v = 0.f;
    for (int p = 0; p < gp.parts; ++p) v += __ldcg(sums + p * kGainBlock + threadIdx.x);
    w[threadIdx.x] += v;
  }
}

// How many CTAs share a block of tokens: enough for four on every SM, each with two stages at least.
int gain_parts(int B, int Hkv, int max_len, long long rows) {
  const long long blocks = static_cast<long long>(B) * Hkv * ((static_cast<long long>(max_len) + kGainBlock - 1) / kGainBlock);
  if (blocks > kGainTickets || blocks == 0) return 1;
  const long long parts = std::min<long long>({8, (4 * kSMs + blocks - 1) / blocks, rows / (2 * kGainPairs * 32)});
  return parts > 1 ? static_cast<int>(parts) : 1;
}

// Workspace: the tickets first, at the same place for every call, then the
// parts, the log-sum-exps, and for the weights the kept scores or the laid out
// queries.
struct Layout {
  size_t gain_ticket, o, ml, lse, scores, laid, info, gain, part_o, part_ml, total;
  int pitch;
};

// Tiles of 8 rows where every sequence's rows fit one, else of 16: 4 rows over 16
// sequences of 8192 (8 kv heads of 128) 57 us, 63 with tiles of 16.
bool few_rows(int Hq, int Hkv, int max_q) { return static_cast<long long>(max_q) * (Hq / Hkv) <= 8; }

// The tensor-memory kernel for more than kDecodeRows rows of a kv head.  Decode
// against it, us, 8 kv heads of 128: 64 rows over one sequence of 32768 tokens 68
// and 65, 128 rows 114 and 67; over four of 32768, 64 rows 185 and 244, 128 rows
// 323 and 246; over 16 of 2048, 64 rows 64 and 65, 96 rows 86 and 65.  But where
// no decode CTA would have more than one step, its launch is the shorter one: a
// prompt of 128, 512 rows, 8.3 and 12.8; (one of 256, two steps and more: 21 and 16).
bool on_prefill(const KvDims& d, int Hq, int B, int max_q, int max_len) {
  const long long rows = static_cast<long long>(max_q) * (Hq / d.Hkv);
  const double steps = static_cast<double>(B) * d.Hkv * ((rows + 15) / 16) * ((static_cast<long long>(max_len) + kSpan - 1) / kSpan);
  return rows > kDecodeRows && steps > kSMs * ctas_per_sm<128, 2>();
}

// Beside it the decode kernel takes the sequences of up to so many rows, where
// there may be some (the shortest has T_q less the others' most); 0: it is not
// launched.  64 sequences of 513 to 8192 tokens, 63 asking for one token and one
// for 512 (8 kv heads of 128): 712 us with one kernel, 280 with both.  32 rows of
// 16, 32 and 64: 48 times 20 rows beside a chunk of 512, all over 4096 tokens, 388,
// 258 and 257 us; 16 sequences of 48 to 96 rows over 32768 945, 945 and 1198; but 12
// times 48 rows beside a chunk, over 8192, 479, 479 and 272.
int beside_prefill(const KvDims& d, int Hq, int B, int T_q, int max_q) {
  const long long least = T_q - static_cast<long long>(B - 1) * max_q;
  return B > 1 && least * (Hq / d.Hkv) <= kBesideRows ? kBesideRows : 0;
}

Layout layout(const KvDims& d, int Hq, int B, int T_q, int max_q, int max_len, bool weights) {
  constexpr size_t slots = static_cast<size_t>(kSMs) * ctas_per_sm<128, 2>() * 2 * 16;
  static_assert(ctas_per_sm<64, 2>() <= ctas_per_sm<128, 2>() && ctas_per_sm<128, 1>() <= ctas_per_sm<64, 1>() &&
                    slots >= static_cast<size_t>(kSMs) * ctas_per_sm<64, 1>() * 2 * 8,
                "slots of either tile size");
  static_assert(kSMs * ctas_per_sm<64, 1>() <= kMostCtas && kSMs * ctas_per_sm<128, 2>() <= kMostCtas, "tickets");
  Layout w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align_up(bytes);
    return r;
  };
  static_assert(align_up(kMostCtas * sizeof(int)) + align_up(kGainTickets * sizeof(int)) == MOE_KV_COUNTER_BYTES, "counters");
  take(kMostCtas * sizeof(int));
  w.gain_ticket = take(kGainTickets * sizeof(int));
  const size_t rows = static_cast<size_t>(T_q) * Hq;
  w.o = take(slots * d.D * sizeof(float));
  w.ml = take(slots * sizeof(float2));
  w.lse = take(rows * sizeof(float));
  if (on_prefill(d, Hq, B, max_q, max_len)) {
    const size_t part_rows = kv_prefill_part_rows(d, Hq, B, T_q, beside_prefill(d, Hq, B, T_q, max_q), max_len);
    w.part_o = take(part_rows * d.D * sizeof(float));
    w.part_ml = take(part_rows * sizeof(float2));
  }
  if (weights && few_rows(Hq, d.Hkv, max_q)) {
    w.pitch = static_cast<int>((static_cast<long long>(max_len) + kTok - 1) / kTok * kTok);
    w.scores = take(rows * w.pitch * sizeof(float));
  } else if (weights) {
    const size_t tiles = laid_tiles(Hq, d.Hkv, B, T_q);
    w.laid = take(tiles * 32 * d.D);
    w.info = take(tiles * 16 * sizeof(float2));
    const int parts = gain_parts(B, d.Hkv, max_len, static_cast<long long>(max_q) * (Hq / d.Hkv));
    const size_t blocks = static_cast<size_t>(B) * d.Hkv * ((static_cast<size_t>(max_len) + kGainBlock - 1) / kGainBlock);
    if (parts > 1) w.gain = take(blocks * parts * kGainBlock * sizeof(float));
  }
  w.total = at;
  return w;
}

template <int D, int R>
int launch_decode(const KvDims& d, const KvPool& pool, const KvSeqs& s, const KvAttention& a, const Parts& parts,
                  int* status, cudaStream_t stream, int* launches) {
  constexpr size_t smem = kWarps * ring_stages<R>() * (Ring<D>::kStageBytes + 16) + 2 * 8 * R * (D + 4) * sizeof(float);
  if (kv_allow_smem<kv_decode_kernel<D, R>>(smem) != cudaSuccess) return MOE_ERR_CUDA;
  // no more CTAs than the longest call of these sizes gives steps to
  long long rows = static_cast<long long>(a.max_q) * (a.Hq / d.Hkv);
  if (a.few) rows = std::min<long long>(rows, a.few);
  const long long tiles = (rows + 8 * R - 1) / (8 * R);
  const double steps = static_cast<double>(s.B) * d.Hkv * tiles * ((static_cast<long long>(s.max_len) + kSpan - 1) / kSpan + 1);
  if (steps > INT_MAX) return MOE_ERR_UNSUPPORTED;
  const int ctas = steps < kSMs * ctas_per_sm<D, R>() ? static_cast<int>(steps) : kSMs * ctas_per_sm<D, R>();
  if (launch_chained(kv_decode_kernel<D, R>, dim3(ctas), dim3(kWarps * 32), smem, stream, d, pool, s, a, parts,
                     status) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

template <int D>
int launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, KvAttention a, void* ws, int* status,
           cudaStream_t stream, int* launches) {
  const Layout w = layout(d, a.Hq, s.B, a.T_q, a.max_q, s.max_len, a.weights != nullptr);
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (a.weights && !a.lse) a.lse = reinterpret_cast<float*>(base + w.lse);
  const bool few = few_rows(a.Hq, d.Hkv, a.max_q);
  const Parts parts{reinterpret_cast<int*>(base), reinterpret_cast<float*>(base + w.o),
                    reinterpret_cast<float2*>(base + w.ml),
                    a.weights && few ? reinterpret_cast<float*>(base + w.scores) : nullptr, w.pitch};
  const long long rows = static_cast<long long>(a.max_q) * (a.Hq / d.Hkv);
  int rc = MOE_OK;
  const bool prefill = on_prefill(d, a.Hq, s.B, a.max_q, s.max_len);
  if (prefill) {
    a.few = beside_prefill(d, a.Hq, s.B, a.T_q, a.max_q);
    rc = kv_prefill_launch(d, pool, s, a, reinterpret_cast<float*>(base + w.part_o),
                           reinterpret_cast<float2*>(base + w.part_ml), status, stream, launches);
  }
  if (rc == MOE_OK && (!prefill || a.few))
    rc = few ? launch_decode<D, 1>(d, pool, s, a, parts, status, stream, launches)
             : launch_decode<D, 2>(d, pool, s, a, parts, status, stream, launches);
  if (rc || !a.weights || s.max_len == 0) return rc;
  if (few) {
    const unsigned blocks = (static_cast<unsigned>(s.max_len) + kGainTokens - 1) / kGainTokens;
    if (launch_chained(kv_gain_kept_kernel, dim3(blocks, d.Hkv, s.B), dim3(kGainThreads), 0, stream, d, s, a,
                       parts.scores, parts.pitch, status) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++*launches;
    return MOE_OK;
  }
  const Laid laid{reinterpret_cast<uint4*>(base + w.laid), reinterpret_cast<float2*>(base + w.info)};
  const unsigned tiles = static_cast<unsigned>((rows + 15) / 16);
  const unsigned blocks = (static_cast<unsigned>(s.max_len) + kGainBlock - 1) / kGainBlock;
  const GainParts gp{gain_parts(s.B, d.Hkv, s.max_len, rows), reinterpret_cast<int*>(base + w.gain_ticket),
                     reinterpret_cast<float*>(base + w.gain)};
  if (launch_chained(kv_lay_kernel<D>, dim3((tiles + 3) / 4, d.Hkv, s.B), dim3(128), 0, stream, d, s, a, laid,
                     status) != cudaSuccess ||
      kv_allow_smem<kv_gain_kernel<D>>(kGainStages * sizeof(GainStage<D>)) != cudaSuccess ||
      launch_chained(kv_gain_kernel<D>, dim3(blocks * gp.parts, d.Hkv, s.B), dim3(kGainWarps * 32),
                     kGainStages * sizeof(GainStage<D>), stream, d, pool, s, a, laid, gp, status) != cudaSuccess)
    return MOE_ERR_CUDA;
  *launches += 2;
  return MOE_OK;
}

}  // namespace

size_t kv_attention_ws_bytes(const KvDims& d, int Hq, int B, int T_q, int max_q, int max_len, bool weights) {
  return layout(d, Hq, B, T_q, max_q, max_len, weights).total;
}

int kv_attention_launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, const KvAttention& a, void* ws,
                        int* status, cudaStream_t stream, int* launches) {
  return d.D == 128 ? launch<128>(d, pool, s, a, ws, status, stream, launches)
                    : launch<64>(d, pool, s, a, ws, status, stream, launches);
}

}  // namespace moe
