// Attention of many query rows over the 8-bit paged KV cache (prompts and
// prompt chunks), on the 5th-generation tensor cores.  The definition is
// kv_attention.cu's; rows are (query, head) pairs of one kv head.
//
// A CTA takes two tiles of 128 rows of one (sequence, kv head) over the tokens
// that they see, 128 at a time:
//  - four warps convert the tokens' codes into shared memory, K to f16 and V to
//    bf16 (both exact), in the 128-byte swizzle of the MMA's operands;
//  - one thread issues the MMAs: S = Q K^T (f16, accumulator in tensor memory),
//    then O += P V (bf16, P from tensor memory, V with its head dimension
//    contiguous);
//  - a warpgroup for each tile turns S into the weights P, a row per thread.
//    P takes the tensor memory of S: the 32 columns of 32 tokens' scores become
//    16 of their weights' high bf16 terms and 16 of the low ones (16 bits in
//    all, at any size, as in the decode kernel), so PV is two MMAs per step.
// The two tiles alternate: one's softmax runs under the other's MMAs.
//
// A page's V scale is 2^e times a mantissa in [1, 2): 2^e goes into the V
// operand (exact), the mantissa into the weights' exponent, and the row's sum
// takes it out again, w / mantissa; for power-of-two scales it is 1.
#include <limits.h>

#include "kv_cache.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;              // rows of a tile, and tokens of a step
constexpr int kThreads = 416;           // 2 x 4 softmax warps, 4 converter warps, 1 MMA warp
constexpr int kConverter0 = 256, kMmaWarp = 12;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;           // see the decode kernel: the maximum follows beyond 2^8 only

struct PrefillArgs {
  KvDims d;
  KvPool pool;
  KvSeqs s;
  KvAttention at;
  int* status;
  uint64_t wait_ns;
};

// What the softmax needs of a step's 16-token groups.
struct Group {
  float ks;    // K scale; kNoPage: the page is not there
  float lv;    // log2 of the V scale's mantissa
  float inv;   // its inverse
  float pad;
};
constexpr uint32_t kNoPage = 0x7FFFFFFFu;   // (a NaN)

template <int D>
struct Smem {
  static constexpr int kOperand = kTile * D * 2;   // a tile of Q, K or V: D / 64 blocks of 128 rows x 128 bytes
  static constexpr int kBlock = kTile * 128;
  static constexpr int q = 0, k = 2 * kOperand, v = 4 * kOperand, ctrl = 6 * kOperand;
  static constexpr int kCtrl = 1024;
  static constexpr int total = ctrl + kCtrl + 1024;   // the tiles start on 1024 bytes
};

struct Ctrl {
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], scale_full[4], drain;
  uint32_t tmem;
  int abort;
  Group group[4][8];   // four steps: a step's are read until the step two later has its scores
};
static_assert(sizeof(Ctrl) <= 1024, "control region");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Instruction descriptor of kind::f16: fp32 accumulator, M x N; bf16 or f16
// operands, B K-major or with its N index contiguous.
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool bf16, bool b_n_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_n_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory descriptor of a 128-byte-swizzled operand whose contiguous
// index is N: blocks of 64 elements (128 bytes) of N, `block` bytes apart, in
// each of them 8-row groups of K, 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_n128(uint32_t saddr, uint32_t block) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(block >> 4) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}

// Two e4m3 codes (the halves of 16 bits) as f16: the hardware conversion, exact.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t v) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(v));
  return r;
}
// Four codes as bf16 times `unit` (a bf16 pair of 2^(120 + e))
__device__ __forceinline__ uint2 e4m3x4_to_bf16x4(uint32_t v, uint32_t unit) {
  return make_uint2(bf16x2_mul((prmt(v, 0u, 0x9180u) << 4) & 0x87F087F0u, unit),
                    bf16x2_mul((prmt(v, 0u, 0xB3A2u) << 4) & 0x87F087F0u, unit));
}

// A V scale's power of two, bounded so that the bf16 operand and the rest stay in range.
__device__ __forceinline__ int v_exponent(float vs) {
  const int e = static_cast<int>(__float_as_uint(vs) >> 23 & 255u) - 127;
  return max(-100, min(e, 7));
}
__device__ __forceinline__ bool v_is_zero(float vs) { return (__float_as_uint(vs) & 0x7F800000u) == 0; }

// The converters' part: K and V of every step, each into a ring of two.
template <int D>
__device__ __forceinline__ void convert(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, int b, int h, int end,
                                        int steps) {
  using S = Smem<D>;
  constexpr int kHalves = D / 64;
  const int tid = threadIdx.x - kConverter0;
  // a quarter warp covers two rows' four chunks: its 16-byte stores meet no bank twice
  const int q4 = tid & 3, r = tid >> 2;
  volatile int* abort = &ctrl->abort;
  int id[4];
  const auto look = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 32 * i + r;
      id[i] = -1;
      if (t < end) {
        id[i] = __ldg(a.s.table + static_cast<size_t>(b) * a.s.width + (t >> a.d.shift));
        if (static_cast<uint32_t>(id[i]) >= static_cast<uint32_t>(a.pool.num_pages)) {
          set_status(a.status, MOE_ERR_DEVICE_CHECK);
          id[i] = -1;
        }
      }
    }
  };
  const auto load = [&](uint4 (&x)[4 * kHalves], const uint8_t* pool, int t0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* row = pool;
      if (id[i] >= 0) row += kv_row(id[i], a.d.Hkv, h, a.d.page, (t0 + 32 * i + r) & (a.d.page - 1), D) + q4 * 16;
#pragma unroll
      for (int f = 0; f < kHalves; ++f)
        x[4 * f + i] = id[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(row + 64 * f)) : make_uint4(0, 0, 0, 0);
    }
  };
  const auto at = [&](int f, int row, int e) {
    return f * S::kBlock + row * 128 + (((2 * q4 + e) ^ (row & 7)) << 4);
  };
  uint4 kx[4 * kHalves], vx[4 * kHalves];
  float vs[4];
  look(0);
  load(kx, a.pool.k, 0);
  for (int j = 0; j < steps; ++j) {
    const int t0 = j * kTile, st = j & 1;
    const uint32_t parity = (j >> 1) & 1;
    load(vx, a.pool.v, t0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vs[i] = id[i] >= 0 ? __ldg(a.pool.v_scale + static_cast<size_t>(id[i]) * a.d.Hkv + h) : 0.f;
    if (tid < 8) {
      const int t = t0 + 16 * tid;
      int page = t < end ? __ldg(a.s.table + static_cast<size_t>(b) * a.s.width + (t >> a.d.shift)) : -1;
      Group g{__uint_as_float(kNoPage), 0.f, 1.f, 0.f};
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pool.num_pages)) {
        const size_t of = static_cast<size_t>(page) * a.d.Hkv + h;
        g.ks = __ldg(a.pool.k_scale + of);
        const float v = __ldg(a.pool.v_scale + of);
        if (!v_is_zero(v)) {
          const float m = v * __uint_as_float(static_cast<uint32_t>(127 - v_exponent(v)) << 23);
          g.lv = log2f(m);
          g.inv = 1.f / m;
        }
      }
      *reinterpret_cast<float4*>(&ctrl->group[j & 3][tid]) = make_float4(g.ks, g.lv, g.inv, 0.f);
      mbar_arrive(&ctrl->scale_full[j & 3]);
    }
    if (!mbar_wait(&ctrl->k_empty[st], parity ^ 1u, abort, a.status, a.wait_ns)) return;
    const uint32_t kt = smem + S::k + st * S::kOperand, vt = smem + S::v + st * S::kOperand;
#pragma unroll
    for (int f = 0; f < kHalves; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = kx[4 * f + i];
        const uint2 c0 = e4m3x4_to_f16x4(x.x), c1 = e4m3x4_to_f16x4(x.y), c2 = e4m3x4_to_f16x4(x.z),
                    c3 = e4m3x4_to_f16x4(x.w);
        sts_u4(kt + at(f, 32 * i + r, 0), make_uint4(c0.x, c0.y, c1.x, c1.y));
        sts_u4(kt + at(f, 32 * i + r, 1), make_uint4(c2.x, c2.y, c3.x, c3.y));
      }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->k_full[st]);
    if (j + 1 < steps) {
      look(t0 + kTile);
      load(kx, a.pool.k, t0 + kTile);
    }
    if (!mbar_wait(&ctrl->v_empty[st], parity ^ 1u, abort, a.status, a.wait_ns)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = v_is_zero(vs[i]) ? 0u : static_cast<uint32_t>(v_exponent(vs[i]) + 247) << 7;
      const uint32_t unit = u | u << 16;
#pragma unroll
      for (int f = 0; f < kHalves; ++f) {
        const uint4 x = vx[4 * f + i];
        const uint2 c0 = e4m3x4_to_bf16x4(x.x, unit), c1 = e4m3x4_to_bf16x4(x.y, unit),
                    c2 = e4m3x4_to_bf16x4(x.z, unit), c3 = e4m3x4_to_bf16x4(x.w, unit);
        sts_u4(vt + at(f, 32 * i + r, 0), make_uint4(c0.x, c0.y, c1.x, c1.y));
        sts_u4(vt + at(f, 32 * i + r, 1), make_uint4(c2.x, c2.y, c3.x, c3.y));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->v_full[st]);
  }
}

// The MMA thread's part.
template <int D>
__device__ __forceinline__ void multiply(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, uint32_t tmem, int tiles,
                                         int steps) {
  using S = Smem<D>;
  constexpr uint32_t kScores = idesc_f32(kTile, kTile, false, false), kOut = idesc_f32(kTile, D, true, true);
  volatile int* abort = &ctrl->abort;
  const auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort, a.status, a.wait_ns); };
  // S of tile t over step j's tokens
  const auto scores = [&](int t, int j) {
    const uint32_t q = smem + S::q + t * S::kOperand, k = smem + S::k + (j & 1) * S::kOperand;
    tc_fence_after();
#pragma unroll
    for (int f = 0; f < D / 64; ++f) {
      const uint64_t dq = smem_desc_k128(q + f * S::kBlock), dk = smem_desc_k128(k + f * S::kBlock);
#pragma unroll
      for (int i = 0; i < 4; ++i) umma_bf16(tmem + t * kTile, dq + 2 * i, dk + 2 * i, kScores, f + i > 0);
    }
    umma_commit(&ctrl->s_full[t]);
  };
  for (int t = 0; t < tiles; ++t)
    if (!wait(&ctrl->q_full[t], 0)) return;
  if (!wait(&ctrl->k_full[0], 0)) return;
  for (int t = 0; t < tiles; ++t) scores(t, 0);
  umma_commit(&ctrl->k_empty[0]);
  for (int j = 0; j < steps; ++j) {
    const uint32_t v = smem + S::v + (j & 1) * S::kOperand;
    for (int t = 0; t < tiles; ++t) {
      if (t == 0 && !wait(&ctrl->v_full[j & 1], (j >> 1) & 1)) return;
      if (!wait(&ctrl->p_full[t], j & 1)) return;
      tc_fence_after();
      const uint32_t o = tmem + 2 * kTile + t * D, p = tmem + t * kTile;
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) {
        const uint64_t dv = smem_desc_n128(v + i * 2048, S::kBlock);
        const uint32_t hi = p + 32 * (i >> 1) + 8 * (i & 1);
        umma_bf16_ts(o, hi, dv, kOut, j + i > 0);
        umma_bf16_ts(o, hi + 16, dv, kOut, 1);
      }
      umma_commit(&ctrl->o_full[t]);
      if (t + 1 == tiles) umma_commit(&ctrl->v_empty[j & 1]);
      if (j + 1 < steps) {
        if (t == 0 && !wait(&ctrl->k_full[(j + 1) & 1], ((j + 1) >> 1) & 1)) return;
        // the next scores overwrite the weights: only once their product is done
        if (!wait(&ctrl->o_full[t], j & 1)) return;
        scores(t, j + 1);
        if (t + 1 == tiles) umma_commit(&ctrl->k_empty[(j + 1) & 1]);
      }
    }
  }
}

// A softmax warpgroup's part: a row per thread.
template <int D>
__device__ __forceinline__ void softmax(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, uint32_t tmem, int t, int b,
                                        int h, int g, int first, int n, int len, int row0, int steps) {
  using S = Smem<D>;
  const KvAttention& at = a.at;
  volatile int* abort = &ctrl->abort;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, in_tile = quad * 32 + lane;
  const int row = row0 + t * kTile + in_tile, rows = n * g;
  const bool real = row < rows;
  const size_t at_row = static_cast<size_t>(first + (real ? row / g : 0)) * at.Hq + h * g + (real ? row % g : 0);
  // (rows beyond the last real one see what it sees)
  const int sees = max(len - n + min(row, rows - 1) / g + 1, 0);
  const int sees_least = max(len - n + min(row - lane, rows - 1) / g + 1, 0);   // of the warp's rows
  float unscale;
  {   // the row to f16 times a power of two, its largest magnitude in [2^7, 2^8)
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(at.q) +
                             static_cast<long long>(first + (real ? row / g : 0)) * at.q_stride +
                             (static_cast<long long>(h) * g + (real ? row % g : 0)) * D;
    uint32_t m = 0;
    uint4 x[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      x[i] = real ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                               __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
    }
    m = max(m & 0xFFFFu, m >> 16);
    const uint32_t e = max(m >> 7, 8u);
    // (the sign of the scale goes with the row, so that larger scores are larger products)
    const float up = copysignf(__uint_as_float((261 - e) << 23), at.scale);
    unscale = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : fabsf(at.scale) * kLog2e * __uint_as_float((e - 7) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(c[k]) : "f"(bf16_hi(w[k]) * up), "f"(bf16_lo(w[k]) * up));
      sts_u4(smem + S::q + t * S::kOperand + (i >> 3) * S::kBlock + in_tile * 128 + (((i & 7) ^ (in_tile & 7)) << 4),
             make_uint4(c[0], c[1], c[2], c[3]));
    }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->q_full[t]);
  }
  const uint32_t lanes = static_cast<uint32_t>(quad) << 21;   // 32 quad in the address's lane field
  const uint32_t sc = tmem + lanes + t * kTile, o = tmem + lanes + 2 * kTile + t * D;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < steps; ++j) {
    const Group* group = ctrl->group[j & 3];
    bool ok = mbar_wait(&ctrl->scale_full[j & 3], (j >> 2) & 1, abort, a.status, a.wait_ns) &&
              mbar_wait(&ctrl->s_full[t], j & 1, abort, a.status, a.wait_ns);
    if (!__all_sync(0xFFFFFFFFu, ok)) return;
    tc_fence_after();
    const int t0 = j * kTile;
    bool masks = t0 + kTile > sees_least;
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t s[32];
      tmem_ld_32cols(sc + 32 * c, s);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ks = group[2 * c + e].ks;
        masks |= __float_as_uint(ks) == kNoPage;
        float x = -INFINITY;
        if (!masks) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x = fmaxf(x, __uint_as_float(s[16 * e + i]));
        } else if (__float_as_uint(ks) != kNoPage) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + 32 * c + 16 * e + i < sees) x = fmaxf(x, __uint_as_float(s[16 * e + i]));
        }
        if (x != -INFINITY) top = fmaxf(top, x * (ks * unscale));
      }
    }
    if (__any_sync(0xFFFFFFFFu, top > m + kSlack)) {
      top = fmaxf(top, m);
      const float f = m == -INFINITY ? 0.f : ex2(m - top);
      m = top;
      l *= f;
      if (j > 0) {   // (the scores of step j came after the product of step j - 1)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld_32cols(o + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
          tmem_st_32cols(o + 32 * c, v);
        }
      }
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t s[32];
      tmem_ld_32cols(sc + 32 * c, s);
      tmem_ld_wait();
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 gr = *reinterpret_cast<const float4*>(&group[2 * c + e]);
        const float f = gr.x * unscale, add = gr.y - base;
        const int t_first = t0 + 32 * c + 16 * e;
        if (masks) {
          const int left = __float_as_uint(gr.x) == kNoPage ? 0 : sees - t_first;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[16 * e + i] = i < left ? __float_as_uint(fmaf(__uint_as_float(s[16 * e + i]), f, add)) : 0xFF800000u;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[16 * e + i] = __float_as_uint(fmaf(__uint_as_float(s[16 * e + i]), f, add));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w0 = ex2(__uint_as_float(s[16 * e + 2 * i])), w1 = ex2(__uint_as_float(s[16 * e + 2 * i + 1]));
          l = fmaf(w0, gr.z, l);
          l = fmaf(w1, gr.z, l);
          const uint32_t u0 = __float_as_uint(w0), u1 = __float_as_uint(w1);
          hi[8 * e + i] = prmt(u0, u1, 0x7632u);
          lo[8 * e + i] = pack_bf16x2(w0 - __uint_as_float(u0 & 0xFFFF0000u), w1 - __uint_as_float(u1 & 0xFFFF0000u));
        }
      }
      tmem_st_16cols(sc + 32 * c, hi);
      tmem_st_16cols(sc + 32 * c + 16, lo);
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&ctrl->p_full[t]);
  }
  if (steps > 0) {
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctrl->o_full[t], (steps - 1) & 1, abort, a.status, a.wait_ns))) return;
    tc_fence_after();
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(at.out) + at_row * D);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t v[32];
    if (steps > 0) {
      tmem_ld_32cols(o + 32 * c, v);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0;
    }
    if (!real) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]) * inv, __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
      out[4 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (real && at.lse) at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(PrefillArgs a, int pairs) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(base + S::ctrl);
  const uint32_t smem = smem_u32(base);
  chain_wait();
  ChainReleaseAtExit release;
  // the rows that see most first: the last CTAs to start are the shortest
  const int heads = a.s.B * a.d.Hkv, unit = blockIdx.x % heads, pair = pairs - 1 - blockIdx.x / heads;
  const int b = unit / a.d.Hkv, h = unit % a.d.Hkv, g = a.at.Hq / a.d.Hkv;
  int first, n, len;
  if (!kv_sequence(a.s, a.at.cu_q, a.at.T_q, b, a.d.page, a.status, &first, &n, &len)) return;
  if (n > a.at.max_q) {
    set_status(a.status, MOE_ERR_DEVICE_CHECK);
    return;
  }
  const int rows = n * g, row0 = pair * 2 * kTile;
  if (row0 >= rows) return;
  const int tiles = row0 + kTile < rows ? 2 : 1;
  const int end = max(len - n + (min(row0 + 2 * kTile, rows) - 1) / g + 1, 0);   // what the last row sees
  const int steps = (end + kTile - 1) / kTile;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctrl->q_full[i], kTile);
      mbar_init(&ctrl->k_full[i], kTile);
      mbar_init(&ctrl->v_full[i], kTile);
      mbar_init(&ctrl->p_full[i], kTile);
      mbar_init(&ctrl->k_empty[i], 1);
      mbar_init(&ctrl->v_empty[i], 1);
      mbar_init(&ctrl->s_full[i], 1);
      mbar_init(&ctrl->o_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ctrl->scale_full[i], 8);
    mbar_init(&ctrl->drain, 1);
    ctrl->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctrl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;
  if (warp < 8) {
    if (warp / 4 < tiles) softmax<D>(a, ctrl, smem, tmem, warp / 4, b, h, g, first, n, len, row0, steps);
  } else if (warp < kMmaWarp) {
    convert<D>(a, ctrl, smem, b, h, end, steps);
  } else {
    if ((threadIdx.x & 31) == 0 && steps > 0) {
      multiply<D>(a, ctrl, smem, tmem, tiles, steps);
      // whatever was issued is done before the tensor memory goes
      umma_commit(&ctrl->drain);
      mbar_wait_timed(&ctrl->drain, 0, a.status);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
int launch(const PrefillArgs& a, cudaStream_t stream, int* launches) {
  if (cudaFuncSetAttribute(kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::total) != cudaSuccess)
    return MOE_ERR_CUDA;
  const long long rows = static_cast<long long>(a.at.max_q) * (a.at.Hq / a.d.Hkv);
  const long long pairs = (rows + 2 * kTile - 1) / (2 * kTile);
  const double ctas = static_cast<double>(pairs) * a.s.B * a.d.Hkv;
  if (ctas > INT_MAX) return MOE_ERR_UNSUPPORTED;
  if (launch_chained(kv_prefill_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), Smem<D>::total, stream, a,
                     static_cast<int>(pairs)) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

}  // namespace

int kv_prefill_launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, const KvAttention& at, int* status,
                      cudaStream_t stream, int* launches) {
  const PrefillArgs a{d, pool, s, at, status, wait_limit_ns()};
  return d.D == 128 ? launch<128>(a, stream, launches) : launch<64>(a, stream, launches);
}

}  // namespace moe
