// Attention of many query rows over the 8-bit paged KV cache (prompts and
// prompt chunks), on the 5th-generation tensor cores.  The definition is
// kv_attention.cu's; rows are (query, head) pairs of one kv head.
//
// A CTA takes two tiles of 128 rows of one (sequence, kv head) over the tokens
// that they see, 64 at a time:
//  - four warps convert the tokens' codes into shared memory, K to f16 and V to
//    bf16 (both exact), in the 128-byte swizzle of the MMA's operands;
//  - two warps a tile issue the MMAs: S = Q K^T (f16, accumulator in tensor
//    memory), and O += P V (bf16, P from tensor memory, V with its head
//    dimension contiguous);
//  - a warpgroup for each tile turns S into the weights P, a row per thread.
//    P takes the tensor memory of S: the 32 columns of 32 tokens' scores become
//    16 of their weights' high bf16 terms and 16 of the low ones (16 bits in
//    all, at any size, as in the decode kernel), so PV is two MMAs per step.
// A tile's S has two buffers, so that the scores of the next step are there when
// a softmax ends, and neither it nor the MMAs wait for each other's last piece.
//
// Bound: instruction issue of the softmax and the converters, in step with the
// MMAs.  One prompt of 8192 (32 heads of 128, 8 kv heads): 784 us, 0.70 PFLOP/s of
// the definition's operations, where the two-term weights alone cost half as many
// MMAs again; the tensor pipe is active 43% of the time, the issue slots 55%.
// What got it there from 1097 us (all same prompt): MMA operands in uniform
// registers and waits tested inline (the MMA warp's own instructions between two
// waits were the longest chain), 64-token steps with two S buffers, the running
// maximum followed only where weights grow (no pass over S for it).  Tried and
// slower: steps of 128 tokens with S in one buffer (815 us: both tiles' softmaxes
// run at once and the tensor cores wait), the same with the tiles taking turns
// (838 us).
//
// Where there are fewer CTAs than half the SMs the key axis is cut in parts, and
// kv_prefill_join_kernel adds what they leave in the workspace.
//
// A page's V scale is 2^e times a mantissa in [1, 2): 2^e goes into the V
// operand (exact), the mantissa into the weights' exponent, and the row's sum
// takes it out again, w / mantissa; for power-of-two scales it is 1.
#include <limits.h>
#include <stddef.h>

#include <algorithm>

#include "kv_cache.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;              // rows of a tile
constexpr int kStep = 64;               // tokens of a step
constexpr int kRing = 4;                // steps of K and of V in shared memory
// Warps: 0 and 1 issue the tiles' score MMAs, 2 and 3 their output MMAs (a warp's
// next barrier test waits behind the MMAs that it has issued), 4 to 7 and 8 to 11
// are the tiles' softmax, 12 to 15 convert.
constexpr int kThreads = 512;
constexpr int kSoftmaxWarp = 4, kConvertWarp = 12;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLarge = 512.f;         // where 32 weights pass it together, the maximum that they are taken against follows

struct PrefillArgs {
  KvDims d;
  KvPool pool;
  KvSeqs s;
  KvAttention at;
  int* status;
  uint64_t wait_ns;
  // The key axis cut in parts, at steps: a part's O (relative to its maximum), its
  // maxima and sums, by [part][unit][row of the unit].
  int most_parts;    // 1: not cut
  float* part_o;     // rows of D
  float2* part_ml;
};

// A unit: two tiles of rows of a (sequence, kv head).  They count by sequence, in
// it from the rows that see most, heads innermost: as many as the real sequences
// have.  A converged warp finds unit u (sequences that fail their checks have
// none) and returns whether there is one; `total`, if asked, is their number.
// Four sequences a lane: 255 sequences of one token and two prompts of 1024 took
// 377 us with one, 364 with four.  (Scanned by the CTA, 337, but a prompt of 8192 took
// 795 us, 782 now.)
struct Unit {
  int b, h, pair, first, n, len;
};
__device__ __forceinline__ bool find_unit(const PrefillArgs& a, int u, Unit* unit, int* total) {
  constexpr int kPer = 4;
  const int lane = threadIdx.x & 31, g = a.at.Hq / a.d.Hkv;
  int before = 0;
  bool found = false;
  for (int base = 0; base < a.s.B && (total || !found); base += 32 * kPer) {
    int first[kPer], n[kPer], len[kPer], pairs[kPer], upto = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int b = base + kPer * lane + k;
      const bool in = b < a.s.B;
      first[k] = in ? __ldg(a.at.cu_q + b) : 0;
      n[k] = in ? __ldg(a.at.cu_q + b + 1) : 0;
      len[k] = in ? __ldg(a.s.seq_lens + b) : 0;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      n[k] -= first[k];
      pairs[k] = 0;
      if (kv_sequence_is(a.s, a.at.T_q, a.d, a.status, first[k], n[k], len[k])) {
        if (n[k] > a.at.max_q)
          set_status(a.status, MOE_ERR_DEVICE_CHECK);
        else if (n[k] * g > a.at.few)
          pairs[k] = (n[k] * g + 2 * kTile - 1) / (2 * kTile);
      }
      upto += pairs[k] * a.d.Hkv;
    }
    const int mine = upto;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, i);
      if (lane >= i) upto += v;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, u - before < upto);
    if (!found && hit) {
      const int from = __ffs(hit) - 1;
      int in = u - before - (upto - mine);   // (what counts is lane `from`'s)
      Unit x{};
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int units = pairs[k] * a.d.Hkv;
        if (in >= 0 && in < units)
          x = Unit{base + kPer * lane + k, in % a.d.Hkv, pairs[k] - 1 - in / a.d.Hkv, first[k], n[k], len[k]};
        in -= units;
      }
      *unit = Unit{__shfl_sync(0xFFFFFFFFu, x.b, from),     __shfl_sync(0xFFFFFFFFu, x.h, from),
                   __shfl_sync(0xFFFFFFFFu, x.pair, from),  __shfl_sync(0xFFFFFFFFu, x.first, from),
                   __shfl_sync(0xFFFFFFFFu, x.n, from),     __shfl_sync(0xFFFFFFFFu, x.len, from)};
      found = true;
    }
    before = min(before + __shfl_sync(0xFFFFFFFFu, upto, 31), 1 << 30);   // (boundaries that overlap: no overflow)
  }
  if (total) *total = before;
  return found;
}

// Parts of `units` units: as many as give each SM a CTA.
__device__ __forceinline__ int parts_of(const PrefillArgs& a, int units) {
  return units == 0 ? 1 : max(1, min(kSMs / units, a.most_parts));
}

// Steps of a part of a unit of `steps`: the same in the kernel and in the join.
__device__ __forceinline__ int part_steps(int steps, int parts) { return (steps + parts - 1) / parts; }

// What the softmax needs of a step's 16-token groups.
struct alignas(16) Group {   // (one 16-byte access)
  float ks;    // K scale; kNoPage: the page is not there
  float lv;    // log2 of the V scale's mantissa
  float inv;   // its inverse
  float pad;
};
constexpr uint32_t kNoPage = 0x7FFFFFFFu;   // (a NaN)

template <int D>
struct Smem {
  // D / 64 blocks of rows of 128 bytes: 128 rows of Q, 64 of K and of V
  static constexpr int kQBlock = kTile * 128, kBlock = kStep * 128;
  static constexpr int kQ = kTile * D * 2, kOperand = kStep * D * 2;
  static constexpr int q = 0, k = 2 * kQ, v = k + kRing * kOperand, ctrl = v + kRing * kOperand;
  static constexpr int kCtrl = 2048;
  static constexpr int total = ctrl + kCtrl + 1024;   // the tiles start on 1024 bytes
};

constexpr int kGroupRing = 8;   // steps whose groups are kept: a step's are read until the step four later is converted
struct Ctrl {
  uint64_t q_full[2], k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing], s_full[2][2], p_full[2][2], o_full[2][2],
      scale_full[kGroupRing], drain[4];
  uint32_t tmem;
  int abort;
  Group group[kGroupRing][kStep / 16];
};
static_assert(sizeof(Ctrl) <= 2048 && sizeof(Group) == 16 && offsetof(Ctrl, group) % 16 == 0, "control region");

// Waits of the pipeline: one test inline, the rest (the barrier's own sleep, up
// to a millisecond at a time, the abort flag and the time limit) out of line,
// so that a wait that is over costs the MMA warp a few instructions.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(limit_ns == 0 ? 0u : 1000000u)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (globaltimer() - t0 >= limit_ns) {
      set_status(status, MOE_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                         uint64_t limit_ns) {
  const uint32_t at = smem_u32(bar);
  return test(at, parity) || wait_on(at, parity, abort, status, limit_ns);
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

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

// Four codes as bf16 times `unit` (a bf16 pair of 2^(120 + e))
__device__ __forceinline__ uint2 e4m3x4_to_bf16x4(uint32_t v, uint32_t unit) {
  return make_uint2(bf16x2_mul((prmt(v, 0u, 0x9180u) << 4) & 0x87F087F0u, unit),
                    bf16x2_mul((prmt(v, 0u, 0xB3A2u) << 4) & 0x87F087F0u, unit));
}

// A V scale's power of two, bounded so that the bf16 operand and the rest stay in
// range (a smaller or subnormal scale's rest is below 1).
__device__ __forceinline__ int v_exponent(float vs) {
  const int e = static_cast<int>(__float_as_uint(vs) >> 23 & 255u) - 127;
  return max(-100, min(e, 7));
}

// The converters' part: K and V of every step, each into a ring of its own.
template <int D>
__device__ __forceinline__ void convert(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, int b, int h, int from,
                                        int end, int steps) {
  using S = Smem<D>;
  constexpr int kHalves = D / 64, kRows = kStep / 32;   // a thread has a chunk of each half of kRows rows
  const int tid = threadIdx.x - kConvertWarp * 32;
  // a quarter warp covers two rows' four chunks: its 16-byte stores meet no bank twice
  const int q4 = tid & 3, r = tid >> 2;
  volatile int* abort = &ctrl->abort;
  // Page ids are asked for two steps ahead, codes and scales one: nothing is
  // waited for when its turn comes.
  const auto look = [&](int (&id)[kRows], int t0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int t = t0 + 32 * i + r;
      id[i] = t < end ? __ldg(a.s.table + static_cast<size_t>(b) * a.s.width + (t >> a.d.shift)) : -1;
    }
  };
  const auto check = [&](int (&id)[kRows], int t0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (static_cast<uint32_t>(id[i]) >= static_cast<uint32_t>(a.pool.num_pages)) {
        if (t0 + 32 * i + r < end) set_status(a.status, MOE_ERR_DEVICE_CHECK);
        id[i] = -1;
      }
  };
  const auto load = [&](uint4 (&x)[kRows * kHalves], const uint8_t* pool, const int (&id)[kRows], int t0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint8_t* row = pool;
      if (id[i] >= 0) row += kv_row(id[i], a.d.Hkv, h, a.d.page, (t0 + 32 * i + r) & (a.d.page - 1), D) + q4 * 16;
#pragma unroll
      for (int f = 0; f < kHalves; ++f)
        x[kRows * f + i] = id[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(row + 64 * f)) : make_uint4(0, 0, 0, 0);
    }
  };
  // The scales of the thread's rows.  Two threads (writes) have the first row of
  // every 16-token group: group 2 i + (r >> 4).
  const bool writes = q4 == 0 && (r & 15) == 0;
  const auto scales = [&](float (&ks)[kRows], float (&vs)[kRows], const int (&id)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const size_t of = static_cast<size_t>(max(id[i], 0)) * a.d.Hkv + h;
      vs[i] = id[i] >= 0 ? __ldg(a.pool.v_scale + of) : 0.f;
      if (writes) ks[i] = id[i] >= 0 ? __ldg(a.pool.k_scale + of) : __uint_as_float(kNoPage);
    }
  };
  const auto at = [&](int f, int row, int e) {
    return f * S::kBlock + row * 128 + (((2 * q4 + e) ^ (row & 7)) << 4);
  };
  uint4 kx[kRows * kHalves], vx[kRows * kHalves];
  float ks[kRows], vs[kRows], ks_next[kRows], vs_next[kRows];
  int id[kRows], id_next[kRows];
  look(id, from);
  look(id_next, from + kStep);
  check(id, from);
  load(kx, a.pool.k, id, from);
  scales(ks, vs, id);
  for (int j = 0; j < steps; ++j) {
    const int t0 = from + j * kStep, st = j % kRing;
    const uint32_t parity = (j / kRing) & 1;
    load(vx, a.pool.v, id, t0);
    if (writes) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        float lv = 0.f, inv = 1.f;
        if (vs[i] != 0.f) {
          const float m = vs[i] * __uint_as_float(static_cast<uint32_t>(127 - v_exponent(vs[i])) << 23);
          lv = log2f(m);
          inv = 1.f / m;
        }
        *reinterpret_cast<float4*>(&ctrl->group[j % kGroupRing][2 * i + (r >> 4)]) = make_float4(ks[i], lv, inv, 0.f);
      }
      mbar_arrive(&ctrl->scale_full[j % kGroupRing]);
    }
    if (!wait_for(&ctrl->k_empty[st], parity ^ 1u, abort, a.status, a.wait_ns)) return;
    const uint32_t kt = smem + S::k + st * S::kOperand, vt = smem + S::v + st * S::kOperand;
#pragma unroll
    for (int f = 0; f < kHalves; ++f)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint4 x = kx[kRows * f + i];
        const uint2 c0 = e4m3x4_to_f16x4(x.x), c1 = e4m3x4_to_f16x4(x.y), c2 = e4m3x4_to_f16x4(x.z),
                    c3 = e4m3x4_to_f16x4(x.w);
        sts_u4(kt + at(f, 32 * i + r, 0), make_uint4(c0.x, c0.y, c1.x, c1.y));
        sts_u4(kt + at(f, 32 * i + r, 1), make_uint4(c2.x, c2.y, c3.x, c3.y));
      }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->k_full[st]);
    check(id_next, t0 + kStep);   // (rows beyond the end have none)
    load(kx, a.pool.k, id_next, t0 + kStep);
    scales(ks_next, vs_next, id_next);
    if (!wait_for(&ctrl->v_empty[st], parity ^ 1u, abort, a.status, a.wait_ns)) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t u = vs[i] == 0.f ? 0u : static_cast<uint32_t>(v_exponent(vs[i]) + 247) << 7;
      const uint32_t unit = u | u << 16;
#pragma unroll
      for (int f = 0; f < kHalves; ++f) {
        const uint4 x = vx[kRows * f + i];
        const uint2 c0 = e4m3x4_to_bf16x4(x.x, unit), c1 = e4m3x4_to_bf16x4(x.y, unit),
                    c2 = e4m3x4_to_bf16x4(x.z, unit), c3 = e4m3x4_to_bf16x4(x.w, unit);
        sts_u4(vt + at(f, 32 * i + r, 0), make_uint4(c0.x, c0.y, c1.x, c1.y));
        sts_u4(vt + at(f, 32 * i + r, 1), make_uint4(c2.x, c2.y, c3.x, c3.y));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->v_full[st]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      id[i] = id_next[i];
      ks[i] = ks_next[i];
      vs[i] = vs_next[i];
    }
    look(id_next, t0 + 2 * kStep);
  }
}

// The MMA warps of a tile.  The whole warp runs each, so that descriptors and
// addresses stay in uniform registers; one elected lane issues.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const PrefillArgs& a, Ctrl* ctrl) {
  if (__all_sync(0xFFFFFFFFu, test(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, wait_on(bar, parity, &ctrl->abort, a.status, a.wait_ns)) != 0;
}

// Scores: S of step j takes the place of step j - 2's weights, once their product is done.
template <int D>
__device__ __forceinline__ void multiply_scores(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, uint32_t tmem, int t,
                                                int steps) {
  using S = Smem<D>;
  constexpr uint32_t kScores = idesc_f32(kTile, kStep, false, false);
  const bool one = elect_one();
  const uint32_t k_full = smem_u32(ctrl->k_full), o_full = smem_u32(ctrl->o_full[t]);
  if (!warp_wait(smem_u32(&ctrl->q_full[t]), 0, a, ctrl)) return;
  const uint64_t dq = smem_desc_k128(smem + S::q + t * S::kQ), k0 = smem_desc_k128(smem + S::k);
  uint32_t stage = 0, phase = 0;
  for (int j = 0; j < steps; ++j) {
    const uint32_t buf = j & 1, to = tmem + t * 2 * kStep + buf * kStep;
    if (!warp_wait(k_full + 8 * stage, phase, a, ctrl)) return;
    if (j > 1 && !warp_wait(o_full + 8 * buf, ((j >> 1) - 1) & 1, a, ctrl)) return;
    tc_fence_after();
    const uint64_t dk = k0 + stage * (S::kOperand >> 4);
    if (one) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        umma_bf16(to, dq + (i >> 2) * (S::kQBlock >> 4) + 2 * (i & 3), dk + (i >> 2) * (S::kBlock >> 4) + 2 * (i & 3),
                  kScores, i > 0);
      umma_commit(&ctrl->s_full[t][buf]);
      umma_commit(&ctrl->k_empty[stage]);
    }
    __syncwarp();
    if (++stage == kRing) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

template <int D>
__device__ __forceinline__ void multiply_out(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, uint32_t tmem, int t,
                                             int steps) {
  using S = Smem<D>;
  constexpr uint32_t kOut = idesc_f32(kTile, D, true, true);
  const bool one = elect_one();
  const uint32_t v_full = smem_u32(ctrl->v_full), p_full = smem_u32(ctrl->p_full[t]);
  const uint64_t v0 = smem_desc_n128(smem + S::v, S::kBlock);
  const uint32_t o = tmem + 4 * kStep + t * D;
  uint32_t stage = 0, phase = 0;
  for (int j = 0; j < steps; ++j) {
    const uint32_t buf = j & 1, p = tmem + t * 2 * kStep + buf * kStep;
    if (!warp_wait(v_full + 8 * stage, phase, a, ctrl)) return;
    if (!warp_wait(p_full + 8 * buf, (j >> 1) & 1, a, ctrl)) return;
    tc_fence_after();
    const uint64_t dv = v0 + stage * (S::kOperand >> 4);
    if (one) {
#pragma unroll
      for (int i = 0; i < kStep / 16; ++i) {
        const uint32_t hi = p + 32 * (i >> 1) + 8 * (i & 1);
        umma_bf16_ts(o, hi, dv + i * (2048 >> 4), kOut, j + i > 0);
        umma_bf16_ts(o, hi + 16, dv + i * (2048 >> 4), kOut, 1);
      }
      umma_commit(&ctrl->o_full[t][buf]);
      umma_commit(&ctrl->v_empty[stage]);
    }
    __syncwarp();
    if (++stage == kRing) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// A softmax warpgroup's part: a row per thread.
template <int D>
__device__ __forceinline__ void softmax(const PrefillArgs& a, Ctrl* ctrl, uint32_t smem, uint32_t tmem, int t, int b,
                                        int h, int g, int first, int n, int len, int row0, int from,
                                        int steps, bool cut) {
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
      sts_u4(smem + S::q + t * S::kQ + (i >> 3) * S::kQBlock + in_tile * 128 + (((i & 7) ^ (in_tile & 7)) << 4),
             make_uint4(c[0], c[1], c[2], c[3]));
    }
    fence_proxy_async_smem();
    mbar_arrive(&ctrl->q_full[t]);
    __syncwarp();
  }
  const uint32_t lanes = static_cast<uint32_t>(quad) << 21;   // 32 quad in the address's lane field
  const uint32_t o = tmem + lanes + 4 * kStep + t * D;
  // m: what the exponents are taken against, a whole number, so that a change
  // of it scales l, O and the weights already written exactly.  It follows the
  // scores only where weights come out above kLarge.
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < steps; ++j) {
    const uint32_t groups = smem_u32(ctrl->group[j % kGroupRing]);
    const uint32_t sc = tmem + lanes + t * 2 * kStep + (j & 1) * kStep;
    const bool ok = wait_for(&ctrl->scale_full[j % kGroupRing], (j / kGroupRing) & 1, abort, a.status, a.wait_ns) &&
                    wait_for(&ctrl->s_full[t][j & 1], (j >> 1) & 1, abort, a.status, a.wait_ns);
    if (!__all_sync(0xFFFFFFFFu, ok)) return;
    __syncwarp();
    tc_fence_after();
    const int t0 = from + j * kStep;
    bool failed = false;
    // 32 tokens (two groups): their scores s to weights, in place
    const auto weigh = [&](int c, uint32_t (&s)[32]) {
      float f[2], lv[2], inv[2];
      bool gone[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 gr = lds_u4(groups + (2 * c + e) * sizeof(Group));
        f[e] = __uint_as_float(gr.x) * unscale;
        lv[e] = __uint_as_float(gr.y);
        inv[e] = __uint_as_float(gr.z);
        gone[e] = gr.x == kNoPage;
      }
      if (t0 + 32 * c + 32 > sees_least || gone[0] || gone[1]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int left = gone[e] ? 0 : sees - (t0 + 32 * c + 16 * e);
          const bool flat = f[e] == 0.f || left <= 0;   // (no -inf times 0, or times a row's NaN)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[16 * e + i] = i >= left ? 0xFF800000u : flat ? 0u : s[16 * e + i];
          if (flat) f[e] = 1.f;
        }
      }
      uint32_t hi[16], lo[16];
      float sum[4];
      bool raised = false;
      for (;;) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float add = lv[e] - (m == -INFINITY ? 0.f : m);
          float part[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float w0 = ex2(fmaf(__uint_as_float(s[16 * e + 2 * i]), f[e], add));
            const float w1 = ex2(fmaf(__uint_as_float(s[16 * e + 2 * i + 1]), f[e], add));
            part[0] += w0;
            part[1] += w1;
            const uint32_t u0 = __float_as_uint(w0), u1 = __float_as_uint(w1);
            hi[8 * e + i] = prmt(u0, u1, 0x7632u);
            lo[8 * e + i] = pack_bf16x2(w0 - __uint_as_float(u0 & 0xFFFF0000u), w1 - __uint_as_float(u1 & 0xFFFF0000u));
          }
          sum[2 * e] = part[0];
          sum[2 * e + 1] = part[1];
        }
        // Too large a sum (or a first one, or a NaN, which stays): m is raised to
        // the scores' maximum and everything so far scaled down to it.
        const bool large = !(sum[0] + sum[1] + sum[2] + sum[3] <= kLarge) || m == -INFINITY;
        if (raised || !__any_sync(0xFFFFFFFFu, large)) break;
        raised = true;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(s[i]) * f[i >> 4]);
        const float to = large && top > m ? ceilf(top) : m;   // (a row goes by its own weights alone)
        const float r = to == m ? 1.f : ex2(m - to);   // (0 for the first)
        m = to;
        l *= r;
        // What this step has stored so far (the weights of the tokens before these, O
        // scaled for them) is read again below, and a load does not wait for a store.
        tmem_st_wait();
        // O so far: once the last step's product is in it (products of a tile end in
        // order, and the next one waits for these weights)
        if (j > 0) {
          failed |= !__all_sync(0xFFFFFFFFu, wait_for(&ctrl->o_full[t][(j - 1) & 1], ((j - 1) >> 1) & 1, abort, a.status, a.wait_ns));
          __syncwarp();   // (the tensor-memory accesses below want the whole warp)
          tc_fence_after();
        }
        const int parts = j > 0 ? D / 16 : 0;
#pragma unroll 1
        for (int k = 0; k < parts; ++k) {
          uint32_t v[16];
          tmem_ld_16cols(o + 16 * k, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * r);
          tmem_st_16cols(o + 16 * k, v);
        }
        const uint32_t r2 = pack_bf16x2(r, r);
#pragma unroll 1
        for (int k = 0; k < 2 * c; ++k) {
          uint32_t v[16];
          tmem_ld_16cols(sc + 16 * k, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = bf16x2_mul(v[i], r2);
          tmem_st_16cols(sc + 16 * k, v);
        }
      }
      l = fmaf(sum[0] + sum[1], inv[0], l);
      l = fmaf(sum[2] + sum[3], inv[1], l);
      tmem_st_16cols(sc + 32 * c, hi);
      tmem_st_16cols(sc + 32 * c + 16, lo);
    };
#pragma unroll 1
    for (int c = 0; c < kStep / 32; ++c) {
      uint32_t s[32];
      tmem_ld_32cols(sc + 32 * c, s);
      tmem_ld_wait();
      weigh(c, s);
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&ctrl->p_full[t][j & 1]);
    if (__any_sync(0xFFFFFFFFu, failed)) return;
  }
  if (steps > 0 && !__all_sync(0xFFFFFFFFu, wait_for(&ctrl->o_full[t][(steps - 1) & 1], ((steps - 1) >> 1) & 1, abort,
                                                    a.status, a.wait_ns)))
    return;
  __syncwarp();
  tc_fence_after();
  const float inv = cut ? 1.f : l == 0.f ? 0.f : 1.f / l;
  const size_t slot = static_cast<size_t>(blockIdx.x) * 2 * kTile + t * kTile + in_tile;
  float4* part = reinterpret_cast<float4*>(a.part_o + slot * D);
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
    if (real && cut) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[8 * c + i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                      __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
    } else if (real) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]) * inv, __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
        out[4 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
  }
  if (real && cut)
    a.part_ml[slot] = make_float2(m, l);
  else if (real && at.lse)
    at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(PrefillArgs a) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(base + S::ctrl);
  const uint32_t smem = smem_u32(base);
  chain_wait();
  ChainReleaseAtExit release;
  int u = blockIdx.x, part = 0, parts = 1;
  Unit unit;
  if (a.most_parts > 1) {
    int units;
    find_unit(a, 0, &unit, &units);
    parts = parts_of(a, units);
    if (u >= units * parts) return;
    part = u / units;
    u %= units;
  }
  if (!find_unit(a, u, &unit, nullptr)) return;
  const int b = unit.b, h = unit.h, first = unit.first, n = unit.n, len = unit.len, g = a.at.Hq / a.d.Hkv;
  const int rows = n * g, row0 = unit.pair * 2 * kTile;
  const int tiles = row0 + kTile < rows ? 2 : 1;
  const int seen = max(len - n + (min(row0 + 2 * kTile, rows) - 1) / g + 1, 0);   // by the last row
  const int all = (seen + kStep - 1) / kStep, per = part_steps(all, parts);
  if (part > 0 && part * per >= all) return;   // (the join does not ask for it)
  const int from = part * per * kStep, steps = min(per, all - part * per), end = min(seen, from + steps * kStep);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctrl->q_full[i], kTile);
      for (int k = 0; k < 2; ++k) {
        mbar_init(&ctrl->o_full[i][k], 1);
        mbar_init(&ctrl->s_full[i][k], 1);
        mbar_init(&ctrl->p_full[i][k], kTile);
      }
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ctrl->k_full[i], 128);
      mbar_init(&ctrl->v_full[i], 128);
      mbar_init(&ctrl->k_empty[i], tiles);
      mbar_init(&ctrl->v_empty[i], tiles);
    }
    for (int i = 0; i < kGroupRing; ++i) mbar_init(&ctrl->scale_full[i], 2);
    for (int i = 0; i < 4; ++i) mbar_init(&ctrl->drain[i], 1);
    ctrl->abort = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(&ctrl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, ctrl->tmem, 0);
  if (warp < kSoftmaxWarp) {
    if ((warp & 1) < tiles && steps > 0) {
      if (warp < 2)
        multiply_scores<D>(a, ctrl, smem, tmem, warp, steps);
      else
        multiply_out<D>(a, ctrl, smem, tmem, warp & 1, steps);
      // whatever was issued is done before the tensor memory goes
      __syncwarp();
      if (elect_one()) {
        umma_commit(&ctrl->drain[warp]);
        mbar_wait_timed(&ctrl->drain[warp], 0, a.status);
      }
      __syncwarp();
    }
  } else if (warp < kConvertWarp) {
    const int t = (warp - kSoftmaxWarp) / 4;
    if (t < tiles) softmax<D>(a, ctrl, smem, tmem, t, b, h, g, first, n, len, row0, from, steps, parts > 1);
  } else {
    convert<D>(a, ctrl, smem, b, h, from, end, steps);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The parts of a row, in order: a warp per row, D / 32 columns a lane.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_prefill_join_kernel(PrefillArgs a) {
  constexpr int kPer = D / 32;
  chain_wait();
  ChainReleaseAtExit release;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, in_unit = blockIdx.x * kJoinWarps + warp;
  const int u = blockIdx.y, g = a.at.Hq / a.d.Hkv;
  Unit unit;
  int units;
  if (!find_unit(a, u, &unit, &units)) return;
  const int parts = parts_of(a, units), rows = unit.n * g, h = unit.h, first = unit.first;
  const int row = unit.pair * 2 * kTile + in_unit;
  if (parts == 1 || row >= rows) return;
  const int seen = max(unit.len - unit.n + (min((unit.pair + 1) * 2 * kTile, rows) - 1) / g + 1, 0);
  const int all = (seen + kStep - 1) / kStep, per = part_steps(all, parts), used = all ? (all + per - 1) / per : 1;
  const auto slot = [&](int p) { return (static_cast<size_t>(p) * units + u) * 2 * kTile + in_unit; };
  float m = -INFINITY;
  for (int p = lane; p < used; p += 32) m = fmaxf(m, a.part_ml[slot(p)].x);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
  float l = 0.f, acc[kPer] = {};
#pragma unroll 4
  for (int p = 0; p < used; ++p) {
    const float2 ml = a.part_ml[slot(p)];
    const float r = ml.x == m ? 1.f : ex2(ml.x - m);   // (a power of two: maxima are whole numbers)
    const float* o = a.part_o + slot(p) * D + lane * kPer;
    float v[kPer];
    if constexpr (kPer == 4) {
      const float4 x = *reinterpret_cast<const float4*>(o);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(o);
      v[0] = x.x, v[1] = x.y;
    }
    l = fmaf(ml.y, r, l);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = fmaf(v[e], r, acc[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t at_row = static_cast<size_t>(first + row / g) * a.at.Hq + h * g + row % g;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.at.out) + at_row * D + lane * kPer);
#pragma unroll
  for (int e = 0; e < kPer; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && a.at.lse) a.at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The units that a call can have, and the parts that they can be cut in: eight
// steps at least, and none where there are too many units for certain.
// 128 rows on 8 kv heads over one sequence of 32768 tokens: 931 us uncut, 67 in 19
// parts; 512 rows 1028 and 136 (9 parts); four of 2048, 512 rows: 64 and 55 (2).
long long most_units(const KvDims& d, int Hq, int B, int T_q, int max_q) {
  const long long g = Hq / d.Hkv, each = (max_q * g + 2 * kTile - 1) / (2 * kTile);
  return std::min(each * B, T_q * g / (2 * kTile) + B) * d.Hkv;
}
int most_parts(const KvDims& d, int Hq, int B, int T_q, int few, int max_len) {
  const long long rows = static_cast<long long>(T_q) * (Hq / d.Hkv) - static_cast<long long>(B) * few;   // at least
  return rows / (2 * kTile) * d.Hkv > kSMs / 2 ? 1 : std::max(1, std::min(kSMs, max_len / (8 * kStep)));
}

template <int D>
int launch(const PrefillArgs& a, cudaStream_t stream, int* launches) {
  if (kv_allow_smem<kv_prefill_kernel<D>>(Smem<D>::total) != cudaSuccess) return MOE_ERR_CUDA;
  const long long units = most_units(a.d, a.at.Hq, a.s.B, a.at.T_q, a.at.max_q);
  if (units > INT_MAX) return MOE_ERR_UNSUPPORTED;
  const bool cut = a.most_parts > 1;
  if (launch_chained(kv_prefill_kernel<D>, dim3(static_cast<unsigned>(cut ? std::max<long long>(units, kSMs) : units)),
                     dim3(kThreads), Smem<D>::total, stream, a) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  if (!cut) return MOE_OK;
  const unsigned joins = static_cast<unsigned>(std::min<long long>(units, kSMs / 2));   // more are not cut
  if (launch_chained(kv_prefill_join_kernel<D>, dim3(2 * kTile / kJoinWarps, joins), dim3(kJoinWarps * 32), 0, stream,
                     a) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

}  // namespace

size_t kv_prefill_part_rows(const KvDims& d, int Hq, int B, int T_q, int few, int max_len) {
  return most_parts(d, Hq, B, T_q, few, max_len) == 1 ? 0 : static_cast<size_t>(kSMs) * 2 * kTile;
}

int kv_prefill_launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, const KvAttention& at, float* part_o,
                      float2* part_ml, int* status, cudaStream_t stream, int* launches) {
  const PrefillArgs a{d, pool, s, at, status, wait_limit_ns(), most_parts(d, at.Hq, s.B, at.T_q, at.few, s.max_len), part_o, part_ml};
  return d.D == 128 ? launch<128>(a, stream, launches) : launch<64>(a, stream, launches);
}

}  // namespace moe
