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
//  - scores: f16.  A K code becomes f16 exactly: its sign at bit 15 and its
//    seven other bits at bits 13..7 read as the code's value times 2^-8
//    (subnormals included); the factor 2^8 goes into the score's scale.  A
//    query row is scaled by a power of two to a largest magnitude in
//    [2^7, 2^8), which keeps all of a bf16's bits down to 2^-21 of it.
//  - output: bf16, which has fp32's range.  A V code becomes bf16 exactly; a
//    weight p * vs enters as two bf16 terms, so that it keeps 16 bits however
//    far it lies below the row's largest (a long sequence's many small weights
//    count as they should, whatever the pages' scales).
// Any code byte reads as a finite value, so what lies beyond a sequence's end
// never turns a masked product into a NaN.
#include "kv_cache.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTok = 32;          // tokens of a warp's step
constexpr int kWarps = 4;
constexpr int kSMs = 152;         // of a GB300: the plan of a call depends on its sizes alone
constexpr int kStages = 3;

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
// copy) as two f16 of 2^-8 times the codes' values.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t v) {
  return (prmt(v, 0u, kSel) << 7) & 0xBF80BF80u;
}
// The same as two bf16 of the codes' values.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t v) {
  return bf16x2_mul((prmt(v, 0u, kSel) << 4) & 0x87F087F0u, 0x7B807B80u);   // times 2^120: e4m3's bias for bf16's
}
constexpr uint32_t kBytes01 = 0x9180u, kBytes23 = 0xB3A2u, kBytes02 = 0xA280u, kBytes13 = 0xB391u;

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

// the same with bf16 inputs
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

// A tile's query rows as MMA operands.  The MMA's K index may stand for any
// order of the head dimension as long as both operands agree: lane (n, c) of a
// K operand holds 16-byte chunk 2c + h of token n's row (chunk c for D = 64),
// four codes d..d+3 per K step, so the query operand of step 4h + r holds
// d = 16 (2c + h) + 4r + {0, 1} and + {2, 3}.  A tile has 8 R rows, R = 1 or 2
// per lane: lane/4 and lane/4 + 8 (zeros for R = 1).
template <int D, int R>
struct QueryTile {
  uint32_t a[D / 16][4];
  float unscale[R];   // scale * log2(e) * 2^8 / (the row's power of two)

  __device__ __forceinline__ void load(const KvAttention& at, int first, int h, int g, int row0, int rows, int lane) {
    const int c = lane & 3;
    uint32_t raw[D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) a[k][1] = a[k][3] = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = row0 + (lane >> 2) + 8 * i;
      const bool real = r < rows;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(at.q) +
                               static_cast<long long>(first + (real ? r / g : 0)) * at.q_stride +
                               (static_cast<long long>(h) * g + (real ? r % g : 0)) * D;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int d0 = (D == 128 ? 16 * (2 * c + (k >> 2)) : 16 * c) + 4 * (k & 3);
        const uint2 v = real ? __ldg(reinterpret_cast<const uint2*>(q + d0)) : make_uint2(0, 0);
        raw[k][i] = v.x;
        raw[k][2 + i] = v.y;
        m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
      }
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      // 2^(7 - floor(log2 max)), kept normal on both sides; a NaN or an
      // infinity in the row makes its scores NaN
      const uint32_t e = max(m >> 7, 8u);   // biased exponent of the largest
      const float up = __uint_as_float((261 - e) << 23), down = __uint_as_float((e - 7) << 23);
      unscale[i] = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : at.scale * kLog2e * 256.f * down;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        a[k][i] = pack_f16x2(bf16_lo(raw[k][i]) * up, bf16_hi(raw[k][i]) * up);
        a[k][2 + i] = pack_f16x2(bf16_lo(raw[k][2 + i]) * up, bf16_hi(raw[k][2 + i]) * up);
      }
    }
  }
};

// s[nt] = raw scores of the tile's rows and 8 tokens each (in units that QueryTile::unscale and the page's scale undo)
template <int D, int R>
__device__ __forceinline__ void scores(float (&s)[kTok / 8][4], const QueryTile<D, R>& q, uint32_t k_tile, int lane) {
  const int n = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < kTok / 8; ++nt) {
    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      const uint4 v = lds_u4(k_tile + swz<D>(nt * 8 + n, D == 128 ? 2 * c + half : c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int r = 0; r < 4; ++r)
        mma_f16(s[nt], q.a[4 * half + r], codes_to_f16x2<kBytes01>(w[r]), codes_to_f16x2<kBytes23>(w[r]));
    }
  }
}

// Where a call's work lies: the row tile's sequence, its rows and what they see.
struct Tile {
  int first, n, len, rows, row0, seen;   // seen: tokens that the tile's last real row sees
  __device__ __forceinline__ bool find(const KvSeqs& s, const KvAttention& at, int b, int g, int mt, int tile_rows,
                                       int page, int* status) {
    if (!kv_sequence(s, at.cu_q, at.T_q, b, page, status, &first, &n, &len)) return false;
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
  // tokens that row r sees (rows beyond the last real one see what it sees)
  __device__ __forceinline__ int sees(int r, int g) const { return max(len - n + min(r, rows - 1) / g + 1, 0); }
};

// One warp's ring of token steps in shared memory.
template <int D>
struct Ring {
  static constexpr int kStageBytes = 2 * kTok * D;
  uint32_t base;       // kStages x (K rows, V rows)
  float* scales;       // kStages x {ks, ks, vs, vs} of the step's two 16-token halves (a page holds whole halves)
  // Starts the copies of tokens [t0, t0 + 32); rows at or beyond `end` are zeros.
  __device__ __forceinline__ void fetch(int stage, const KvDims& d, const KvPool& pool, const KvSeqs& s, int b, int h,
                                        int t0, int end, int lane, int* status) const {
    constexpr int kChunks = D / 16, kRowsAtOnce = 32 / kChunks;
    int id[2];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 16 * i;
      id[i] = t < end ? __ldg(s.table + static_cast<size_t>(b) * s.width + t / d.page) : -1;
      ok[i] = id[i] >= 0 && id[i] < pool.num_pages;
      if (t < end && !ok[i]) set_status(status, MOE_ERR_DEVICE_CHECK);
    }
    const uint32_t k = base + stage * kStageBytes, v = k + kTok * D;
#pragma unroll
    for (int j = 0; j < kTok / kRowsAtOnce; ++j) {
      const int r = j * kRowsAtOnce + lane / kChunks, c = lane % kChunks, i = j * kRowsAtOnce >> 4;
      const bool in = ok[i] && t0 + r < end;
      const size_t at = in ? kv_row(id[i], d.Hkv, h, d.page, (t0 + r) % d.page, D) + c * 16 : 0;
      cp_async16(k + swz<D>(r, c), pool.k + at, in);
      cp_async16(v + swz<D>(r, c), pool.v + at, in);
    }
    if (lane < 4) {
      const int i = lane & 1;
      // a page that is not there: a NaN of its own, taken as masked
      scales[stage * 4 + lane] = ok[i] ? __ldg((lane < 2 ? pool.k_scale : pool.v_scale) +
                                               static_cast<size_t>(id[i]) * d.Hkv + h)
                                       : (lane < 2 ? __uint_as_float(0x7FFFFFFFu) : 0.f);
    }
  }
};

__device__ __forceinline__ bool no_page(float k_scale) { return __float_as_uint(k_scale) == 0x7FFFFFFFu; }

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
};

// 2^(a - b), 0 where a is -inf (also against b = -inf)
__device__ __forceinline__ float exp2_diff(float a, float b) { return a == -INFINITY ? 0.f : exp2_approx(a - b); }

// Partial results of one (row, head) of one chunk, relative to its own maximum: in the workspace, [T_q * Hq][chunks].
struct Partials {
  float* o;      // [..][D]
  float2* ml;    // running maximum (base 2) and sum
  int chunks;    // per row
  int chunk;     // tokens of a chunk
};

// Grid: (chunk, row tile) x kv head x sequence.  Each warp takes every
// kWarps-th 32-token step of the chunk through its own ring, with its own
// running softmax; the warps' states meet in shared memory at the end.
template <int D, int R>
__global__ void __launch_bounds__(kWarps * 32, 2) kv_attention_kernel(KvDims d, KvPool pool, KvSeqs s, KvAttention at,
                                                                      Partials part, int* status) {
  constexpr int kRows = 8 * R;
  extern __shared__ __align__(128) uint8_t smem[];
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x % part.chunks, mt = blockIdx.x / part.chunks, h = blockIdx.y, b = blockIdx.z;
  const int g = at.Hq / d.Hkv;
  Tile tile;
  if (!tile.find(s, at, b, g, mt, kRows, d.page, status)) return;
  const int begin = chunk * part.chunk;
  if (begin >= tile.seen && chunk > 0) return;
  const int end = min(begin + part.chunk, tile.seen);
  const int steps = (end - begin + kTok - 1) / kTok;   // may be 0: rows that see nothing

  Ring<D> ring{smem_u32(smem) + warp * kStages * Ring<D>::kStageBytes,
               reinterpret_cast<float*>(smem + kWarps * kStages * Ring<D>::kStageBytes) + warp * kStages * 4};
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    const int st = warp + i * kWarps;
    if (st < steps) ring.fetch(i, d, pool, s, b, h, begin + st * kTok, end, lane, status);
    cp_async_commit();
  }
  QueryTile<D, R> q;
  q.load(at, tile.first, h, g, tile.row0, tile.rows, lane);
  State<D, R> x;
  x.clear();
  int sees[R];
#pragma unroll
  for (int i = 0; i < R; ++i) sees[i] = tile.sees(tile.row0 + (lane >> 2) + 8 * i, g);
  const int sees_least = tile.sees(tile.row0, g);
  int stage = 0;
  for (int st = warp; st < steps; st += kWarps) {
    {
      const int next = st + (kStages - 1) * kWarps;
      __syncwarp();   // every lane is done with the stage that is filled now
      if (next < steps)
        ring.fetch(stage == 0 ? kStages - 1 : stage - 1, d, pool, s, b, h, begin + next * kTok, end, lane, status);
      cp_async_commit();
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t k_tile = ring.base + stage * Ring<D>::kStageBytes, v_tile = k_tile + kTok * D;
    const float ks0 = ring.scales[stage * 4], ks1 = ring.scales[stage * 4 + 1];
    const float vs0 = ring.scales[stage * 4 + 2], vs1 = ring.scales[stage * 4 + 3];
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float sc[kTok / 8][4];
    scores<D, R>(sc, q, k_tile, lane);
    const int t0 = begin + st * kTok;
    const bool masks = t0 + kTok > sees_least || no_page(ks0) || no_page(ks1);
    float m[R];
    bool grew = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = x.m[i];
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) {
        const float ks = nt < 2 ? ks0 : ks1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& v = sc[nt][2 * i + e];
          v *= ks * q.unscale[i];
          if (masks && (t0 + nt * 8 + 2 * (lane & 3) + e >= sees[i] || no_page(ks))) v = -INFINITY;
          m[i] = fmaxf(m[i], v);
        }
      }
      m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 1));
      m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 2));
      grew |= m[i] != x.m[i];
    }
    if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float f = exp2_diff(x.m[i], m[i]);
        x.m[i] = m[i];
        x.l[i] *= f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 2 * i; e < (R == 1 ? 4 : 2 * i + 2); ++e) x.o[j][p][e] *= f;
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
        x.l[i] += p0 + p1;
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
        mma_bf16(x.o[j][0], hi[k], even0, even1);
        mma_bf16(x.o[j][1], hi[k], odd0, odd1);
        if (R == 2) {
          mma_bf16(x.o[j][0], lo[k], even0, even1);
          mma_bf16(x.o[j][1], lo[k], odd0, odd1);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();   // the rings become the meeting place: kWarps x kRows x (D + 4 outputs, {m, l})
  constexpr int kPitch = D + 4;
  float* all_o = reinterpret_cast<float*>(smem);
  float2* all_ml = reinterpret_cast<float2*>(smem + kWarps * kRows * kPitch * sizeof(float));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float l = x.l[i];
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    const int r = (lane >> 2) + 8 * i;
    if ((lane & 3) == 0) all_ml[warp * kRows + r] = make_float2(x.m[i], l);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {   // even and odd columns of the V bytes interleave: d = 16 j + 4 c + 0..3
      float v[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) v[p][e] = x.o[j][p][2 * i + e] + (R == 1 ? x.o[j][p][2 + e] : 0.f);
      *reinterpret_cast<float4*>(all_o + (warp * kRows + r) * kPitch + 16 * j + 4 * (lane & 3)) =
          make_float4(v[0][0], v[1][0], v[0][1], v[1][1]);
    }
  }
  __syncthreads();
  const bool alone = tile.seen <= part.chunk;   // the only chunk of this tile: the result, not a part
  for (int i = threadIdx.x; i < kRows * D / 4; i += kWarps * 32) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    if (tile.row0 + r >= tile.rows) break;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, all_ml[w * kRows + r].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = all_ml[w * kRows + r];
      const float f = exp2_diff(ml.x, m);
      const float4 v = *reinterpret_cast<const float4*>(all_o + (w * kRows + r) * kPitch + c);
      l += ml.y != ml.y ? ml.y : f * ml.y;   // (a NaN sum belongs to a row of NaN scores, whose maximum is -inf)
      o.x += f * v.x;
      o.y += f * v.y;
      o.z += f * v.z;
      o.w += f * v.w;
    }
    const int row = tile.row0 + r;
    const size_t at_row = static_cast<size_t>(tile.first + row / g) * at.Hq + h * g + row % g;
    if (alone) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(at.out) + at_row * D + c) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (c == 0 && at.lse) at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      const size_t slot = at_row * part.chunks + chunk;
      *reinterpret_cast<float4*>(part.o + slot * D + c) = o;
      if (c == 0) part.ml[slot] = make_float2(m, l);
    }
  }
}

// Joins the chunks of every row whose tile had more than one: a warp per (row, head), the chunks in order.
template <int D>
__global__ void __launch_bounds__(128) kv_join_kernel(KvDims d, KvSeqs s, KvAttention at, Partials part, int tile_rows,
                                                      int* status) {
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, g = at.Hq / d.Hkv;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);   // (query, head) of sequence b
  const int b = blockIdx.y;
  const int query = i / at.Hq, head = i % at.Hq;
  Tile tile;
  if (query >= at.max_q || !tile.find(s, at, b, g, 0, tile_rows, d.page, status) || query >= tile.n) return;
  tile.find(s, at, b, g, (query * g + head % g) / tile_rows, tile_rows, d.page, status);
  if (tile.seen <= part.chunk) return;
  const int n = (tile.seen + part.chunk - 1) / part.chunk;
  const size_t at_row = static_cast<size_t>(tile.first + query) * at.Hq + head;
  const float2* ml = part.ml + at_row * part.chunks;
  float m = -INFINITY;
  for (int c = lane; c < n; c += 32) m = fmaxf(m, ml[c].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  constexpr int kPer = D / 32;
  float acc[kPer] = {};
  float l = 0.f;
  for (int c = 0; c < n; ++c) {
    const float2 x = ml[c];
    const float f = exp2_diff(x.x, m);
    l += x.y != x.y ? x.y : f * x.y;
    const float* o = part.o + (at_row * part.chunks + c) * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += f * o[e];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(at.out) + at_row * D + lane * kPer);
#pragma unroll
  for (int e = 0; e < kPer; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && at.lse) at.lse[at_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// weights[b][h][t] += sum over the rows of (b, h) of exp(s_t - lse): a warp per
// 32 tokens, all rows in order, so the sums do not depend on scheduling.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_weights_kernel(KvDims d, KvPool pool, KvSeqs s, KvAttention at,
                                                                 int* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  chain_wait();
  ChainReleaseAtExit release;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y, b = blockIdx.z, g = at.Hq / d.Hkv;
  const int t0 = (blockIdx.x * kWarps + warp) * kTok;
  Tile tile;
  if (!tile.find(s, at, b, g, 0, 16, d.page, status) || t0 >= tile.len) return;
  Ring<D> ring{smem_u32(smem) + warp * Ring<D>::kStageBytes,
               reinterpret_cast<float*>(smem + kWarps * Ring<D>::kStageBytes) + warp * 4};
  ring.fetch(0, d, pool, s, b, h, t0, tile.len, lane, status);
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  const float ks0 = ring.scales[0], ks1 = ring.scales[1];
  float sum[kTok / 8][2] = {};
  for (int mt = 0; mt * 16 < tile.rows; ++mt) {
    tile.find(s, at, b, g, mt, 16, d.page, status);
    if (t0 >= tile.seen) continue;
    QueryTile<D, 2> q;
    q.load(at, tile.first, h, g, tile.row0, tile.rows, lane);
    float sc[kTok / 8][4];
    scores<D, 2>(sc, q, ring.base, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = tile.row0 + (lane >> 2) + 8 * i;
      const bool real = r < tile.rows;
      const float lse = real ? at.lse[static_cast<size_t>(tile.first + r / g) * at.Hq + h * g + r % g] : INFINITY;
      const float lse2 = lse * kLog2e;
      const int sees = real ? tile.sees(r, g) : 0;
#pragma unroll
      for (int nt = 0; nt < kTok / 8; ++nt) {
        const float ks = nt < 2 ? ks0 : ks1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = t0 + nt * 8 + 2 * (lane & 3) + e;
          if (t < sees && !no_page(ks)) sum[nt][e] += exp2_approx(sc[nt][2 * i + e] * (ks * q.unscale[i]) - lse2);
        }
      }
    }
  }
  float* w = at.weights + (static_cast<long long>(b) * d.Hkv + h) * at.w_stride;
#pragma unroll
  for (int nt = 0; nt < kTok / 8; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = sum[nt][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      const int t = t0 + nt * 8 + 2 * (lane & 3) + e;
      if ((lane >> 2) == 0 && t < tile.len) w[t] += v;
    }
}

// How a call is cut: tokens of a chunk, chunks of a row, and the workspace behind them.
struct Plan {
  int rows;   // of a tile: 8 where every sequence's rows fit, else 16
  int chunk, chunks, tiles;
  size_t o, ml, lse, total;
};

Plan plan(const KvDims& d, int Hq, int B, int T_q, int max_q, int max_len) {
  Plan p{};
  const int g = Hq / d.Hkv;
  p.rows = static_cast<long long>(max_q) * g <= 8 ? 8 : 16;
  p.tiles = static_cast<int>((static_cast<long long>(max_q) * g + p.rows - 1) / p.rows);
  // enough CTAs for four rounds of two per SM, chunks of at least 256 tokens
  const long long units = static_cast<long long>(B) * d.Hkv * p.tiles;
  const long long want = (8ll * kSMs + units - 1) / (units > 0 ? units : 1);
  long long chunk = (max_len + want - 1) / want;
  chunk = (chunk + kWarps * kTok - 1) / (kWarps * kTok) * (kWarps * kTok);
  p.chunk = static_cast<int>(chunk < 256 ? 256 : chunk);
  p.chunks = max_len > p.chunk ? static_cast<int>((static_cast<long long>(max_len) + p.chunk - 1) / p.chunk) : 1;
  const size_t rows = static_cast<size_t>(T_q) * Hq;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align_up(bytes);
    return r;
  };
  p.lse = take(rows * sizeof(float));
  if (p.chunks > 1) {
    p.ml = take(rows * p.chunks * sizeof(float2));
    p.o = take(rows * p.chunks * d.D * sizeof(float));
  }
  p.total = at;
  return p;
}

template <int D>
int launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, KvAttention a, void* ws, int* status,
           cudaStream_t stream, int* launches) {
  const Plan p = plan(d, a.Hq, s.B, a.T_q, a.max_q, s.max_len);
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (a.weights && !a.lse) a.lse = reinterpret_cast<float*>(base + p.lse);
  const Partials part{reinterpret_cast<float*>(base + p.o), reinterpret_cast<float2*>(base + p.ml), p.chunks, p.chunk};
  const size_t ring = kWarps * kStages * (Ring<D>::kStageBytes + 4 * sizeof(float));
  const size_t meet = kWarps * p.rows * ((D + 4) * sizeof(float) + sizeof(float2));
  const size_t smem = ring > meet ? ring : meet;
  const auto kernel = p.rows == 8 ? kv_attention_kernel<D, 1> : kv_attention_kernel<D, 2>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (launch_chained(kernel, dim3(static_cast<unsigned>(p.chunks) * p.tiles, d.Hkv, s.B), dim3(kWarps * 32), smem,
                     stream, d, pool, s, a, part, status) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  if (p.chunks > 1) {
    const unsigned rows = static_cast<unsigned>((static_cast<long long>(a.max_q) * a.Hq + 3) / 4);
    if (launch_chained(kv_join_kernel<D>, dim3(rows, s.B), dim3(128), 0, stream, d, s, a, part, p.rows, status) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++*launches;
  }
  if (a.weights) {
    const unsigned blocks = (static_cast<unsigned>(s.max_len) + kWarps * kTok - 1) / (kWarps * kTok);
    if (launch_chained(kv_weights_kernel<D>, dim3(blocks, d.Hkv, s.B), dim3(kWarps * 32),
                       kWarps * (Ring<D>::kStageBytes + 4 * sizeof(float)), stream, d, pool, s, a,
                       status) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++*launches;
  }
  return MOE_OK;
}

}  // namespace

size_t kv_attention_ws_bytes(const KvDims& d, int Hq, int B, int T_q, int max_q, int max_len) {
  return plan(d, Hq, B, T_q, max_q, max_len).total;
}

int kv_attention_launch(const KvDims& d, const KvPool& pool, const KvSeqs& s, const KvAttention& a, void* ws,
                        int* status, cudaStream_t stream, int* launches) {
  return d.D == 128 ? launch<128>(d, pool, s, a, ws, status, stream, launches)
                    : launch<64>(d, pool, s, a, ws, status, stream, launches);
}

}  // namespace moe
