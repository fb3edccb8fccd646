// Product of two 8-bit matrices with block scales for up to 16 rows of A: a stream of
// the weights through registers.
//
// A CTA has 16 weight rows, its eight warps an eighth of K each, and adds their sums
// in shared memory in the order of the warps: no barrier, copy engine or tensor
// memory stands before the loads, and all of them are in flight at once (up to
// 2048 values of K; beyond, a block at a time, with more CTAs an SM).  The codes
// become f16, exactly, in registers, and are multiplied by 16 x 8 x 16 MMAs with
// fp32 sums: any order of K serves the sum, so a thread's 16 neighbouring codes of a
// row are its part of four MMAs.  A block's sum takes its scales when the block is
// done.
#include "linear8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;   // weight rows of a CTA

__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {   // two codes, the first in the low byte
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(codes)));
  return d;
}

// d += a b over 16 values of K: a 16 rows, b 8 columns.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x += d times the scales of two exponent bytes, whose product may pass what one fp32 factor holds: then by two.
__device__ __forceinline__ void add_scaled(float& x0, float d0, float& x1, float d1, int a, int w) {
  const int e = a + w - 127;   // biased
  if (a != 255 && w != 255 && e > 0 && e < 255) {
    const float f = __int_as_float(e << 23);
    x0 = fmaf(d0, f, x0);
    x1 = fmaf(d1, f, x1);
    return;
  }
  const int e1 = max(1, min(254, e)), e2 = max(1, e - e1 + 127);
  const float f1 = __int_as_float(e1 << 23), f2 = a == 255 || w == 255 ? __int_as_float(0x7FFFFFFF) : __int_as_float(e2 << 23);
  x0 = fmaf(d0 * f1, f2, x0);
  x1 = fmaf(d1 * f1, f2, x1);
}

// kBatch blocks of K whose loads a warp issues together, kTiles of eight tokens.
template <int kBatch, int kTiles>
__global__ void __launch_bounds__(kThreads, kBatch == 1 ? 3 : 2) linear8_few_kernel(Linear8 a) {
  __shared__ float part[kWarps][8 * kTiles][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows;
  const int blocks = (a.K + kBlockK - 1) / kBlockK;
  const int b0 = blocks * warp / kWarps, b1 = blocks * (warp + 1) / kWarps;
  // rows beyond the last weight read it again; their sums are not stored
  const uint8_t* w0 = a.w + min(n0 + g, a.N - 1) * a.ldw + 16 * t;
  const uint8_t* w1 = a.w + min(n0 + g + 8, a.N - 1) * a.ldw + 16 * t;
  const uint8_t* sw = a.w_scales + static_cast<long long>(n0 >> 7) * a.lws;
  // (columns beyond the last token have its sums, which are not stored)
  const uint8_t *x[kTiles], *sa[kTiles][2];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) {
    x[c] = a.a + min(8 * c + g, a.T - 1) * a.lda + 16 * t;
    sa[c][0] = a.a_scales + min(8 * c + 2 * t, a.T - 1) * a.las;
    sa[c][1] = a.a_scales + min(8 * c + 2 * t + 1, a.T - 1) * a.las;
  }
  float total[kTiles][4] = {};
  chain_wait();
  chain_release();
  for (int b = b0; b < b1; b += kBatch) {
    uint4 w[kBatch][2][2], v[kBatch][kTiles][2];
    int ew[kBatch], ea[kBatch][kTiles][2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = (b + i) * kBlockK, left = b + i < b1 ? a.K - k - 16 * t : 0;   // values from this lane's on
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool in = left > 64 * j;
        w[i][j][0] = in ? __ldcs(reinterpret_cast<const uint4*>(w0 + k + 64 * j)) : zero;
        w[i][j][1] = in ? __ldcs(reinterpret_cast<const uint4*>(w1 + k + 64 * j)) : zero;
#pragma unroll
        for (int c = 0; c < kTiles; ++c) v[i][c][j] = in ? *reinterpret_cast<const uint4*>(x[c] + k + 64 * j) : zero;
      }
      const int at = min(b + i, b1 - 1);
      ew[i] = sw[at];
#pragma unroll
      for (int c = 0; c < kTiles; ++c) {
        ea[i][c][0] = sa[c][0][at];
        ea[i][c][1] = sa[c][1][at];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b + i >= b1) break;
      float d[kTiles][4] = {};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t p[4] = {w[i][j][0].x, w[i][j][0].y, w[i][j][0].z, w[i][j][0].w};
        const uint32_t q[4] = {w[i][j][1].x, w[i][j][1].y, w[i][j][1].z, w[i][j][1].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a0 = f16x2_of(p[m]), a1 = f16x2_of(q[m]), a2 = f16x2_of(p[m] >> 16), a3 = f16x2_of(q[m] >> 16);
#pragma unroll
          for (int c = 0; c < kTiles; ++c) {
            const uint32_t y[4] = {v[i][c][j].x, v[i][c][j].y, v[i][c][j].z, v[i][c][j].w};
            mma16(d[c], a0, a1, a2, a3, f16x2_of(y[m]), f16x2_of(y[m] >> 16));
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kTiles; ++c) {
        add_scaled(total[c][0], d[c][0], total[c][2], d[c][2], ea[i][c][0], ew[i]);
        add_scaled(total[c][1], d[c][1], total[c][3], d[c][3], ea[i][c][1], ew[i]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kTiles; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][8 * c + 2 * t + (k & 1)][g + 8 * (k >> 1)] = total[c][k];
  __syncthreads();
  const int n = threadIdx.x & 15, tok = threadIdx.x >> 4;
  if (tok < a.T && n0 + n < a.N) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += part[i][tok][n];
    a.out[tok * a.ldo + n0 + n] = __float2bfloat16_rn(s);
  }
}

}  // namespace

// Where it is the faster one (the tensor-memory kernel's time in parentheses; replays over several sets of operands, more
// than L2 holds).  Up to 8 rows while the CTAs fit at once, three an SM, and a warp has four blocks of K at most:
// 1 x 2048 x 2048 2.3 (4.0) us, 1 x 4096 x 2048 3.2 (4.9), 8 x 7296 x 4096 6.9 (8.0), but 1 x 8192 x 8192 17.2 (12.7),
// 1 x 16384 x 4096 14.8 (12.8) and 1 x 8192 x 4096 9.7 (8.2).  Up to 16 rows with two an SM and two blocks: 16 x 4096 x 2048
// 3.9 (5.1), 16 x 4864 x 2048 4.0 (5.3), but 16 x 7296 x 2048 6.4 (6.0).  (With more blocks it would still be the faster one at
// 16 x 4096 x 4096, 6.0 (6.4).)
bool linear8_few_takes(const Linear8& a, int sms) {
  const int ctas = (a.N + kRows - 1) / kRows;
  return a.T <= 8 ? a.K <= 4 * kWarps * kBlockK && ctas <= 3 * sms : a.T <= 16 && a.K <= 2 * kWarps * kBlockK && ctas <= 2 * sms;
}

int linear8_few_launch(const Linear8& a, int sms, cudaStream_t stream) {
  const int ctas = (a.N + kRows - 1) / kRows;
  // two blocks at once where a warp has two and two CTAs fit (1 x 2048 x 2048 2.4 us, one at a time 3.0; 1 x 7296 x
  // 2048 5.1 and 4.3, 1 x 7296 x 1024 4.0 and 3.1)
  const bool two = a.K > kWarps * kBlockK && a.K <= 2 * kWarps * kBlockK && ctas <= 2 * sms;
  auto kernel = a.T > 8 ? linear8_few_kernel<2, 2> : two ? linear8_few_kernel<2, 1> : linear8_few_kernel<1, 1>;
  return launch_chained(kernel, dim3(ctas), dim3(kThreads), 0, stream, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
