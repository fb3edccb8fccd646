// Rows and weights in 8 bits: RMS norm with the residual's addition, and
// quantisation of rows (plain, or SiLU(gate) * up) and of weights.
//
// Format: e4m3 codes with one power of two s per block (128 values of a row;
// 128 x 128 of a weight), the least with max|x| <= 448 s, 2^-126 at least, held
// as its exponent byte.  A power of two costs e4m3 no precision (its own
// exponent takes up the rest; only values under 2^-14 of the block's largest
// lose bits), scaling by it is exact, and it is the scale that the tensor
// cores' block-scaled MMA multiplies by itself.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// The exponent byte of a block whose largest finite magnitude is m: with m =
// 1.f * 2^(x - 127), m <= 448 * 2^e = 1.75 * 2^(e + 8) is e >= x - 135, one
// more where 1.f > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}
// 2^(127 - byte), by which a block's values are multiplied (exact)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// An infinity as a NaN, anything else as it is: fmaxf then leaves both out of
// the maximum, and the conversion gives the NaN code.
__device__ __forceinline__ float no_inf(float v) { return fmaf(v, 0.f, v); }

// Two values as e4m3 codes (to nearest even), lo in the low byte; NaN as 0x7f.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16,
                    e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float absmax8(float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = no_inf(v[i]);
    m = fmaxf(m, fabsf(v[i]));
  }
  return m;
}
// The largest of 16 neighbouring lanes: a block of 128 values, eight a lane.
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// ---------------------------------------------------------------- norm
constexpr int kMaxNormWarps = 32;

// h = bf16(x + r); y = h rsqrt(mean h^2 + eps) w.  A CTA per row; thread i has
// the row's vectors i, i + blockDim, ... in registers, so that x and r are read
// once.  The sum of squares is held in fp32; y is rounded once, to e4m3 or bf16.
// Bound: memory (7 bytes a value with a residual and codes): 8192 x 4096 in 34.8 us,
// 6.75 TB/s; one row of 2048 is latency, 1.4 us.  About two vectors a thread and
// 256 threads: with one vector and 512 threads 8192 x 4096 takes 40 us, with four
// and 128 threads 36 and 4096 x 8192 63 instead of 36 (too few loads in flight).
// Rows of more than 8192 values (many rows) or 16384 have eight vectors a thread, of which 84
// bytes are spilled at the 64 registers that 1024 threads leave: 2048 x 16384 takes 48 us.
// Of short rows the CTAs' launches are the bound, 1.0 ns a row: 65536 x 512 takes 66 us,
// 262144 x 128 262.
template <int kVecs>
__global__ void __launch_bounds__(1024) rms_norm8_kernel(Norm8 a) {
  chain_wait();
  chain_release();
  __shared__ float part[kMaxNormWarps];
  const long long row = blockIdx.x;
  const int n = a.H >> 3;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + row * a.x_stride;
  const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(a.r) + row * a.r_stride;
  uint4 keep[kVecs];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    keep[i] = make_uint4(0, 0, 0, 0);
    if (j < n) keep[i] = *reinterpret_cast<const uint4*>(x + 8 * j);
  }
  // the weight: asked for before the row's sum is waited for, where registers are left for it
  constexpr bool kEarly = kVecs <= 4;
  auto load_weight = [&](int j) {
    uint4 w = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
    if (a.w && j < n) w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w) + 8 * j);
    return w;
  };
  uint4 weight[kVecs];
  if (kEarly)
#pragma unroll
    for (int i = 0; i < kVecs; ++i) weight[i] = load_weight(threadIdx.x + i * blockDim.x);
  if (a.r) {
    uint4 add[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int j = threadIdx.x + i * blockDim.x;
      add[i] = make_uint4(0, 0, 0, 0);
      if (j < n) add[i] = *reinterpret_cast<const uint4*>(r + 8 * j);
    }
    __nv_bfloat16* h = static_cast<__nv_bfloat16*>(a.h) + row * a.h_stride;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int j = threadIdx.x + i * blockDim.x;
      float u[8], v[8];
      unpack8(keep[i], u);
      unpack8(add[i], v);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] += v[k];
      keep[i] = pack8(u);
      if (j < n) *reinterpret_cast<uint4*>(h + 8 * j) = keep[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[8];
    unpack8(keep[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < blockDim.x >> 5; ++w) sum += part[w];
  const float scale = rsqrtf(sum / static_cast<float>(a.H) + a.eps);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = threadIdx.x + i * blockDim.x;
    float v[8], w[8];
    unpack8(keep[i], v);
    unpack8(kEarly ? weight[i] : load_weight(j), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * scale * w[k];
    if (a.y && j < n) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * a.y_stride + 8 * j) = pack8(v);
    if (a.codes) {
      const uint32_t byte = scale_byte(max16(absmax8(v)));
      if (j < n) {
        *reinterpret_cast<uint2*>(a.codes + row * a.ld + 8 * j) = codes8(v, inv_scale(byte));
        if ((j & 15) == 0) a.scales[row * a.lds + (j >> 4)] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// ---------------------------------------------------------------- rows
// x / (1 + e^-x) * u, with e^-|x| = h^2: of a negative x it is (x h / (1 + h^2)) u h, which passes the fp32
// range only where the result does (e^-x alone would from x = -88 on, and the quotient be lost from -87).
// h = 2^(-|x| c), c = log2(e) / 2 in two parts: the first has 16 bits, so that its product with a bf16 is exact, and
// the second's, 2^-10 at most, comes in as 1 - |x| c2 ln 2.  (With c in one part the product's rounding alone is up to 2^-17
// of the result at x = -90; this way all errors together stay under 20 2^-24.  16384 x 4096 by replays over two sets of
// operands 59.6 -> 61.8 us.)
// Subnormal results of ex2 are taken as 0, which saves its special cases (16384 x 4096 66 -> 57.6 us): h is
// one from x = -174 on, where no up of bf16 brings the product over 2^-116.
__device__ __forceinline__ float silu_mul(float x, float u) {
  constexpr float kHigh = 47274.f / 65536.f, kLow = -2.44424758e-6f;   // kLow = (kHigh - c) ln 2
  const float a = fabsf(x);
  float h, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(a * -kHigh));
  h = fmaf(h, a * kLow, h);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.f)));
  const float f = x < 0.f ? h : 1.f;
  return x * f * r * (u * f);
}

constexpr int kQuantizeThreads = 256;
constexpr uint32_t kQuantizeMany = 1u << 16;   // blocks of 128: from here on several a thread

// 16 lanes a block of 128; blocks are numbered along the rows.  A thread has
// kPer blocks' vectors in flight at once.  Bound: memory (3 bytes a value, 5 with
// SiLU): 16384 x 4096 in 31.1 us, 6.5 TB/s (one block a thread 39.6, two 33.0, eight
// 40.3: registers), with SiLU in 59.8 us, 5.6 TB/s (before its exponent came in two parts 57.6, with two blocks 59.8).
template <int kAct, int kPer>
__global__ void __launch_bounds__(kQuantizeThreads) quantize8_kernel(Quantize8 a, uint32_t blocks_per_row, uint32_t blocks) {
  chain_wait();
  chain_release();
  constexpr uint32_t kStep = kQuantizeThreads / 16;
  const uint32_t b0 = blockIdx.x * (kStep * kPer) + (threadIdx.x >> 4), in_block = (threadIdx.x & 15u) * 8u;
  uint4 x[kPer], up[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t b = b0 + i * kStep, row = b / blocks_per_row, col = (b - row * blocks_per_row) * 128u + in_block;
    x[i] = up[i] = make_uint4(0, 0, 0, 0);
    if (b < blocks && col < static_cast<uint32_t>(a.K)) {
      const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.x) + static_cast<long long>(row) * a.x_stride + col;
      x[i] = *reinterpret_cast<const uint4*>(from);
      if (kAct) up[i] = *reinterpret_cast<const uint4*>(from + a.K);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t b = b0 + i * kStep, row = b / blocks_per_row, col = (b - row * blocks_per_row) * 128u + in_block;
    float v[8];
    unpack8(x[i], v);
    if (kAct) {
      float u[8];
      unpack8(up[i], u);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = silu_mul(v[k], u[k]);
    }
    const uint32_t byte = scale_byte(max16(absmax8(v)));
    if (b < blocks && col < static_cast<uint32_t>(a.K)) {
      *reinterpret_cast<uint2*>(a.codes + static_cast<long long>(row) * a.ld + col) = codes8(v, inv_scale(byte));
      if (in_block == 0) a.scales[static_cast<long long>(row) * a.lds + (col >> 7)] = static_cast<uint8_t>(byte);
    }
  }
}

// ---------------------------------------------------------------- weights
// A CTA per block of 128 x 128: 16 lanes a row, eight rows a thread, kept packed between the maximum and the
// rounding so that four CTAs fit an SM (8192 x 4096 in 16.9 us, 5.9 TB/s; three CTAs 19.7), though 52 bytes a
// thread are spilled at the 64 registers that this leaves.
__global__ void __launch_bounds__(256, 4) quantize8_weight_kernel(Quantize8 a, int N) {
  chain_wait();
  chain_release();
  __shared__ float part[8];
  const int col = blockIdx.x * 128 + (threadIdx.x & 15) * 8, row0 = blockIdx.y * 128 + (threadIdx.x >> 4);
  uint4 x[8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    if (row0 + 16 * i < N && col < a.K)
      x[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (row0 + 16 * i) * a.x_stride + col);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(x[i], v);
    m = fmaxf(m, absmax8(v));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
  const uint32_t byte = scale_byte(m);
  const float inv = inv_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(x[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = no_inf(v[k]);
    if (row0 + 16 * i < N && col < a.K)
      *reinterpret_cast<uint2*>(a.codes + (row0 + 16 * i) * a.ld + col) = codes8(v, inv);
  }
  if (threadIdx.x == 0) a.scales[blockIdx.y * a.lds + blockIdx.x] = static_cast<uint8_t>(byte);
}

inline int done(cudaError_t e, int* launches) {
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

}  // namespace

int rms_norm8_launch(const Norm8& a, int T, cudaStream_t stream, int* launches) {
  const int n = a.H / 8;
  // few rows: more threads for each (64 x 4096: 2.2 -> 1.9 us; 8192 x 4096 with as many: 35 -> 40)
  const int per = T <= 256 ? 512 : 256;
  int vecs = 1;
  while (vecs < 8 && n > per * vecs) vecs *= 2;
  const int threads = ((n + vecs - 1) / vecs + 31) / 32 * 32;
  auto kernel = vecs == 1 ? rms_norm8_kernel<1> : vecs == 2 ? rms_norm8_kernel<2> : vecs == 4 ? rms_norm8_kernel<4> : rms_norm8_kernel<8>;
  return done(launch_chained(kernel, dim3(T), dim3(threads), 0, stream, a), launches);
}

int quantize8_launch(const Quantize8& a, int T, int act, cudaStream_t stream, int* launches) {
  const uint32_t per_row = (a.K + 127) / 128, blocks = per_row * static_cast<uint32_t>(T);
  // several blocks a thread once there is work for every SM's threads
  const bool many = blocks >= kQuantizeMany;
  auto kernel = act ? (many ? quantize8_kernel<1, 4> : quantize8_kernel<1, 1>) : (many ? quantize8_kernel<0, 4> : quantize8_kernel<0, 1>);
  const uint32_t per = 16 * (many ? 4 : 1);
  return done(launch_chained(kernel, dim3((blocks + per - 1) / per), dim3(kQuantizeThreads), 0, stream, a, per_row, blocks), launches);
}

int quantize8_weight_launch(const Quantize8& a, int N, cudaStream_t stream, int* launches) {
  return done(launch_chained(quantize8_weight_kernel, dim3((a.K + 127) / 128, (N + 127) / 128), dim3(256), 0, stream, a, N),
              launches);
}

}  // namespace moe
