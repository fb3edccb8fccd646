// Product of two 8-bit matrices with block scales: out[t][n] = sum over the
// 128-wide blocks b of K of 2^(ea[t][b] + ew[n / 128][b]) * sum_{k in b} a[t][k] w[n][k].
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

__device__ __forceinline__ float value(uint32_t code) {
  return (code & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FFFFFFFu) : e4m3_to_f32(code);
}

// 64 x 64 outputs a CTA, 4 x 4 a thread, fp32 FMAs; a block's sum takes its scales when the block is done.
__global__ void __launch_bounds__(256) linear8_kernel(Linear8 a) {
  chain_wait();
  ChainReleaseAtExit release;
  __shared__ float sa[16][65], sw[16][65];
  const int t0 = blockIdx.y * 64, n0 = blockIdx.x * 64, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float acc[4][4] = {}, sub[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 16) {
    __syncthreads();
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 4;
    const uint32_t va = t0 + r < a.T ? *reinterpret_cast<const uint32_t*>(a.a + (t0 + r) * a.lda + k0 + c) : 0u;
    const uint32_t vw = n0 + r < a.N ? *reinterpret_cast<const uint32_t*>(a.w + (n0 + r) * a.ldw + k0 + c) : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sa[c + j][r] = value(va >> (8 * j) & 0xFFu);
      sw[c + j][r] = value(vw >> (8 * j) & 0xFFu);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sub[i][j] = fmaf(sa[k][ty * 4 + i], sw[k][tx * 4 + j], sub[i][j]);
    if ((k0 & 127) == 112 || k0 + 16 == a.K) {
      const int b = k0 >> 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ea = t0 + ty * 4 + i < a.T ? a.a_scales[(t0 + ty * 4 + i) * a.las + b] : 127;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ew = n0 + tx * 4 + j < a.N ? a.w_scales[((n0 + tx * 4 + j) >> 7) * a.lws + b] : 127;
          acc[i][j] += ea == 255 || ew == 255 ? __uint_as_float(0x7FFFFFFFu) : ldexpf(sub[i][j], ea + ew - 254);
          sub[i][j] = 0.f;
        }
      }
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (t0 + ty * 4 + i < a.T && n0 + tx * 4 + j < a.N)
        a.out[(t0 + ty * 4 + i) * a.ldo + n0 + tx * 4 + j] = __float2bfloat16_rn(acc[i][j]);
}

}  // namespace

int linear8_launch(const Linear8& a, int* status, int sms, cudaStream_t stream, int* launches) {
  if (launch_chained(linear8_kernel, dim3((a.N + 63) / 64, (a.T + 63) / 64), dim3(256), 0, stream, a) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++*launches;
  return MOE_OK;
}

}  // namespace moe
