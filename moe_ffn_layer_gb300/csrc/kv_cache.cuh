// Device helpers shared by the kernels of the 8-bit paged KV cache: where a
// token lies, the cache's scale rule, and e4m3 in registers.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kSMs = 152;   // of a GB300: the plan of a call depends on its sizes alone

// Allows a kernel its dynamic shared memory, once per device and kernel.
template <auto kKernel>
inline cudaError_t kv_allow_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t r = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (r == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
  return r;
}

// Row of a code pool ([num_pages][Hkv][page][D]) that holds slot `slot` of a
// page for one head, as a byte offset (64 bits: a pool can pass 4 GB; its rows
// fit 32, which the host checks).
__device__ __forceinline__ size_t kv_row(int page_id, int Hkv, int h, int page, int slot, int D) {
  const uint32_t row = (static_cast<uint32_t>(page_id) * Hkv + h) * page + slot;
  return static_cast<size_t>(row) * static_cast<uint32_t>(D);
}

// The least power of two s with amax <= 448 s (448 = 1.75 * 2^8, the largest
// e4m3 value), 2^-126 at least.  amax is finite and not negative.  A power of
// two loses nothing in a floating code (a code's relative step does not depend
// on its scale) and makes x / s and a later change of scale exact except where
// a code becomes subnormal.
__device__ __forceinline__ float kv_pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased exponent of s
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// Two floats to two e4m3 codes (lo in the low byte), to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four e4m3 codes as f16 pairs (codes 0 and 1, 2 and 3): the hardware's conversion, exact.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t v) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(v));
  return r;
}

// Sixteen codes times a ratio, rounded to codes again (the codes 0x7f and 0xff, which the cache never holds, read as +-480).
__device__ __forceinline__ uint4 e4m3x16_scaled(const uint4& v, float ratio) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = e4m3x2_of(e4m3_to_f32(w[i]) * ratio, e4m3_to_f32(w[i] >> 8) * ratio) |
           e4m3x2_of(e4m3_to_f32(w[i] >> 16) * ratio, e4m3_to_f32(w[i] >> 24) * ratio) << 16;
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A sequence's length, checked: in [0, max_len] with its pages inside the table's width.
__device__ __forceinline__ bool kv_length_is(const KvSeqs& s, const KvDims& d, int len) {
  return len >= 0 && len <= s.max_len && (static_cast<long long>(len) + d.page - 1) >> d.shift <= s.width;
}

// The packed cu_* boundaries and length of sequence b, checked: first row,
// rows n >= 0 of T, and the length.  False (and MOE_ERR_DEVICE_CHECK) where
// they are not what they have to be.
__device__ __forceinline__ bool kv_sequence_is(const KvSeqs& s, int T, const KvDims& d, int* status, int first, int n,
                                               int len) {
  if (first < 0 || n < 0 || n > T - first || !kv_length_is(s, d, len)) {
    set_status(status, MOE_ERR_DEVICE_CHECK);
    return false;
  }
  return true;
}
__device__ __forceinline__ bool kv_sequence(const KvSeqs& s, const int32_t* cu, int T, int b, const KvDims& d, int* status,
                                            int* first, int* n, int* len) {
  *first = cu[b];
  *n = cu[b + 1] - cu[b];
  *len = s.seq_lens[b];
  return kv_sequence_is(s, T, d, status, *first, *n, *len);
}

}  // namespace moe
