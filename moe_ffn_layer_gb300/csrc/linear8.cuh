// What the kernels of the 8-bit product share: block-scaled MMAs, their scales in
// tensor memory, cluster addresses, tensor maps.
//
// The tensor cores' mxf8f6f4 MMA multiplies each row's product over 32 values of
// K by two powers of two, A's and B's, that it takes as exponent bytes from
// tensor memory, and adds the fp32 results into D.  The scales of 128 rows are
// four columns: row r's 32-bit word in lane r % 32 of column r / 32, the same in
// each quarter of the lanes; the instruction descriptor says which byte of the word
// an MMA uses.  A word here is a row's scales of four neighbouring blocks of
// 128, as they lie in memory, and all four MMAs of a block use its byte.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kBlockK = 128;          // values of K per scale, and per row of a staged tile (128 bytes, 128-byte swizzle)
constexpr uint32_t kSfBytes = 512;    // scale words of 128 rows in shared memory: 32 rows of 16 bytes
constexpr uint32_t kSfCols = 4;       // and in tensor memory

// D[tmem] (+)= (A sfa) (B sfb)^T over 32 values of K.
template <int kGroup>
__device__ __forceinline__ void umma_mx8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if (kGroup == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor of it: e4m3 A and B, both K-major, shape M x N, e8m0
// scales; `byte` is added by mx8_byte.
__host__ __device__ constexpr uint32_t idesc_mx8(int M, int N) {
  return (static_cast<uint32_t>(N >> 3) << 17)      // N / 8
         | (1u << 23)                               // scales are e8m0
         | (static_cast<uint32_t>(M >> 7) << 27);   // M / 128
}
// The byte of the scale words that an MMA uses, A's and B's.
__device__ __forceinline__ uint32_t mx8_byte(uint32_t byte) { return byte << 4 | byte << 29; }

// 32 rows of 16 bytes in shared memory (scale words of 128 rows) to four
// columns of tensor memory, the same in each quarter of the lanes.  Runs in the order
// of issue with the MMAs.
template <int kGroup>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t saddr) {
  // rows of 16 bytes, groups of eight rows 128 bytes apart, no swizzle
  const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 32) |
                        (static_cast<uint64_t>(1u) << 46);
  if (kGroup == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// The address of `saddr` (shared memory of this CTA) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// (relaxed: what it is to make visible, barriers just made, was fenced for that)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The MMA warps run whole, so that descriptors and addresses stay in uniform registers, as the
// MMA takes them; one elected lane issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// Such a warp's wait: tested again and again, since a suspended wait is woken late, within mbar_wait's limits.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns) {
  if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) return true;
  uint64_t from = 0;
  for (uint32_t it = 1; limit_ns; ++it) {
    if (__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) return true;
    if ((it & 255u) == 0) {
      if (__any_sync(0xFFFFFFFFu, *abort)) return false;
      const uint64_t now = globaltimer();
      if (from == 0) from = now;
      if (__any_sync(0xFFFFFFFFu, now - from > limit_ns)) break;
    }
  }
  set_status(status, MOE_ERR_TIMEOUT);
  *abort = 1;
  return false;
}

// The scales of the blocks 4 g .. 4 g + 3 of kRows rows as words, from the aligned words that hold them: one each
// where rows of scales are words, else two, of which a byte at least is of the row (what lies beside it, beyond the last
// block too, is not used).  All loads are issued together, for the scales' warp has as long as the MMAs of four blocks:
// 8192 x 4096 x 2176 takes 53 us (17 scales a row; 47.7 us with 16, which are words), and 76 us where each row's
// second load waits for its first.
template <int kRows>
__device__ __forceinline__ void scale_words(uint32_t (&w)[kRows], const uint8_t* const (&row)[kRows], const bool (&in)[kRows], int g,
                                            int blocks, bool words) {
  if (words) {
#pragma unroll
    for (int c = 0; c < kRows; ++c) w[c] = in[c] ? reinterpret_cast<const uint32_t*>(row[c])[g] : 0x7F7F7F7Fu;   // (1.0)
  } else {
    uint32_t lo[kRows], hi[kRows];
#pragma unroll
    for (int c = 0; c < kRows; ++c) {
      const uint8_t* p = row[c] + 4 * g;
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
      const uint32_t* at = reinterpret_cast<const uint32_t*>(p - off);
      lo[c] = in[c] ? at[0] : 0u;
      hi[c] = in[c] ? at[off && 4 * g + 4 - off < blocks ? 1 : 0] : 0u;
    }
#pragma unroll
    for (int c = 0; c < kRows; ++c)
      w[c] = in[c] ? __funnelshift_r(lo[c], hi[c], 8 * static_cast<int>(reinterpret_cast<uintptr_t>(row[c] + 4 * g) & 3)) : 0x7F7F7F7Fu;
  }
}
__device__ __forceinline__ bool scales_are_words(const uint8_t* scales, long long lds, int rows) {
  return (reinterpret_cast<uintptr_t>(scales) & 3) == 0 && (rows == 1 || (lds & 3) == 0);
}
// Those of rows row0 + lane + 32 c (c < 4) of `rows` (rows beyond have 1.0: their codes read as 0).
__device__ __forceinline__ uint4 scale_words_of_rows(const uint8_t* scales, long long lds, int row0, int rows, int g, int blocks, bool words) {
  const int r = row0 + static_cast<int>(threadIdx.x & 31);
  const uint8_t* row[4];
  bool in[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    row[c] = scales + (r + 32 * c) * lds;
    in[c] = r + 32 * c < rows;
  }
  uint32_t w[4];
  scale_words(w, row, in, g, blocks, words);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A byte matrix [rows][cols], rows `ld` bytes apart, in boxes of 128 bytes x
// box_rows in the 128-byte swizzle; what lies outside reads as 0.
bool linear8_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows);

// The output in boxes of 32 columns x box_rows (64-byte swizzle), N a multiple of 8; what lies outside is not written.
bool linear8_out_map(CUtensorMap* m, const Linear8& a, uint32_t box_rows);

// Up to 16 rows, of the sizes that it takes: a stream of the weights.
bool linear8_few_takes(const Linear8& a, int sms);
int linear8_few_launch(const Linear8& a, int sms, cudaStream_t stream);
// Many rows: tiles of 256 tokens by pairs of CTAs.
int linear8_wide_launch(const Linear8& a, int* status, int sms, cudaStream_t stream);

}  // namespace moe
