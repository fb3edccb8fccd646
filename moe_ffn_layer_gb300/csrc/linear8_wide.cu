// Product of two 8-bit matrices with block scales, many rows of A: tiles of 256
// tokens x kBN weight rows, computed by pairs of CTAs (two-CTA MMAs, M = 256).
//
// Each CTA of a pair stages its tokens and half of the tile's weight rows, and holds
// its tokens' sums in tensor memory; the first one's MMA warp issues for both.  Tensor
// memory holds two accumulators of 256 x 224 and the scales beside them (two of 256
// columns would leave the scales no room).
//
// Bound: 16384 x 8192 x 4096 in 317 us, 3.46 PFLOP/s, at 2070 MHz: copies and MMAs
// beside each other, which meet in shared memory (the copies without MMAs take 237 us of
// it, the MMAs without copies 264), and then the power cap: run back to back the
// clock settles at 1.45 GHz and a call at 368 us.  A tile has 512 tokens where that
// many fill the pairs, since it then moves (512 + 224) rows a block of K instead of
// 2 (256 + 224) for the same products.  (Its kernel spills 28 bytes: an epilogue thread
// holds 112 packed pairs beside the 32 columns that it reads.)
// What it took (16384 x 8192 x 4096): pairs instead of single CTAs 997 -> 408 us; the
// MMA warp run whole, descriptors in uniform registers -> 356; two accumulators of a
// 512-token tile -> 327; copies issued by a whole warp, the accumulators in turn
// block by block instead of by twos -> 317.
#include <mutex>

#include "linear8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 384;   // 4 warps: copies, MMAs, scales, tensor memory; 8 warps: the epilogue
constexpr int kRows = 256;      // tokens of an accumulator, 128 in each CTA

// Two accumulators of 256 x kBN: kAcc == 1, a tile's, in turn; kAcc == 2, the halves of a tile of 512 tokens.
template <int kBN, int kAcc>
struct Cfg {
  static constexpr int kM = kAcc * kRows;
  static constexpr uint32_t kABytes = kRows / 2 * kBlockK, kBBytes = kBN / 2 * kBlockK;
  static constexpr uint32_t kStageBytes = kAcc * kABytes + kBBytes;
  static constexpr int kSlots = 2;   // of scale words, four blocks of K each
  static constexpr int kCopies = kAcc + (kBN + 127) / 128;   // of 128 rows: the tokens', the weights'
  static constexpr uint32_t kSlotBytes = kCopies * kSfBytes;
  static constexpr uint32_t kOutBytes = 8 * 2 * 32 * 64;   // an epilogue warp's 32 rows of 32 bf16, twice
  static constexpr int kStages = (232448 - 1024 - 512 - kOutBytes - kSlots * kSlotBytes) / kStageBytes;
  static constexpr uint32_t kOut = kStages * kStageBytes;
  static constexpr uint32_t kSf = kOut + kOutBytes;
  static constexpr uint32_t kCtl = kSf + kSlots * kSlotBytes;
  static constexpr uint32_t kSmem = kCtl + 512 + 1024;   // (1024: the ring's alignment)
  static constexpr uint32_t kSfBase = 2 * kBN;
  static constexpr uint32_t kSlotCols = kCopies * kSfCols;
  static_assert(kSfBase + kSlots * kSlotCols <= 512, "tensor memory");
  static_assert((2 * kStages + 2 * kSlots + 4 + 1) * 8 + 16 <= 512, "control region");
  static_assert(kStageBytes % 1024 == 0 && kBN % 32 == 0, "swizzled tiles, scale words by 32 rows");
};

// A wait for a barrier that threads of the other CTA arrive on.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                                  uint64_t limit_ns) {
  // (the second test, of a phase that is complete, has the other CTA's writes acquired)
  return warp_wait(bar, parity, abort, status, limit_ns) && __all_sync(0xFFFFFFFFu, try_wait_cluster(bar, parity));
}
__device__ __forceinline__ void arrive_first(uint64_t* bar) {   // on the first CTA's barrier
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(smem_u32(bar), 0)) : "memory");
}

// A box into this CTA's shared memory, its bytes counted on the first CTA's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
// Arrives on `bar` of both CTAs when the MMAs and copies issued so far by this thread are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Tiles in groups of eight rows of tiles, so that the tiles that run at once share operands in L2.
struct Tiles {
  int mt, nt;
  __device__ __forceinline__ void at(int tile, int* m, int* n) const {
    const int per = 8 * nt, g = tile / per, r = tile - g * per, high = min(8, mt - 8 * g);
    *n = r / high;
    *m = 8 * g + r - *n * high;
  }
};

// 32 rows of bf16 pairs, a lane's each, to rows of any alignment, ldo apart: each lane the elements up to its
// row's first 16-byte boundary; the rest, moved down so that vectors begin there, through shared memory (32 rows of
// 128 bytes at `staging`), from where eight lanes store a row's vectors side by side.  (16384 x 2047 x 64: 149 us by
// single elements.)
template <int kPairs>
__device__ __forceinline__ void store_rows(__nv_bfloat16* first, long long ldo, int rows, int cols, uint32_t staging,
                                           uint32_t (&v)[kPairs]) {
  const int lane = threadIdx.x & 31;
  auto head_of = [&](const __nv_bfloat16* to) { return static_cast<int>(-(reinterpret_cast<uintptr_t>(to) >> 1) & 7); };
  __nv_bfloat16* own = first + lane * ldo;
  const int head = head_of(own);
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < min(head, cols) && lane < rows) *reinterpret_cast<uint16_t*>(own + i) = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const uint32_t next = i + 1 < kPairs ? v[i + 1] : 0u;
    v[i] = head & 1 ? __byte_perm(v[i], next, 0x5432) : v[i];
  }
#pragma unroll
  for (int i = 0; i + 1 < kPairs; ++i) v[i] = head & 2 ? v[i + 1] : v[i];
#pragma unroll
  for (int i = 0; i + 2 < kPairs; ++i) v[i] = head & 4 ? v[i + 2] : v[i];
#pragma unroll
  for (int c = 0; c < kPairs; c += 32) {   // 32 pairs: 8 vectors of a row
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + 4 * j < kPairs)
        sts_u4(staging + lane * 128 + ((j ^ (lane & 7)) << 4), make_uint4(v[c + 4 * j], v[c + 4 * j + 1], v[c + 4 * j + 2], v[c + 4 * j + 3]));
    __syncwarp();
    const int j = lane & 7;
    if (c + 4 * j < kPairs)
#pragma unroll 2
      for (int r = lane >> 3; r < rows; r += 4) {
        __nv_bfloat16* to = first + r * ldo;
        const int at = head_of(to) + 2 * c + 8 * j;
        if (at >= cols) continue;
        const uint4 x = lds_u4(staging + r * 128 + ((j ^ (r & 7)) << 4));
        if (at + 8 <= cols) {
          *reinterpret_cast<uint4*>(to + at) = x;
        } else {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (at + i < cols) *reinterpret_cast<uint16_t*>(to + at + i) = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
      }
  }
}

template <int kBN, int kAcc>
__global__ void __launch_bounds__(kThreads, 1) linear8_wide_kernel(const __grid_constant__ CUtensorMap ma,
                                                                   const __grid_constant__ CUtensorMap mw,
                                                                   const __grid_constant__ CUtensorMap mo, Linear8 a, int tma_out,
                                                                   int* status, uint64_t wait_ns) {
  using C = Cfg<kBN, kAcc>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kCtl);   // (the first CTA's)
  uint64_t* empty = full + C::kStages;
  uint64_t* sf_full = empty + C::kStages;                         // (the first CTA's)
  uint64_t* sf_empty = sf_full + C::kSlots;
  uint64_t* acc_full = sf_empty + C::kSlots;
  uint64_t* acc_empty = acc_full + 2;                             // (the first CTA's)
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int blocks = (a.K + kBlockK - 1) / kBlockK;
  const Tiles order{(a.T + C::kM - 1) / C::kM, (a.N + kBN - 1) / kBN};
  const int tiles = order.mt * order.nt, step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&sf_full[i], 2);
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kAcc == 1 ? 16 : 8);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 3) {
    // both CTAs of the pair, and only one CTA fits an SM: no other can hold the columns for good
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mw);
    if (tma_out) tma_prefetch_desc(&mo);
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int issued = 0;   // blocks of K whose copies were started
  if (warp == 0) {
    const bool one = elect_one();
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t ring = smem_u32(smem), bars = cluster_addr(smem_u32(full), 0);
    int stage = 0, m, n;
    uint32_t phase = 0;
    bool ok = true;
    order.at(blockIdx.x >> 1, &m, &n);
    chain_wait();
    for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += step) {
      const int row_a = m * C::kM + rank * (kRows / 2), row_b = n * kBN + rank * (kBN / 2);
      for (int kb = 0; kb < blocks; ++kb) {
        if (!(ok = warp_wait(&empty[stage], phase ^ 1u, abort_flag, status, wait_ns))) break;
        const uint32_t at = ring + stage * C::kStageBytes, bar = bars + stage * 8;
        if (one) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
#pragma unroll
          for (int h = 0; h < kAcc; ++h) tma_load_pair(at + h * C::kABytes, &ma, bar, kb * kBlockK, row_a + h * kRows, pol);
          tma_load_pair(at + kAcc * C::kABytes, &mw, bar, kb * kBlockK, row_b, pol);
        }
        __syncwarp();
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (tile + step < tiles) order.at(tile + step, &m, &n);
    }
  } else if (warp == 1 && rank == 0) {
    const bool one = elect_one();
    int stage = 0, slot = 0, tile_no = 0;
    uint32_t phase = 0, sf_phase = 0;
    bool ok = true;
    chain_wait();   // (it touches no memory of the launch before, but its waits are not to count, or spin through, that one's time)
    for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += step, ++tile_no) {
      for (int kb = 0; kb < blocks; ++kb) {
        const uint32_t sfa = tmem + C::kSfBase + slot * C::kSlotCols, sfb = sfa + kAcc * kSfCols;
        const bool last = kb == blocks - 1, slot_done = (kb & 3) == 3 || last;
        if ((kb & 3) == 0 && !(ok = warp_wait_cluster(&sf_full[slot], sf_phase, abort_flag, status, wait_ns))) break;
        if (!(ok = warp_wait(&full[stage], phase, abort_flag, status, wait_ns))) break;
        const uint32_t sf_at = smem_u32(smem + C::kSf + slot * C::kSlotBytes), at = smem_u32(smem + stage * C::kStageBytes);
        const uint64_t da = smem_desc_k128(at), db = smem_desc_k128(at + kAcc * C::kABytes);
        const uint32_t idesc = idesc_mx8(kRows, kBN) | mx8_byte(kb & 3);
#pragma unroll
        for (int h = 0; h < kAcc; ++h) {
          // the accumulator: given back by the epilogue before a tile's first block
          const int acc = kAcc == 1 ? tile_no & 1 : h;
          const uint32_t uses = kAcc == 1 ? tile_no >> 1 : tile_no;
          if (kb == 0 && !(ok = warp_wait_cluster(&acc_empty[acc], (uses & 1) ^ 1u, abort_flag, status, wait_ns))) break;
          tc_fence_after();
          if (one) {
            if (h == 0 && (kb & 3) == 0) {
#pragma unroll
              for (int c = 0; c < C::kCopies; ++c) scales_to_tmem<2>(sfa + c * kSfCols, sf_at + c * kSfBytes);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)   // 32 values of K: 32 bytes, 2 in the descriptor's units
              umma_mx8<2>(tmem + acc * kBN, da + h * (C::kABytes >> 4) + 2 * k, db + 2 * k, idesc, sfa + h * kSfCols, sfb, kb > 0 || k > 0);
            if (last) commit_pair(&acc_full[acc]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (one) {
          commit_pair(&empty[stage]);
          if (slot_done) commit_pair(&sf_empty[slot]);
        }
        __syncwarp();
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (slot_done && ++slot == C::kSlots) {
          slot = 0;
          sf_phase ^= 1u;
        }
      }
    }
    if (one) commit_pair(drained);   // (whatever was issued)
  } else if (warp == 2) {
    int slot = 0;
    uint32_t phase = 0;
    const int groups = (blocks + 3) >> 2;
    bool ok = true;
    const bool words_a = scales_are_words(a.a_scales, a.las, a.T), words_w = scales_are_words(a.w_scales, a.lws, (a.N + 127) >> 7);
    chain_wait();
    for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += step) {
      int m, n;
      order.at(tile, &m, &n);
      for (int g = 0; g < groups; ++g) {
        uint4 w[C::kCopies];
#pragma unroll
        for (int h = 0; h < kAcc; ++h)
          w[h] = scale_words_of_rows(a.a_scales, a.las, m * C::kM + h * kRows + rank * (kRows / 2), a.T, g, blocks, words_a);
        // one scale for 128 weight rows: the same for 32 rows of a tile
        constexpr int kParts = 4 * (C::kCopies - kAcc);
        const uint8_t* row[kParts];
        bool in[kParts];
        uint32_t v[kParts];
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          row[c] = a.w_scales + ((n * kBN + 32 * c) >> 7) * a.lws;
          in[c] = 32 * c < kBN && n * kBN + 32 * c < a.N;
        }
        scale_words(v, row, in, g, blocks, words_w);
#pragma unroll
        for (int i = 0; i < C::kCopies - kAcc; ++i) w[kAcc + i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sf_empty[slot], phase ^ 1u, abort_flag, status, wait_ns)))) break;
        const uint32_t at = smem_u32(smem + C::kSf + slot * C::kSlotBytes) + lane * 16;
#pragma unroll
        for (int i = 0; i < C::kCopies; ++i) sts_u4(at + i * kSfBytes, w[i]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_first(&sf_full[slot]);
        if (++slot == C::kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 3) {
    // The next launch may set itself up meanwhile: this CTA holds its tensor memory (one that still
    // had to get it could wait for a CTA that waits for this launch).
    chain_release();
  } else if (warp >= 4) {
    chain_wait();
    const int quad = warp & 3, group = (warp >> 2) - 1;
    const uint32_t stage_out = smem_u32(smem + C::kOut) + (warp - 4) * 2 * 32 * 64;
    uint32_t half = 0;   // of the staging rows: one is written while the other leaves
    // 32 columns of this lane's row, as 16 pairs, through staging rows that leave by TMA
    auto store = [&](const uint32_t* v, int col, int row0) {
      if (col >= a.N || row0 >= a.T) return;
      const uint32_t at = stage_out + half;
      half ^= 32 * 64;
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j)   // rows of 64 bytes in the 64-byte swizzle
        sts_u4(at + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4), make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(&mo)), "r"(at), "r"(col), "r"(row0)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    };
    // A group of four warps has an accumulator of its own (kAcc == 2), or half the columns of each in turn.
    constexpr int kCols = kAcc == 2 ? kBN : (kBN + 63) / 64 * 32;
    const int from = kAcc == 2 ? 0 : group * kCols, cols = min(kCols, kBN - from);
    int acc_no = kAcc == 2 ? group : 0;
    uint32_t phase = 0;
    for (int tile = blockIdx.x >> 1; tile < tiles; tile += step) {
      int m, n;
      order.at(tile, &m, &n);
      const int row0 = m * C::kM + (kAcc == 1 ? 0 : group * kRows) + rank * (kRows / 2) + quad * 32, col0 = n * kBN + from;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[acc_no], phase, abort_flag, status, wait_ns))) break;
      tc_fence_after();
      const uint32_t acc = tmem + acc_no * kBN + from + (static_cast<uint32_t>(quad * 32) << 16);
      // packed to bf16 at once, so that the accumulator is given back before anything is stored
      uint32_t v[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        if (c >= cols) {   // (the second group's part is smaller; store_rows moves all of v)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[c / 2 + i] = 0u;
          continue;
        }
        uint32_t r[32];
        tmem_ld_32cols(acc + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c / 2 + i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(&acc_empty[acc_no]);
      if (kAcc == 2 || (acc_no ^= 1) == 0) phase ^= 1u;
      if (tma_out) {
#pragma unroll
        for (int c = 0; c < kCols; c += 32)
          if (c < cols) store(v + c / 2, col0 + c, row0);
      } else {
        store_rows(a.out + row0 * a.ldo + col0, a.ldo, min(32, a.T - row0), min(cols, a.N - col0), stage_out, v);
      }
    }
    if (tma_out && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_timed(drained, 0, status);   // nothing more arrives here from the MMAs
  if (*abort_flag && threadIdx.x == 0) {
    // given up: the copies in flight end before the CTAs do (bounded waits); what the other CTA has
    // in flight is counted on the first one's barriers, in part perhaps: a while more for that
    if (rank == 0)
      for (int i = 0; i < C::kStages && i < issued; ++i)
        mbar_wait_timed(&full[i], ((issued - 1 - i) / C::kStages) & 1, status);
    const uint64_t from = globaltimer();
    while (globaltimer() - from < 1000000) __nanosleep(1000);
  }
  // neither CTA leaves while the other may still reach its barriers or read its operands
  tc_fence_before();
  cluster_sync_all();
  if (warp == 3) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int kBN, int kAcc>
int launch_wide(const Linear8& a, int* status, cudaStream_t stream) {
  using C = Cfg<kBN, kAcc>;
  static std::mutex mu;
  static int pairs_of[64] = {};   // the pairs that fit a device at once
  int dev = 0, pairs = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return MOE_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!pairs_of[dev]) {
      if (cudaFuncSetAttribute(linear8_wide_kernel<kBN, kAcc>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
        return MOE_ERR_CUDA;
      cudaLaunchConfig_t q = {};
      q.gridDim = dim3(2);
      q.blockDim = dim3(kThreads);
      q.dynamicSmemBytes = C::kSmem;
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = 2;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      q.attrs = &at;
      q.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&pairs, linear8_wide_kernel<kBN, kAcc>, &q) != cudaSuccess || pairs < 1) return MOE_ERR_CUDA;
      pairs_of[dev] = pairs;
    }
    pairs = pairs_of[dev];
  }
  const long long tiles = static_cast<long long>((a.T + C::kM - 1) / C::kM) * ((a.N + kBN - 1) / kBN);
  if (tiles > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  CUtensorMap ma, mw, mo = {};
  if (!linear8_map(&ma, a.a, a.T, a.K, a.lda, kRows / 2) || !linear8_map(&mw, a.w, a.N, a.K, a.ldw, kBN / 2)) return MOE_ERR_CUDA;
  // by TMA where the rows lie as it takes them, and are whole vectors of 16 bytes: it writes such a vector whole where
  // a row ends inside it
  const bool tma_out = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.N % 8 == 0 && (a.T == 1 || a.ldo % 8 == 0);
  if (tma_out && !linear8_out_map(&mo, a, 32)) return MOE_ERR_CUDA;
  const int grid = 2 * static_cast<int>(tiles < pairs ? tiles : pairs);
  return launch_chained_cluster(linear8_wide_kernel<kBN, kAcc>, dim3(grid), dim3(kThreads), C::kSmem, stream, 2, ma, mw, mo, a,
                                tma_out ? 1 : 0, status, wait_limit_ns()) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int linear8_wide_launch(const Linear8& a, int* status, int sms, cudaStream_t stream) {
  // A tile of 512 tokens takes 7/4 of the time of one of 256.
  const long long n = (a.N + 223) / 224, pairs = sms / 2;
  const long long one = (n * ((a.T + 255) / 256) + pairs - 1) / pairs, two = (n * ((a.T + 511) / 512) + pairs - 1) / pairs;
  return 4 * one < 7 * two ? launch_wide<224, 1>(a, status, stream) : launch_wide<224, 2>(a, status, stream);
}

}  // namespace moe
