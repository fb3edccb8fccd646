// Product of two 8-bit matrices with block scales, few rows of A: out[t][n] =
// sum over the 128-wide blocks b of K of 2^(ea[t][b] + ew[n / 128][b] - 254) *
// sum_{k in b} a[t][k] w[n][k].
//
// The weights are the MMA's A operand, 128 of their rows a tile, and the tokens
// its B operand, 16 to 128 columns, so that few tokens waste little of the MMA.
// K is cut between the CTAs of a cluster, enough of them to draw the weights'
// stream over every SM; each then sums its share of the tokens' partial sums, which
// the others copy into its shared memory, in the order of the ranks.
//
// Bound: of 17 to 64 rows the latency of one pass (launch, a round trip to memory, the
// exchange between CTAs: 4.5 us before any streaming) and then the weights' stream
// (64 x 6144 x 4096 in 8.5 us, 3.1 TB/s); of more rows the operands' way from L2 and
// the MMAs, which take 122 clocks each however narrow (777 x 2500 x 2000 in 10.8 us).
// Times are of replayed graphs over several sets of operands, together more than L2 holds; over one set, which L2
// holds, 64 x 6144 x 4096 takes 7.9 us and 777 x 2500 x 2000 9.9.
// What it took: copies started before the tensor memory is allocated and the next
// launch set up meanwhile (1 x 4096 x 2048, which was computed here then, 6.7 -> 5.4 us); bulk
// copies between the CTAs instead of single stores (64 x 6144 x 4096 12.2 -> 10.8);
// MMAs issued by a whole warp that spins on its barriers (10.7 -> 9.9); arrivals at the
// cluster's barrier that order nothing by themselves (9.8 -> 8.6).
#include <mutex>

#include "linear8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWideM = 128;   // weight rows of a tile

template <int kNT>
struct Cfg {
  // accumulators that the MMAs of a block take in turn (16 x 512 x 8192 6.2 us, one 6.5; 64 x 6144 x 4096, with waits that
  // took longer, 10.0 and 9.9)
  static constexpr int kChains = kNT <= 32 ? 4 : 1;
  // stages of the ring: so many that one CTA fills an SM, or two do
  static constexpr int kDeep = kNT == 16 ? 9 : kNT == 32 ? 8 : kNT == 64 ? 6 : 4;
  static constexpr int kShallow = kNT == 16 ? 5 : kNT == 32 ? 4 : kNT == 64 ? 3 : 4;
  static constexpr int kSlots = 2;   // of scale words, four blocks of K each
  static constexpr uint32_t kStageBytes = kWideM * kBlockK + kNT * kBlockK;
  // behind the ring: the others' partial sums [rank][token of the share][128] fp32, scale words (weights, tokens), barriers
  static constexpr uint32_t kSf = (kNT + 8) * kWideM * 4;
  static constexpr uint32_t kCtl = kSf + kSlots * 2 * kSfBytes;
  static constexpr uint32_t kBehind = kCtl + (2 * kDeep + 2 * kSlots + 2) * 8 + 8;
  static constexpr uint32_t smem(int stages) { return stages * kStageBytes + kBehind + 1024; }   // (1024: the ring's alignment)
  static constexpr int kCols = kChains * kNT + kSlots * 2 * kSfCols;
  static constexpr int kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr uint32_t kSfBase = kChains * kNT;
  static_assert(kNT * kWideM * 4 <= kShallow * kStageBytes, "this CTA's partial sums take the ring's place");
  // No two clusters' CTAs may each wait for tensor memory that a CTA of the other holds: as many CTAs
  // as an SM's shared memory takes (of this kernel, or the others here) find room for their columns.
  static_assert(smem(kShallow) > 75 * 1024 && kTmemCols * (smem(kShallow) <= 113 * 1024 ? 2 : 1) <= 512, "tensor memory of an SM's CTAs");
};

template <int kNT>
__global__ void __launch_bounds__(kThreads) linear8_narrow_kernel(const __grid_constant__ CUtensorMap mw,
                                                                  const __grid_constant__ CUtensorMap ma, Linear8 a, int split, int stages,
                                                                  int* status, uint64_t wait_ns) {
  using C = Cfg<kNT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* behind = smem + stages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(behind + C::kCtl);
  uint64_t* empty = full + C::kDeep;
  uint64_t* sf_full = empty + C::kDeep;
  uint64_t* sf_empty = sf_full + C::kSlots;
  uint64_t* done = sf_empty + C::kSlots;
  uint64_t* parts = done + 1;   // the others' partial sums have come
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(parts + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split;   // == rank in the cluster
  const int n0 = blockIdx.x / split * kWideM, t0 = blockIdx.y * kNT;
  const int blocks = (a.K + kBlockK - 1) / kBlockK;
  const int kb0 = static_cast<int>(static_cast<long long>(blocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / split);
  // the tile's tokens, and those of them that each CTA sums, and this one
  const int tokens = min(kNT, a.T - t0), share = (tokens + split - 1) / split;
  const int first = rank * share, mine = min(share, tokens - first);

  // the copies: started before the tensor memory is there, by the thread that made their barriers
  int issued = 0;   // blocks of K whose copies were started
  // (the weights are read once where one tile holds all tokens)
  const uint64_t pol_w = gridDim.y == 1 ? l2_policy_evict_first() : l2_policy_evict_normal(), pol_a = l2_policy_evict_last();
  auto load = [&](int kb, int stage) {
    mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
    uint8_t* at = smem + stage * C::kStageBytes;
    tma_load_2d(at, &mw, &full[stage], kb * kBlockK, n0, pol_w);
    tma_load_2d(at + kWideM * kBlockK, &ma, &full[stage], kb * kBlockK, t0, pol_a);
    ++issued;
  };
  // a group's scale words: the tokens', and the tile's weight rows', which share one
  uint4 sf_a;
  uint32_t sf_w;
  const bool words_a = scales_are_words(a.a_scales, a.las, a.T), words_w = scales_are_words(a.w_scales, a.lws, (a.N + 127) >> 7);
  auto scales = [&](int g) {
    sf_a = scale_words_of_rows(a.a_scales, a.las, t0, a.T, g, blocks, words_a);
    const uint8_t* row[1] = {a.w_scales + static_cast<long long>(n0 >> 7) * a.lws};
    const bool in[1] = {true};
    uint32_t w[1];
    scale_words(w, row, in, g, blocks, words_w);
    sf_w = w[0];
  };
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&mw);
    tma_prefetch_desc(&ma);
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&sf_full[i], 1);
      mbar_init(&sf_empty[i], 1);
    }
    mbar_init(done, 1);
    mbar_init(parts, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (mine > 0 && split > 1) mbar_arrive_expect_tx(parts, (split - 1) * mine * kWideM * 4);
    chain_wait();
    for (int i = 0; i < stages && kb0 + i < kb1; ++i) load(kb0 + i, i);
  }
  if (warp == 2) {
    chain_wait();
    scales(kb0 >> 2);
  }
  if (warp == 3) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (split > 1) cluster_arrive();   // (waited for before the first access to another CTA)

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0 + stages; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase, abort_flag, status, wait_ns)) break;
        load(kb, stage);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    int stage = 0, slot = 0;
    uint32_t phase = 0, sf_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint32_t sfa = tmem + C::kSfBase + slot * 2 * kSfCols, sfb = sfa + kSfCols;
      const bool group = kb == kb0 || (kb & 3) == 0;
      if (group && !warp_wait(&sf_full[slot], sf_phase, abort_flag, status, wait_ns)) break;
      if (!warp_wait(&full[stage], phase, abort_flag, status, wait_ns)) break;
      tc_fence_after();
      const uint32_t sf_at = smem_u32(behind + C::kSf + slot * 2 * kSfBytes), at = smem_u32(smem + stage * C::kStageBytes);
      const uint64_t da = smem_desc_k128(at), db = smem_desc_k128(at + kWideM * kBlockK);
      const uint32_t idesc = idesc_mx8(kWideM, kNT) | mx8_byte(kb & 3);
      if (one) {
        if (group) {
          scales_to_tmem<1>(sfa, sf_at);
          scales_to_tmem<1>(sfb, sf_at + kSfBytes);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)   // 32 values of K: 32 bytes, 2 in the descriptor's units
          umma_mx8<1>(tmem + (k % C::kChains) * kNT, da + 2 * k, db + 2 * k, idesc, sfa, sfb, kb > kb0 || k >= C::kChains);
        umma_commit(&empty[stage]);
        if ((kb & 3) == 3) umma_commit(&sf_empty[slot]);
      }
      __syncwarp();
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      if ((kb & 3) == 3 && ++slot == C::kSlots) {
        slot = 0;
        sf_phase ^= 1u;
      }
    }
    if (one) umma_commit(done);   // (whatever was issued)
  } else if (warp == 2) {
    int slot = 0;
    uint32_t phase = 0;
    const int g1 = (kb1 + 3) >> 2;
    for (int g = kb0 >> 2; g < g1; ++g) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sf_empty[slot], phase ^ 1u, abort_flag, status, wait_ns))) break;
      const uint32_t at = smem_u32(behind + C::kSf + slot * 2 * kSfBytes) + lane * 16;
      sts_u4(at, make_uint4(sf_w, sf_w, sf_w, sf_w));
      sts_u4(at + kSfBytes, sf_a);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sf_full[slot]);
      if (g + 1 < g1) scales(g + 1);
      if (++slot == C::kSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else {
    // The next launch may set itself up meanwhile: this CTA holds its tensor memory (one that still
    // had to get it could wait for a CTA that waits for this launch).
    chain_release();
  }
  __syncwarp();

  // every warp: its 32 weight rows of the accumulators
  const bool in_time = mbar_wait(done, 0, abort_flag, status, wait_ns);
  const bool ok = __syncthreads_and(in_time && !*abort_flag);
  if (!ok && threadIdx.x == 0) {
    // given up: the MMAs and copies in flight end before the CTA does (bounded waits)
    mbar_wait_timed(done, 0, status);
    for (int i = 0; i < stages && i < issued; ++i)
      mbar_wait_timed(&full[i], ((issued - 1 - i) / stages) & 1, status);
  }
  tc_fence_after();
  float* own = reinterpret_cast<float*>(smem);   // [token][128], where the ring was
  if (ok) {
    const uint32_t at = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // 64 registers at once: 16 columns of four accumulators, 64 of one
    constexpr int kStep = C::kChains == 4 ? 16 : 64;
#pragma unroll
    for (int c = 0; c < kNT; c += kStep) {
      if (c >= tokens) break;
      uint32_t r[4][16];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld_16cols(at + (C::kChains == 4 ? i * kNT + c : c + 16 * i), r[i]);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float v[4] = {__uint_as_float(r[0][j]), __uint_as_float(r[1][j]), __uint_as_float(r[2][j]), __uint_as_float(r[3][j])};
        if (C::kChains == 4) {
          own[(c + j) * kWideM + threadIdx.x] = v[0] + v[1] + v[2] + v[3];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) own[(c + 16 * i + j) * kWideM + threadIdx.x] = v[i];
        }
      }
    }
  }
  tc_fence_before();
  bool whole = ok;
  if (split > 1) {
    fence_proxy_async_smem();
    cluster_wait();   // (every CTA has made its barrier; and this one's sums are in shared memory)
    __syncthreads();
    if (ok && threadIdx.x < split && threadIdx.x != rank) {
      // to CTA r the sums of its tokens, counted on its barrier
      const int r = threadIdx.x, n = min(share, tokens - r * share);
      if (n > 0) {
        const uint32_t to = cluster_addr(smem_u32(behind) + rank * share * kWideM * 4, r);
        asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                     "r"(smem_u32(own + r * share * kWideM)), "r"(n * kWideM * 4), "r"(cluster_addr(smem_u32(parts), r))
                     : "memory");
      }
    }
    if (mine > 0) whole = mbar_wait(parts, 0, abort_flag, status, wait_ns) && ok;
    __syncwarp();
    cluster_arrive();   // what was sent here has come
  } else {
    __syncthreads();
  }
  if (whole) {
    // a lane's four weight rows: neighbours, stored as a vector, or 32 apart where the rows of `out` do not lie so
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 7) == 0 && ((a.ldo & 3) == 0 || a.T == 1) && n0 + kWideM <= a.N;
    const int at = vec ? lane * 4 : lane, n = n0 + at;
    const float* part = reinterpret_cast<const float*>(behind) + at;
    const float* here = own + first * kWideM + at;
    for (int j0 = warp; j0 < mine; j0 += 16) {   // four tokens at a time, in the order of the ranks
      float4 s[4] = {};
      for (int r = 0; r < split; ++r) {
        const float* from = r == rank ? here : part + r * share * kWideM;
        float4 p[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* q = from + (j0 + 4 * i) * kWideM;
          if (j0 + 4 * i >= mine) continue;
          if (vec) p[i] = *reinterpret_cast<const float4*>(q);
          else p[i] = make_float4(q[0], q[32], q[64], q[96]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i].x += p[i].x;
          s[i].y += p[i].y;
          s[i].z += p[i].z;
          s[i].w += p[i].w;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (j0 + 4 * i >= mine) break;
        __nv_bfloat16* to = a.out + (t0 + first + j0 + 4 * i) * a.ldo + n;
        if (vec) {
          *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(s[i].x, s[i].y), pack_bf16x2(s[i].z, s[i].w));
        } else {
          const float v[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + 32 * k < a.N) to[32 * k] = __float2bfloat16_rn(v[k]);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (split > 1) {
    cluster_wait();   // no CTA leaves before its sums have been taken
    if (!whole || wait_ns == 0) {   // given up: what the others sent may still be on its way
      const uint64_t from = globaltimer();
      while (globaltimer() - from < 1000000) __nanosleep(1000);
    }
  }
}

// How many clusters of `split` CTAs a device takes at once, with deep rings.
template <int kNT>
int clusters_at_once(int split) {
  using C = Cfg<kNT>;
  static std::mutex mu;
  static int known[64][9] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(mu);
  int& n = known[dev][split];
  if (!n) {
    if (cudaFuncSetAttribute(linear8_narrow_kernel<kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(C::kDeep)) != cudaSuccess)
      return 0;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(split);
    q.blockDim = dim3(kThreads);
    q.dynamicSmemBytes = C::smem(C::kDeep);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    q.attrs = &at;
    q.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, linear8_narrow_kernel<kNT>, &q) != cudaSuccess) n = 0;
  }
  return n;
}

template <int kNT>
int launch_narrow(const Linear8& a, int* status, cudaStream_t stream) {
  using C = Cfg<kNT>;
  const int blocks = (a.K + kBlockK - 1) / kBlockK;
  const long long tiles = static_cast<long long>((a.N + kWideM - 1) / kWideM) * ((a.T + kNT - 1) / kNT);
  if ((a.T + kNT - 1) / kNT > 65535 || !clusters_at_once<kNT>(1)) return MOE_ERR_CUDA;
  // The most CTAs a tile that fit at once; 16 and 32 tokens: four, two CTAs an SM, where that many fit.
  int split = 1, stages = C::kDeep;
  if (kNT <= 32 && tiles <= 2 * clusters_at_once<kNT>(4) && tiles > clusters_at_once<kNT>(8)) {
    split = 4;
    if (tiles > clusters_at_once<kNT>(4)) stages = C::kShallow;
  } else {
    for (int s : {8, 4, 2})
      if (tiles <= clusters_at_once<kNT>(s)) {
        split = s;
        break;
      }
    if (tiles > clusters_at_once<kNT>(1)) stages = C::kShallow;
  }
  if (split > blocks) split = blocks;
  const int most = (blocks + split - 1) / split;   // no deeper than a CTA's blocks (so that the next launch finds room)
  if (stages > most) stages = most < C::kShallow ? C::kShallow : most;
  CUtensorMap mw, ma;
  if (!linear8_map(&mw, a.w, a.N, a.K, a.ldw, kWideM) || !linear8_map(&ma, a.a, a.T, a.K, a.lda, kNT)) return MOE_ERR_CUDA;
  const dim3 grid((a.N + kWideM - 1) / kWideM * split, (a.T + kNT - 1) / kNT);
  return launch_chained_cluster(linear8_narrow_kernel<kNT>, grid, dim3(kThreads), C::smem(stages), stream, split, mw, ma, a, split,
                                stages, status, wait_limit_ns()) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t rows, uint64_t cols, uint64_t ld_bytes,
            uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  if (!fn) return false;
  // (a single row has no stride, but the map wants one)
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {rows == 1 ? 16 : ld_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool linear8_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, cols, ld, kBlockK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool linear8_out_map(CUtensorMap* m, const Linear8& a, uint32_t box_rows) {
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, a.T, a.N, 2 * a.ldo, 32, box_rows, CU_TENSOR_MAP_SWIZZLE_64B);
}

int linear8_launch(const Linear8& a, int* status, int sms, cudaStream_t stream, int* launches) {
  // Tiles of 64 tokens while an SM each is enough for them, or, up to 24 blocks of K, half an SM.  By blocks of K (16, 22,
  // 24, 26, 32), tiles of 64 tokens and of 128: 256 x 6144 10.3, 12.8, 13.3, 14.3, 16.0 and 10.7, 12.9, 13.1, 14.2, 15.4 us;
  // 512 x 4096 10.0, 12.6, 13.0, 13.8, 15.4 and 10.5, 12.8, 12.9, 13.9, 15.1; 300 x 6144 10.2, 12.8, 13.1, 14.2, 15.9 and
  // 10.7, 12.9, 13.2, 14.1, 15.5; 777 x 2500, whose last tiles are less full, 10.3, 12.7, 13.1, 14.0, 15.5 and 11.3, 13.5,
  // 13.6, 14.6, 15.9.  Then of 128, then the pairs' tiles (512 x 6144 x 4096 26.5, 27.8 and 17.7; 1024 x 4096 x 2048 18.9,
  // 19.7 and 11.8; of the sizes above the pairs' take 1.2 to 4.5 us longer than the better of the others).
  const long long wide = (a.N + kWideM - 1) / kWideM, most = a.K <= 24 * kBlockK ? 2 * sms : sms;
  int rc;
  if (linear8_few_takes(a, sms)) rc = linear8_few_launch(a, sms, stream);
  else if (a.T <= 16) rc = launch_narrow<16>(a, status, stream);
  else if (a.T <= 32) rc = launch_narrow<32>(a, status, stream);
  else if (a.T <= 64 || wide * ((a.T + 63) / 64) <= most) rc = launch_narrow<64>(a, status, stream);
  else if (wide * ((a.T + 127) / 128) <= sms) rc = launch_narrow<128>(a, status, stream);
  else rc = linear8_wide_launch(a, status, sms, stream);
  if (rc == MOE_OK) ++*launches;
  return rc;
}

}  // namespace moe
