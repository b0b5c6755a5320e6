// gemm16_pair.cuh -- the large dense linear on pairs of SMs.
//
// A cluster of two CTAs works on one tile of 256 rows of x and two 128-row
// blocks of the weights (256 outputs, or gate and up of 128 features) with
// tcgen05.mma.cta_group::2: CTA r holds rows 128 r .. of x (operand A) and weight
// block r (half of operand B) in its shared memory, and receives its rows' 256
// columns in its own tensor memory.  Per stage of 64 inputs an SM loads 32 KB
// where a tile of its own of 128 rows x 256 outputs takes 48 KB, and that
// traffic is power, which is what holds a long run of large products.
//
// The even CTA leads: both CTAs' loads count on its barriers, its thread issues
// the products of both, and their completion (tcgen05.commit, to both CTAs)
// frees the stages and hands the accumulators to the epilogues.  Two
// accumulator sets; the epilogue is the one of gemm16.cuh with the rows on M.
// Every wait is bounded; both CTAs meet at the end whatever happened.
#pragma once
#include "gemm16.cuh"

namespace moe {

struct Gemm16PairCfg {
  static constexpr int kStages = 6;
  static constexpr uint32_t kStage = 2 * 128 * 128;  // 128 rows of x, 128 of the weights, 64 inputs each
  static constexpr uint32_t kTailOff = kStages * kStage;
  static constexpr uint32_t kSmemBytes = kTailOff + 1024 /* alignment */ + 256;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

// Address of this CTA's shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// A TMA load into this CTA whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The issued products' completion arrives at this barrier of both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, uint32_t limit) {
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}

template <bool kGated, bool kF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kG16Threads, 1)
    gemm16_pair_kernel(Gemm16Args a, const __grid_constant__ CUtensorMap w_map,
                       const __grid_constant__ CUtensorMap x64_map, const __grid_constant__ CUtensorMap x16_map) {
  using C = Gemm16PairCfg;
  constexpr int kOut = kGated ? 128 : 256;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kTailOff);  // used in the even CTA
  uint64_t *empty = full + C::kStages;
  uint64_t *acc_full = empty + C::kStages;  // [2]
  uint64_t *acc_empty = acc_full + 2;       // [2], used in the even CTA
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(acc_empty + 2);
  volatile int *abort_s = reinterpret_cast<volatile int *>(tmem_base_s + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kG16EpiWarps);
    }
    *abort_s = 0;
    fence_mbar_init();
    tma_prefetch_map(&w_map);
    tma_prefetch_map(&x64_map);
    tma_prefetch_map(&x16_map);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_base_s)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers and tensor memory are ready
  tc_fence_after();
  grid_dep_trigger();
  const uint32_t tmem = *tmem_base_s;
  const int ntiles = ((a.rows + 255) / 256) * a.nfb;
  const int t0 = blockIdx.x >> 1, G = gridDim.x >> 1;
  const int KB = (a.K + kG16BK - 1) / kG16BK;
  auto fail = [&]() {
    atomicExch(a.err, DEVERR_PREFILL_WAIT);
    *abort_s = 1;
  };
  // valid rows of CTA r of tile t's rows, in whole boxes of 16
  auto valid = [&](int row0, int r) { return min(max(a.rows - row0 - 128 * r, 0), 128); };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int t = t0; t < ntiles && ok && !*abort_s; t += G) {
        const int row0 = t / a.nfb * 256, n0 = t % a.nfb * kOut;
        const int nrows = (valid(row0, rank) + 15) & ~15, mine = row0 + 128 * rank;
        const uint32_t bytes = 2u * 128u * 128u + 128u * (uint32_t)(((valid(row0, 0) + 15) & ~15) + ((valid(row0, 1) + 15) & ~15));
        const int wrow = n0 + rank * a.mat_off;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_cluster(&empty[s], ph ^ 1u, kG16WaitPolls)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t at = smem_u32(smem + s * C::kStage), wt = at + 128 * 128;
          const uint32_t bar = mapa_u32(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          tma_load_2d_pair(wt, &w_map, kb * kG16BK, wrow, bar);
          int r = 0;
          for (; r + 64 <= nrows; r += 64) tma_load_2d_pair(at + r * 128, &x64_map, kb * kG16BK, mine + r, bar);
          for (; r < nrows; r += 16) tma_load_2d_pair(at + r * 128, &x16_map, kb * kG16BK, mine + r, bar);
          if (++s == C::kStages) s = 0, ph ^= 1u;
        }
      }
      // The leader's products also arrive on the other CTA's `empty` barriers: a
      // CTA stays until the last arrival of each stage has come.
      for (int i = 0; i < C::kStages && ok && !*abort_s; ++i) {
        if (!mbar_wait_cluster(&empty[s], ph ^ 1u, kG16WaitPolls)) {
          fail();
          ok = false;
        }
        if (++s == C::kStages) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
      // M = 256 over the pair, N = 256
      const uint32_t idesc = (idesc_16_f32(256, kF16) & ~(31u << 24)) | ((256u >> 4) << 24);
      uint32_t s = 0, ph = 0, tc = 0;
      bool ok = true;
      for (int t = t0; t < ntiles && ok && !*abort_s; t += G, ++tc) {
        const uint32_t acc = tmem + (tc & 1u) * 256u;
        if (!mbar_wait_cluster(&acc_empty[tc & 1u], ((tc >> 1) & 1u) ^ 1u, kG16WaitPolls)) {
          fail();
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_cluster(&full[s], ph, kG16WaitPolls)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + (s * C::kStage >> 4), bd = ad + (128 * 128 >> 4);
#pragma unroll
          for (int kk = 0; kk < kG16BK / 16; ++kk)
            tc_mma_pair(acc, ad + (kk * 32 >> 4), bd + (kk * 32 >> 4), idesc, (kb | kk) ? 1u : 0u);
          tc_commit_pair(&empty[s]);
          if (++s == C::kStages) s = 0, ph ^= 1u;
        }
        if (ok) tc_commit_pair(&acc_full[tc & 1u]);
      }
    }
  } else {
    // epilogue: lane: row 32 q + lane of this CTA's 128; the quarter's warps take 16 outputs in turn
    const int q = warp & 3, sub = (warp - 2) >> 2;
    constexpr int kStep = 16 * (kG16EpiWarps / 4);
    const uint32_t free0 = mapa_u32(smem_u32(acc_empty), 0);
    uint32_t tc = 0;
    for (int t = t0; t < ntiles && !*abort_s; t += G, ++tc) {
      const int row0 = t / a.nfb * 256 + 128 * rank, n0 = t % a.nfb * kOut;
      const int nvalid = valid(row0, 0), outs = min(kOut, a.N - n0), row = q * 32 + lane;
      const bool live = row < nvalid;
      const uint16_t *rrow = a.residual + (int64_t)(row0 + row) * a.ldr + n0;
      uint32_t rr[8] = {};
      if (a.residual && live && sub * 16 < outs) gemm16_load16(rrow + sub * 16, outs - sub * 16, rr);
      if (!mbar_wait_cluster(&acc_full[tc & 1u], (tc >> 1) & 1u, kG16WaitPolls)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + (tc & 1u) * 256u + ((uint32_t)(q * 32) << 16);
      if (q * 32 < nvalid)
        for (int c0 = sub * 16; c0 < outs; c0 += kStep) {
          uint32_t v[2][16], rnext[8] = {};
          tmem_ld16_async(acc + c0, v[0]);
          if (kGated) tmem_ld16_async(acc + 128 + c0, v[1]);
          if (a.residual && live && c0 + kStep < outs) gemm16_load16(rrow + c0 + kStep, outs - c0 - kStep, rnext);
          tmem_ld_wait();
          float p[2][16];
#pragma unroll
          for (int m = 0; m < (kGated ? 2 : 1); ++m) {
            tmem_regs_after_wait(v[m]);
#pragma unroll
            for (int i = 0; i < 16; ++i) p[m][i] = __uint_as_float(v[m][i]);
          }
          if (live) gemm16_emit_row<kGated, kF16, false>(a, n0 + c0, row0 + row, rr, p[0], p[kGated ? 1 : 0]);
#pragma unroll
          for (int i = 0; i < 8; ++i) rr[i] = rnext[i];
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(free0 + (tc & 1u) * 8u) : "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // Aborted CTAs come here too.  The loads that a CTA still has in flight land
  // in its own shared memory and count on the even CTA's barriers, so neither
  // may leave before the other has arrived, and an aborted one waits a while.
  if (*abort_s) {
    for (int i = 0; i < 100; ++i) __nanosleep(1000000);
  }
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <bool kGated, bool kF16>
static moe_status gemm16_pair_launch(const Gemm16Args &a, int pairs, const CUtensorMap &w, const CUtensorMap &x64,
                                     const CUtensorMap &x16, int dev, cudaStream_t stream) {
  using C = Gemm16PairCfg;
  auto kern = gemm16_pair_kernel<kGated, kF16>;
  static std::atomic<bool> attr_done[64];  // per device; the attribute call is idempotent
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    attr_done[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kG16Threads), C::kSmemBytes, stream, a, w, x64, x16);
}

}  // namespace moe
