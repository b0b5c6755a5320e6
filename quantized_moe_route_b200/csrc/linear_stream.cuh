// linear_stream.cuh -- the linear for up to 32 rows of x: a weight stream.
//
// With few rows the product is as fast as its weights arrive.  A CTA takes
// strips of R outputs (R <= 16, chosen so that the strips divide evenly over
// the SMs; gated: R / 2 gate rows and their up rows) and a group of its warps
// splits a strip's K by pairs of 64-input columns: every warp runs a private
// ring, in which its own lane 0 brings a pair of the weights (R x 128) and of x
// (its valid rows; the others and everything past K arrive as zeros) by TMA, so
// nothing is shared between warps until the strip's partial sums meet in
// shared memory (added in warp order) for the epilogue.  The next strip's
// columns are on their way meanwhile.  A pair is 256 consecutive bytes of each
// row: with single columns neighbouring halves of a DRAM burst were fetched at
// different times (16384 x 4096, one row: 30 to 42 us).
// The products run on m16n8k16 with the weights as A and the rows of x as B;
// a lane takes the 16-byte pieces 2t and 2t + 1 of a 64-input column, each as
// the fragments of two instructions (any order of k will do), which in the
// 128-byte swizzle touches every bank once.
#pragma once
#include "gemm16.cuh"

namespace moe {

constexpr int kLsWarps = 8;
constexpr int kLsCols = 2;    // 64-input columns of a stage
// Pairs of columns of a warp between additions of its accumulators to its sums:
// the tensor core's fp32 additions truncate, by up to a unit in the last place
// each (K = 2^20 without: 1.7e-4 too small), so an accumulation has at most 16.
constexpr int kLsFold = 8;
constexpr uint32_t kLsPolls = 1u << 20;

struct LinearStreamArgs {
  Gemm16Args g;
  int strips, R;       // strips of R outputs (gated: R / 2 features)
  int group_log2;      // warps to a strip
  int whole;           // K is a multiple of 64: one box brings a stage's columns, R rows each
};

template <int NB>
struct LinearStreamCfg {
  static constexpr int kStages = NB == 1 ? 4 : NB == 2 ? 3 : 2;                     // per warp: 96 to 128 KB of weights in flight
  static constexpr uint32_t kXOff = kLsCols * 2048;                   // 16 weight rows, then 8 NB rows of x
  static constexpr uint32_t kStage = kXOff + kLsCols * NB * 1024;
  static constexpr uint32_t kPartOff = kLsWarps * kStages * kStage;
  static constexpr uint32_t kPart = 16 * 8 * NB * 4;    // a warp's partial sums
  static constexpr uint32_t kBarOff = kPartOff + 2 * kLsWarps * kPart;
  static constexpr uint32_t kSmemBytes = kBarOff + kLsWarps * kStages * 8 + 1024 /* alignment */;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

template <bool kF16>
__device__ __forceinline__ void mma_w16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_bf16_pure(d, a, b0, b1);
}

template <bool kGated, bool kF16, int NB>
__global__ void __launch_bounds__(kLsWarps * 32, 1)
    linear_stream_kernel(LinearStreamArgs a, const __grid_constant__ CUtensorMap w_map,
                         const __grid_constant__ CUtensorMap x_map) {
  using C = LinearStreamCfg<NB>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff) + warp * C::kStages;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_map(&w_map);
    tma_prefetch_map(&x_map);
  }
  __syncwarp();
  grid_dep_wait();
  grid_dep_trigger();

  const int T = a.g.rows, K = a.g.K, R = a.R, G = gridDim.x;
  const int gs = 1 << a.group_log2, group = warp >> a.group_log2, wg = warp & (gs - 1);
  const int ngroups = kLsWarps >> a.group_log2;
  const int KC = (K + 64 * kLsCols - 1) / (64 * kLsCols);
  const int cols = wg < KC ? (KC - 1 - wg) / gs + 1 : 0;  // this warp's pairs of columns of a strip
  // the group's strips: every ngroups-th of the CTA's
  const int first = (int)blockIdx.x + group * G, step = ngroups * G;
  const int nstrips = first < a.strips ? (a.strips - 1 - first) / step + 1 : 0;
  uint8_t *ring = smem + warp * (C::kStages * C::kStage);
  const int per = kGated ? R / 2 : R;
  const uint32_t bytes = kLsCols * ((uint32_t)R * 128u + NB * 1024u);
  // lines of 128 bytes from a column to the next, in one box or in boxes of their own
  const int wline = a.whole ? per : kGated ? 8 : 16;

  // position of the next pair to load: strip is, column ic, ring stage ss
  int is = 0, ic = 0, ss = 0;
  auto issue = [&]() {
    if (is >= nstrips || cols == 0) return;
    if (lane == 0) {
      uint8_t *st = ring + ss * C::kStage;
      const int c = (wg + ic * gs) * kLsCols, n0 = (first + is * step) * per;
      mbar_arrive_expect_tx(&bars[ss], bytes);
      if (a.whole) {
        tma_load_3d(st, &w_map, 0, n0, c, &bars[ss]);
        if (kGated) tma_load_3d(st + kLsCols * 1024, &w_map, 0, a.g.N + n0, c, &bars[ss]);
        tma_load_3d(st + C::kXOff, &x_map, 0, 0, c, &bars[ss]);
      } else {
#pragma unroll
        for (int i = 0; i < kLsCols; ++i) {
          tma_load_2d(st + i * wline * 128, &w_map, (c + i) * 64, n0, &bars[ss]);
          if (kGated) tma_load_2d(st + kLsCols * 1024 + i * wline * 128, &w_map, (c + i) * 64, a.g.N + n0, &bars[ss]);
          tma_load_2d(st + C::kXOff + i * NB * 1024, &x_map, (c + i) * 64, 0, &bars[ss]);
        }
      }
    }
    if (++ss == C::kStages) ss = 0;
    if (++ic == cols) ic = 0, ++is;
  };
  for (int i = 0; i < C::kStages; ++i) issue();

  // pieces 2 t and 2 t + 1 of row g: of x, and of the weights, whose swizzle is the line's place among eight
  const uint32_t xo[2] = {(uint32_t)(g * 128 + (((2 * t4) ^ g) << 4)), (uint32_t)(g * 128 + (((2 * t4 + 1) ^ g) << 4))};
  uint32_t wo[kLsCols][2];
#pragma unroll
  for (int j = 0; j < kLsCols; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      wo[j][i] = (uint32_t)((j * wline + g) * 128 + (((2 * t4 + i) ^ ((j * wline + g) & 7)) << 4));
  constexpr uint32_t kRow8 = kGated ? kLsCols * 1024 : 1024;  // from row g to row g + 8 (its up row)
  auto ld16 = [](const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); };
  int cs = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int s = 0; s < nstrips; ++s) {
    float acc[NB][4][4] = {}, sum[NB][4] = {};
    auto fold = [&]() {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[nb][i] += (acc[nb][0][i] + acc[nb][1][i]) + (acc[nb][2][i] + acc[nb][3][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nb][j][i] = 0.f;
        }
    };
    for (int c = 0; c < cols && ok; ++c) {
      if (c && c % kLsFold == 0) fold();
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[cs], parity, kLsPolls))) {
        if (lane == 0) atomicExch(a.g.err, DEVERR_PREFILL_WAIT);
        ok = false;
        break;
      }
      const uint8_t *st = ring + cs * C::kStage;
#pragma unroll
      for (int j = 0; j < kLsCols; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w0 = ld16(st + wo[j][i]), w1 = ld16(st + wo[j][i] + kRow8);
          const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint4 v = ld16(st + C::kXOff + (j * NB + nb) * 1024 + xo[i]);
            mma_w16<kF16>(acc[nb][2 * i], f0, v.x, v.y);
            mma_w16<kF16>(acc[nb][2 * i + 1], f1, v.z, v.w);
          }
        }
      __syncwarp();  // the stage is read
      issue();
      if (++cs == C::kStages) cs = 0, parity ^= 1u;
    }
    fold();
    // partial sums [row][token], two buffers in turn: one barrier a strip
    float *part = reinterpret_cast<float *>(smem + C::kPartOff + (s & 1) * (kLsWarps * C::kPart));
    float *mine = part + warp * (C::kPart / 4);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = nb * 8 + 2 * t4;
      *reinterpret_cast<float2 *>(mine + g * 8 * NB + n) = make_float2(sum[nb][0], sum[nb][1]);
      *reinterpret_cast<float2 *>(mine + (g + 8) * 8 * NB + n) = make_float2(sum[nb][2], sum[nb][3]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * gs) : "memory");
    const int n0 = (first + s * step) * per;
    const float *pg = part + (group << a.group_log2) * (C::kPart / 4);
    for (int v = wg * 32 + lane; v < 16 * T; v += 32 * gs) {
      const int row = v & 15, t = v >> 4;
      if (row >= per || n0 + row >= a.g.N) continue;
      float p0[1] = {0.f}, p1[1] = {0.f};
      for (int w = 0; w < gs; ++w) {
        p0[0] += pg[w * (C::kPart / 4) + row * 8 * NB + t];
        if (kGated) p1[0] += pg[w * (C::kPart / 4) + (row + 8) * 8 * NB + t];
      }
      float b0, b1;
      uint16_t r[1] = {0};
      gemm16_bias<kGated, kF16>(a.g, n0 + row, b0, b1);
      if (a.g.residual) gemm16_residual(a.g, n0 + row, t, 1, r);
      gemm16_emit<kGated, kF16, 1, true>(a.g, n0 + row, t, 1, b0, b1, r, p0, p1);
    }
  }
  if (!ok)  // let the copies in flight land before the CTA leaves: stages cs, cs + 1, ... in order of issue
    for (int i = 0; i < C::kStages; ++i) {
      mbar_wait_bounded(&bars[cs], parity, 1u << 16);
      if (++cs == C::kStages) cs = 0, parity ^= 1u;
    }
}

template <bool kGated, bool kF16, int NB>
static moe_status linear_stream_launch(const LinearStreamArgs &a, int grid, const CUtensorMap &wm, const CUtensorMap &xm,
                                       int dev, cudaStream_t stream) {
  using C = LinearStreamCfg<NB>;
  auto kern = linear_stream_kernel<kGated, kF16, NB>;
  static std::atomic<bool> attr_done[64];  // per device; the attribute call is idempotent
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    attr_done[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kLsWarps * 32), C::kSmemBytes, stream, a, wm, xm);
}

}  // namespace moe
