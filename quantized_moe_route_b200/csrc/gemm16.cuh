// gemm16.cuh -- the tensor-core product behind moe_linear and the grouped
// FFN with bf16 experts: y = epilogue(x W^T) for 16-bit x [rows][K] and W
// [outputs][K], both K-major as they lie in memory, dense or with the rows
// of x grouped by expert.
//
// The weights are the MMA's A operand (M = 128 outputs), the rows of x its N
// (up to kNT, trimmed to the valid rows rounded up to 16), so one kernel fits
// any number of rows and a lane of tensor memory is an output: bias is one
// value a lane, and a warp's store is 32 consecutive outputs of one row.  A
// tile is a chunk of rows of one expert and kMats blocks of 128 outputs that
// share the chunk's operand: gate and up of 128 features, or 256 consecutive
// outputs, or (kMats = 1, kNT = 256) 128 outputs.
//
// Grouped, a tile holds at most 128 rows, and one of more than `flip` rows is
// issued the other way round: the rows are M, the tile's two weight blocks one
// N = 256 operand, and a lane of tensor memory is a row.  An MMA of M = 128, K =
// 16 takes about 111 cycles for any N up to 200 and about 135 for 256, so
// that is one product of 256 for two of up to 128, but it multiplies 128 rows
// whatever is valid, and a long run of these kernels is held by the board's
// power.  With flip = 32 the skewed prompt of 2048 tokens over 256 experts
// takes 246 us (0: 258, 128: 258), one of 100 tokens 253 (0: 267, 128: 253).

// Warp 0 loads 64-channel stages by TMA (128-byte swizzle; out-of-range rows
// and channels arrive as zeros), warp 1 issues tcgen05.mma into one of two
// accumulator sets in tensor memory, warps 2-13 run the epilogue of the other
// set.  Products with too few tiles for the GPU split K over a cluster of
// CTAs instead of looping over tiles: each leaves its fp32 partial in shared
// memory, and every CTA adds up its share of the rows in rank order through
// distributed shared memory (a fixed order: the same bits every call).
#pragma once
#include "w16.cuh"

namespace moe {

constexpr int kG16BK = 64;
constexpr uint32_t kG16Ring = 216 * 1024;  // bytes of the stage ring: 4 stages of the largest tiles, more of smaller ones
constexpr int kG16MaxStages = 12;
constexpr int kG16Seg = 8;          // k blocks that one accumulation runs over where y is fp32 or K long
constexpr int kG16EpiWarps = 12;  // three to a lane quarter of tensor memory
constexpr int kG16Threads = (2 + kG16EpiWarps) * 32;
constexpr uint32_t kG16WaitPolls = 1u << 18;  // sleeping polls of up to 10 us: a bound of seconds

struct Gemm16Args {
  const int32_t *offsets;  // grouped: [E + 1]; dense: NULL
  int E;                   // grouped: experts; dense: 1
  int rows, N, K;          // N: outputs (features when gated)
  int w_rows;              // weight rows per expert
  int mat_off;             // weight rows from a tile's block 0 to its block 1
  int nfb;                 // output blocks per row chunk
  int nt;                  // rows per chunk (at most kNT, a multiple of 16)
  int stages;              // of the ring (set by the launch)
  int flip;                // tiles of more rows are issued with the rows on M (two blocks of up to 128 rows)
  int splits;              // CTAs of a cluster that share a tile (1: none, persistent over tiles)
  const uint16_t *bias, *residual;
  void *y;
  int64_t ldr, ldy;
  int act, y_f32;
  int *err;
};

template <int kMats, int kNT>
struct Gemm16Cfg {
  static constexpr uint32_t kABytes = kMats * 128 * 128;  // 128 rows of 64 channels per block
  static constexpr uint32_t kBBytes = kNT * 128;
  static constexpr uint32_t kTailOff = kG16Ring;
  static_assert(4 * (kABytes + kBBytes) <= kG16Ring, "four stages");
  static constexpr uint32_t kTableInts = 1024 + 1;
  static constexpr uint32_t kSmemBytes = kTailOff + 1024 /* alignment */ + 256 + kTableInts * 4;
  static constexpr uint32_t kAccCols = kMats * kNT;
  static constexpr uint32_t kTmemCols = 2 * kAccCols <= 256 ? 256 : 512;  // a power of two
  static_assert(2 * kAccCols <= 512, "two accumulator sets in tensor memory");
  static_assert(kMats * 128 * kNT * 4 <= kTailOff, "split partials fit in the ring");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

struct Gemm16Tile {
  int row0, nvalid, n0, wrow;  // rows of x, first output, first weight row
};

// Tile t: chunk t / nfb, output block t % nfb.  start[e]: first chunk of expert e.
template <bool kGrouped, int kOut>
__device__ __forceinline__ Gemm16Tile gemm16_tile(const Gemm16Args &a, const int *start, int t) {
  Gemm16Tile ti;
  const int chunk = t / a.nfb;
  ti.n0 = (t - chunk * a.nfb) * kOut;
  if (kGrouped) {
    const int e = last_at_or_below(start, a.E, chunk);
    const int o0 = clamped_offset(a.offsets, e, a.rows), o1 = clamped_offset(a.offsets, e + 1, a.rows);
    ti.row0 = o0 + (chunk - start[e]) * a.nt;
    ti.nvalid = min(a.nt, o1 - ti.row0);
    ti.wrow = e * a.w_rows + ti.n0;
  } else {
    ti.row0 = chunk * a.nt;
    ti.nvalid = min(a.nt, a.rows - ti.row0);
    ti.wrow = ti.n0;
  }
  return ti;
}

template <bool kExact, int kN>
__device__ __forceinline__ void activate_all(float (&v)[kN], int act) {
  switch (act) {  // the branch is uniform: one loop each
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = activate<kExact>(v[i], MOE_ACT_SILU);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = activate<kExact>(v[i], MOE_ACT_GELU);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = activate<kExact>(v[i], MOE_ACT_GELU_TANH);
      break;
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = activate<kExact>(v[i], MOE_ACT_RELU);
      break;
    case MOE_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = activate<kExact>(v[i], MOE_ACT_SIGMOID);
      break;
    default: break;
  }
}

// The residual of output n in kN rows from row0 on (the first nv of them exist),
// as stored.  Issued a batch ahead of its use: its latency is the epilogue's.
template <int kN>
__device__ __forceinline__ void gemm16_residual(const Gemm16Args &a, int n, int64_t row0, int nv, uint16_t (&r)[kN]) {
  const uint16_t *rp = a.residual + row0 * a.ldr + n;
#pragma unroll
  for (int i = 0; i < kN; ++i) r[i] = i < nv && n < a.N ? rp[i * a.ldr] : (uint16_t)0;
}

// kN rows of output n from their products p0 (and, gated, p1) and residual r:
// bias (b0, b1), activation, gate, residual, store.
template <bool kGated, bool kF16, int kN, bool kExact, bool kBare = false>
__device__ __forceinline__ void gemm16_emit(const Gemm16Args &a, int n, int64_t row0, int nv, float b0, float b1,
                                            const uint16_t (&r)[kN], float (&p0)[kN], float (&p1)[kN]) {
  if (n >= a.N) return;
  if (!kBare) {
#pragma unroll
    for (int i = 0; i < kN; ++i) p0[i] += b0;
    activate_all<kExact>(p0, a.act);
  }
  if (kGated) {
#pragma unroll
    for (int i = 0; i < kN; ++i) p0[i] = (kBare ? activate(p0[i], MOE_ACT_SILU) : p0[i]) * (kBare ? p1[i] : p1[i] + b1);
  }
  if (!kBare && a.residual) {
#pragma unroll
    for (int i = 0; i < kN; ++i) p0[i] += w16_to_f32<kF16>(r[i]);
  }
  const int64_t o = row0 * a.ldy + n;
  if (!kBare && a.y_f32) {
    float *y = static_cast<float *>(a.y) + o;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < nv) y[i * a.ldy] = p0[i];
  } else {
    uint16_t *y = static_cast<uint16_t *>(a.y) + o;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < nv) y[i * a.ldy] = f32_to_w16<kF16>(p0[i]);
  }
}

// The biases of output n (gated: of its gate and up rows).
template <bool kGated, bool kF16>
__device__ __forceinline__ void gemm16_bias(const Gemm16Args &a, int n, float &b0, float &b1) {
  b0 = a.bias && n < a.N ? w16_to_f32<kF16>(a.bias[n]) : 0.f;
  b1 = kGated && a.bias && n < a.N ? w16_to_f32<kF16>(a.bias[a.N + n]) : 0.f;
}

// Four consecutive outputs n .. n + 3 of row `row` (those below a.N), from their
// products: as gemm16_emit, with the row's outputs in one vector where they
// lie on its boundary.
template <bool kGated, bool kF16, bool kExact>
__device__ __forceinline__ void gemm16_emit4(const Gemm16Args &a, int n, int64_t row, float (&p0)[4], float (&p1)[4]) {
  if (n >= a.N) return;
  const int nv = min(4, a.N - n);
  float b[2][4] = {};
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < nv) b[0][i] = w16_to_f32<kF16>(a.bias[n + i]);
      if (kGated && i < nv) b[1][i] = w16_to_f32<kF16>(a.bias[a.N + n + i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) p0[i] += b[0][i];
  activate_all<kExact>(p0, a.act);
  if (kGated) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p0[i] *= p1[i] + b[1][i];
  }
  if (a.residual) {
    const uint16_t *r = a.residual + row * a.ldr + n;
    if (nv == 4 && reinterpret_cast<uintptr_t>(r) % 8 == 0) {
      const uint2 v = *reinterpret_cast<const uint2 *>(r);
      const uint32_t u[2] = {v.x, v.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) p0[i] += w16_to_f32<kF16>((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
    } else {
      for (int i = 0; i < nv; ++i) p0[i] += w16_to_f32<kF16>(r[i]);
    }
  }
  if (a.y_f32) {
    float *y = static_cast<float *>(a.y) + row * a.ldy + n;
    if (nv == 4 && reinterpret_cast<uintptr_t>(y) % 16 == 0)
      *reinterpret_cast<float4 *>(y) = make_float4(p0[0], p0[1], p0[2], p0[3]);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < nv) y[i] = p0[i];
  } else {
    uint16_t *y = static_cast<uint16_t *>(a.y) + row * a.ldy + n;
    uint16_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32_to_w16<kF16>(p0[i]);
    if (nv == 4 && reinterpret_cast<uintptr_t>(y) % 8 == 0)
      *reinterpret_cast<uint2 *>(y) = make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < nv) y[i] = o[i];
  }
}

// Sixteen consecutive 16-bit values of a row (those below nv), as stored, in two
// vectors where they lie on a 16-byte boundary.
__device__ __forceinline__ void gemm16_load16(const uint16_t *p, int nv, uint32_t (&v)[8]) {
  if (nv >= 16 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = (2 * i < nv ? p[2 * i] : 0u) | (2 * i + 1 < nv ? (uint32_t)p[2 * i + 1] << 16 : 0u);
  }
}
template <bool kF16>
__device__ __forceinline__ float gemm16_half(uint32_t v, int hi) {
  if (kF16) return w16_to_f32<true>((uint16_t)(v >> (16 * hi)));
  return __uint_as_float(hi ? v & 0xFFFF0000u : v << 16);
}

// Sixteen consecutive outputs n .. n + 15 (those below a.N) of row `row`, from
// their products and the row's residual: as gemm16_emit, y 16-bit.  kBare: the grouped
// FFN's, SiLU on the gate or nothing, bf16 outputs in whole vectors (a kernel's
// first pass over its code is a walk through the instruction cache: with the
// linear's epilogue in its place a small prompt takes 3 us more).
template <bool kGated, bool kF16, bool kBare>
__device__ __forceinline__ void gemm16_emit_row(const Gemm16Args &a, int n, int64_t row, const uint32_t (&r)[8],
                                                float (&p0)[16], float (&p1)[16]) {
  const int nv = a.N - n;
  if (kBare) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f0 = kGated ? activate(p0[2 * i], MOE_ACT_SILU) * p1[2 * i] : p0[2 * i];
      const float f1 = kGated ? activate(p0[2 * i + 1], MOE_ACT_SILU) * p1[2 * i + 1] : p0[2 * i + 1];
      o[i] = cvt_bf16x2(f0, f1);
    }
    uint16_t *y = static_cast<uint16_t *>(a.y) + row * a.ldy + n;
    reinterpret_cast<uint4 *>(y)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4 *>(y)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    return;
  }
  if (a.bias) {
    uint32_t b[8];
    gemm16_load16(a.bias + n, nv, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) p0[i] += gemm16_half<kF16>(b[i >> 1], i & 1);
  }
  activate_all<false>(p0, a.act);
  if (kGated) {
    uint32_t b[8] = {};
    if (a.bias) gemm16_load16(a.bias + a.N + n, nv, b);
#pragma unroll
    for (int i = 0; i < 16; ++i) p0[i] *= p1[i] + gemm16_half<kF16>(b[i >> 1], i & 1);
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < 16; ++i) p0[i] += gemm16_half<kF16>(r[i >> 1], i & 1);
  }
  uint16_t *y = static_cast<uint16_t *>(a.y) + row * a.ldy + n;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = kF16 ? (uint32_t)f32_to_w16<true>(p0[2 * i]) | (uint32_t)f32_to_w16<true>(p0[2 * i + 1]) << 16
                : cvt_bf16x2(p0[2 * i], p0[2 * i + 1]);
  if (nv >= 16 && reinterpret_cast<uintptr_t>(y) % 16 == 0) {
    reinterpret_cast<uint4 *>(y)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4 *>(y)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < nv) y[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
  }
}

// A cluster's epilogue: CTA `rank` of kS adds up its share of the tile's rows
// over the partials of all kS CTAs, in rank order: a warp takes a row, a lane
// four of its 128 outputs, with the loads from all CTAs in flight together.
template <int kS, bool kGated, int kMats, int kNT, bool kF16, bool kExact>
__device__ __forceinline__ void gemm16_join(const Gemm16Args &a, const Gemm16Tile &ti, uint32_t part, int rank) {
  static_assert(kMats == 1 || kGated, "128 outputs a tile");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (ti.nvalid + kS - 1) / kS, c1 = min(ti.nvalid, (rank + 1) * per);
  part += (uint32_t)lane * 16u;
  for (int c = rank * per + warp - 2; c < c1; c += kG16EpiWarps) {
    float4 v[kS][kMats];
#pragma unroll
    for (int k = 0; k < kS; ++k)
#pragma unroll
      for (int m = 0; m < kMats; ++m) v[k][m] = ld_dsmem_f32x4(part + (uint32_t)(m * kNT + c) * 512u, k);
    float p[kMats][4];
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      float4 t = v[0][m];
#pragma unroll
      for (int k = 1; k < kS; ++k) t.x += v[k][m].x, t.y += v[k][m].y, t.z += v[k][m].z, t.w += v[k][m].w;
      p[m][0] = t.x, p[m][1] = t.y, p[m][2] = t.z, p[m][3] = t.w;
    }
    gemm16_emit4<kGated, kF16, kExact>(a, ti.n0 + 4 * lane, ti.row0 + c, p[0], p[kMats - 1]);
  }
}

template <bool kGrouped, bool kGated, int kMats, int kNT, bool kF16, bool kSeg = false>
__global__ void __launch_bounds__(kG16Threads, 1)
    gemm16_kernel(Gemm16Args a, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x64_map,
                  const __grid_constant__ CUtensorMap x16_map) {
  using C = Gemm16Cfg<kMats, kNT>;
  static_assert(!kGated || kMats == 2, "gate and up");
  constexpr bool kCanFlip = kMats == 2 && kNT == 128;  // rows on M, two weight blocks on N
  constexpr bool kOnlyFlip = kCanFlip && !kGrouped && !kGated;  // the dense linear's two blocks of outputs: flip = 0
  constexpr bool kSplits = !kGrouped && !kOnlyFlip;             // K may be shared by a cluster
  constexpr int kOut = kGated ? 128 : 128 * kMats;  // outputs per tile
  auto flipped = [&](const Gemm16Tile &ti) { return kCanFlip && (kOnlyFlip || ti.nvalid > a.flip); };
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (keeps the address space known)
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kTailOff);
  uint64_t *empty = full + kG16MaxStages;
  uint64_t *acc_full = empty + kG16MaxStages;  // [2]
  uint64_t *acc_empty = acc_full + 2;       // [2]
  uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(acc_empty + 2);
  volatile int *abort_s = reinterpret_cast<volatile int *>(tmem_base_s + 1);
  int *start = reinterpret_cast<int *>(smem + C::kTailOff + 256);  // [E + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a stage holds the weights and the nt rows that a chunk has at most
  const uint32_t stage = C::kABytes + (uint32_t)a.nt * 128u;
  const int nst = a.stages;
  if (tid == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kG16EpiWarps * 32);
    }
    *abort_s = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_base_s, C::kTmemCols);
  if (tid == 0) {
    tma_prefetch_map(&w_map);
    tma_prefetch_map(&x64_map);
    tma_prefetch_map(&x16_map);
  }
  grid_dep_wait();
  if (kGrouped && warp == 2) {  // chunk table: exclusive scan of the experts' chunk counts
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? max(clamped_offset(a.offsets, e + 1, a.rows) - clamped_offset(a.offsets, e, a.rows), 0) : 0;
      const int c = (n + a.nt - 1) / a.nt;
      int v = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e < a.E) start[e] = carry + v - c;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) start[a.E] = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_trigger();
  const uint32_t tmem = *tmem_base_s;
  const int nchunks = kGrouped ? start[a.E] : (a.rows + a.nt - 1) / a.nt;
  const int ntiles = nchunks * a.nfb;
  const int S = kSplits ? a.splits : 1, rank = S > 1 ? (int)cluster_rank() : 0;
  const int t0 = blockIdx.x / S, G = gridDim.x / S;
  const int KB = (a.K + kG16BK - 1) / kG16BK;
  const int kb0 = KB * rank / S, kb1 = KB * (rank + 1) / S;  // S <= KB: never empty
  auto fail = [&]() {
    atomicExch(a.err, DEVERR_PREFILL_WAIT);
    *abort_s = 1;
  };

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int t = t0; t < ntiles && !*abort_s; t += G) {
        const Gemm16Tile ti = gemm16_tile<kGrouped, kOut>(a, start, t);
        const int nrows = (ti.nvalid + 15) & ~15;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait_sleep(&empty[s], ph ^ 1u, kG16WaitPolls)) {
            fail();
            break;
          }
          uint8_t *at = smem + s * stage, *bt = at + C::kABytes;
          mbar_arrive_expect_tx(&full[s], C::kABytes + (uint32_t)nrows * 128u);
#pragma unroll
          for (int m = 0; m < kMats; ++m)
            tma_load_2d(at + m * 128 * 128, &w_map, kb * kG16BK, ti.wrow + m * a.mat_off, &full[s]);
          int r = 0;  // boxes of 64 rows, then of 16
          for (; r + 64 <= nrows; r += 64) tma_load_2d(bt + r * 128, &x64_map, kb * kG16BK, ti.row0 + r, &full[s]);
          for (; r < nrows; r += 16) tma_load_2d(bt + r * 128, &x16_map, kb * kG16BK, ti.row0 + r, &full[s]);
          if (++s == nst) s = 0, ph ^= 1u;
        }
      }
      // the last load issued into each stage lands before the CTA leaves: from
      // stage s on in the order of issue (a stage not used yet: its barrier's
      // phase before the first counts as complete)
      if (*abort_s)
        for (int i = 0; i < nst; ++i) {
          mbar_wait_sleep(&full[s], ph ^ 1u, kG16WaitPolls);
          if (++s == nst) s = 0, ph ^= 1u;
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
      int s = 0;
      uint32_t ph = 0, tc = 0;
      for (int t = t0; t < ntiles && !*abort_s; t += G) {
        const Gemm16Tile ti = gemm16_tile<kGrouped, kOut>(a, start, t);
        const uint32_t idesc = idesc_16_f32(flipped(ti) ? 256 : (ti.nvalid + 15) & ~15, kF16);
        bool ok = true;
        for (int kb = kb0; kb < kb1 && ok; ++tc) {  // accumulations: one, or one a segment
          const uint32_t acc = tmem + (tc & 1u) * C::kAccCols;
          if (!mbar_wait_sleep(&acc_empty[tc & 1u], ((tc >> 1) & 1u) ^ 1u, kG16WaitPolls)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const int first = kb, last = kSeg ? min(kb1, kb + kG16Seg) : kb1;
          for (; kb < last; ++kb) {
            if (!mbar_wait_sleep(&full[s], ph, kG16WaitPolls)) {
              fail();
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = desc0 + ((uint32_t)s * stage >> 4), bd = ad + (C::kABytes >> 4);
            if (flipped(ti)) {
#pragma unroll
              for (int kk = 0; kk < kG16BK / 16; ++kk)
                tc_mma_bf16(acc, bd + (kk * 32 >> 4), ad + (kk * 32 >> 4), idesc, (kb > first || kk) ? 1u : 0u);
            } else {
#pragma unroll
              for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int kk = 0; kk < kG16BK / 16; ++kk)
                  tc_mma_bf16(acc + m * kNT, ad + ((m * 128 * 128 + kk * 32) >> 4), bd + (kk * 32 >> 4), idesc,
                              (kb > first || kk) ? 1u : 0u);
            }
            tc_commit(&empty[s]);
            if (++s == nst) s = 0, ph ^= 1u;
          }
          if (ok) tc_commit(&acc_full[tc & 1u]);
        }
        if (!ok) break;
      }
    }
  } else {
    // epilogue warps: lane quarter q holds outputs 32 q + lane of each block;
    // the quarter's warps take groups of 16 rows in turn
    const int q = warp & 3, sub = (warp - 2) >> 2;
    constexpr int kStep = 16 * (kG16EpiWarps / 4);
    uint32_t tc = 0;
    for (int t = t0; t < ntiles && !*abort_s; t += G, ++tc) {
      const Gemm16Tile ti = gemm16_tile<kGrouped, kOut>(a, start, t);
      const int n = ti.n0 + q * 32 + lane;
      if constexpr (kSeg) {
        // The tensor core's fp32 additions truncate: after 128 steps of k a sum is
        // 1.9e-6 too small, which an fp32 result shows, and a 16-bit one after many
        // more.  So here an accumulation runs over 512 inputs, and the segments
        // are added in registers (K = 2048: 4e-7).
        static_assert(!kGrouped && !kCanFlip, "weights on M");
        constexpr int kB = (kNT + kStep - 1) / kStep;
        float sum[kB][kMats][16] = {};
        bool ok = true;
        for (int k0 = kb0; k0 < kb1; k0 += kG16Seg, ++tc) {
          if (!mbar_wait_sleep(&acc_full[tc & 1u], (tc >> 1) & 1u, kG16WaitPolls)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + (tc & 1u) * C::kAccCols + ((uint32_t)(q * 32) << 16);
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            const int c0 = sub * 16 + b * kStep;
            if (c0 >= ti.nvalid) break;
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
              uint32_t v[16];
              tmem_ld16(acc + m * kNT + c0, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[b][m][i] += __uint_as_float(v[i]);
            }
          }
          tc_fence_before();
          mbar_arrive(&acc_empty[tc & 1u]);
        }
        --tc;  // (the loop counts accumulations)
        if (!ok) break;
        float b0 = 0.f, b1 = 0.f;
        if (S == 1) gemm16_bias<kGated, kF16>(a, n, b0, b1);
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const int c0 = sub * 16 + b * kStep;
          if (c0 >= ti.nvalid) break;
          if (S > 1) {
            float *part = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
              for (int i = 0; i < 16; ++i) part[(m * kNT + c0 + i) * 128 + q * 32 + lane] = sum[b][m][i];
          } else {
            uint16_t r[16] = {};
            if (a.residual) gemm16_residual(a, n, ti.row0 + c0, ti.nvalid - c0, r);
            gemm16_emit<kGated, kF16, 16, true>(a, n, ti.row0 + c0, ti.nvalid - c0, b0, b1, r, sum[b][0], sum[b][kMats - 1]);
          }
        }
        continue;
      }
      float b0 = 0.f, b1 = 0.f;
      uint16_t r[16] = {};
      if (!kGrouped && S == 1 && !flipped(ti)) {  // what does not depend on the products, before waiting for them
        gemm16_bias<kGated, kF16>(a, n, b0, b1);
        if (a.residual) gemm16_residual(a, n, ti.row0 + sub * 16, ti.nvalid - sub * 16, r);
      }
      if (!mbar_wait_sleep(&acc_full[tc & 1u], (tc >> 1) & 1u, kG16WaitPolls)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + (tc & 1u) * C::kAccCols + ((uint32_t)(q * 32) << 16);
      if (flipped(ti)) {
        // lane: row 32 q + lane; columns: the tile's outputs (gated: gate, then up)
        const int row = q * 32 + lane, outs = min(kOut, a.N - ti.n0);
        const bool live = row < ti.nvalid;
        const uint16_t *rrow = a.residual + (int64_t)(ti.row0 + row) * a.ldr + ti.n0;
        uint32_t rr[8] = {};
        if (!kGrouped && a.residual && live && sub * 16 < outs) gemm16_load16(rrow + sub * 16, outs - sub * 16, rr);
        if (q * 32 < ti.nvalid)
          for (int c0 = sub * 16; c0 < outs; c0 += kStep) {
            uint32_t v[2][16], rnext[8] = {};
            tmem_ld16_async(acc + c0, v[0]);
            if (kGated) tmem_ld16_async(acc + 128 + c0, v[1]);
            if (!kGrouped && a.residual && live && c0 + kStep < outs) gemm16_load16(rrow + c0 + kStep, outs - c0 - kStep, rnext);
            tmem_ld_wait();
            float p[2][16];
#pragma unroll
            for (int m = 0; m < (kGated ? 2 : 1); ++m) {
              tmem_regs_after_wait(v[m]);
#pragma unroll
              for (int i = 0; i < 16; ++i) p[m][i] = __uint_as_float(v[m][i]);
            }
            if (live) gemm16_emit_row<kGated, kF16, kGrouped>(a, ti.n0 + c0, ti.row0 + row, rr, p[0], p[kGated ? 1 : 0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) rr[i] = rnext[i];
          }
      } else if constexpr (!kOnlyFlip) {
        for (int c0 = sub * 16; c0 < ti.nvalid; c0 += kStep) {
          uint32_t v[kMats][16];
#pragma unroll
          for (int m = 0; m < kMats; ++m) tmem_ld16_async(acc + m * kNT + c0, v[m]);
          uint16_t rn[16] = {};
          if (!kGrouped && a.residual && S == 1)  // the next batch's
            gemm16_residual(a, n, ti.row0 + c0 + kStep, ti.nvalid - c0 - kStep, rn);
          tmem_ld_wait();
          float p[2][16];
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            tmem_regs_after_wait(v[m]);
#pragma unroll
            for (int i = 0; i < 16; ++i) p[m][i] = __uint_as_float(v[m][i]);
          }
          if (S > 1) {  // partials: [block][row][128 outputs]
            float *part = reinterpret_cast<float *>(smem);
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
              for (int i = 0; i < 16; ++i) part[(m * kNT + c0 + i) * 128 + q * 32 + lane] = p[m][i];
          } else {
            gemm16_emit<kGated, kF16, 16, false, kGrouped>(a, n, ti.row0 + c0, ti.nvalid - c0, b0, b1, r, p[0], p[kMats - 1]);
            if (kMats == 2 && !kGated)  // grouped: outputs n and n + 128
              gemm16_emit<false, kF16, 16, false, true>(a, n + 128, ti.row0 + c0, ti.nvalid - c0, 0.f, 0.f, r, p[1], p[1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = rn[i];
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[tc & 1u]);
    }
  }
  if constexpr (kSplits) {
    if (S > 1) {  // one tile per cluster; every thread of every CTA comes here, aborted or not
      __syncwarp();
      cluster_sync_all();
      if (warp >= 2 && t0 < ntiles) {
        const Gemm16Tile ti = gemm16_tile<kGrouped, kOut>(a, start, t0);
        const uint32_t part = smem_u32(smem);
        if (S == 8) gemm16_join<8, kGated, kMats, kNT, kF16, kSeg>(a, ti, part, rank);
        else if (S == 4) gemm16_join<4, kGated, kMats, kNT, kF16, kSeg>(a, ti, part, rank);
        else gemm16_join<2, kGated, kMats, kNT, kF16, kSeg>(a, ti, part, rank);
      }
      cluster_sync_all();  // no CTA leaves while another may read its partials
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- host side
// 16-bit [rows][cols] with a row stride of ld elements, boxes of 64 columns x
// box_rows rows, 128-byte swizzle, zeros outside.
inline bool gemm16_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f16) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for cols a multiple of 64, as 64-column blocks: boxes of 64 columns x
// box_rows rows x `blocks` consecutive blocks.
inline bool gemm16_map3(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows, int blocks,
                        bool f16) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DeviceInfo {
  int dev, sms;
};
// The current device and its SM count (looked up once per device).
inline bool device_info(DeviceInfo *d) {
  static std::atomic<int> sms[64];
  cudaError_t e = cudaGetDevice(&d->dev);
  if (e == cudaSuccess && (d->dev < 0 || d->dev >= 64)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess && (d->sms = sms[d->dev].load(std::memory_order_acquire)) == 0) {
    e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->dev);
    if (e == cudaSuccess) sms[d->dev].store(d->sms, std::memory_order_release);
  }
  if (e != cudaSuccess) set_cuda_error(e);
  return e == cudaSuccess;
}

// How many clusters of `splits` CTAs the device holds at once (looked up once
// per device and size; every configuration has the same threads and all but
// the same shared memory).
template <bool kGrouped, bool kGated, int kMats, int kNT, bool kF16, bool kSeg = false>
int gemm16_clusters(int splits, int dev) {
  using C = Gemm16Cfg<kMats, kNT>;
  static std::atomic<int> most[64][4];
  const int i = splits == 8 ? 3 : splits == 4 ? 2 : 1;
  int n = most[dev][i].load(std::memory_order_acquire);
  if (n == 0) {
    auto kern = gemm16_kernel<kGrouped, kGated, kMats, kNT, kF16, kSeg>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)splits);
    cfg.blockDim = dim3(kG16Threads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();  // (not an error of the call: it runs without clusters)
      n = -1;
    }
    most[dev][i].store(n, std::memory_order_release);
  }
  return n < 0 ? 0 : n;
}

template <bool kGrouped, bool kGated, int kMats, int kNT, bool kF16, bool kSeg = false>
moe_status gemm16_launch(Gemm16Args a, int grid, const CUtensorMap &w, const CUtensorMap &x64,
                         const CUtensorMap &x16, int dev, cudaStream_t stream) {
  using C = Gemm16Cfg<kMats, kNT>;
  auto kern = gemm16_kernel<kGrouped, kGated, kMats, kNT, kF16, kSeg>;
  static std::atomic<bool> attr_done[64];  // per device; the attribute call is idempotent
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    attr_done[dev].store(true, std::memory_order_release);
  }
  const int fit = (int)(kG16Ring / (C::kABytes + (uint32_t)a.nt * 128u));
  a.stages = fit < kG16MaxStages ? fit : kG16MaxStages;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kG16Threads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, w, x64, x16);
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace moe
