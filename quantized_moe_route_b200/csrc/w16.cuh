// w16.cuh -- pieces shared by the 16-bit-weight kernels (linear, decode layer
// and grouped FFN with bf16 / f16 weights).
#pragma once
#include <atomic>

#include "tcgen05.cuh"

namespace moe {

__device__ __forceinline__ float sigmoid_f32(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The activations of moe_act in fp32.  __expf and __fdividef are within a few
// fp32 ulps here, far below the rounding of a 16-bit result; 1 + exp(-v)
// overflowing to infinity gives the limit 0.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU: return __fdividef(v, 1.0f + __expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH: {  // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
      const float z2 = 1.5957691216057308f * (v + 0.044715f * v * v * v);
      return __fdividef(v, 1.0f + __expf(-z2));
    }
    case MOE_ACT_RELU: return v < 0.0f ? 0.0f : v;  // (fmaxf would make a NaN 0)
    case MOE_ACT_SIGMOID: return sigmoid_f32(v);
    default: return v;
  }
}

// 16-bit storage types: bf16 and f16 bit patterns
template <bool kF16>
__device__ __forceinline__ float w16_to_f32(uint16_t b) {
  return kF16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}
template <bool kF16>
__device__ __forceinline__ uint16_t f32_to_w16(float f) {
  return kF16 ? __half_as_ushort(__float2half_rn(f)) : f32_to_bf16_bits(f);
}

// D[16x8] (fp32) += A[16x16] (row) * B[16x8] (col), bf16 operands: a pure
// function of its registers, for the compiler to schedule.
__device__ __forceinline__ void mma_bf16_pure(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Instruction descriptor of kind::f16 with bf16 or f16 operands (M = 128, N = n).
__host__ __device__ constexpr uint32_t idesc_16_f32(int n, bool f16) {
  return idesc_bf16_f32(n) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

// Bring a tensor map (a kernel parameter) into the descriptor cache.
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// TMA loads with an L2 cache policy.
__device__ __forceinline__ void tma_load_4d_hint(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                 int c3, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_hint(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                 int c3, int c4, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

}  // namespace moe
