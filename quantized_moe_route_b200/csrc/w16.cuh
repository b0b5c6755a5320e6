// w16.cuh -- pieces shared by the 16-bit-weight kernels (linear, decode layer
// and grouped FFN with bf16 / f16 weights).
#pragma once
#include <atomic>

#include "tcgen05.cuh"

namespace moe {

__device__ __forceinline__ float sigmoid_f32(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The activations of moe_act in fp32, NaN for NaN.
// kExact, for fp32 results: expf (1 ulp).  Otherwise, for results of at most 16
// bits: __expf (2 + 1.2 |z| ulps at z): 2^-19 of the value at |v| = 10, 2^-16.7 at
// 60, where half a step of f16 is 2^-11.  Divisions are __fdividef (2 ulps; 0 for
// a quotient by 2^126 and more, so magnitudes below 10^-36 become 0; with IEEE
// division an fp32 SiLU of 2048 x 5000 takes 100 us for 94).
// GELU is v times the normal distribution's Phi, and the lower tail is computed
// for itself, Phi(-a) = exp(-a^2 / 2) t P(t), t = 1 / (1 + 0.32 a): a relative
// error of 2^-20.3 for every a >= 0 (P of degree 7 is this file's own minimax fit
// of exp(a^2 / 2) Phi(-a) / t over 0 <= a <= 40, where (1 + erff) / 2 is 6 %
// off at a = 5).  In both GELUs the rounded argument of exp adds its own
// magnitude in ulps: 2^-17 at v = -9.
template <bool kExact = false>
__device__ __forceinline__ float activate(float v, int act) {
  auto exp_of = [](float z) { return kExact ? expf(z) : __expf(z); };
  switch (act) {
    case MOE_ACT_SILU: return __fdividef(v, 1.0f + exp_of(-v));
    case MOE_ACT_GELU: {
      const float t = __fdividef(1.0f, 1.0f + 0.32f * fabsf(v));
      float q = fmaf(0.0345206335f, t, -0.1224306f);
      q = fmaf(q, t, 0.106114104f);
      q = fmaf(q, t, 0.0155905411f);
      q = fmaf(q, t, 0.097373195f);
      q = fmaf(q, t, 0.113439046f);
      q = fmaf(q, t, 0.127733395f);
      q = fmaf(q, t, 0.127659902f);
      const float tail = exp_of(-0.5f * v * v) * (t * q);
      return v * (v < 0.0f ? tail : 1.0f - tail);
    }
    case MOE_ACT_GELU_TANH:  // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
      return __fdividef(v, 1.0f + exp_of(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_RELU: return v < 0.0f ? 0.0f : v;  // (fmaxf would make a NaN 0)
    case MOE_ACT_SIGMOID: return __fdividef(1.0f, 1.0f + exp_of(-v));
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
