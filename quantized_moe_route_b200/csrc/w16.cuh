// w16.cuh -- pieces shared by the 16-bit-weight kernels (linear, decode layer
// and grouped FFN with bf16 / f16 weights).
#pragma once
#include "common.cuh"

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
    case MOE_ACT_RELU: return fmaxf(v, 0.0f);
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

}  // namespace moe
