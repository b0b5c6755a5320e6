// linear.cu -- y = act(x w^T + bias) + residual on 16-bit weights.
//
// One warp per output feature (and its gate) and four tokens: the lanes walk
// the rows 32 elements at a time, fp32 FMAs, then a shuffle tree.
#include "w16.cuh"

namespace moe {

struct LinearArgs {
  const uint16_t *x, *w, *bias, *residual;
  void *y;
  int64_t ldx, ldw, ldr, ldy;
  int T, N, K, act, gated, y_f32;
};

template <bool kF16>
__global__ void __launch_bounds__(256) linear_kernel(LinearArgs a) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  for (int64_t t0 = 4 * (int64_t)blockIdx.y; t0 < a.T; t0 += 4 * (int64_t)gridDim.y) {
    float acc[2][4] = {};
    for (int c = lane; c < a.K; c += 32) {
      const float w0 = w16_to_f32<kF16>(a.w[n * a.ldw + c]);
      const float w1 = a.gated ? w16_to_f32<kF16>(a.w[(n + a.N) * a.ldw + c]) : 0.f;
      for (int i = 0; i < 4 && t0 + i < a.T; ++i) {
        const float xv = w16_to_f32<kF16>(a.x[(t0 + i) * a.ldx + c]);
        acc[0][i] = __fmaf_rn(xv, w0, acc[0][i]);
        acc[1][i] = __fmaf_rn(xv, w1, acc[1][i]);
      }
    }
    for (int i = 0; i < 4; ++i)
      for (int m = 0; m < 2; ++m)
        for (int o = 16; o > 0; o >>= 1) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], o);
    for (int i = 0; i < 4 && t0 + i < a.T; ++i) {
      if (lane != i) continue;
      float v = acc[0][i] + (a.bias ? w16_to_f32<kF16>(a.bias[n]) : 0.f);
      v = activate(v, a.act);
      if (a.gated) v *= acc[1][i] + (a.bias ? w16_to_f32<kF16>(a.bias[n + a.N]) : 0.f);
      if (a.residual) v += w16_to_f32<kF16>(a.residual[(t0 + i) * a.ldr + n]);
      if (a.y_f32) static_cast<float *>(a.y)[(t0 + i) * a.ldy + n] = v;
      else static_cast<uint16_t *>(a.y)[(t0 + i) * a.ldy + n] = f32_to_w16<kF16>(v);
    }
  }
}

}  // namespace moe

using namespace moe;

extern "C" MOE_API moe_status moe_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, int T, int N, int K,
                                         int dtype, const void *bias, int act, int gated, const void *residual,
                                         int64_t ldr, void *y, int64_t ldy, int y_dtype, moe_stream_t stream) {
  if (T < 0 || N < 0 || K <= 0 || (dtype != MOE_BF16 && dtype != MOE_F16) || (y_dtype != dtype && y_dtype != MOE_F32) ||
      act < MOE_ACT_NONE || act > MOE_ACT_SIGMOID || gated < 0 || gated > 1)
    return MOE_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return MOE_OK;
  if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldy < N || (residual && ldr < N)) return MOE_ERR_INVALID_ARG;
  const int64_t ld_max = (int64_t)1 << 38;
  if (ldx % 8 || ldw % 8 || ldx > ld_max || ldw > ld_max || ldy > ld_max || (residual && ldr > ld_max) || N > (1 << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t ymask = y_dtype == MOE_F32 ? 3 : 1;
  if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(w) % 16 ||
      (reinterpret_cast<uintptr_t>(y) & ymask) || reinterpret_cast<uintptr_t>(bias) % 2 ||
      reinterpret_cast<uintptr_t>(residual) % 2)
    return MOE_ERR_INVALID_ARG;
  if (residual == y && (y_dtype == MOE_F32 || ldr != ldy)) return MOE_ERR_INVALID_ARG;
  LinearArgs a;
  a.x = static_cast<const uint16_t *>(x);
  a.w = static_cast<const uint16_t *>(w);
  a.bias = static_cast<const uint16_t *>(bias);
  a.residual = static_cast<const uint16_t *>(residual);
  a.y = y;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldr = ldr;
  a.ldy = ldy;
  a.T = T;
  a.N = N;
  a.K = K;
  a.act = act;
  a.gated = gated;
  a.y_f32 = y_dtype == MOE_F32;
  const dim3 grid((unsigned)((N + 7) / 8), (unsigned)min((T + 3) / 4, 65535));
  if (dtype == MOE_F16) return launch_pdl(linear_kernel<true>, grid, dim3(256), 0, as_stream(stream), a);
  return launch_pdl(linear_kernel<false>, grid, dim3(256), 0, as_stream(stream), a);
}
