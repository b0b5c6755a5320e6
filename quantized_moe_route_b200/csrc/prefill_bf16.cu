// prefill_bf16.cu -- grouped expert FFN with bf16 experts.
//
// Two launches, one warp per row and output: h = SiLU(W_gate x) * W_up x,
// then y = W_down h.
#include "w16.cuh"

namespace moe {

__device__ __forceinline__ float pb16_dot(const uint16_t *a, const uint16_t *b, int n) {
  float s = 0.f;
  for (int c = threadIdx.x & 31; c < n; c += 32) s = __fmaf_rn(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c]), s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <bool kGU>
__global__ void __launch_bounds__(256) pb16_kernel(const uint16_t *w, const uint16_t *in, const int32_t *offsets,
                                                   int E, int rows, int K, int N, uint16_t *out) {
  grid_dep_wait();
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = blockIdx.y + blockIdx.z * 65535;
  if (n >= N || r >= rows) return;
  int e = 0;
  while (e < E && !(min(max(offsets[e], 0), rows) <= r && r < min(max(offsets[e + 1], 0), rows))) ++e;
  if (e == E) return;
  const uint16_t *we = w + (size_t)e * (kGU ? 2 : 1) * N * K, *xr = in + (size_t)r * K;
  float v = pb16_dot(xr, we + (size_t)n * K, K);
  if (kGU) v = activate(v, MOE_ACT_SILU) * pb16_dot(xr, we + (size_t)(N + n) * K, K);
  if ((threadIdx.x & 31) == 0) out[(size_t)r * N + n] = f32_to_bf16_bits(v);
}

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_prefill_bf16_workspace_bytes(int rows, int F) {
  if (rows <= 0 || F <= 0) return 0;
  return (size_t)rows * F * 2;
}

extern "C" MOE_API moe_status moe_ffn_grouped_prefill_bf16(const moe_bf16_layer *layer, const uint16_t *x_perm,
                                                           const int32_t *offsets, int rows, uint16_t *y_perm, void *ws,
                                                           size_t ws_bytes, moe_stream_t stream) {
  if (!layer || rows < 0) return MOE_ERR_INVALID_ARG;
  const int E = layer->E, H = layer->H, F = layer->F;
  if (E <= 0 || H <= 0 || F <= 0) return MOE_ERR_INVALID_ARG;
  if (H % 64 || F % 64 || E > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!layer->gate_up || !layer->down || !x_perm || !offsets || !y_perm) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_prefill_bf16_workspace_bytes(rows, F)) return MOE_ERR_WORKSPACE;
  for (const void *p : {(const void *)layer->gate_up, (const void *)layer->down, (const void *)x_perm,
                        (const void *)y_perm, (const void *)ws})
    if (reinterpret_cast<uintptr_t>(p) % 16) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(offsets) % 4) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  uint16_t *h = static_cast<uint16_t *>(ws);
  const unsigned ry = (unsigned)min(rows, 65535), rz = (unsigned)((rows + 65534) / 65535);
  moe_status st = launch_pdl(pb16_kernel<true>, dim3((F + 7) / 8, ry, rz), dim3(256), 0, s, layer->gate_up, x_perm,
                             offsets, E, rows, H, F, h);
  if (st != MOE_OK) return st;
  return launch_pdl(pb16_kernel<false>, dim3((H + 7) / 8, ry, rz), dim3(256), 0, s, layer->down, (const uint16_t *)h,
                    offsets, E, rows, F, H, y_perm);
}
