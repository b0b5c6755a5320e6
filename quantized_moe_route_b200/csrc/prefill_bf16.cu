// prefill_bf16.cu -- grouped expert FFN with bf16 experts: two launches of
// the tensor-core product, h = SiLU(W_gate x) * W_up x and y = W_down h.
#include "gemm16.cuh"

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
  DeviceInfo d;
  if (!device_info(&d)) return MOE_ERR_CUDA;
  Gemm16Args a = {};
  a.err = device_error_word();
  if (!a.err) return MOE_ERR_CUDA;
  CUtensorMap gum, dnm, x64, x16, h64, h16;
  if (!gemm16_map(&gum, layer->gate_up, (int64_t)E * 2 * F, H, H, 128, false) ||
      !gemm16_map(&dnm, layer->down, (int64_t)E * H, F, F, 128, false) ||
      !gemm16_map(&x64, x_perm, rows, H, H, 64, false) || !gemm16_map(&x16, x_perm, rows, H, H, 16, false) ||
      !gemm16_map(&h64, h, rows, F, F, 64, false) || !gemm16_map(&h16, h, rows, F, F, 16, false)) {
    set_cuda_error(cudaErrorInvalidValue);
    return MOE_ERR_CUDA;
  }
  a.offsets = offsets;
  a.E = E;
  a.rows = rows;
  a.nt = 128;
  a.splits = 1;
  a.N = F;
  a.K = H;
  a.w_rows = 2 * F;
  a.mat_off = F;
  a.nfb = (F + 127) / 128;
  // a tile to an SM at most: latency counts, and the rows' own epilogue (16
  // outputs a lane) is the shorter one (8 experts, 37 tokens: 11.7 against 14.9 us)
  auto flip = [&]() { return ((int64_t)E + rows / 128) * a.nfb <= d.sms ? 0 : 32; };
  a.flip = flip();
  a.y = h;
  a.ldy = F;
  a.act = MOE_ACT_SILU;
  moe_status st = gemm16_launch<true, true, 2, 128, false>(a, d.sms, gum, x64, x16, d.dev, s);
  if (st != MOE_OK) return st;
  a.N = H;
  a.K = F;
  a.w_rows = H;
  a.mat_off = 128;
  a.nfb = (H + 255) / 256;
  a.flip = flip();
  a.y = y_perm;
  a.ldy = H;
  a.act = MOE_ACT_NONE;
  return gemm16_launch<true, false, 2, 128, false>(a, d.sms, dnm, h64, h16, d.dev, s);
}
