// decode_bf16.cu -- one MoE layer with bf16 experts for up to 16 tokens.
//
// Four launches: the router's logits (one warp per token and expert), the
// routing (one warp per token), h (one warp per routed row and feature), and
// the down projection with the combine (one warp per token and output).
#include "route.cuh"
#include "w16.cuh"

namespace moe {

constexpr size_t kB16CtrlBytes = 4096;

struct DecodeBf16Args {
  const uint16_t *gu, *dn, *x, *wr, *sg, *residual;
  const float *logits;
  float *logits_ws, *w;  // w: routing weights [T][k]
  float *sgate;          // [T] shared gate
  int32_t *idx;          // [T][k]
  float *h;  // [T (k + shared)][F]
  uint16_t *y;
  int T, k, shared, E, H, F;
};

__device__ __forceinline__ float warp_dot(const uint16_t *a, const uint16_t *b, int n) {
  float s = 0.f;
  for (int c = threadIdx.x & 31; c < n; c += 32) s = __fmaf_rn(bf16_bits_to_f32(a[c]), bf16_bits_to_f32(b[c]), s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__global__ void __launch_bounds__(256) db16_logits_kernel(DecodeBf16Args a) {
  grid_dep_wait();
  const int Er = a.E - a.shared, e = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
  if (e > Er || (e < Er && !a.wr) || (e == Er && !a.sg)) return;
  const float v = warp_dot(a.x + (size_t)t * a.H, e < Er ? a.wr + (size_t)e * a.H : a.sg, a.H);
  if ((threadIdx.x & 31) == 0) {
    if (e < Er) a.logits_ws[(size_t)t * Er + e] = v;
    else a.sgate[t] = sigmoid_f32(v);
  }
}

__global__ void __launch_bounds__(256) db16_h_kernel(DecodeBf16Args a) {
  grid_dep_wait();
  const int kk = a.k + a.shared, f = blockIdx.x * 8 + (threadIdx.x >> 5), r = blockIdx.y, t = r / kk, j = r % kk;
  if (f >= a.F) return;
  const int e = j < a.k ? a.idx[t * a.k + j] : a.E - 1;
  const uint16_t *w = a.gu + (size_t)e * 2 * a.F * a.H, *xr = a.x + (size_t)t * a.H;
  const float g = warp_dot(xr, w + (size_t)f * a.H, a.H), u = warp_dot(xr, w + (size_t)(a.F + f) * a.H, a.H);
  if ((threadIdx.x & 31) == 0) a.h[(size_t)r * a.F + f] = activate(g, MOE_ACT_SILU) * u;
}

__global__ void __launch_bounds__(256) db16_y_kernel(DecodeBf16Args a) {
  grid_dep_wait();
  const int kk = a.k + a.shared, c = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
  if (c >= a.H) return;
  float acc = 0.f;
  for (int j = 0; j < kk; ++j) {
    const int e = j < a.k ? a.idx[t * a.k + j] : a.E - 1;
    const float *h = a.h + ((size_t)t * kk + j) * a.F;
    const uint16_t *d = a.dn + ((size_t)e * a.H + c) * a.F;
    float v = 0.f;
    for (int f = threadIdx.x & 31; f < a.F; f += 32) v = __fmaf_rn(h[f], bf16_bits_to_f32(d[f]), v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    acc += (j < a.k ? a.w[t * a.k + j] : a.sg ? a.sgate[t] : 1.0f) * v;
  }
  if (a.residual) acc += bf16_bits_to_f32(a.residual[(size_t)t * a.H + c]);
  if ((threadIdx.x & 31) == 0) a.y[(size_t)t * a.H + c] = f32_to_bf16_bits(acc);
}

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_decode_layer_bf16_workspace_bytes(int T, int k, int shared, int E, int H, int F) {
  if (T <= 0 || k <= 0 || shared < 0 || shared > 1 || E <= shared || H <= 0 || F <= 0) return 0;
  // control words, h words of every routed row, logit words of every expert
  return kB16CtrlBytes + sizeof(unsigned long long) * ((size_t)T * (k + shared) * F + (size_t)T * E);
}

extern "C" MOE_API moe_status moe_decode_layer_bf16(const moe_bf16_layer *layer, const uint16_t *x, const uint16_t *wr,
                                                    float *logits, int T, int k, int shared,
                                                    const uint16_t *shared_gate, const uint16_t *residual, uint16_t *y,
                                                    int32_t *idx, float *w, void *ws, size_t ws_bytes,
                                                    moe_stream_t stream) {
  if (!layer || T < 0 || k <= 0 || shared < 0 || shared > 1) return MOE_ERR_INVALID_ARG;
  const int E = layer->E, H = layer->H, F = layer->F, kk = k + shared, Er = E - shared;
  if (Er <= 0 || H <= 0 || F <= 0 || k > Er || (shared_gate && !shared)) return MOE_ERR_INVALID_ARG;
  if (H % 64 || F % 64 || E > 1024 || T > 16 || T * kk > 256 || kk > 32) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!layer->gate_up || !layer->down || !x || (!wr && !logits) || !y) return MOE_ERR_INVALID_ARG;
  if ((idx == nullptr) != (w == nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)layer->gate_up, (const void *)layer->down, (const void *)x, (const void *)wr,
                        (const void *)shared_gate, (const void *)residual, (const void *)y, (const void *)ws})
    if (reinterpret_cast<uintptr_t>(p) % 16) return MOE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)logits, (const void *)idx, (const void *)w})
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_decode_layer_bf16_workspace_bytes(T, k, shared, E, H, F)) return MOE_ERR_WORKSPACE;
  uint8_t *base = static_cast<uint8_t *>(ws) + kB16CtrlBytes;
  DecodeBf16Args a;
  a.gu = layer->gate_up;
  a.dn = layer->down;
  a.x = x;
  a.wr = wr;
  a.sg = shared_gate;
  a.residual = residual;
  a.h = reinterpret_cast<float *>(base);
  a.logits_ws = wr && logits ? logits : reinterpret_cast<float *>(base + sizeof(uint64_t) * (size_t)T * kk * F);
  a.logits = wr ? a.logits_ws : logits;
  a.y = y;
  // routing outputs and the shared gate: in the control words when not asked for
  a.idx = idx ? idx : static_cast<int32_t *>(ws);
  a.w = w ? w : static_cast<float *>(ws) + 256;
  a.sgate = static_cast<float *>(ws) + 512;
  a.T = T;
  a.k = k;
  a.shared = shared;
  a.E = E;
  a.H = H;
  a.F = F;
  cudaStream_t s = as_stream(stream);
  moe_status st = MOE_OK;
  if (wr || shared_gate) st = launch_pdl(db16_logits_kernel, dim3(Er / 8 + 1, T), dim3(256), 0, s, a);
  if (st == MOE_OK) st = route_rows(a.logits, T, Er, k, a.idx, a.w, s);
  if (st == MOE_OK) st = launch_pdl(db16_h_kernel, dim3(F / 8, T * kk), dim3(256), 0, s, a);
  if (st == MOE_OK) st = launch_pdl(db16_y_kernel, dim3(H / 8, T), dim3(256), 0, s, a);
  return st;
}
