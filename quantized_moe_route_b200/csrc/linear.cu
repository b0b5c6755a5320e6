// linear.cu -- y = act(x w^T + bias) + residual on 16-bit weights: few rows of
// x as a weight stream, more on the 5th-generation tensor cores.
#include "gemm16.cuh"
#include "gemm16_pair.cuh"
#include "linear_stream.cuh"

namespace moe {

// Rows of x up to which a linear is a weight stream: 16; and 32 where each SM
// has one strip of outputs and K >= 512, so that x is loaded once (2048 x 2048,
// 32 rows: 5.3 us against 6.6 on the tensor-core tiles, 2048 x 8192 10.3 / 13.6;
// 8192 x 2048 15.1 / 10.5, 1000 x 100 5.8 / 3.9).
inline bool linear_streams(int T, int N, int K, bool gated, int sms) {
  return T <= 16 || (T <= 32 && K >= 512 && N <= (gated ? 8 : 16) * sms);
}

template <bool kGated, bool kF16>
static moe_status linear_stream(const Gemm16Args &g, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                const DeviceInfo &d, cudaStream_t s) {
  // equal strips: as few to an SM as 16 rows each allow, of as few rows as that takes
  const int most = kGated ? 8 : 16;
  const int per_sm = (g.N + most * d.sms - 1) / (most * d.sms), per = (g.N + per_sm * d.sms - 1) / (per_sm * d.sms);
  LinearStreamArgs a;
  a.g = g;
  a.R = kGated ? 2 * per : per;
  a.strips = (g.N + per - 1) / per;
  a.group_log2 = g.K > 512 ? 3 : g.K > 256 ? 2 : 1;  // a pair of 64-input columns a warp at least
  a.whole = g.K % 64 == 0;
  CUtensorMap wm, xm;
  const int nb = g.rows > 16 ? 4 : g.rows > 8 ? 2 : 1;
  const int64_t wrows = (int64_t)g.N * (kGated ? 2 : 1);
  const int xrows = 8 * nb;
  if (!(a.whole ? gemm16_map3(&wm, w, wrows, g.K, ldw, per, kLsCols, kF16) && gemm16_map3(&xm, x, g.rows, g.K, ldx, xrows, kLsCols, kF16)
                : gemm16_map(&wm, w, wrows, g.K, ldw, per, kF16) && gemm16_map(&xm, x, g.rows, g.K, ldx, xrows, kF16))) {
    set_cuda_error(cudaErrorInvalidValue);
    return MOE_ERR_CUDA;
  }
  const int grid = a.strips < d.sms ? a.strips : d.sms;
  return nb == 4   ? linear_stream_launch<kGated, kF16, 4>(a, grid, wm, xm, d.dev, s)
         : nb == 2 ? linear_stream_launch<kGated, kF16, 2>(a, grid, wm, xm, d.dev, s)
                   : linear_stream_launch<kGated, kF16, 1>(a, grid, wm, xm, d.dev, s);
}

// The rows of a tile and the CTAs that share its K: the least of a model of
// the time in us, fitted to a sweep of both over N 512 to 8192, K 512 to 8192
// and T 32 to 1024 (within 10 % of the sweep's best at most sizes).  A CTA
// loads 94 KB/us, a k block's products take 0.16 us a block of weights (0.26
// above 128 rows), joining a cluster's partials 0.4 us and 8 ns a row, and an
// epilogue that nothing overlaps 5 ns a row.  (2048 x 2048, 256 rows: one chunk
// over 8 CTAs 20.3 us, two over 4 each 8.8, eight whole ones 11.6.)
template <bool kGated, int kMats, int kNT, bool kF16, bool kSeg>
static void gemm16_plan(Gemm16Args &a, const DeviceInfo &d) {
  const int KB = (a.K + kG16BK - 1) / kG16BK;
  const int most = gemm16_clusters<false, kGated, kMats, kNT, kF16, kSeg>(8, d.dev) * 8 >= 64 ? 8 : 4;
  float best = 1e30f;
  for (int nt = min(kNT, (a.rows + 15) / 16 * 16); nt >= 16; nt -= 16) {
    const int chunks = (a.rows + nt - 1) / nt;
    if (chunks > 1 && nt > ((a.rows + chunks - 1) / chunks + 15) / 16 * 16) continue;  // a smaller nt has as few chunks
    const int64_t tiles = (int64_t)a.nfb * chunks;
    for (int S = 1; S <= most && (S == 1 || S * 2 <= KB); S *= 2) {
      if (S > 1 && tiles > gemm16_clusters<false, kGated, kMats, kNT, kF16, kSeg>(S, d.dev)) break;
      const float kb = (float)((KB + S - 1) / S);
      const float load = kb * (128 * kMats + nt) * (128.f / 94e3f), mma = kb * kMats * (nt > 128 ? 0.26f : 0.16f);
      const int64_t waves = (tiles * S + d.sms - 1) / d.sms;
      float t = (float)waves * (load > mma ? load : mma) +
                      (S > 1 ? 0.4f + 0.008f * nt * kMats : 0.005f * nt * kMats);
      if (kSeg && nt > 128 / kMats) t *= 1.12f;  // more sums than the registers hold
      if (t < best) best = t, a.nt = nt, a.splits = S;
    }
    if (tiles > 4 * d.sms) break;  // finer tiles only add waves
  }
}

template <bool kGated, bool kF16, bool kSegments>
static moe_status linear_gemm(Gemm16Args &a, const void *x, int64_t ldx, const void *w, int64_t ldw, const DeviceInfo &d,
                              cudaStream_t s) {
  // gated: gate and up of 128 features and 128 rows a tile; else 128 outputs and 256 rows
  // (in segments the sums stand in the epilogue's registers: three quarters of the rows)
  constexpr int kMats = kGated ? 2 : 1, kNT = (kSegments ? 192 : 256) / kMats;
  CUtensorMap wm, x64, x16;
  if (!gemm16_map(&wm, w, (int64_t)a.N * (kGated ? 2 : 1), a.K, ldw, 128, kF16) ||
      !gemm16_map(&x64, x, a.rows, a.K, ldx, 64, kF16) || !gemm16_map(&x16, x, a.rows, a.K, ldx, 16, kF16)) {
    set_cuda_error(cudaErrorInvalidValue);
    return MOE_ERR_CUDA;
  }
  // Tiles of 128 rows and two weight blocks (256 outputs, or gate and up of 128)
  // for most SMs: the rows go on M, and a lane of the epilogue holds 16 outputs
  // of a row, one vector, where the other way round it has one output of 16
  // rows.  (2048 x 2048, 2048 rows = 128 tiles: 16.6 us against 21.5; 1280 rows =
  // 80 tiles: 16.6 / 15.7; gated, 640 rows = 80 tiles: 16.7 / 17.8.)
  // Rows of y and of the residual that are no whole vectors would be 16 accesses
  // of 2 bytes a lane, each in a row of its own; with the weights on M they are 32
  // consecutive outputs of a row.  (5001 x 2048, 2048 rows with bias, GELU and
  // residual: 145 us with the rows on M, 53.5 with the weights; 5000: 52.6 / 53.5.)
  const bool vectors = a.ldy % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                       (!a.residual || (a.ldr % 8 == 0 && reinterpret_cast<uintptr_t>(a.residual) % 16 == 0));
  const int nfb = (a.N + (kGated ? 127 : 255)) / (kGated ? 128 : 256);
  const int64_t tiles1 = (int64_t)nfb * ((a.rows + 127) / 128), tiles2 = (int64_t)nfb * ((a.rows + 255) / 256);
  if (!kSegments && vectors && tiles1 >= (kGated ? d.sms / 2 : 3 * d.sms / 4)) {
    a.mat_off = kGated ? a.N : 128;
    a.nfb = nfb;
    a.nt = 128;
    a.splits = 1;
    a.flip = 0;
    // Pairs of SMs where there is a tile for every pair, no more rounds of them,
    // and K is long enough to pay for the pairing: 8192 rows of 2048 x 8192 with
    // bias, GELU and residual 248 us against 270 one after another (plain 207 /
    // 240); 2048 x 512, 4096 rows 14.7 / 14.1.
    const int pairs = d.sms / 2;
    if (a.K >= 1024 && tiles2 >= pairs && (tiles2 + pairs - 1) / pairs <= (tiles1 + d.sms - 1) / d.sms)
      return gemm16_pair_launch<kGated, kF16>(a, pairs, wm, x64, x16, d.dev, s);
    return gemm16_launch<false, kGated, 2, 128, kF16>(a, (int)(tiles1 < d.sms ? tiles1 : d.sms), wm, x64, x16, d.dev, s);
  }
  a.mat_off = a.N;
  a.nfb = (a.N + 127) / 128;
  a.flip = 128;
  gemm16_plan<kGated, kMats, kNT, kF16, kSegments>(a, d);
  const int64_t tiles = (int64_t)a.nfb * ((a.rows + a.nt - 1) / a.nt);
  const int grid = a.splits > 1 ? (int)tiles * a.splits : (int)(tiles < d.sms ? tiles : d.sms);
  if constexpr (kSegments) {
    // up to two thirds of the rows: fewer sums in registers (5 % faster there; of
    // these kernels only the gated one spills, 28 bytes a thread)
    constexpr int kFew = 128 / kMats;
    if (a.nt <= kFew) return gemm16_launch<false, kGated, kMats, kFew, kF16, true>(a, grid, wm, x64, x16, d.dev, s);
  }
  return gemm16_launch<false, kGated, kMats, kNT, kF16, kSegments>(a, grid, wm, x64, x16, d.dev, s);
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
  if (ldx % 8 || ldw % 8 || ldx > ld_max || ldw > ld_max || ldy > ld_max || (residual && ldr > ld_max) || N > (1 << 29) || T > (1 << 30) || K > (1 << 30))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t ymask = y_dtype == MOE_F32 ? 3 : 1;
  if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(w) % 16 ||
      (reinterpret_cast<uintptr_t>(y) & ymask) || reinterpret_cast<uintptr_t>(bias) % 2 ||
      reinterpret_cast<uintptr_t>(residual) % 2)
    return MOE_ERR_INVALID_ARG;
  if (y == x || y == w || y == bias || (residual == y && (y_dtype == MOE_F32 || ldr != ldy))) return MOE_ERR_INVALID_ARG;
  Gemm16Args a = {};
  a.E = 1;
  a.rows = T;
  a.N = N;
  a.K = K;
  a.bias = static_cast<const uint16_t *>(bias);
  a.residual = static_cast<const uint16_t *>(residual);
  a.y = y;
  a.ldr = ldr;
  a.ldy = ldy;
  a.act = act;
  a.y_f32 = y_dtype == MOE_F32;
  a.err = device_error_word();
  if (!a.err) return MOE_ERR_CUDA;
  cudaStream_t s = as_stream(stream);
  DeviceInfo d;
  if (!device_info(&d)) return MOE_ERR_CUDA;
  // Sums in segments where the tensor core's truncating additions would show:
  // they leave a sum 6e-9 K too small (K = 32768: 1.9e-4, two fifths of half a
  // step of f16; K = 2^18: 1.6e-3, two fifths of half a step of bf16).  It costs
  // time only where rows are many (f16, 2048 x 40960: 2048 rows 273 -> 374 us, 300
  // rows 71 -> 73, 40 rows 46.3 -> 46.8).
  const bool segments = a.y_f32 || K > (dtype == MOE_F16 ? 1 << 15 : 1 << 18);
  const bool f16 = dtype == MOE_F16, stream_w = linear_streams(T, N, K, gated, d.sms);
#define MOE_LINEAR(GATED, F16)                                                        \
  (stream_w    ? linear_stream<GATED, F16>(a, x, ldx, w, ldw, d, s)                   \
   : segments  ? linear_gemm<GATED, F16, true>(a, x, ldx, w, ldw, d, s)               \
               : linear_gemm<GATED, F16, false>(a, x, ldx, w, ldw, d, s))
  if (f16) return gated ? MOE_LINEAR(true, true) : MOE_LINEAR(false, true);
  return gated ? MOE_LINEAR(true, false) : MOE_LINEAR(false, false);
#undef MOE_LINEAR
}
