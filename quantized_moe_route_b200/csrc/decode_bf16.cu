// decode_bf16.cu -- one MoE layer with bf16 experts for up to 16 tokens, in
// one launch: the router, the routing, every selected expert's gate/up,
// SwiGLU and down projection, the shared expert, the combine and the
// residual.
//
// A decode step reads each selected expert's weights once (6 H F bytes) and
// does little else, so the kernel is a stream: a persistent grid, one CTA per
// SM, whose producer thread brings weight tiles by TMA through a ring of 16 KB
// stages, and 15 consumer warps that each take whole units of work from it, so
// no barrier between warps sits on the stream.  (One TMA box per 16 KB streams
// 7.1 TB/s over 148 CTAs with nothing else to do; the same bytes as 16 row
// copies of 1 KB reach 2.8 TB/s, as four of 4 KB 4.5 TB/s.)
//   phase A  unit = 4 or 8 features of one expert (their gate and up rows, all
//            H inputs).  Units go round the CTAs; h is published as 16-byte
//            words {four values of 24 bits, call epoch}, stored and loaded as one
//            .b128 each (single-copy atomic: a reader polls the words
//            themselves, no fence or counter on the path).  Every CTA of phase B
//            reads all of h, so its bytes count: with 8-byte words {bf16 pair,
//            epoch}, twice as many, 16 tokens take 128 us for 124, 4 tokens 45 / 42,
//            one 20.1 / 19.9.
//   phase B  a CTA owns R output channels (H / CTAs, at most 16) and runs
//            every selected expert's rows of them, a warp per expert, four
//            tokens and 512 inputs (a busier expert's tile is loaded again, from L2): all k
//            rows of a token meet in the CTA's shared memory, so the combine
//            needs no second handoff.  The producer runs ahead: these weights
//            do not depend on h and are loaded while h is still on its way.
// Dot products run on m16n8k16 tensor-core instructions with the weight rows
// as A and the tokens as B.  A sum over k may take k in any order, so lane
// (g, t) reads the 16-byte pieces 2t and 2t + 1 of its row's 64 inputs and uses
// each as the fragments of two instructions.  Weight rows arrive in the
// 128-byte swizzle (piece p of row r at p ^ (r mod 8)) and token rows lie 16
// bytes (mod 128) apart, so in both the eight lanes of a 16-byte read touch
// every bank once.  The down projection takes h as a pair of bf16 values (hi +
// lo, 16 significant bits) in two token columns of the same instruction, which
// costs nothing with at most four tokens to a job.
//
// The router's logits are computed over the grid (each CTA its experts' rows,
// K split over the warps, partial sums added in warp order), published as
// words {logit, epoch}, and every CTA routes for itself.  Every CTA is
// resident (cooperative launch) and every wait is bounded.
#include <atomic>

#include "decode_common.cuh"
#include "decode_items.cuh"
#include "route.cuh"
#include "w16.cuh"

namespace moe {

constexpr int kB16All = 16;                           // warps: 15 consumers and the producer
constexpr int kB16Warps = kB16All - 1;                // (a 17th warp would cost every thread 32 registers)
constexpr int kB16Threads = kB16All * 32;
constexpr int kB16KC = 512;                           // inputs of a 16-row stage (an 8-row stage: twice that)
constexpr uint32_t kB16Stage = 16 * kB16KC * 2;       // bytes of a stage
constexpr int kB16MaxStages = 8;                      // a power of two, like every smaller ring
constexpr int kB16JobTok = 4;                         // tokens of a phase B job
constexpr int kB16MaxF = 1 << 20;
constexpr int kB16MaxX = 166000;                      // bytes of x rows that fit beside two stages
constexpr size_t kB16CtrlBytes = 4096;                // workspace head: epoch, done counter
// The logit words lie between the head and h, at one place whatever the call's sizes: both kinds of words keep
// their epoch where a call of other sizes would look for one.
constexpr size_t kB16LogitBytes = 16 * 1025 * 8;
constexpr uint32_t kB16Polls = 1u << 22;              // bound of a poll loop (of >= 32 ns sleeps)
constexpr uint32_t kB16BarPolls = 1u << 19;           // bound of a barrier wait (polls suspend for some us)

struct DecodeBf16Args {
  const uint16_t *gu, *dn, *x, *wr, *sg, *residual;
  float *logits;             // [T][Er]: the input, or with wr an optional output
  ulonglong2 *hbuf;          // [T kk][F / 4] words {epoch, upper 16 bits of four values of h, their next 8 bits each}
  unsigned long long *lbuf;  // [T][Er + 1] words {fp32 logit, epoch}; entry Er: the shared expert's gate
  unsigned int *ctrl;        // [0] last epoch, [1] CTAs done
  uint16_t *y;
  int32_t *idx;
  float *w;
  int *err;
  int T, kk, shared, E, H, F;  // kk: rows per token (k + shared)
  uint32_t h_polls;            // bound of phase B's wait for h (polls of about 1 us)
  int starve;                  // test hook: phase A publishes no h
  int nst_log2;                // ring stages
  int R;                       // output channels of a phase B strip (at most 16)
  uint32_t hb_bytes;           // per-warp h buffer
  int shared_xh;               // the h buffers take x's place after phase A (both do not fit)
};

struct B16Smem {
  uint32_t x, h, rows, tables, total;  // byte offsets; the ring is at 0
};
__host__ __device__ inline uint32_t b16_hb_bytes(int T) {  // 512 h values (hi and lo) of a token or two, 256 of four
  return T == 1 ? 2080u : 4224u;
}
__host__ __device__ inline B16Smem b16_layout(int T, int kk, int H, int nst, int shared_xh) {
  B16Smem L;
  L.x = (uint32_t)nst * kB16Stage;
  const uint32_t xb = (uint32_t)T * (uint32_t)(H * 2 + 16), hb = kB16Warps * b16_hb_bytes(T);
  L.h = shared_xh ? L.x : L.x + xb;  // x in phase A, the warps' h in phase B
  L.rows = L.x + (shared_xh ? (xb > hb ? xb : hb) : xb + hb);
  L.tables = L.rows + (uint32_t)(T * kk) * 64u;
  L.total = L.tables + 32 * 4 + 256 * 4 + 256 * 16 + 256 * 4 + 256 * 4 + 256 * 4 + 320 * 2 + 320 * 4 + 2 * 8 * kB16MaxStages + 64 + 1024 /* alignment of the ring */;
  return L;
}

__device__ __forceinline__ void b16_consumer_sync() { asm volatile("bar.sync 1, 480;" ::: "memory"); }
__device__ __forceinline__ void st_relaxed_u64(unsigned long long *p, unsigned long long v) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void st_relaxed_b128(ulonglong2 *p, unsigned long long a, unsigned long long b) {
  asm volatile("{\n\t.reg .b128 t;\n\tmov.b128 t, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], t;\n\t}" ::"l"(p), "l"(a),
               "l"(b)
               : "memory");
}
__device__ __forceinline__ void ld_relaxed_b128(const ulonglong2 *p, ulonglong2 &v) {
  asm volatile("{\n\t.reg .b128 t;\n\tld.relaxed.gpu.global.b128 t, [%2];\n\tmov.b128 {%0, %1}, t;\n\t}"
               : "=l"(v.x), "=l"(v.y)
               : "l"(p)
               : "memory");
}
// What 24 bits of a value leave beside its upper 16: hi, the value's upper half in
// place, next, the next 8 bits in byte `at` of r.  An infinity, less the largest
// finite value, leaves itself: its products then are as infinite as the upper
// half's and of their sign, so no sum of the two halves is inf - inf.
__device__ __forceinline__ float b16_rest(uint32_t hi, uint32_t r, int at) {
  const float most = 3.4028234663852886e38f, finite = fmaxf(fminf(__uint_as_float(hi), most), -most);
  return __uint_as_float(__byte_perm(hi, r, 0x3200 | (4 + at) << 4)) - finite;
}
// the n-th set bit of m (n < popc(m))
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (int i = 0; i < n; ++i) m &= m - 1u;
  return __ffs(m) - 1;
}

// kRows: weight rows of a phase A unit, half gate and half up.  8 serves up to
// 4 tokens: the finer units balance the little work there is, and the idle
// halves of the instruction (rows 8-15, token columns 4-7) take the second
// half of the unit's inputs, so that one instruction does the work of two.
// PER: logits per lane in the routing.
template <int kRows, int PER>
__global__ void __launch_bounds__(kB16Threads, 1)
    decode_bf16_kernel(DecodeBf16Args a, const __grid_constant__ CUtensorMap gu_map,
                       const __grid_constant__ CUtensorMap dn_map) {
  constexpr int NB = kRows == 16 ? 2 : 1;        // token blocks of 8
  constexpr bool kJobs = kRows == 16;            // phase B jobs are groups of an expert's tokens
  constexpr int FPU = kRows / 2;                 // features of a unit
  constexpr int KCA = kRows == 16 ? kB16KC : 2 * kB16KC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (keeps the address space known)
  const B16Smem L = b16_layout(a.T, a.kk, a.H, 1 << a.nst_log2, a.shared_xh);
  float *rowbuf = reinterpret_cast<float *>(smem + L.rows);            // [T kk][16]
  uint32_t *emask = reinterpret_cast<uint32_t *>(smem + L.tables);     // [32] expert presence bits
  uint32_t *tokmask = emask + 32;                                      // [256] tokens of a slot
  uint8_t *slot_j = reinterpret_cast<uint8_t *>(tokmask + 256);        // [256][16] row of (slot, token) within the token
  int *slot_expert = reinterpret_cast<int *>(slot_j + 256 * 16);       // [256]
  int *ridx = slot_expert + 256;                                       // [256] expert of a row
  float *rw = reinterpret_cast<float *>(ridx + 256);                   // [256] weight of a row
  uint16_t *jobs = reinterpret_cast<uint16_t *>(rw + 256);             // [320] phase B: slot + 256 * group of tokens
  volatile int *joined = reinterpret_cast<volatile int *>(jobs + 320);   // [320] phase B: chunks of a job in rowbuf, over all strips
  uint64_t *full = reinterpret_cast<uint64_t *>(jobs + 320 + 640);
  uint64_t *empty = full + kB16MaxStages;
  volatile int *misc = reinterpret_cast<volatile int *>(empty + kB16MaxStages);  // [0] abort, [1] epoch, [2] stages issued, [3] jobs listed, [4] jobs

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int T = a.T, kk = a.kk, H = a.H, F = a.F, Er = a.E - a.shared, G = gridDim.x, nst = 1 << a.nst_log2;
  const uint32_t xpitch = (uint32_t)(H * 2 + 16);

  if (tid == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    misc[0] = 0;
    misc[2] = 0;
    misc[3] = 0;
    fence_mbar_init();
    tma_prefetch_map(&gu_map);
    tma_prefetch_map(&dn_map);
  }
  if (tid < 32) emask[tid] = 0u;
  if (tid < 256) tokmask[tid] = 0u;
  if (tid < 320) joined[tid] = 0;
  pdl_wait();
  if (tid == kB16Threads - 1) {
    const unsigned int ep = a.ctrl[0] + 1u;  // this call's epoch; never 0 (zeroed words never match)
    misc[1] = (int)(ep == 0u ? 1u : ep);
  }
  auto fail = [&](int code) {
    atomicExch(a.err, code);
    misc[0] = 1;
  };

  // ---- router: rows blockIdx.x + G i of {wr, shared gate}, 16 at a time
  const bool have_rows = a.wr != nullptr || a.sg != nullptr;
  if (have_rows) {
    const int lo = a.wr ? 0 : Er, hi = a.sg ? Er + 1 : Er;  // experts' rows, then the gate's
    float *part = reinterpret_cast<float *>(smem);          // the ring is idle: [16 warps][16 rows][16 tokens]
    for (int e0 = lo + (int)blockIdx.x; e0 < hi; e0 += 16 * G) {
      const uint16_t *r0 = nullptr, *r1 = nullptr;  // this lane's rows g and g + 8
      const int ea = e0 + g * G, eb = e0 + (g + 8) * G;
      if (ea < hi) r0 = ea < Er ? a.wr + (size_t)ea * H : a.sg;
      if (eb < hi) r1 = eb < Er ? a.wr + (size_t)eb * H : a.sg;
      float d[2][4] = {};
      const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 4
      for (int b = warp; b < H / 32; b += kB16All) {
        const int c = 32 * b + 8 * t4;
        const uint4 w0 = r0 ? *reinterpret_cast<const uint4 *>(r0 + c) : z;
        const uint4 w1 = r1 ? *reinterpret_cast<const uint4 *>(r1 + c) : z;
        const uint4 q0 = g < T ? *reinterpret_cast<const uint4 *>(a.x + (size_t)g * H + c) : z;
        const uint4 q1 = g + 8 < T ? *reinterpret_cast<const uint4 *>(a.x + (size_t)(g + 8) * H + c) : z;
        const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
        mma_bf16_pure(d[0], f0, q0.x, q0.y);
        mma_bf16_pure(d[0], f1, q0.z, q0.w);
        if (NB == 2) {
          mma_bf16_pure(d[1], f0, q1.x, q1.y);
          mma_bf16_pure(d[1], f1, q1.z, q1.w);
        }
      }
      float *p = part + warp * 256;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n = nb * 8 + 2 * t4;
        p[g * 16 + n] = d[nb][0];
        p[g * 16 + n + 1] = d[nb][1];
        p[(g + 8) * 16 + n] = d[nb][2];
        p[(g + 8) * 16 + n + 1] = d[nb][3];
      }
      __syncthreads();
      if (tid < 256) {
        const int r = tid >> 4, t = tid & 15, e = e0 + r * G;
        if (t < T && e < hi) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kB16All; ++w) v += part[w * 256 + tid];
          st_relaxed_u64(a.lbuf + (size_t)t * (Er + 1) + e,
                         ((unsigned long long)__float_as_uint(v) << 32) | (unsigned int)misc[1]);
          if (e < Er && a.logits) a.logits[(size_t)t * Er + e] = v;
          __threadfence();  // every CTA polls these words: push them out now
        }
      }
      __syncthreads();
    }
    fence_proxy_async_smem();  // the ring's next writers are the weight copies
  }
  if (warp < T) {  // token `warp` of x; awaited after the routing
    const uint16_t *src = a.x + (size_t)warp * H;
    for (int c = lane; c < H / 8; c += 32) cp_async_16(smem + L.x + (size_t)warp * xpitch + 16 * c, src + 8 * c);
    cp_async_commit();
  }
  __syncthreads();  // barrier initialisation, table clears, the epoch
  const unsigned int epoch = (unsigned int)misc[1];

  // ---- routing: warp t routes token t
  if (warp < T) {
    const int k = kk - a.shared;
    const unsigned long long *lw = a.lbuf + (size_t)warp * (Er + 1);
    uint32_t key[PER];
    if (a.wr) {
      unsigned long long wv[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) wv[i] = lane + 32 * i < Er ? ld_relaxed_u64(lw + lane + 32 * i) : 0ull;
      uint32_t spins = 0;
      while (true) {  // reload all of the lane's words still from an earlier call
        uint32_t pending = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (lane + 32 * i < Er && (unsigned int)wv[i] != epoch) pending |= 1u << i;
        if (!pending) break;
        if (++spins > kB16Polls) {
          fail(DEVERR_DECODE_ROUTER_WAIT);
          break;
        }
        __nanosleep(32);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if ((pending >> i) & 1u) wv[i] = ld_relaxed_u64(lw + lane + 32 * i);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = lane + 32 * i < Er ? route_key(__uint_as_float((unsigned int)(wv[i] >> 32))) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = lane + 32 * i < Er ? route_key(a.logits[(size_t)warp * Er + lane + 32 * i]) : 0u;
    }
    int j_idx;
    float j_w;
    route_token_keys<PER>(key, k, &j_idx, &j_w);
    j_idx = min(max(j_idx, 0), Er - 1);  // (NaN logits are outside the contract; stay memory safe)
    if (lane < k && blockIdx.x == 0 && a.idx) {
      a.idx[warp * k + lane] = j_idx;
      a.w[warp * k + lane] = j_w;
    }
    if (a.shared && lane == k) {
      j_idx = Er;
      j_w = 1.0f;
      if (a.sg) {
        unsigned long long v = ld_relaxed_u64(lw + Er);
        for (uint32_t spins = 0; (unsigned int)v != epoch; v = ld_relaxed_u64(lw + Er)) {
          if (++spins > kB16Polls) {
            fail(DEVERR_DECODE_ROUTER_WAIT);
            break;
          }
          __nanosleep(32);
        }
        j_w = sigmoid_f32(__uint_as_float((unsigned int)(v >> 32)));
      }
    }
    if (lane < kk) {
      ridx[warp * kk + lane] = j_idx;
      rw[warp * kk + lane] = j_w;
      atomicOr(&emask[j_idx >> 5], 1u << (j_idx & 31));
    }
  }
  cp_async_wait_all();  // this thread's part of x
  __syncthreads();
  pdl_launch_dependents();
  // slots: the selected experts in increasing id; every warp scans the presence words for itself
  const uint32_t em = emask[lane];
  const int incl = warp_inclusive_scan(__popc(em)), ebase = incl - __popc(em);
  const int U = __shfl_sync(0xffffffffu, incl, 31);
  const int UA = F / FPU, nUnits = U * UA;
  const int myUnits = (int)blockIdx.x < nUnits ? (nUnits - 1 - (int)blockIdx.x) / G + 1 : 0;
  const int CA = (H + KCA - 1) / KCA, CB = (F + kB16KC - 1) / kB16KC;
  const int nA = myUnits * CA;  // stages of phase A
  const int R = a.R;
  const int nStrips = (H + R - 1) / R;
  const int myStrips = (int)blockIdx.x < nStrips ? (nStrips - 1 - (int)blockIdx.x) / G + 1 : 0;

  auto wait_bar = [&](uint64_t *bar, uint32_t parity) {
    for (uint32_t i = 0; i < kB16BarPolls; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if (misc[0]) return false;
    }
    fail(DEVERR_DECODE_H_WAIT);
    return false;
  };
  // Wait for stage use `ord`.  A warp may be several uses of a stage ahead of
  // its barrier, whose parity alone would then say "done" for an earlier use,
  // so the producer's count comes first: once use `ord` is issued, every
  // earlier use of its stage has been consumed.
  auto wait_full = [&](int ord) {
    for (uint32_t i = 0; misc[2] <= ord; ++i) {
      if (misc[0]) return false;
      if (i > kB16Polls) {
        fail(DEVERR_DECODE_H_WAIT);
        return false;
      }
      __nanosleep(32);
    }
    return wait_bar(&full[ord & (nst - 1)], (ord >> a.nst_log2) & 1);
  };

  if (warp == kB16Warps) {
    // ------------------------------------------------------------ producer
    {
      uint32_t m = em;
      int b = ebase;
      while (m) {  // slots in order of expert id
        slot_expert[b++] = 32 * lane + __ffs(m) - 1;
        m &= m - 1u;
      }
    }
    __syncwarp();
    int ord = 0;
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      bool ok = true;
      // the stage of use `ord`, free and armed for `bytes`
      auto arm = [&](uint32_t bytes) {
        const int s = ord & (nst - 1);
        if (!wait_bar(&empty[s], ((ord >> a.nst_log2) & 1) ^ 1)) return false;
        mbar_arrive_expect_tx(&full[s], bytes);
        misc[2] = ++ord;
        return true;
      };
      for (int q = 0; q < myUnits && ok; ++q) {
        const int unit = blockIdx.x + q * G, slot = unit / UA, f0 = (unit - slot * UA) * FPU, e = slot_expert[slot];
        for (int c = 0; c < CA && (ok = arm(kB16Stage)); ++c) {
          const int s = (ord - 1) & (nst - 1);
          tma_load_5d_hint(smem + (size_t)s * kB16Stage, &gu_map, 0, f0, 0, c * (KCA / 64), e, &full[s], pol);
        }
      }
      int nJobs = U;
      if (ok && myStrips && kJobs) {
        for (uint32_t i = 0; !misc[3] && ok; ++i) {
          if (i > kB16Polls) fail(DEVERR_DECODE_H_WAIT);
          ok = !misc[0];
          __nanosleep(32);
        }
        __threadfence_block();
        nJobs = misc[4];
      }
      for (int si = 0; si < myStrips && ok; ++si) {
        const int row0 = (blockIdx.x + si * G) * R;
        for (int j = 0; j < nJobs && ok; ++j) {
          const int e = slot_expert[kJobs ? jobs[j] & 255 : j];
          for (int c = 0; c < CB && (ok = arm((uint32_t)R * (kB16KC * 2))); ++c) {
            const int s = (ord - 1) & (nst - 1);
            tma_load_4d_hint(smem + (size_t)s * kB16Stage, &dn_map, 0, row0, c * (kB16KC / 64), e, &full[s], pol);
          }
        }
      }
    }
    // the last copies issued into each stage land before the CTA leaves, also
    // when the consumers gave up
    if (lane == 0)
      for (int o = max(0, ord - nst); o < ord; ++o) mbar_wait_bounded(&full[o & (nst - 1)], (o >> a.nst_log2) & 1, 1u << 20);
  } else {
    // ------------------------------------------------------------ consumers
    if (warp * 32 < T * kk) {
      const int r = min(tid, T * kk - 1), t = r / kk, e = ridx[r];
      const int below = __shfl_sync(0xffffffffu, ebase, e >> 5);
      const uint32_t word = __shfl_sync(0xffffffffu, em, e >> 5);
      const int slot = below + __popc(word & ((1u << (e & 31)) - 1u));
      if (tid < T * kk) {
        atomicOr(&tokmask[slot], 1u << t);
        slot_j[slot * 16 + t] = (uint8_t)(r - t * kk);
      }
    }
    b16_consumer_sync();
    if (kJobs && warp == kB16Warps - 1) {  // the jobs of phase B; eight slots a lane
      int n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n += (__popc(tokmask[8 * lane + i]) + kB16JobTok - 1) / kB16JobTok;
      const int end = warp_inclusive_scan(n);
      int at = end - n;
      for (int i = 0; i < 8; ++i)
        for (int sub = 0; sub * kB16JobTok < __popc(tokmask[8 * lane + i]); ++sub)
          jobs[at++] = (uint16_t)(8 * lane + i + 256 * sub);
      if (lane == 31) misc[4] = end;
      __threadfence_block();
      __syncwarp();
      if (lane == 0) misc[3] = 1;  // for the producer; the consumers meet at the barrier after phase A
    }
    bool ok = true;
    // ---- phase A
    const uint8_t *xs = smem + L.x;
    auto ld16 = [](const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); };
    // this lane's pieces 2 t and 2 t + 1 of row g (or g + 8) of a swizzled 8-row group
    const uint32_t wo[2] = {(uint32_t)(g * 128 + (((2 * t4) ^ g) << 4)), (uint32_t)(g * 128 + (((2 * t4 + 1) ^ g) << 4))};
    for (int q = warp; q < myUnits && ok; q += kB16Warps) {
      const int unit = blockIdx.x + q * G, slot = unit / UA, f0 = (unit - slot * UA) * FPU;
      const uint32_t mask = tokmask[slot];
      const int ntok = __popc(mask);
      const uint8_t *xa[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n = kRows == 16 ? nb * 8 + g : (g & 3);
        xa[nb] = xs + (uint32_t)nth_bit(mask, n < ntok ? n : 0) * xpitch + 32u * t4;
      }
      const bool two = NB == 2 && ntok > 8;
      float acc[NB][4][4] = {};  // four independent chains
      for (int c = 0; c < CA; ++c) {
        const int o = q * CA + c, s = o & (nst - 1);
        if (!__all_sync(0xffffffffu, wait_full(o))) {
          ok = false;
          break;
        }
        const uint8_t *wa = smem + (uint32_t)s * kB16Stage;
        const int nch = min(KCA, H - c * KCA) / 64;
        uint32_t xo = (uint32_t)(c * KCA * 2);
        if (kRows == 16) {
#pragma unroll 4
          for (int b = 0; b < nch; ++b, wa += 2048, xo += 128) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 w0 = ld16(wa + wo[i]), w1 = ld16(wa + 1024 + wo[i]);
              const uint32_t f0r[4] = {w0.x, w1.x, w0.y, w1.y}, f1r[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if (nb == 1 && !two) continue;
                const uint4 v = ld16(xa[nb] + xo + 16 * i);
                mma_bf16_pure(acc[nb][2 * i], f0r, v.x, v.y);
                mma_bf16_pure(acc[nb][2 * i + 1], f1r, v.z, v.w);
              }
            }
          }
        } else {
          // rows 0-7 with tokens 0-3: columns b; rows 8-15 (the same weight rows)
          // with tokens in 4-7: columns b + half.  An odd last column has no
          // second: its weights are zeros (out of range, filled by the copy) and so
          // is its x (any other may hold an infinity).
          const int half = (nch + 1) / 2;
#pragma unroll 4
          for (int b = 0; b < half; ++b, wa += 1024, xo += 128) {
            const bool none = g >= 4 && b + half >= nch;
            const uint8_t *xv = xa[0] + xo + (g >= 4 && !none ? half * 128 : 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 w0 = ld16(wa + wo[i]), w1 = ld16(wa + half * 1024 + wo[i]);
              const uint32_t f0r[4] = {w0.x, w1.x, w0.y, w1.y}, f1r[4] = {w0.z, w1.z, w0.w, w1.w};
              uint4 v = ld16(xv + 16 * i);
              if (none) v = make_uint4(0, 0, 0, 0);
              mma_bf16_pure(acc[0][2 * i], f0r, v.x, v.y);
              mma_bf16_pure(acc[0][2 * i + 1], f1r, v.z, v.w);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      if (!ok) break;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (acc[nb][0][i] + acc[nb][1][i]) + (acc[nb][2][i] + acc[nb][3][i]);
        if (kRows == 8) {  // the halves' sums; rows 0-3 gate, 4-7 up: the partner is 16 lanes up
          v[0] += __shfl_down_sync(0xffffffffu, v[2], 2);
          v[1] += __shfl_down_sync(0xffffffffu, v[3], 2);
          v[2] = __shfl_down_sync(0xffffffffu, v[0], 16);
          v[3] = __shfl_down_sync(0xffffffffu, v[1], 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = nb * 8 + 2 * t4 + i;
          const float h = activate(v[i], MOE_ACT_SILU) * v[2 + i];
          // 24 bits, rounded (a NaN as it is: its payload would carry into the sign); four features to a word
          const uint32_t h0 = (__float_as_uint(h) + (h == h ? 0x80u : 0u)) >> 8, h1 = __shfl_down_sync(0xffffffffu, h0, 4),
                         h2 = __shfl_down_sync(0xffffffffu, h0, 8), h3 = __shfl_down_sync(0xffffffffu, h0, 12);
          if (n < ntok && (g & 3) == 0 && g < FPU && !a.starve) {
            const int t = nth_bit(mask, n);
            const uint32_t p0 = __byte_perm(h0, h1, 0x6521), p1 = __byte_perm(h2, h3, 0x6521),
                           p2 = __byte_perm(__byte_perm(h0, h1, 0x0040), __byte_perm(h2, h3, 0x0040), 0x5410);
            st_relaxed_b128(a.hbuf + (size_t)(t * kk + slot_j[slot * 16 + t]) * (F / 4) + (f0 + g) / 4,
                            (unsigned long long)p0 << 32 | epoch, (unsigned long long)p2 << 32 | p1);
          }
        }
      }
    }
    if (a.shared_xh || kJobs) b16_consumer_sync();  // x is consumed and the jobs are listed

    // ---- phase B
    uint8_t *hbp = smem + L.h + (uint32_t)warp * a.hb_bytes;
    const int nJobs = kJobs ? misc[4] : U;
    for (int si = 0; si < myStrips; ++si) {
      const int row0 = (blockIdx.x + si * G) * R, nr = min(R, H - row0);
      // the units are a job's chunks of inputs, each for the next warp: the ring holds
      // few jobs of many chunks (12 tokens, 16 experts, 2560 x 1088: 167 us with
      // whole jobs to a warp, 108 so; 4 tokens, 64 experts, 2048 x 1536: 104, 87)
      const int units = nJobs * CB, base = si * units;
      for (int q = (2 * kB16Warps - 1 - warp - base % kB16Warps) % kB16Warps; q < units && ok; q += kB16Warps) {
        const int j = CB == 1 ? q : q / CB, c = q - j * CB;
        int u = j;
        uint32_t mask;  // the job's tokens
        if (kJobs) {
          u = jobs[j] & 255;
          mask = tokmask[u];
          for (int i = 0; i < (jobs[j] >> 8) * kB16JobTok; ++i) mask &= mask - 1u;
        } else {
          mask = tokmask[u];
        }
        const int m = min(__popc(mask), kB16JobTok);
        const int my_t = nth_bit(mask, min(lane, m - 1));  // lane n: token n of the job and its row
        const int my_row = my_t * kk + slot_j[u * 16 + my_t];
        int fc = kB16KC, sh = 2;  // inputs whose h fits the warp's buffer; log2(fc / 128)
        while ((uint32_t)(m * (fc * 2 + 16) * 2) > a.hb_bytes) fc >>= 1, --sh;
        const int o = nA + base + q, cc = min(kB16KC, F - c * kB16KC);
        const uint8_t *wa = smem + (uint32_t)(o & (nst - 1)) * kB16Stage;
        bool landed = false;
        float acc[4][4] = {};
        for (int k1 = 0; k1 < cc && ok; k1 += fc) {
          const int kc = min(fc, cc - k1), words = kc / 4;
          const uint32_t hp = (uint32_t)(kc * 2 + 16), lo_off = (uint32_t)m * hp;
          const ulonglong2 *hw = a.hbuf + (c * kB16KC + k1) / 4;
          for (int n0 = 0; n0 < m && ok; n0 += 4 >> sh) {
            ulonglong2 wv[4];  // four loads a lane in flight (eight: spills, and slower)
            uint32_t spins = 0;
            while (true) {  // all of the words, again until all are this call's
              bool mine = true;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = n0 + (i >> sh), p = (i & ((1 << sh) - 1)) * 32 + lane;
                const int row = __shfl_sync(0xffffffffu, my_row, n);
                if (n < m && p < words) ld_relaxed_b128(hw + (size_t)row * (F / 4) + p, wv[i]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n0 + (i >> sh) < m && (i & ((1 << sh) - 1)) * 32 + lane < words && (unsigned int)wv[i].x != epoch) mine = false;
              if (__all_sync(0xffffffffu, mine)) break;
              if (++spins > a.h_polls && lane == 0) fail(DEVERR_DECODE_H_WAIT);
              if (__any_sync(0xffffffffu, spins > a.h_polls || misc[0])) {
                ok = false;
                break;
              }
              // warps that are early (no barrier before phase B) poll 16 words of a
              // row while h is far off: all of them would crowd the stream
              while (!a.shared_xh && spins <= a.h_polls) {
                ld_relaxed_b128(hw + (size_t)__shfl_sync(0xffffffffu, my_row, n0) * (F / 4) + (lane & 15), wv[0]);
                if (__all_sync(0xffffffffu, (unsigned int)wv[0].x == epoch)) break;
                if (++spins > a.h_polls || __any_sync(0xffffffffu, misc[0])) break;  // (the outer loop ends the wait)
                __nanosleep(100);
              }
              if (a.shared_xh) __nanosleep(64);
            }
            if (!ok) break;
            __syncwarp();  // the buffer's last reads are over
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = n0 + (i >> sh), p = (i & ((1 << sh) - 1)) * 32 + lane;
              if (n < m && p < words) {
                uint8_t *at = hbp + (uint32_t)n * hp + (uint32_t)p * 8u;
                const uint32_t p0 = (uint32_t)(wv[i].x >> 32), p1 = (uint32_t)wv[i].y, r = (uint32_t)(wv[i].y >> 32);
                const float l0 = b16_rest(p0 << 16, r, 0), l1 = b16_rest(p0 & 0xFFFF0000u, r, 1),
                            l2 = b16_rest(p1 << 16, r, 2), l3 = b16_rest(p1 & 0xFFFF0000u, r, 3);
                *reinterpret_cast<uint2 *>(at) = make_uint2(p0, p1);
                *reinterpret_cast<uint2 *>(at + lo_off) =
                    make_uint2(__byte_perm(__float_as_uint(l0), __float_as_uint(l1), 0x7632),
                               __byte_perm(__float_as_uint(l2), __float_as_uint(l3), 0x7632));
              }
            }
          }
          __syncwarp();
          if (ok && !landed) {
            ok = __all_sync(0xffffffffu, wait_full(o));
            landed = true;
          }
          if (!ok) break;
          // token columns 0-3 take hi, 4-7 lo of the job's tokens
          const uint8_t *ha = hbp + (uint32_t)min(g & 3, m - 1) * hp + (g >= 4 ? lo_off : 0u) + 32u * t4;
          int line = (k1 / 64) * R + g;  // 128-byte line of row g; its swizzle is the line's place among eight
#pragma unroll 4
          for (int b = 0; b < kc / 64; ++b, line += R, ha += 128) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint8_t *wk = wa + (line * 128 + (((2 * t4 + i) ^ (line & 7)) << 4));
              const uint4 w0 = ld16(wk), w1 = ld16(wk + 1024);
              const uint4 v = ld16(ha + 16 * i);
              const uint32_t f0r[4] = {w0.x, w1.x, w0.y, w1.y}, f1r[4] = {w0.z, w1.z, w0.w, w1.w};
              mma_bf16_pure(acc[2 * i], f0r, v.x, v.y);
              mma_bf16_pure(acc[2 * i + 1], f1r, v.z, v.w);
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[o & (nst - 1)]);
        // this chunk's sums (hi + lo), added to those of the earlier inputs in their order
        if (c) {
          for (uint32_t i = 0; joined[j] != si * CB + c; ++i) {
            if (i > kB16Polls && lane == 0) fail(DEVERR_DECODE_H_WAIT);
            if (misc[0]) {
              ok = false;
              break;
            }
            __nanosleep(20);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          __threadfence_block();
        }
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = (acc[0][i] + acc[1][i]) + (acc[2][i] + acc[3][i]);
          v[i] += __shfl_down_sync(0xffffffffu, v[i], 2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * t4 + i, row = __shfl_sync(0xffffffffu, my_row, n);
          if (n < m) {
            float *rb = rowbuf + row * 16 + g;
            rb[0] = c ? rb[0] + v[i] : v[i];
            rb[8] = c ? rb[8] + v[2 + i] : v[2 + i];
          }
        }
        if (CB > 1) {
          __threadfence_block();
          __syncwarp();
          if (lane == 0) joined[j] = si * CB + c + 1;
        }
      }
      b16_consumer_sync();  // every expert's rows of this strip are in rowbuf
      if (!misc[0]) {
        for (int v = tid; v < T * nr; v += kB16Warps * 32) {
          const int t = v / nr, o = v - t * nr;
          float s = 0.f;
          for (int j = 0; j < kk; ++j) s = __fmaf_rn(rw[t * kk + j], rowbuf[(t * kk + j) * 16 + o], s);
          const size_t at = (size_t)t * H + row0 + o;
          if (a.residual) s += bf16_bits_to_f32(a.residual[at]);
          a.y[at] = f32_to_bf16_bits(s);
        }
      }
      b16_consumer_sync();  // rowbuf is free for the next strip
    }
  }
  __syncthreads();
  // the last CTA out records this call's epoch for the next call
  if (tid == 0) {
    const unsigned int done = atomicAdd(&a.ctrl[1], 1u);
    if (done == (unsigned int)G - 1u) {
      a.ctrl[0] = epoch;
      a.ctrl[1] = 0u;
      __threadfence();
    }
  }
}

// gate_up [E][2][F][H] as 64-input columns: box = 64 inputs x kRows / 2
// features x {gate, up} x the stage's columns; down [E][H][F]: box = 64 inputs
// x R outputs x 8 columns.  128-byte swizzle, zeros outside.
static bool b16_maps(CUtensorMap *gu, CUtensorMap *dn, const DecodeBf16Args &a, int rows) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t E = a.E, H = a.H, F = a.F;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const cuuint64_t d1[5] = {64, F, 2, H / 64, E}, s1[4] = {H * 2, F * H * 2, 128, 2 * F * H * 2};
  const cuuint32_t b1[5] = {64, (cuuint32_t)rows / 2, 2, (cuuint32_t)(kB16Stage / 128 / rows), 1};
  const cuuint64_t d2[4] = {64, H, F / 64, E}, s2[3] = {F * 2, 128, H * F * 2};
  const cuuint32_t b2[4] = {64, (cuuint32_t)a.R, kB16KC / 64, 1};
  return fn(gu, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t *>(a.gu), d1, s1, b1, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         fn(dn, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(a.dn), d2, s2, b2, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kRows, int PER>
static moe_status decode_bf16_launch(DecodeBf16Args &a, cudaStream_t stream) {
  auto kern = decode_bf16_kernel<kRows, PER>;
  int dev = 0, sms = 0, smem_max = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  const uint32_t cap = (uint32_t)smem_max;
  a.hb_bytes = b16_hb_bytes(a.T);
  a.nst_log2 = 3;
  a.shared_xh = 0;
  if (b16_layout(a.T, a.kk, a.H, 1 << a.nst_log2, a.shared_xh).total > cap) a.shared_xh = 1;
  while (a.nst_log2 > 1 && b16_layout(a.T, a.kk, a.H, 1 << a.nst_log2, a.shared_xh).total > cap) --a.nst_log2;
  const B16Smem L = b16_layout(a.T, a.kk, a.H, 1 << a.nst_log2, a.shared_xh);
  if (L.total > cap) return MOE_ERR_UNSUPPORTED_SHAPE;
  static std::atomic<int> per_sm[64];  // per device: the shared-memory opt-in and the CTAs per SM it allows
  if (dev < 0 || dev >= 64) {
    set_cuda_error(cudaErrorInvalidDevice);
    return MOE_ERR_CUDA;
  }
  if (per_sm[dev].load(std::memory_order_acquire) == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cap);
    int occ = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kB16Threads, cap);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    if (occ < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
    per_sm[dev].store(occ, std::memory_order_release);
  }
  // phase B strips: equal shares of the outputs, at most 16 a strip
  const int G = sms * per_sm[dev].load(std::memory_order_acquire), per_cta = (a.H + 16 * G - 1) / (16 * G);
  a.R = (a.H + per_cta * G - 1) / (per_cta * G);
  CUtensorMap gu_map, dn_map;
  if (!b16_maps(&gu_map, &dn_map, a, kRows)) {
    set_cuda_error(cudaErrorInvalidValue);
    return MOE_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G);
  cfg.blockDim = dim3(kB16Threads);
  cfg.dynamicSmemBytes = L.total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, gu_map, dn_map);
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_decode_layer_bf16_workspace_bytes(int T, int k, int shared, int E, int H, int F) {
  if (T <= 0 || k <= 0 || shared < 0 || shared > 1 || E <= shared || H <= 0 || F <= 0) return 0;
  // control words, logit words, h words of every routed row
  return kB16CtrlBytes + kB16LogitBytes + ((size_t)T * (k + shared) * F + 3) / 4 * sizeof(ulonglong2);
}

// polls: bound of phase B's wait for h; starve: the test hook
static moe_status decode_layer_bf16(const moe_bf16_layer *layer, const uint16_t *x, const uint16_t *wr, float *logits,
                                    int T, int k, int shared, const uint16_t *shared_gate, const uint16_t *residual,
                                    uint16_t *y, int32_t *idx, float *w, void *ws, size_t ws_bytes, unsigned int polls,
                                    int starve, moe_stream_t stream) {
  if (!layer || T < 0 || k <= 0 || shared < 0 || shared > 1) return MOE_ERR_INVALID_ARG;
  const int E = layer->E, H = layer->H, F = layer->F, kk = k + shared, Er = E - shared;
  if (Er <= 0 || H <= 0 || F <= 0 || k > Er || (shared_gate && !shared)) return MOE_ERR_INVALID_ARG;
  if (H % 64 || F % 64 || F > kB16MaxF || E > 1024 || T > 16 || T * kk > 256 || kk > 32 ||
      T * (2 * (int64_t)H + 64) > kB16MaxX)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!layer->gate_up || !layer->down || !x || (!wr && !logits) || !y) return MOE_ERR_INVALID_ARG;
  if ((idx == nullptr) != (w == nullptr) || y == x) return MOE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)layer->gate_up, (const void *)layer->down, (const void *)x, (const void *)wr,
                        (const void *)shared_gate, (const void *)residual, (const void *)y, (const void *)ws})
    if (reinterpret_cast<uintptr_t>(p) % 16) return MOE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)logits, (const void *)idx, (const void *)w})
    if (reinterpret_cast<uintptr_t>(p) % 4) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_decode_layer_bf16_workspace_bytes(T, k, shared, E, H, F)) return MOE_ERR_WORKSPACE;
  DecodeBf16Args a = {};
  a.gu = layer->gate_up;
  a.dn = layer->down;
  a.x = x;
  a.wr = wr;
  a.sg = shared_gate;
  a.residual = residual;
  a.logits = logits;
  a.ctrl = static_cast<unsigned int *>(ws);
  a.lbuf = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(ws) + kB16CtrlBytes);
  a.hbuf = reinterpret_cast<ulonglong2 *>(static_cast<uint8_t *>(ws) + kB16CtrlBytes + kB16LogitBytes);
  a.y = y;
  a.idx = idx;
  a.w = w;
  a.err = device_error_word();
  if (!a.err) return MOE_ERR_CUDA;
  a.T = T;
  a.kk = kk;
  a.shared = shared;
  a.E = E;
  a.H = H;
  a.F = F;
  a.h_polls = polls;
  a.starve = starve;
  cudaStream_t s = as_stream(stream);
  if (T <= kB16JobTok) return Er <= 256 ? decode_bf16_launch<8, 8>(a, s) : decode_bf16_launch<8, 32>(a, s);
  return Er <= 256 ? decode_bf16_launch<16, 8>(a, s) : decode_bf16_launch<16, 32>(a, s);
}

extern "C" MOE_API moe_status moe_decode_layer_bf16(const moe_bf16_layer *layer, const uint16_t *x, const uint16_t *wr,
                                                    float *logits, int T, int k, int shared,
                                                    const uint16_t *shared_gate, const uint16_t *residual, uint16_t *y,
                                                    int32_t *idx, float *w, void *ws, size_t ws_bytes,
                                                    moe_stream_t stream) {
  return decode_layer_bf16(layer, x, wr, logits, T, k, shared, shared_gate, residual, y, idx, w, ws, ws_bytes, kB16Polls,
                           0, stream);
}

extern "C" MOE_API moe_status moe_debug_starve_decode_bf16(const moe_bf16_layer *layer, const uint16_t *x, float *logits,
                                                           int T, int k, uint16_t *y, void *ws, size_t ws_bytes,
                                                           unsigned int polls, moe_stream_t stream) {
  if (polls == 0) return MOE_ERR_INVALID_ARG;
  return decode_layer_bf16(layer, x, nullptr, logits, T, k, 0, nullptr, nullptr, y, nullptr, nullptr, ws, ws_bytes, polls,
                           1, stream);
}
