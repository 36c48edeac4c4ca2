// The whole MoE layer for 1 to 16 tokens in two kernels: router scores, then everything else.
#include "beam_moe_few.cuh"

#include <math_constants.h>

#include <type_traits>

namespace beam {
namespace {

// ------------------------------------------------------------------ router scores

// logits = h W_r^T, s = sigmoid(logit), sb = s + bias.  The sums run in FP64 and are rounded to
// FP32 once, and so is the sigmoid, so that the scores are the exactly rounded ones and near ties
// fall as the definition has them.
//
// Two experts per CTA: 128 CTAs for 256 experts.  Their rows and all tokens are copied into shared
// memory (2 bulk copies), and a warp takes a pair of tokens and a part of K.  Operands are widened
// with integer operations: the conversion instruction takes about 20 clocks of an SM a warp (at
// T = 16 the kernel took 39 us with it).  Bound by latency: 5.2 MB in all, and code that runs once.
//
// The kernel also clears the status words and marks as unwritten what the layer kernel exchanges.
constexpr int kRtThreads = 256, kRtExperts = 2, kRtWarps = kRtThreads / 32;

// x 2^-896 in FP64, exactly, zero and subnormals too: the exponent field as it is.  Infinity becomes what
// 2^128 does (as large a logit); NaN, which also becomes a number, is looked for apart.
constexpr double kUnscale = 0x1p+896;
__device__ __forceinline__ double widen_scaled(uint32_t u) {
  return __hiloint2double((static_cast<int>(u) >> 3) & static_cast<int>(0x8fffffffu), static_cast<int>(u << 29));
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__global__ void __launch_bounds__(kRtThreads) few_router_kernel(const FewRouterArgs a) {
  extern __shared__ __align__(128) uint8_t rt_smem[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ double part[kRtWarps][2 * kRtExperts];
  __shared__ int abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  const int e0 = blockIdx.x * kRtExperts;
  const uint32_t w_bytes = kRtExperts * a.d * 4, h_bytes = a.T * a.d * 2;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(smem_u32(&bar), 1);
    fence_mbarrier_init();
    mbar_arrive_expect_tx(smem_u32(&bar), w_bytes + h_bytes);
    bulk_load(smem_u32(rt_smem), a.W + static_cast<size_t>(e0) * a.d, w_bytes, smem_u32(&bar));
    bulk_load(smem_u32(rt_smem) + w_bytes, a.h, h_bytes, smem_u32(&bar));
  }
  if (blockIdx.x == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0u;
  if (blockIdx.x == 0 && threadIdx.x == 4) a.status[kFewMarkWord] = kFewMark;
  for (int64_t i = blockIdx.x * kRtThreads + threadIdx.x; i < a.unwritten_n;
       i += static_cast<int64_t>(gridDim.x) * kRtThreads)
    a.unwritten[i] = make_uint4(kUnwritten32, kUnwritten32, kUnwritten32, kUnwritten32);
  __syncthreads();
  const bool landed = a.wait_limit_ns == 0
                          ? mbar_test_wait(smem_u32(&bar), 0)  // gives up at once
                          : mbar_wait_bounded(smem_u32(&bar), 0, &abort_sh, a.wait_limit_ns, nullptr, 0);
  const float* W = reinterpret_cast<const float*>(rt_smem);
  const __nv_bfloat16* h = reinterpret_cast<const __nv_bfloat16*>(rt_smem + w_bytes);
  // warps: pairs of tokens, and parts of K while there are warps to spare
  const int pairs = (a.T + 1) / 2;
  const int log_parts = pairs == 1 ? 3 : pairs == 2 ? 2 : pairs <= 4 ? 1 : 0;
  const int pair = warp >> log_parts, t0 = pair * 2, t1 = t0 + 1 < a.T ? t0 + 1 : t0;
  const int span = a.d >> log_parts;
  if (pair < pairs) {
    double acc[2][kRtExperts] = {};  // of h and W 2^-896
    uint32_t h_top[2] = {};
    float w_top[kRtExperts] = {};
    const int k0 = (warp & ((1 << log_parts) - 1)) * span;
#pragma unroll 1
    for (int k = k0 + lane * 4; k < k0 + span; k += 128) {
      const uint2 x[2] = {*reinterpret_cast<const uint2*>(h + static_cast<size_t>(t0) * a.d + k),
                          *reinterpret_cast<const uint2*>(h + static_cast<size_t>(t1) * a.d + k)};
      double hd[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        hd[t][0] = widen_scaled(x[t].x << 16) * kUnscale;
        hd[t][1] = widen_scaled(x[t].x & 0xffff0000u) * kUnscale;
        hd[t][2] = widen_scaled(x[t].y << 16) * kUnscale;
        hd[t][3] = widen_scaled(x[t].y & 0xffff0000u) * kUnscale;
        h_top[t] = max_nan_bf16x2(h_top[t], max_nan_bf16x2(x[t].x, x[t].y));
      }
#pragma unroll
      for (int j = 0; j < kRtExperts; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(W + j * a.d + k);
        const double wd[4] = {widen_scaled(w.x), widen_scaled(w.y), widen_scaled(w.z), widen_scaled(w.w)};
        w_top[j] = max_nan(w_top[j], max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                                             max_nan(__uint_as_float(w.z), __uint_as_float(w.w))));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[0][j] = fma(wd[i], hd[0][i], acc[0][j]);
          acc[1][j] = fma(wd[i], hd[1][i], acc[1][j]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float top = max_nan(bf16_lo(h_top[t]), bf16_hi(h_top[t]));
#pragma unroll
      for (int j = 0; j < kRtExperts; ++j)
        if (top != top || w_top[j] != w_top[j]) acc[t][j] = CUDART_NAN;
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < kRtExperts; ++j) acc[t][j] += __shfl_xor_sync(0xffffffffu, acc[t][j], o);
    if (lane < 2 * kRtExperts)
      part[warp][lane] = lane == 0 ? acc[0][0] : lane == 1 ? acc[0][1] : lane == 2 ? acc[1][0] : acc[1][1];
  }
  // After a wait that ran out the scores are marked as unwritten, and the layer kernel, which chooses such
  // an expert before any other, reports it (the status words are only being cleared).
  const bool lost = __syncthreads_or(!landed);
  if (threadIdx.x < kRtExperts * a.T) {
    const int j = threadIdx.x % kRtExperts, t = threadIdx.x / kRtExperts;
    double v = 0.0;
    for (int p = 0; p < 1 << log_parts; ++p)
      v += part[((t >> 1) << log_parts) + p][(t & 1) * kRtExperts + j];
    const float logit = static_cast<float>(v * kUnscale);
    float s = static_cast<float>(1.0 / (1.0 + exp(-static_cast<double>(logit))));
    if (s != s) s = __uint_as_float(0x7fffffffu);  // not the mark
    const float2 nan = make_float2(__uint_as_float(kUnwritten32), __uint_as_float(0x7fffffffu));
    a.sc[static_cast<size_t>(t) * a.E + e0 + j] = lost ? nan : make_float2(s, s + a.bias[e0 + j]);
  }
  if (lost) {  // copies in flight must land before this CTA's shared memory is given up
    volatile int never = 0;
    mbar_wait_bounded(smem_u32(&bar), 0, &never, 2000000000ull, nullptr, 0);
  }
}

// ------------------------------------------------------------------ the layer

// A store of what other CTAs poll for.  A NaN is stored as the one that is not kUnwritten32.
__device__ __forceinline__ void st_relaxed32(float* p, float v) {
  uint32_t u = __float_as_uint(v);
  if (u == kUnwritten32) u = 0x7fffffffu;
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(u) : "memory");
}

// Order-preserving map of a score to unsigned; NaN above everything, nothing maps to 0.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v != v) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kWhereFew = 20;  // status sites of the layer kernel: 20..26

constexpr uint8_t kNoSlot = 255;
constexpr int kEntryMax = 4;  // tokens of an entry, at most
static_assert(kEntryMax * 3 <= 2 * kFewCols, "the BF16 pieces of an entry's activations are columns of two MMAs");
constexpr int kSlotTable = kFewMaxTokens * kMaxE * 8;  // offset in the ring, behind the scores

struct FewShared {
  uint64_t full_bar[kFewMaxStages], empty_bar[kFewMaxStages];
  uint64_t red_full[kFewRed], red_empty[kFewRed];
  float wts[kFewMaxSlots];              // routing weight of slot t * k + j
  uint32_t mask[kMaxE];                 // tokens of each expert
  uint8_t chosen[kFewMaxTokens][kMaxTopK];  // chosen experts of each token, ascending
  uint8_t entry_e[kFewMaxSlots];        // expert of each entry
  uint8_t entry_n[kFewMaxSlots];        // its token columns, 1..4
  uint8_t entry_slot[kFewMaxSlots][kEntryMax];  // their slots, or kNoSlot
  int warp_entries[kFewWarps];
  alignas(16) uint8_t zeros[16];
  int n_entries, abort_flag;
};

// Selection of token `t` by one warp from its E (score, biased score) pairs in `sc`:
// the Gk groups with the largest sums of their two best biased scores, the k best experts in
// them, ties to the lower index; ascending experts and normalised weights out.
// slot_of[t * E + e]: the slot j of expert e.
__device__ void few_select(const FewLayerArgs& a, const float2* sc, uint8_t* slot_of, FewShared& sh,
                           int t, int lane) {
  const int P = a.E / a.G;
  uint32_t gkey = 0;
  if (lane < a.G) {  // lane g: the sum of group g's two best
    float m1 = -CUDART_INF_F, m2 = -CUDART_INF_F, n = 0.f;
    int jj = lane % P;  // start at different banks
#pragma unroll 4
    for (int j = 0; j < P; ++j) {
      const float v = sc[lane * P + jj].y;
      if (++jj == P) jj = 0;
      n = v != v ? v : n;  // NaN if a score is; infinities (a bias of -inf masks an expert) have their order
      m2 = fmaxf(m2, fminf(m1, v));
      m1 = fmaxf(m1, v);
    }
    gkey = score_key((P >= 2 ? m1 + m2 : m1) + n);
  }
  int grank = 0;
#pragma unroll 1
  for (int g = 0; g < a.G; ++g) {
    const uint32_t o = __shfl_sync(0xffffffffu, gkey, g);
    grank += o > gkey || (o == gkey && g < lane);
  }
  const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.G && grank < a.Gk);
  // experts lane, lane + 32, ...
  const uint32_t inv = (65536u + P - 1) / P;  // e / P = e inv / 65536 for e, P <= 256
  uint32_t key[kMaxE / 32];
#pragma unroll
  for (int i = 0; i < kMaxE / 32; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < a.E && ((kept >> ((e * inv) >> 16)) & 1u) ? score_key(sc[e].y) : 0u;
  }
  // k times the best; ties to the lower expert
  uint32_t at = 0;  // experts chosen, in the lane's registers: bit i of `chosen`
  uint32_t chosen = 0;
#pragma unroll 1
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kMaxE / 32; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    uint32_t cand = kMaxE;  // the lane's lowest expert with that key
#pragma unroll
    for (int i = kMaxE / 32 - 1; i >= 0; --i) cand = key[i] == m ? static_cast<uint32_t>(32 * i + lane) : cand;
    cand = __reduce_min_sync(0xffffffffu, cand);
    const uint32_t mine = (cand & 31u) == static_cast<uint32_t>(lane) ? cand >> 5 : kMaxE;
    chosen |= mine < 32u ? 1u << mine : 0u;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i) key[i] = mine == static_cast<uint32_t>(i) ? 0u : key[i];
  }
  // slots: chosen experts in ascending order
#pragma unroll 1
  for (int i = 0; i < (a.E + 31) / 32; ++i) {
    const bool c = (chosen >> i) & 1u;
    const uint32_t b = __ballot_sync(0xffffffffu, c);
    if (c) {
      const int e = lane + 32 * i, j = at + __popc(b & ((1u << lane) - 1u));
      sh.chosen[t][j] = static_cast<uint8_t>(e);
      slot_of[t * a.E + e] = static_cast<uint8_t>(j);
      atomicOr(&sh.mask[e], 1u << t);
    }
    at += __popc(b);
  }
  __syncwarp();
  const int e = lane < a.k ? sh.chosen[t][lane] : 0;
  const float s = lane < a.k ? sc[e].x : 0.f;
  float sum = 0.f;  // in ascending order
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, s, j);
  if (lane < a.k) {
    if (__float_as_uint(s) == kUnwritten32) {  // a wait of the router ran out: no CTA writes outputs
      sh.abort_flag = 1;
      record_status(a.status, kDevTimeout, kWhereFew + 6);
    }
    const float w = a.norm ? a.scale * s / sum : a.scale * s;
    sh.wts[t * a.k + lane] = w;
    if (blockIdx.x == 0) {
      if (a.idx) a.idx[t * a.k + lane] = e;
      if (a.wts) a.wts[t * a.k + lane] = w;
    }
  }
}

// Lists the touched experts ascending, run by the consumer warps, a thread to an expert.
//   by_token: an entry's column t is token t (kNoSlot where the token has other experts), so that all
//             entries share the token fragments of gate|up;
//   else      its columns are its tokens, entry_max at most; one more opens a second entry that reads
//             the weights again (16 tokens that choose 8 of 64 experts at random: for 4 experts in 100).
__device__ void few_entries(const FewLayerArgs& a, const uint8_t* slot_of, FewShared& sh, bool by_token) {
  const int e = threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kFewWarps * 32 == kMaxE, "a thread to an expert");
  uint32_t m = e < a.E ? sh.mask[e] : 0u;
  if (blockIdx.x == 0 && e < a.E) a.cnt[e] = __popc(m);
  const int shift = 31 - __clz(a.entry_max);  // 2 or 4 tokens
  const int need = by_token ? m != 0u : (__popc(m) + a.entry_max - 1) >> shift;
  int incl = need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.warp_entries[warp] = incl;
  asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
  int at = incl - need;
  for (int w = 0; w < warp; ++w) at += sh.warp_entries[w];
  if (e == kMaxE - 1) sh.n_entries = at + need;
  for (int p = 0; p < need; ++p, ++at) {
    int n = 0;
    if (by_token) {
      for (; n < a.T; ++n)
        sh.entry_slot[at][n] = (m >> n) & 1u ? static_cast<uint8_t>(n * a.k + slot_of[n * a.E + e]) : kNoSlot;
    } else {
      while (m && n < a.entry_max) {
        const int t = __ffs(m) - 1;
        m &= m - 1;
        sh.entry_slot[at][n++] = static_cast<uint8_t>(t * a.k + slot_of[t * a.E + e]);
      }
    }
    sh.entry_e[at] = static_cast<uint8_t>(e);
    sh.entry_n[at] = static_cast<uint8_t>(n);
  }
}

// Everything after the router scores, in one cooperative persistent kernel:
//   selection        every CTA for itself (E scores per token; no exchange needed)
//   gate|up          items (entry, 8 intermediate rows): a 16-row tile holds 8 gate rows and the
//                    same 8 up rows, so one lane ends up with both and applies SwiGLU;
//                    FP32 activations
//   down             items (entry, 16 output rows): the entry's activations, polled for; FP32
//                    partial outputs per slot
//   combine          every CTA an even share of the output columns: each token's k slots, polled
//                    for, in ascending expert order, FP32, rounded to BF16 once
// Each CTA takes one contiguous run of items of either phase, cut so that both runs together are
// the same number of weight bytes for every CTA; its producer goes from the first into the second
// without waiting for anything but ring space, so the weights keep streaming while activations
// cross the GPU.  GROUP = 0: BF16 weights.  MODE: the arrangement of digits, 1 or 2 (0 for BF16).
//
// Bound by HBM, the bytes of the touched experts.  d = 5120, I = 2560, 64 experts, 8 chosen: BF16 1 token
// 114 us and 16 tokens 745 (5.5 and 6 TB/s), 4-bit weights 8 tokens 180.  4-bit, 1 token, 42 us: 26 of
// them the bytes, 6 the selection and the first copies, 4 the exchange of the activations (the ring holds
// 4 us of weights, and the slowest CTA's last rows take that long to reach everyone), 4 the combine.
template <int GROUP, int MODE>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const FewLayerArgs a) {
  constexpr bool kI4 = GROUP != 0;
  constexpr int kUnit = kI4 ? kI4Unit : kBf16Unit;                       // K elements
  constexpr int kUnitBytes = kI4 ? i4_unit_bytes(kI4 ? GROUP : 128) : 0;  // packed bytes
  constexpr int kRuns = kFewMaxK / kFewWarps / 32;                       // runs of 32 per warp
  constexpr int kStep = kI4 ? 2 : 1;  // tiles of one step, which share a ring slot, waits and hand-over
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ FewShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem);
  const uint32_t red = ring + a.stages * a.slot_bytes;
  volatile int* abort_flag = &sh.abort_flag;

  for (int e = threadIdx.x; e < kMaxE; e += kFewThreads) sh.mask[e] = 0u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_u32(&sh.full_bar[i]), 1);
      mbar_init(smem_u32(&sh.empty_bar[i]), kFewWarps);
    }
    for (int i = 0; i < kFewRed; ++i) {
      mbar_init(smem_u32(&sh.red_full[i]), kFewWarps);
      mbar_init(smem_u32(&sh.red_empty[i]), 1);
    }
    sh.abort_flag = 0;
    *reinterpret_cast<uint4*>(sh.zeros) = make_uint4(0u, 0u, 0u, 0u);
    fence_mbarrier_init();
  }
  // the tokens' scores, in the ring's space until the weights need it
  float2* sc = reinterpret_cast<float2*>(smem);
  uint8_t* slot_of = smem + kSlotTable;
  // With few enough tokens the columns of every entry are the tokens: the fragments of gate|up are
  // loaded once, while other warps select.
  const bool by_token = a.T <= a.entry_max;
  auto select = [&](int first, int step) {
    for (int t = first; t < a.T; t += step) few_select(a, sc + t * a.E, slot_of, sh, t, lane);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // generic accesses before bulk writes
  };
  pdl_wait();
  for (int i = threadIdx.x; i < a.T * a.E; i += kFewThreads) sc[i] = a.sc[i];
  __syncthreads();

  // ---- this CTA's items
  const int n_gu = a.I / 8, n_dn = a.d / 16;
  int i1, j1, i2, j2;
  auto cut = [&] {
    // 32 bits suffice: at most 128 entries, and K in units of 128
    const uint32_t N1 = sh.n_entries * n_gu, N2 = sh.n_entries * n_dn, K1 = a.d / 128, K2 = a.I / 128;
    const uint32_t grid = gridDim.x;
    // Lanes 0, 1: this CTA's and the next one's first gate|up item; 2, 3: down items.  Those start
    // where the CTAs before b have b / grid of all bytes (an item's are 16 K; gate|up: K = d, down:
    // K = I).  That is monotone in b as long as a CTA's down bytes cover the one gate|up item by
    // which the first runs differ; below that, an even cut.
    const uint32_t b = blockIdx.x + (lane & 1);
    const bool even = N2 * K2 < grid * K1;
    uint32_t v = b * N1 / grid;
    if (lane & 2) {
      const uint32_t w = (even ? b * N2 : b * (N1 * K1 + N2 * K2)) / grid;
      v = even ? w : (w - v * K1) / K2;
      if (b == grid || v > N2) v = N2;
    }
    i1 = __shfl_sync(0xffffffffu, v, 0);
    j1 = __shfl_sync(0xffffffffu, v, 1);
    i2 = __shfl_sync(0xffffffffu, v, 2);
    j2 = __shfl_sync(0xffffffffu, v, 3);
  };

  // tiles of the next step, of one entry
  auto step_len = [](int left, int of_entry) {
    const int n = left < of_entry ? left : of_entry;
    return n < kStep ? n : kStep;
  };

  if (warp < kFewWarps) {
    more_registers<kFewRegsConsumer>();
    // ---- consumers
    // token fragments: BF16 4 registers a run of 32; INT8 digits 2 or 4 (4: up to 20 runs)
    uint32_t b[kI4 ? i4_mode_regs(kI4 ? MODE : 1) : 128];
    [[maybe_unused]] I4Factor factor[2];
    uint8_t* const raw = smem + a.stages * a.slot_bytes + kFewRed * kFewWarps * kStep * 512 + warp * a.stage_bytes;
    auto load = [&](int ph, int entry) {  // entry < 0: all tokens
      const KSplit ks = ph > 0 ? a.k2 : a.k1;
      const int units = ks.count(warp), n = entry < 0 ? a.T : sh.entry_n[entry];
      const size_t k0 = ks.start(warp) * kUnit;
      TokenSource src{ph > 0, abort_flag, a.wait_limit_ns, a.status, kWhereFew + 1};
      auto row = [&](int col) -> const void* {
        if (entry < 0) return a.h + static_cast<size_t>(col) * a.d + k0;
        const int s = sh.entry_slot[entry][col];
        if (s == kNoSlot) return nullptr;
        if (ph > 0) return a.act + static_cast<size_t>(s) * a.I + k0;
        return a.h + static_cast<size_t>(s / a.k) * a.d + k0;
      };
      if constexpr (kI4)
        i4_load_tokens<(kI4 ? MODE : 1)>(b, factor, src, row, ph > 0, n, units, raw, sh.zeros, lane);
      else
        load_tokens<kRuns>(b, src, row, ph > 0, a.room, n, units * kUnit, raw, sh.zeros, lane);
      return __all_sync(0xffffffffu, src.ok) != 0;
    };
    int slot = 0, rb = 0;
    uint32_t par = 0, rpar = 1;
    bool ok = true, seen = false;  // seen: the current slot's phase
    // Phase -1 is the selection, with the loading of all tokens if they stay; as a turn of the same
    // loop so that there is one copy of the loading code.
#pragma unroll 1
    for (int ph = -1; ph < 2 && ok; ++ph) {
      const KSplit ks = ph > 0 ? a.k2 : a.k1;
      const int per = ph > 0 ? n_dn : n_gu;
      const int first = ph < 0 ? 0 : ph ? i2 : i1, last = ph < 0 ? 1 : ph ? j2 : j1;
      const int units = ks.count(warp), mine = warp / ks.cw, chunks = ks.chunks();
      const int cstart = ks.start(mine * ks.cw);
      const int cunits = ks.start((mine + 1) * ks.cw) - cstart;
      const int uoff = ks.start(warp) - cstart;
      const uint32_t off = kI4 ? uoff * kUnitBytes : uoff * 64;
      const int stride = bf16_row_stride(cunits);
      int entry = first / per, tile = first % per, loaded = -1, len = 1;
#pragma unroll 1
      for (int it = first; it < last; it += len) {
        if (ph < 0 ? by_token : entry != loaded && !(ph == 0 && by_token)) {
          loaded = entry;
          ok = load(ph, ph < 0 ? -1 : entry);
          if (!ok) break;
        }
        if (ph < 0) {
          if (!by_token) select(warp, kFewThreads / 32);
          __syncthreads();  // every token's selection is there
          few_entries(a, slot_of, sh, by_token);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncthreads();  // and the entries; the ring is the producer's
          cut();
          continue;
        }
        len = step_len(last - it, per - tile);
        // of each tile: rows g, g of two tokens, then g + 8; BF16 weights: of each set of columns
        float4 part[2] = {};
        static_assert(kStep <= 2, "parts");
        const bool two_sets = !kI4 && ph > 0 && sh.entry_n[entry] > 2;
        bool red_seen = false;
        if (!kI4) red_seen = mbar_test_wait(smem_u32(&sh.red_empty[rb]), rpar);
        // every warp passes every chunk in order: a phase may only be waited for by who has seen
        // the slot's phase before
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          ok = mbar_wait_seen(seen, smem_u32(&sh.full_bar[slot]), par, abort_flag, a.wait_limit_ns, a.status,
                              kWhereFew + 2);
          if (!ok) break;
          const int next = slot + 1 == a.stages ? 0 : slot + 1;
          if (next == 0) par ^= 1;
          // 4-bit weights: the tests of barriers come after the slice's loads from shared memory, which
          // wait for the answer of a test ahead of them.
          auto test = [&] {
            seen = mbar_test_wait(smem_u32(&sh.full_bar[next]), par);
            if (kI4 && ch + 1 == chunks) red_seen = mbar_test_wait(smem_u32(&sh.red_empty[rb]), rpar);
          };
          if (!kI4 || ch != mine) test();
          if (ch == mine) {
            const uint32_t base = ring + slot * a.slot_bytes + off;
            if constexpr (kI4) {
              // Both tiles are multiplied even where the step has one: the second is then what the slot
              // held before, and its sums are not stored.
              I4Acc<(kI4 ? MODE : 1)> acc[kStep] = {};
              i4_slice<(kI4 ? GROUP : 128)>(acc, b, base, cunits * kUnitBytes, units, lane);
              test();
#pragma unroll
              for (int r = 0; r < kStep; ++r) part[r] = i4_result(acc[r], factor, lane);
            } else {
              if (two_sets) {
                float acc[2][4] = {};
                bf16_slice<kRuns / 2>(acc, b, base, stride, units, lane);
#pragma unroll
                for (int r = 0; r < 2; ++r) part[r] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
              } else {
                float acc[1][4] = {};
                bf16_slice<kRuns>(acc, b, base, stride, units, lane);
                part[0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty_bar[slot]));
          slot = next;
        }
        if (!ok) break;
        if (!kI4 && ph > 0) {
          part[0] = sum_pieces(part[0]);
          // both sets go into one partial tile: lanes c = 0 keep tokens 0 and 1, lanes c = 1 the others
          if (two_sets) {
            const float4 other = sum_pieces(part[1]);
            if (lane & 1) part[0] = other;
          }
        }
        ok = mbar_wait_seen(red_seen, smem_u32(&sh.red_empty[rb]), rpar, abort_flag, a.wait_limit_ns, a.status,
                            kWhereFew + 3);
        if (!ok) break;
        if (units > 0) {
#pragma unroll
          for (int r = 0; r < kStep; ++r)
            sts128(red + ((rb * kFewWarps + warp) * kStep + r) * 512 + lane * 16, part[r]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.red_full[rb]));
        if (++rb == kFewRed) {
          rb = 0;
          rpar ^= 1;
        }
        if ((tile += len) == per) {
          tile = 0;
          ++entry;
        }
      }
    }
    __syncwarp();
    fewer_registers<kFewRegsLaunch>();
  } else {
    fewer_registers<kFewRegsOther>();
    if (by_token)
      select(warp - kFewWarps, kFewThreads / 32 - kFewWarps);
    else
      select(warp, kFewThreads / 32);
    __syncthreads();
    __syncthreads();
    cut();
  if (warp == kFewWarps) {
    // ---- producer
    int slot = 0;
    uint32_t par = 1, issued = 0;
    bool ok = true;
#pragma unroll 1
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const KSplit ks = ph ? a.k2 : a.k1;
      const int per = ph ? n_dn : n_gu, K = ph ? a.I : a.d;
      int entry = (ph ? i2 : i1) / per, tile = (ph ? i2 : i1) % per;
      const int last = ph ? j2 : j1;
      int len;
#pragma unroll 1
      for (int it = ph ? i2 : i1; it < last && ok; it += len) {
        len = step_len(last - it, per - tile);
        const int e = sh.entry_e[entry];
        const uint8_t* src;
        if (kI4) {
          src = static_cast<const uint8_t*>(ph ? a.w_down : a.w_gate) +
                (static_cast<size_t>(e) * per + tile) * ks.n * kUnitBytes;
        } else {  // lane r < 16 copies row r of the tile
          const int r = lane & 15;
          const void* m = ph ? a.w_down : (r < 8 ? a.w_gate : a.w_up);
          const size_t row = ph ? static_cast<size_t>(e) * a.d + tile * 16 + r
                                : static_cast<size_t>(e) * a.I + tile * 8 + (r & 7);
          src = static_cast<const uint8_t*>(m) + row * K * 2;
        }
        for (int w = 0; w < kFewWarps; w += ks.cw) {
          ok = mbar_wait_warp(smem_u32(&sh.empty_bar[slot]), par, abort_flag, a.wait_limit_ns,
                              a.status, kWhereFew);
          if (!ok) break;
          const int s = ks.start(w), n = ks.start(w + ks.cw) - s;
          const uint32_t bar = smem_u32(&sh.full_bar[slot]);
          const uint32_t dst = ring + slot * a.slot_bytes;
          if (lane == 0) mbar_arrive_expect_tx(bar, kI4 ? len * n * kUnitBytes : 16 * n * 64);
          __syncwarp();
          if (kI4) {
            if (lane < len)  // lane r copies the chunk of tile r
              bulk_load(dst + lane * n * kUnitBytes, src + static_cast<size_t>(lane * ks.n + s) * kUnitBytes,
                        n * kUnitBytes, bar);
          } else if (lane < 16 && n > 0) {
            bulk_load(dst + lane * bf16_row_stride(n), src + static_cast<size_t>(s) * 64, n * 64, bar);
          }
          ++issued;
          if (++slot == a.stages) {
            slot = 0;
            par ^= 1;
          }
        }
        if ((tile += len) == per) {
          tile = 0;
          ++entry;
        }
      }
    }
    if (!ok) {  // copies in flight must land before this CTA's shared memory is given up
      volatile int never = 0;
      const uint32_t back = issued < static_cast<uint32_t>(a.stages) ? issued : a.stages;
      for (uint32_t i = issued - back; i < issued; ++i)
        mbar_wait_bounded(smem_u32(&sh.full_bar[i % a.stages]), (i / a.stages) & 1, &never,
                          2000000000ull, nullptr, 0);
    }
  } else {
    // ---- finishing warps, steps in turn: no more warps than buffers, so that who waits for a buffer
    // has seen its phase before (or a later step's)
    const int mine = warp - kFewWarps - 1;
    const bool idle = mine >= kFewRed;
    const int g = lane >> 2, c = lane & 3;
    int rb = 0;
    uint32_t rpar = 0;
    bool ok = true;
#pragma unroll 1
    for (int ph = 0; ph < 2 && ok && !idle; ++ph) {
      const KSplit ks = ph ? a.k2 : a.k1;
      const int per = ph ? n_dn : n_gu;
      const int first = ph ? i2 : i1, last = ph ? j2 : j1;
      const int active = ks.n < kFewWarps ? ks.n : kFewWarps;
      int entry = first / per, tile = first % per, len;
#pragma unroll 1
      for (int it = first; it < last; it += len) {
        len = step_len(last - it, per - tile);
        if (rb == mine) {  // a buffer to each finishing warp
          ok = mbar_wait_warp(smem_u32(&sh.red_full[rb]), rpar, abort_flag, a.wait_limit_ns, a.status,
                              kWhereFew + 4);
          if (!ok) break;
          float4 v[kStep] = {};
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) {
            if (w >= active) break;
#pragma unroll
            for (int r = 0; r < kStep; ++r) {
              const float4 p = lds_f4(red + ((rb * kFewWarps + w) * kStep + r) * 512 + lane * 16);
              v[r].x += p.x;
              v[r].y += p.y;
              v[r].z += p.z;
              v[r].w += p.w;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.red_empty[rb]));
          const int n = sh.entry_n[entry];
#pragma unroll
          for (int r = 0; r < kStep; ++r) {
            if (r >= len) break;
            const float lo[2] = {v[r].x, v[r].y}, hi[2] = {v[r].z, v[r].w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int col = c * 2 + h;
              if (col < n && sh.entry_slot[entry][col] != kNoSlot) {
                const size_t s = sh.entry_slot[entry][col];
                if (ph == 0) {
                  st_relaxed32(a.act + s * a.I + (tile + r) * 8 + g, swiglu(lo[h], hi[h]));
                } else {
                  float* y = a.y + s * a.d + (tile + r) * 16 + g;
                  st_relaxed32(y, lo[h]);
                  st_relaxed32(y + 8, hi[h]);
                }
              }
            }
          }
        }
        if (++rb == kFewRed) {
          rb = 0;
          rpar ^= 1;
        }
        if ((tile += len) == per) {
          tile = 0;
          ++entry;
        }
      }
    }
    }
    __syncwarp();
    more_registers<kFewRegsLaunch>();
  }

  // ---- combine: every CTA an even share of the output columns, four to a thread; the partial
  // outputs come from all CTAs
  __syncthreads();
  if (sh.abort_flag) return;
  const int q0 = blockIdx.x * (a.d / 4) / gridDim.x, nq = (blockIdx.x + 1) * (a.d / 4) / gridDim.x - q0;
  TokenSource poll{true, abort_flag, a.wait_limit_ns, a.status, kWhereFew + 5};
  for (int u = threadIdx.x; u < nq * a.T; u += kFewThreads) {
    const int t = u / nq, col = (q0 + u % nq) * 4;
    const float* y = a.y + static_cast<size_t>(t) * a.k * a.d + col;
    uint4 v[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
      if (j < a.k) v[j] = ld_relaxed(y + static_cast<size_t>(j) * a.d);
    float o[4] = {};
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= a.k) break;
      uint64_t t0 = 0;
      while ((v[j].x == kUnwritten32 || v[j].y == kUnwritten32 || v[j].z == kUnwritten32 ||
              v[j].w == kUnwritten32) && poll.ok && poll.again(t0))
        v[j] = ld_relaxed(y + static_cast<size_t>(j) * a.d);
      const float w = sh.wts[t * a.k + j];
      o[0] = fmaf(w, __uint_as_float(v[j].x), o[0]);
      o[1] = fmaf(w, __uint_as_float(v[j].y), o[1]);
      o[2] = fmaf(w, __uint_as_float(v[j].z), o[2]);
      o[3] = fmaf(w, __uint_as_float(v[j].w), o[3]);
    }
    __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<size_t>(t) * a.d + col);
    out[0] = __floats2bfloat162_rn(o[0], o[1]);
    out[1] = __floats2bfloat162_rn(o[2], o[3]);
  }
}

using LayerKernel = void (*)(FewLayerArgs);
template <int GROUP>
LayerKernel layer_kernel_of(int mode) {
  return mode == 1 ? few_layer_kernel<GROUP, 1> : few_layer_kernel<GROUP, 2>;
}
LayerKernel layer_kernel(int group, int mode) {
  return group == 0    ? few_layer_kernel<0, 0>
         : group == 32 ? layer_kernel_of<32>(mode)
         : group == 64 ? layer_kernel_of<64>(mode)
                       : layer_kernel_of<128>(mode);
}

constexpr size_t kFewDynamicSmem = kFewSmemMax - 4096;  // the rest: FewShared
static_assert(sizeof(FewShared) <= 4096, "FewShared must fit beside the ring");
// Scores and slots lie in the ring while tokens are selected.  The smallest slot is two tiles of one
// superblock (or one tile of four BF16 units), and there are kFewMaxStages of them.  Only the scores of
// calls whose columns are not the tokens may reach into the partial-tile buffers behind: nothing uses
// those before the selection is done.
constexpr int kSmallestRing = kFewMaxStages * 2 * i4_unit_bytes(128);
static_assert(16 * bf16_row_stride(4) >= 2 * i4_unit_bytes(128), "BF16 rings are no smaller");
static_assert(kSlotTable + kEntryMax * kMaxE <= kSmallestRing, "scores and slots must fit in the ring");
static_assert(kFewMaxTokens * kMaxE * 9 <= kSmallestRing + kFewRed * kFewWarps * 512,
              "scores and slots must fit in the ring and the partial-tile buffers");

constexpr int kRtSmemMax = kFewSmemMax - 1024;

}  // namespace

cudaError_t launch_few_router(const FewRouterArgs& a, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kRtExperts) * a.d * 4 + static_cast<size_t>(a.T) * a.d * 2;
  few_router_kernel<<<a.E / kRtExperts, kRtThreads, smem, s>>>(a);
  return cudaGetLastError();
}

int few_router_tokens(int d) { return (kRtSmemMax - kRtExperts * d * 4) / (d * 2); }

cudaError_t launch_few_layer(FewLayerArgs a, int group, int sms, cudaStream_t s) {
  const int unit = group ? kI4Unit : kBf16Unit, unit_bytes = group ? i4_unit_bytes(group) : 0;
  // Tokens of an entry: 4, or 2 where the registers of a warp do not hold the fragments of 4 (the three
  // pieces of FP32 activations; the digits of 4-bit products, and there also where there are no more
  // tokens).  With 8 the weights of an expert of 5 to 8 tokens are read once, but every 4-bit product then
  // takes three MMAs instead of two (16 tokens over 64 experts, BF16 activations: 267 us, with 4 to an entry
  // 249).
  a.entry_max = (group ? a.T <= 2 || a.d > 5120 || a.I > 5120 : a.I > kFewMaxK / 2) ? 2 : kEntryMax;
  const int step = group ? 2 : 1;  // tiles
  a.k1 = make_ksplit(a.d / unit, group ? kI4SlotBytes : kBf16SlotBytes, step * unit_bytes);
  a.k2 = make_ksplit(a.I / unit, group ? kI4SlotBytes : kBf16SlotBytes, step * unit_bytes);
  const int c1 = chunk_bytes(a.k1, step * unit_bytes), c2 = chunk_bytes(a.k2, step * unit_bytes);
  a.slot_bytes = c1 > c2 ? c1 : c2;
  const int b1 = stage_bytes((a.d / unit + kFewWarps - 1) / kFewWarps * unit, group != 0, false);
  const int b2 = stage_bytes((a.I / unit + kFewWarps - 1) / kFewWarps * unit, group != 0, true);
  size_t red = 0;
  auto plan_stages = [&](int bytes) {
    a.stage_bytes = bytes;
    red = static_cast<size_t>(kFewRed) * kFewWarps * step * 512 + static_cast<size_t>(kFewWarps) * bytes;
    a.stages = static_cast<int>((kFewDynamicSmem - red) / a.slot_bytes);
    if (a.stages > kFewMaxStages) a.stages = kFewMaxStages;
    return a.stages;
  };
  const int without = plan_stages(b1 > b2 ? b1 : b2);
  if (!group) {  // room for all three BF16 pieces of a row, unless it costs a ring slot (as at I = 2560)
    const int pieces = b2 / 2 * 3;
    a.room = plan_stages(b1 > pieces ? b1 : pieces) == without;
    if (!a.room) plan_stages(b1 > b2 ? b1 : b2);
  }
  // no more CTAs than gate|up items can exist
  const int64_t items = static_cast<int64_t>(a.T) * a.k * (a.I / 8);
  const int grid = items < sms ? static_cast<int>(items) : sms;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = a.stages * static_cast<size_t>(a.slot_bytes) + red;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, layer_kernel(group, i4_mode(a.entry_max)), a);
}

cudaError_t prepare_few_kernels() {
  const cudaError_t r = cudaFuncSetAttribute(few_router_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kRtSmemMax);
  if (r != cudaSuccess) return r;
  for (int group : {0, 32, 64, 128})
    for (int mode : {1, 2}) {
      const cudaError_t e = cudaFuncSetAttribute(layer_kernel(group, mode),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kFewDynamicSmem));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace beam
