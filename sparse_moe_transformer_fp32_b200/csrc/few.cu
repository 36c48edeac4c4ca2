// The whole MoE layer for 1 to 16 tokens in two kernels: router scores, then everything else.
#include "beam_moe_few.cuh"

#include <math_constants.h>

#include <type_traits>

namespace beam {
namespace {

// ------------------------------------------------------------------ router scores

// logits = h W_r^T, s = sigmoid(logit), sb = s + bias.  The sums run in FP64 and are rounded to
// FP32 once, and so is the sigmoid, so that the scores are the exactly rounded ones and near ties
// fall as the definition has them.  Operands are widened with integer operations: the conversion
// instruction takes about 20 clocks of an SM a warp (at T = 16 the kernel took 39 us with it).  Two
// experts per CTA: 128 CTAs for 256 experts, each reading 2 d FP32 weights; latency-bound at 5.2 MB
// in all.
//
// The kernel also clears the status words and marks as unwritten what the layer kernel exchanges.
constexpr int kRtThreads = 256, kRtExperts = 2;

// FP32 to FP64: exponent rebiased by 896; subnormals count as zero (they are below 2^-126).
__device__ __forceinline__ double widen(float v) {
  const uint32_t u = __float_as_uint(v), m = u & 0x7fffffffu;
  uint32_t hi = (m >> 3) + 0x38000000u;
  if (m < 0x00800000u) hi = 0u;
  if (m >= 0x7f800000u) hi |= 0x7ff00000u;
  return __hiloint2double(static_cast<int>(hi | (u & 0x80000000u)),
                          m < 0x00800000u ? 0 : static_cast<int>(u << 29));
}

template <int TM>
__global__ void __launch_bounds__(kRtThreads) few_router_kernel(const FewRouterArgs a) {
  __shared__ double part[kRtThreads / 32][kRtExperts * TM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0u;
  for (int64_t i = blockIdx.x * kRtThreads + threadIdx.x; i < a.unwritten_n;
       i += static_cast<int64_t>(gridDim.x) * kRtThreads)
    a.unwritten[i] = make_uint4(kUnwritten32, kUnwritten32, kUnwritten32, kUnwritten32);
  const int e0 = blockIdx.x * kRtExperts;
  double acc[kRtExperts][TM];
#pragma unroll
  for (int j = 0; j < kRtExperts; ++j)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[j][t] = 0.0;
#pragma unroll(TM <= 2 ? 5 : 2)
  for (int k = threadIdx.x * 4; k < a.d; k += kRtThreads * 4) {
    float4 w[kRtExperts];
    uint2 h[TM];
#pragma unroll
    for (int j = 0; j < kRtExperts; ++j)
      w[j] = __ldg(reinterpret_cast<const float4*>(a.W + static_cast<size_t>(e0 + j) * a.d + k));
#pragma unroll
    for (int t = 0; t < TM; ++t)
      h[t] = t < a.T ? __ldg(reinterpret_cast<const uint2*>(a.h + static_cast<size_t>(t) * a.d + k))
                     : make_uint2(0u, 0u);
    double wd[kRtExperts][4];
#pragma unroll
    for (int j = 0; j < kRtExperts; ++j) {
      wd[j][0] = widen(w[j].x);
      wd[j][1] = widen(w[j].y);
      wd[j][2] = widen(w[j].z);
      wd[j][3] = widen(w[j].w);
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const double hd[4] = {widen(bf16_lo(h[t].x)), widen(bf16_hi(h[t].x)), widen(bf16_lo(h[t].y)),
                            widen(bf16_hi(h[t].y))};
#pragma unroll
      for (int j = 0; j < kRtExperts; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][t] = fma(wd[j][i], hd[i], acc[j][t]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRtExperts; ++j)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      double v = acc[j][t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) part[warp][j * TM + t] = v;
    }
  __syncthreads();
  if (threadIdx.x < kRtExperts * TM) {
    const int j = threadIdx.x / TM, t = threadIdx.x % TM;
    if (t < a.T) {
      double v = 0.0;
#pragma unroll
      for (int w = 0; w < kRtThreads / 32; ++w) v += part[w][threadIdx.x];
      const float logit = static_cast<float>(v);
      const float s = static_cast<float>(1.0 / (1.0 + exp(-static_cast<double>(logit))));
      a.sc[static_cast<size_t>(t) * a.E + e0 + j] = make_float2(s, s + a.bias[e0 + j]);
    }
  }
}

// ------------------------------------------------------------------ the layer

// Stores of what other CTAs poll for.  A NaN is stored as the one that is not kUnwritten.
__device__ __forceinline__ void st_relaxed16(__nv_bfloat16* p, __nv_bfloat16 v) {
  unsigned short u = __bfloat16_as_ushort(v);
  if (u == kUnwritten16) u = 0x7fff;
  asm volatile("st.relaxed.gpu.global.u16 [%0], %1;" ::"l"(p), "h"(u) : "memory");
}
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

constexpr int kWhereFew = 20;  // status sites of the layer kernel: 20..24

struct FewShared {
  uint64_t full_bar[kFewMaxStages], empty_bar[kFewMaxStages];
  uint64_t red_full[kFewRed], red_empty[kFewRed];
  float wts[kFewMaxSlots];              // routing weight of slot t * k + j
  uint32_t mask[kMaxE];                 // tokens of each expert
  uint8_t chosen[kFewMaxTokens][kMaxTopK];  // chosen experts of each token, ascending
  uint8_t entry_e[kFewMaxSlots];        // expert of each entry
  uint8_t entry_n[kFewMaxSlots];        // its tokens, 1..8
  uint8_t entry_slot[kFewMaxSlots][kFewCols];  // their slots
  int n_entries, abort_flag;
};

// Selection of token `t` by one warp from its E (score, biased score) pairs in `sc`:
// the Gk groups with the largest sums of their two best biased scores, the k best experts in
// them, ties to the lower index; ascending experts and normalised weights out.
__device__ void few_select(const FewLayerArgs& a, const float2* sc, FewShared& sh, int t, int lane) {
  const int P = a.E / a.G;
  uint32_t gkey = 0;
  if (lane < a.G) {
    float m1 = -CUDART_INF_F, m2 = -CUDART_INF_F;
    bool nan = false;
    int jj = lane % P;  // start at different banks
#pragma unroll 4
    for (int j = 0; j < P; ++j) {
      const float v = sc[lane * P + jj].y;
      if (++jj == P) jj = 0;
      nan |= v != v;
      if (v > m1) {
        m2 = m1;
        m1 = v;
      } else if (v > m2) {
        m2 = v;
      }
    }
    gkey = nan ? 0xffffffffu : score_key(P >= 2 ? m1 + m2 : m1);
  }
  int grank = 0;
  for (int g = 0; g < a.G; ++g) {
    const uint32_t o = __shfl_sync(0xffffffffu, gkey, g);
    if (o > gkey || (o == gkey && g < lane)) ++grank;
  }
  const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.G && grank < a.Gk);
  // experts lane, lane + 32, ...: ties between lanes fall to the lower expert below
  uint32_t key[kMaxE / 32];
#pragma unroll
  for (int i = 0; i < kMaxE / 32; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < a.E && ((kept >> (e / P)) & 1u) ? score_key(sc[e].y) : 0u;
  }
  uint32_t chosen = 0;  // bit i: expert lane + 32 i
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    const uint32_t cand = best == m ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffffffu;
    const uint32_t win = __reduce_min_sync(0xffffffffu, cand);
    if (cand == win) {
      chosen |= 1u << bi;
#pragma unroll
      for (int i = 0; i < kMaxE / 32; ++i)
        if (i == bi) key[i] = 0u;
    }
  }
  // ascending expert ids, and the sum of the chosen scores in that order
  int at = 0;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxE / 32; ++i) {
    uint32_t b = __ballot_sync(0xffffffffu, (chosen >> i) & 1u);
    while (b) {
      const int e = (__ffs(b) - 1) + 32 * i;
      b &= b - 1;
      sum += sc[e].x;
      if (lane == 0) {
        sh.chosen[t][at] = static_cast<uint8_t>(e);
        atomicOr(&sh.mask[e], 1u << t);
      }
      ++at;
    }
  }
  __syncwarp();
  if (lane < a.k) {
    const int e = sh.chosen[t][lane];
    const float s = sc[e].x;
    const float w = a.norm ? a.scale * s / sum : a.scale * s;
    sh.wts[t * a.k + lane] = w;
    if (blockIdx.x == 0) {
      if (a.idx) a.idx[t * a.k + lane] = e;
      if (a.wts) a.wts[t * a.k + lane] = w;
    }
  }
}

// Lists the touched experts ascending, entry_max tokens at most to an entry (one more token of an
// expert opens a second entry that reads its weights again: with 8 to an entry and at most 16 tokens
// that takes a routing where more than half of them agree).  Run by one warp.
__device__ void few_entries(const FewLayerArgs& a, FewShared& sh, int lane) {
  int base = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    uint32_t m = e < a.E ? sh.mask[e] : 0u;
    const int need = (__popc(m) + a.entry_max - 1) / a.entry_max;
    int incl = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int at = base + incl - need;
    for (int p = 0; p < need; ++p, ++at) {
      int n = 0;
      while (m && n < a.entry_max) {
        const int t = __ffs(m) - 1;
        m &= m - 1;
        int j = 0;
        while (sh.chosen[t][j] != e) ++j;
        sh.entry_slot[at][n++] = static_cast<uint8_t>(t * a.k + j);
      }
      sh.entry_e[at] = static_cast<uint8_t>(e);
      sh.entry_n[at] = static_cast<uint8_t>(n);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) sh.n_entries = base;
}

// Everything after the router scores, in one cooperative persistent kernel:
//   selection        every CTA for itself (E scores per token; no exchange needed)
//   gate|up          items (entry, 8 intermediate rows): a 16-row tile holds 8 gate rows and the
//                    same 8 up rows, so one lane ends up with both and applies SwiGLU; BF16
//                    activations, the down product's MMA operand, as the layer defines them
//   down             items (entry, 16 output rows): the entry's activations, polled for; FP32
//                    partial outputs per slot
//   combine          every CTA an even share of the output columns: each token's k slots, polled
//                    for, in ascending expert order, FP32, rounded to BF16 once
// Each CTA takes one contiguous run of items of either phase, cut so that both runs together are
// the same number of weight bytes for every CTA; its producer goes from the first into the second
// without waiting for anything but ring space, so the weights keep streaming while activations
// cross the GPU.  GROUP = 0: BF16 weights.  MODES: the largest i4_mode of an entry.  HBM-bound on the touched experts' bytes.
template <int GROUP, int MODES>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const FewLayerArgs a) {
  constexpr bool kI4 = GROUP != 0;
  constexpr int kUnit = kI4 ? kI4Unit : kBf16Unit;                       // K elements
  constexpr int kUnitBytes = kI4 ? i4_unit_bytes(kI4 ? GROUP : 128) : 0;  // packed bytes
  constexpr int kRuns = kFewMaxK / kFewWarps / 32;                       // runs of 32 per warp
  constexpr int kRed = kI4 ? kFewRed : kBf16Red;
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
    for (int i = 0; i < kRed; ++i) {
      mbar_init(smem_u32(&sh.red_full[i]), kFewWarps);
      mbar_init(smem_u32(&sh.red_empty[i]), 1);
    }
    sh.abort_flag = 0;
    fence_mbarrier_init();
  }
  // the tokens' scores, in the ring's space until the weights need it
  float2* sc = reinterpret_cast<float2*>(smem);
  for (int i = threadIdx.x; i < a.T * a.E; i += kFewThreads) sc[i] = a.sc[i];
  __syncthreads();
  for (int t = warp; t < a.T; t += kFewThreads / 32) few_select(a, sc + t * a.E, sh, t, lane);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // generic reads before bulk writes
  __syncthreads();
  if (warp == 0) few_entries(a, sh, lane);
  __syncthreads();

  // ---- this CTA's items
  const int n_gu = a.I / 8, n_dn = a.d / 16;
  // 32 bits suffice: at most 128 entries, and K in units of 128
  const uint32_t N1 = sh.n_entries * n_gu, N2 = sh.n_entries * n_dn, K1 = a.d / 128, K2 = a.I / 128;
  const uint32_t grid = gridDim.x;
  auto first1 = [&](uint32_t b) { return b * N1 / grid; };
  // Down items start where the CTAs before b have b / grid of all bytes (an item's are 16 K;
  // gate|up: K = d, down: K = I).  That is monotone in b as long as a CTA's down bytes cover the
  // one gate|up item by which the first runs differ; below that, an even cut.
  auto first2 = [&](uint32_t b) {
    if (N2 * K2 < grid * K1) return b * N2 / grid;
    const uint32_t v = (b * (N1 * K1 + N2 * K2) / grid - first1(b) * K1) / K2;
    return b == grid || v > N2 ? N2 : v;
  };
  const int i1 = first1(blockIdx.x), j1 = first1(blockIdx.x + 1);
  const int i2 = first2(blockIdx.x), j2 = first2(blockIdx.x + 1);

  if (warp < kFewWarps) {
    more_registers<kFewRegsConsumer>();
    // ---- consumers
    // token fragments: BF16 4 registers a run of 32; INT8 digits 2, 4 or 6 (4 and 6: up to 20 runs)
    uint32_t b[!kI4 ? 128 : MODES == 1 ? 64 : MODES == 2 ? 80 : 120];
    [[maybe_unused]] I4Factor factor[2];
    [[maybe_unused]] uint8_t* const split =
        smem + a.stages * a.slot_bytes + kRed * kFewWarps * 512 + warp * kI4SplitBytes;
    int n_tok = 0;
    int slot = 0, rb = 0;
    uint32_t par = 0, rpar = 1;
    bool ok = true;
#pragma unroll 1
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const KSplit ks = ph ? a.k2 : a.k1;
      const int per = ph ? n_dn : n_gu, K = ph ? a.I : a.d;
      const int first = ph ? i2 : i1, last = ph ? j2 : j1;
      const int units = ks.count(warp), mine = warp / ks.cw, chunks = ks.chunks();
      const int cstart = ks.start(mine * ks.cw);
      const int cunits = ks.start((mine + 1) * ks.cw) - cstart;
      const int uoff = ks.start(warp) - cstart;
      const uint32_t off = kI4 ? uoff * kUnitBytes : uoff * 64;
      const int stride = bf16_row_stride(cunits);
      const int k0 = ks.start(warp) * kUnit;
      int entry = first / per, tile = first % per, loaded = -1;
#pragma unroll 1
      for (int it = first; it < last; ++it) {
        if (entry != loaded) {  // token fragments of the entry
          loaded = entry;
          n_tok = sh.entry_n[entry];
          auto row = [&](int col) {
            const int s = sh.entry_slot[entry][col];
            return ph ? a.act + static_cast<size_t>(s) * K + k0
                      : a.h + static_cast<size_t>(s / a.k) * K + k0;
          };
          auto load = [&](auto& src) {
            if constexpr (kI4) {
              if (MODES == 1 || n_tok <= 2)
                i4_load_tokens<1>(b, factor, src, row, n_tok, units, split, lane);
              else if (MODES == 2 || n_tok <= 4)
                i4_load_tokens<(MODES > 1 ? 2 : 1)>(b, factor, src, row, n_tok, units, split, lane);
              else
                i4_load_tokens<MODES>(b, factor, src, row, n_tok, units, split, lane);
            } else {
              const int col = lane >> 2;
              load_tokens<kRuns>(b, src, col < n_tok ? row(col) : nullptr, units, lane & 3);
            }
          };
          if (ph) {
            PolledRow src{abort_flag, a.wait_limit_ns, a.status, kWhereFew + 1};
            load(src);
            ok = __all_sync(0xffffffffu, src.ok);
            if (!ok) break;
          } else {
            TokenRow src;
            load(src);
          }
        }
        float4 part = make_float4(0.f, 0.f, 0.f, 0.f);  // rows g, g of two tokens, then g + 8
        // every warp passes every chunk in order: a phase may only be waited for by who has seen
        // the slot's phase before
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          ok = mbar_wait_warp(smem_u32(&sh.full_bar[slot]), par, abort_flag, a.wait_limit_ns, a.status,
                              kWhereFew + 2);
          if (!ok) break;
          if (ch == mine) {
            const uint32_t base = ring + slot * a.slot_bytes + off;
            if constexpr (kI4) {
              constexpr std::integral_constant<int, kI4 ? GROUP : 128> kG{};
              auto product = [&](auto acc) {
                i4_slice<kG.value>(acc, b, base, units, lane);
                part = i4_result(acc, factor, lane);
              };
              if (MODES == 1 || n_tok <= 2)
                product(I4Acc<1>{});
              else if (MODES == 2 || n_tok <= 4)
                product(I4Acc<(MODES > 1 ? 2 : 1)>{});
              else
                product(I4Acc<MODES>{});
            } else {
              float acc[4] = {};
              bf16_slice<kRuns>(acc, b, base, stride, units, lane);
              part = make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.empty_bar[slot]));
          if (++slot == a.stages) {
            slot = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        ok = mbar_wait_warp(smem_u32(&sh.red_empty[rb]), rpar, abort_flag, a.wait_limit_ns, a.status,
                            kWhereFew + 3);
        if (!ok) break;
        if (units > 0)
          sts128(red + (rb * kFewWarps + warp) * 512 + lane * 16, part);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.red_full[rb]));
        if (++rb == kRed) {
          rb = 0;
          rpar ^= 1;
        }
        if (++tile == per) {
          tile = 0;
          ++entry;
        }
      }
    }
    __syncwarp();
    fewer_registers<kFewRegsLaunch>();
  } else {
    fewer_registers<kFewRegsOther>();
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
#pragma unroll 1
      for (int it = ph ? i2 : i1; it < (ph ? j2 : j1) && ok; ++it) {
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
          if (lane == 0) mbar_arrive_expect_tx(bar, kI4 ? n * kUnitBytes : 16 * n * 64);
          __syncwarp();
          if (kI4) {
            if (lane == 0)
              bulk_load(dst, src + static_cast<size_t>(s) * kUnitBytes, n * kUnitBytes, bar);
          } else if (lane < 16 && n > 0) {
            bulk_load(dst + lane * bf16_row_stride(n), src + static_cast<size_t>(s) * 64, n * 64, bar);
          }
          ++issued;
          if (++slot == a.stages) {
            slot = 0;
            par ^= 1;
          }
        }
        if (++tile == per) {
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
  } else if (warp <= kFewWarps + 2) {
    // ---- finishing warps, tiles in turn
    const int g = lane >> 2, c = lane & 3;
    int rb = 0;
    uint32_t rpar = 0, turn = warp - kFewWarps - 1;
    bool ok = true;
#pragma unroll 1
    for (int ph = 0; ph < 2 && ok; ++ph) {
      const KSplit ks = ph ? a.k2 : a.k1;
      const int per = ph ? n_dn : n_gu;
      const int first = ph ? i2 : i1, last = ph ? j2 : j1;
      const int active = ks.n < kFewWarps ? ks.n : kFewWarps;
      int entry = first / per, tile = first % per;
#pragma unroll 1
      for (int it = first; it < last; ++it, turn ^= 1) {
        if (turn) {
          if (++rb == kRed) {
            rb = 0;
            rpar ^= 1;
          }
          if (++tile == per) {
            tile = 0;
            ++entry;
          }
          continue;
        }
        ok = mbar_wait_warp(smem_u32(&sh.red_full[rb]), rpar, abort_flag, a.wait_limit_ns, a.status,
                            kWhereFew + 4);
        if (!ok) break;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < active; ++w) {
          const uint4 p = lds128(red + (rb * kFewWarps + w) * 512 + lane * 16);
          v.x += __uint_as_float(p.x);
          v.y += __uint_as_float(p.y);
          v.z += __uint_as_float(p.z);
          v.w += __uint_as_float(p.w);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.red_empty[rb]));
        if (++rb == kRed) {
          rb = 0;
          rpar ^= 1;
        }
        const int n = sh.entry_n[entry];
        const float lo[2] = {v.x, v.y}, hi[2] = {v.z, v.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = c * 2 + h;
          if (col < n) {
            const size_t s = sh.entry_slot[entry][col];
            if (ph == 0) {
              st_relaxed16(a.act + s * a.I + tile * 8 + g, __float2bfloat16_rn(swiglu(lo[h], hi[h])));
            } else {
              float* y = a.y + s * a.d + tile * 16 + g;
              st_relaxed32(y, lo[h]);
              st_relaxed32(y + 8, hi[h]);
            }
          }
        }
        if (++tile == per) {
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
  PolledRow poll{abort_flag, a.wait_limit_ns, a.status, kWhereFew + 5};
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
LayerKernel layer_kernel_of(int modes) {
  return modes == 1 ? few_layer_kernel<GROUP, 1> : modes == 2 ? few_layer_kernel<GROUP, 2>
                                                              : few_layer_kernel<GROUP, 3>;
}
LayerKernel layer_kernel(int group, int modes) {
  return group == 0    ? few_layer_kernel<0, 0>
         : group == 32 ? layer_kernel_of<32>(modes)
         : group == 64 ? layer_kernel_of<64>(modes)
                       : layer_kernel_of<128>(modes);
}

constexpr size_t kFewDynamicSmem = kFewSmemMax - 6144;  // the rest: FewShared
static_assert(sizeof(FewShared) <= 6144, "FewShared must fit beside the ring");
// the scores of 16 tokens fit in the ring
static_assert(kFewMaxTokens * kMaxE * 8 <= kI4SlotBytes && kFewMaxTokens * kMaxE * 8 <= kBf16SlotBytes, "scores must fit in the ring");

}  // namespace

cudaError_t launch_few_router(const FewRouterArgs& a, cudaStream_t s) {
  const dim3 grid(a.E / kRtExperts);
  if (a.T <= 1)
    few_router_kernel<1><<<grid, kRtThreads, 0, s>>>(a);
  else if (a.T <= 2)
    few_router_kernel<2><<<grid, kRtThreads, 0, s>>>(a);
  else if (a.T <= 4)
    few_router_kernel<4><<<grid, kRtThreads, 0, s>>>(a);
  else if (a.T <= 8)
    few_router_kernel<8><<<grid, kRtThreads, 0, s>>>(a);
  else
    few_router_kernel<16><<<grid, kRtThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_few_layer(FewLayerArgs a, int group, int sms, cudaStream_t s) {
  const int unit = group ? kI4Unit : kBf16Unit, unit_bytes = group ? i4_unit_bytes(group) : 0;
  // the digits of 3 to 8 tokens fit in a warp's registers up to K = 5120, those of 2 up to 8192
  a.entry_max = group && (a.d > 5120 || a.I > 5120) ? 2 : kFewCols;
  a.slot_bytes = group ? kI4SlotBytes : kBf16SlotBytes;
  a.k1 = make_ksplit(a.d / unit, a.slot_bytes, unit_bytes);
  a.k2 = make_ksplit(a.I / unit, a.slot_bytes, unit_bytes);
  const size_t red = static_cast<size_t>(group ? kFewRed : kBf16Red) * kFewWarps * 512 +
                     (group ? static_cast<size_t>(kFewWarps) * kI4SplitBytes : 0);
  a.stages = static_cast<int>((kFewDynamicSmem - red) / a.slot_bytes);
  if (a.stages > kFewMaxStages) a.stages = kFewMaxStages;
  // no more CTAs than gate|up items can exist
  const int64_t most = static_cast<int64_t>(a.T) * a.k * (a.I / 8);
  const int grid = most < sms ? static_cast<int>(most) : sms;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = a.stages * static_cast<size_t>(a.slot_bytes) + red;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_kernel(group, i4_mode(a.T < a.entry_max ? a.T : a.entry_max)), a);
}

cudaError_t prepare_few_kernels() {
  for (int group : {0, 32, 64, 128})
    for (int modes : {1, 2, 3}) {
      const cudaError_t e = cudaFuncSetAttribute(layer_kernel(group, modes),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kFewDynamicSmem));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace beam
