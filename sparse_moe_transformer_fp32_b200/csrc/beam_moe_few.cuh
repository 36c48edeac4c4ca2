// Few-token operators (1 to 16 tokens): 4-bit weights with group scales, their products, and the
// whole MoE layer in two kernels.  Constants, kernel arguments, launchers, and the device code the
// kernels share.
//
// Every one of these operators is a product of a large weight matrix with a handful of token rows:
// each weight is read once and used for at most 8 tokens (16 in the linear product), far below the
// arithmetic intensity at which the tensor cores bound anything, so the design is about streaming
// weights without a pause:
//
//  - one persistent CTA per SM: a producer warp moves weights into a shared-memory ring of
//    about 190 KB with bulk copies (4 us of one SM's share of the HBM bandwidth in flight, so
//    synchronisation between phases does not stop the stream), 16 consumer warps multiply, one
//    warp finishes outputs;
//  - a tile is 16 weight rows by the whole K range of the CTA; the 16 consumer warps split K.
//    Each keeps its K slice of the token rows in registers, as B fragments of
//    mma.sync.m16n8k16 (weights are the 16-row A operand, tokens the 8 columns), for as long as
//    the CTA stays with the same tokens, so that shared memory carries weights only;
//  - the 16 partial tiles go through a small shared-memory buffer to the finishing warp, which
//    adds them in warp order (results do not depend on timing).
//
// tcgen05 is not used here: its smallest tile is 128 weight rows by 8 tokens with both operands
// in shared memory, which would need the 4-bit codes expanded to BF16 in shared memory (four
// times the bytes) and gives 320 m-tiles of 16 rows only 40 tiles to spread over 148 SMs.
#pragma once
#include "beam_moe_internal.cuh"

namespace beam {

constexpr int kFewMaxTokens = 16;     // tokens per call
constexpr int kFewCols = 8;           // token columns of one MMA
constexpr int kFewMaxK = 8192;        // K of one tile: 16 warps x 512 elements (64 B registers)
constexpr int kFewMaxSlots = kFewMaxTokens * kMaxTopK;  // (token, expert) slots = most entries
constexpr int kFewWarps = 16;         // consumer warps
constexpr int kFewThreads = (kFewWarps + 2) * 32;  // + producer + finishing warp
constexpr int kFewSlotBytes = 21504;  // ring slot: 16 rows x (1280 + 64) bytes of BF16 weights
constexpr int kFewRed = 3;            // partial-tile buffers
constexpr int kFewMaxStages = 16;
constexpr int kFewSmemMax = 232448;   // 227 KB
constexpr int kBf16Unit = 32;         // K elements of the smallest BF16 slice of a warp

// 4-bit weights: superblocks of 16 rows x 128 K elements, in K order inside a 16-row tile.
// A superblock holds two 512-byte code blocks (64 K elements each) and then its BF16 scales.
// Code block: 16 bytes per lane of the MMA fragment, lane = 4 g + c: word v (0..3) holds, with
// k = 32 (v / 2) + 8 c + 4 (v % 2), the nibbles (bits 4i..4i+3)
//   i = 0, 4: row g     k, k + 1        i = 1, 5: row g + 8  k, k + 1
//   i = 2, 6: row g     k + 2, k + 3    i = 3, 7: row g + 8  k + 2, k + 3
// each storing code + 8.  Scales: for every group of the superblock 16 BF16, position 2 g for row
// g and 2 g + 1 for row g + 8.
constexpr int kI4Unit = 128;
__host__ __device__ constexpr int i4_unit_bytes(int group) {
  return kI4Unit * 16 / 2 + (kI4Unit / group) * 32;
}

// Slices of n K units over the 16 consumer warps: the first n % 16 warps hold one more.
struct KSplit {
  int n;        // units of the tile's K range
  int log_cw;   // log2 of the warps that share one ring slot ("chunk")
  __host__ __device__ int start(int w) const {
    const int q = n / kFewWarps, r = n % kFewWarps;
    return w * q + (w < r ? w : r);
  }
  __host__ __device__ int count(int w) const { return start(w + 1) - start(w); }
  __host__ __device__ int chunks() const { return kFewWarps >> log_cw; }
};

// Ring bytes of a BF16 chunk of u units: 16 rows at a stride of 64 bytes modulo 128, so that the
// eight rows of a fragment load fall into different banks.
__host__ __device__ constexpr int bf16_row_stride(int u) { return u * 64 + ((u & 1) ? 0 : 64); }

inline KSplit make_ksplit(int units, int slot_bytes, int unit_bytes_i4 /* 0: BF16 */) {
  KSplit s{units, 4};
  auto bytes = [&](int u) { return unit_bytes_i4 ? u * unit_bytes_i4 : 16 * bf16_row_stride(u); };
  for (; s.log_cw > 0; --s.log_cw) {
    int most = 0;
    for (int w = 0; w < kFewWarps; w += 1 << s.log_cw) {
      const int u = s.start(w + (1 << s.log_cw)) - s.start(w);
      if (u > most) most = u;
    }
    if (bytes(most) <= slot_bytes) break;
  }
  return s;
}

// ------------------------------------------------------------------ kernel arguments

struct Int4QuantArgs {
  const __nv_bfloat16* a;  // [groups, rows, cols]
  const __nv_bfloat16* b;  // same, or null
  uint8_t* packed;         // [groups, tiles, cols / 128, superblock]
  int64_t units;           // groups * tiles * cols / 128
  int rows, cols, tiles;   // tiles: 16-row tiles per group (8 rows of a and 8 of b with b)
  int group;
};

enum Int4Out { kI4OutBf16 = 0, kI4OutF32 = 1, kI4OutSwiglu = 2 };

struct Int4LinearArgs {
  const __nv_bfloat16* x;  // [T, K]
  const uint8_t* w;        // packed [tiles, K / 128, superblock]
  void* out;               // [T, N] (SwiGLU: [T, N / 2] BF16)
  uint64_t wait_limit_ns;
  int T, N, K, tiles;
  int out_kind;            // Int4Out
  int cluster;             // CTAs that split K
  int log_cw;              // KSplit::log_cw of the largest K range
  int stages, slot_bytes;
};

struct FewRouterArgs {
  const __nv_bfloat16* h;  // [T, d]
  const float* W;          // [E, d]
  const float* bias;       // [E]
  float2* sc;              // [T, E] out: score, biased score
  uint32_t* ctl;           // control words cleared for the layer kernel
  int ctl_words;
  int T, d, E;
};

struct FewLayerArgs {
  const __nv_bfloat16* h;  // [T, d]
  const float2* sc;        // [T, E]
  const void* w_gate;      // BF16 [E, I, d], or packed gate|up
  const void* w_up;        // BF16 [E, I, d], or null
  const void* w_down;      // BF16 [E, d, I], or packed
  __nv_bfloat16* act;      // [T * k, I]
  float* y;                // [T * k, d]
  __nv_bfloat16* out;      // [T, d]
  int32_t* idx;            // [T, k] out, or null
  float* wts;              // [T, k] out, or null
  uint32_t* ready;         // [kFewMaxSlots] finished gate/up tiles per entry; zero on entry
  uint32_t* done;          // [d / 16] finished down tiles per output tile; zero on entry
  uint32_t* status;
  uint64_t wait_limit_ns;
  KSplit k1, k2;           // gate/up and down K slices
  int T, d, E, G, Gk, k, I;
  float scale;
  int norm;
  int stages, slot_bytes;
};

cudaError_t launch_int4_quantize(const Int4QuantArgs& a, cudaStream_t s);
cudaError_t launch_int4_linear(Int4LinearArgs a, int group, int sms, cudaStream_t s);
cudaError_t launch_few_router(const FewRouterArgs& a, cudaStream_t s);
cudaError_t launch_few_layer(FewLayerArgs a, int group /* 0: BF16 */, int sms, cudaStream_t s);
cudaError_t prepare_int4_kernels();
cudaError_t prepare_few_kernels();

// ------------------------------------------------------------------ device code

#ifdef __CUDACC__

// Bulk copy global -> shared, completing on mbarrier `bar`; 16-byte aligned addresses and size.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp; every lane polls (each must see the phase complete before it reads
// what the barrier guards).  False on all lanes when any lane gave up.  A limit of 0 gives up at
// the first open phase (a try_wait may park the thread long enough to miss it).
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, uint64_t limit_ns,
                                               uint32_t* status, uint32_t where) {
  bool ok = mbar_test_wait(bar, parity);
  if (!ok) {
    if (limit_ns != 0) {
      ok = mbar_wait_bounded(bar, parity, abort_flag, limit_ns, status, where);
    } else {
      *abort_flag = 1;
      record_status(status, kDevTimeout, where);
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// D (16 x 8, FP32) += A (16 x 16, BF16) * B (16 x 8, BF16).
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The MMA sums over k in any order as long as both operands agree: in each run of 32 elements
// lane column c owns elements 8 c .. 8 c + 7 (one 16-byte load) and spends the first four on
// the first MMA, the last four on the second.

// B fragments of one token row's K slice: `row` points at the slice (null: an unused column,
// zeros), 4 registers per 32 elements.
template <int RUNS, bool COHERENT>
__device__ __forceinline__ void load_tokens(uint32_t (&b)[RUNS * 4], const __nv_bfloat16* row,
                                            int runs, int c) {
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row != nullptr && j < runs) {
      const uint4* p = reinterpret_cast<const uint4*>(row + j * 32 + c * 8);
      v = COHERENT ? __ldcg(p) : __ldg(p);
    }
    b[j * 4 + 0] = v.x;
    b[j * 4 + 1] = v.y;
    b[j * 4 + 2] = v.z;
    b[j * 4 + 3] = v.w;
  }
}

// acc += 16 BF16 weight rows (`base`: row 0 of the warp's slice, rows `stride` bytes apart) times
// the token columns, over `runs` runs of 32 K elements.
template <int RUNS>
__device__ __forceinline__ void bf16_slice(float (&acc)[4], const uint32_t (&b)[RUNS * 4],
                                           uint32_t base, int stride, int runs, int lane) {
  const uint32_t lo = base + (lane >> 2) * stride + (lane & 3) * 16;
  const uint32_t hi = lo + 8 * stride;
  float d0[4] = {}, d1[4] = {};  // two chains of dependent MMAs
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
    if (j < runs) {
      const uint4 r = lds128(lo + j * 64), s = lds128(hi + j * 64);
      mma_bf16(d0, r.x, s.x, r.y, s.y, b[j * 4], b[j * 4 + 1]);
      mma_bf16(d1, r.z, s.z, r.w, s.w, b[j * 4 + 2], b[j * 4 + 3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += d0[i] + d1[i];
}

// Two codes (nibbles at bits 0..3 and 16..19 of v) as exact BF16: 0x4300 | n is 128 + n, so
// subtracting 136 leaves n - 8.
__device__ __forceinline__ uint32_t i4_pair(uint32_t v) {
  uint32_t u, d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(u) : "r"(v), "r"(0x000f000fu), "r"(0x43004300u));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(u), "r"(0x43084308u));
  return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// acc[nt] += 16 rows of 4-bit weights (`base`: the warp's first superblock) times the token
// columns, over `units` superblocks.  The products of one group (or of the 64 elements of a
// code block, if the group is longer) are summed exactly scaled: codes and tokens are exact in
// BF16, the sum is FP32, and the group's scale multiplies it in FP32.
template <int NT, int UNITS, int GROUP>
__device__ __forceinline__ void i4_slice(float (&acc)[NT][4], const uint32_t (&b)[NT][UNITS * 16],
                                         uint32_t base, int units, int lane) {
  constexpr int kUnitBytes = i4_unit_bytes(GROUP);
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if (u < units) {
      const uint32_t ub = base + u * kUnitBytes;
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint4 w4 = lds128(ub + blk * 512 + lane * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        constexpr int kScaled = GROUP == 32 ? 2 : 1;  // scale changes inside a code block
#pragma unroll
        for (int p = 0; p < kScaled; ++p) {
          const int gi = GROUP == 32 ? blk * 2 + p : GROUP == 64 ? blk : 0;
          const uint32_t sc = lds32(ub + 1024 + gi * 32 + (lane >> 2) * 4);
          float d[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[nt][i] = 0.f;
#pragma unroll
          for (int v = p * (4 / kScaled); v < (p + 1) * (4 / kScaled); ++v) {
            const uint32_t a0 = i4_pair(w[v]), a1 = i4_pair(w[v] >> 4), a2 = i4_pair(w[v] >> 8),
                           a3 = i4_pair(w[v] >> 12);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(d[nt], a0, a1, a2, a3, b[nt][(u * 2 + blk) * 8 + v * 2],
                       b[nt][(u * 2 + blk) * 8 + v * 2 + 1]);
          }
          const float s0 = bf16_lo(sc), s1 = bf16_hi(sc);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = fmaf(s0, d[nt][0], acc[nt][0]);
            acc[nt][1] = fmaf(s0, d[nt][1], acc[nt][1]);
            acc[nt][2] = fmaf(s1, d[nt][2], acc[nt][2]);
            acc[nt][3] = fmaf(s1, d[nt][3], acc[nt][3]);
          }
        }
      }
    }
  }
}

// SiLU(g) * u in FP32.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

#endif  // __CUDACC__

}  // namespace beam
