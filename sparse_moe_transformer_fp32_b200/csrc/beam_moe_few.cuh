// Few-token operators (1 to 16 tokens): 4-bit weights with group scales, their products, and the
// whole MoE layer in two kernels.  Constants, kernel arguments, launchers, and the device code the
// kernels share.
//
// Every one of these operators is a product of a large weight matrix with a handful of token rows:
// each weight is read once and used for at most 4 tokens (16 in the linear product), far below the
// arithmetic intensity at which the tensor cores bound anything, so the design is about streaming
// weights without a pause:
//
//  - one persistent CTA per SM: a producer warp moves weights into a shared-memory ring (at Beam's
//    sizes 169 KB with 4-bit weights in groups of 128, 210 KB with BF16) with bulk copies (4 us of one
//    SM's share of the HBM bandwidth in flight, so synchronisation between phases does not stop the
//    stream), 8 consumer warps multiply, three finish outputs;
//  - a tile is 16 weight rows by the whole K range of the CTA; the 8 consumer warps split K.
//    Each keeps its K slice of the token rows in registers, as B fragments of mma.sync (weights are
//    the 16-row A operand, tokens the 8 columns), for as long as the CTA stays with the same
//    tokens, so that shared memory carries weights only;
//  - with 4-bit weights a step is two tiles where there are enough of them: waits, hand-over and
//    branches cost a warp about as much as its products of a tile;
//  - the 8 partial tiles go through a small shared-memory buffer to a finishing warp, which
//    adds them in warp order (results do not depend on timing).
//
// tcgen05 is not used here: its smallest tile is 128 weight rows by 8 tokens with both operands
// in shared memory, which would need the 4-bit codes expanded to BF16 in shared memory (four
// times the bytes) and gives 320 m-tiles of 16 rows only 40 tiles to spread over 148 SMs.
#pragma once
#include <type_traits>

#include "beam_moe_internal.cuh"

namespace beam {

constexpr int kFewMaxTokens = 16;     // tokens per call
constexpr int kFewCols = 8;           // token columns of an MMA
constexpr int kFewMaxK = 8192;        // K of one tile: 8 warps x 1024 elements (128 B registers)
constexpr int kFewMaxSlots = kFewMaxTokens * kMaxTopK;  // (token, expert) slots = most entries
constexpr int kFewWarps = 8;          // consumer warps
// Consumers, then a warp group of the producer and three finishing warps: register budgets are given
// per warp group.  Launched with 168 registers a thread; while the roles run,
// consumers hold 216 and the others 72 (256 * 216 + 128 * 72 = 384 * 168).
constexpr int kFewThreads = (kFewWarps + 4) * 32;
constexpr int kFewRegsLaunch = 168, kFewRegsConsumer = 216, kFewRegsOther = 72;
static_assert(kFewWarps == 8 && kFewWarps * kFewRegsConsumer + 4 * kFewRegsOther ==
                                    (kFewWarps + 4) * kFewRegsLaunch, "register budgets must add up");
// Ring slot, 4-bit weights, at most: two tiles of K = 2560 or halves of two of K = 5120, any group.  A
// warp's waits, hand-over and branches take about 1100 clocks a slot, its products 400 clocks a tile of
// K = 2560, and a tile of that size arrives every 900: with one tile to a slot a layer of one token took
// 46.7 us and one of 8 tokens 268, with two 41.6 and 212 (d = 5120, I = 2560, 64 experts, 8 chosen).
constexpr int kI4SlotBytes = 46080;
// Ring slot, BF16 weights: 16 rows x (2560 + 64) bytes.  Each row of a slot is a bulk copy, and one
// SM starts a copy about every 39 ns whatever its size: segments of 640, 1280 and 2560 bytes
// stream at 2.4, 4.8 and 7.4 TB/s over the GPU.
constexpr int kBf16SlotBytes = 41984;
constexpr int kFewRed = 2;            // buffers of partial tiles, each with a finishing warp
constexpr int kFewMaxStages = 16;
constexpr int kFewSmemMax = 232448;   // 227 KB
constexpr int kBf16Unit = 32;         // K elements of the smallest BF16 slice of a warp

// 4-bit weights: superblocks of 16 rows x 128 K elements, in K order inside a 16-row tile.
// A superblock holds two 512-byte code blocks (64 K elements each) and then its BF16 scales.
// Code block: 16 bytes per lane of the MMA fragment, lane = 4 g + c: byte i of word v (0..3) holds
// the codes (two's complement) of column 32 (v / 2) + 8 c + 4 (v % 2) + i: row g in the high four
// bits, row g + 8 in the low four.  The word masked with 0xf0f0f0f0, and the word shifted up by four
// and masked, are A registers of an 8-bit MMA with the values 16 q.
// Scales: for every group of the superblock 16 BF16, position 2 g for row g and 2 g + 1 for row
// g + 8.
constexpr int kI4Unit = 128;
__host__ __device__ constexpr int i4_unit_bytes(int group) {
  return kI4Unit * 16 / 2 + (kI4Unit / group) * 32;
}

// Slices of n K units over the consumer warps: the first n % kFewWarps warps hold one more.
struct KSplit {
  int n;   // units of the tile's K range
  int cw;  // warps that share one ring slot (a "chunk" of the tile)
  __host__ __device__ int start(int w) const {
    if (w > kFewWarps) w = kFewWarps;
    const int q = n / kFewWarps, r = n % kFewWarps;
    return w * q + (w < r ? w : r);
  }
  __host__ __device__ int count(int w) const { return start(w + 1) - start(w); }
  __host__ __device__ int chunks() const { return (kFewWarps + cw - 1) / cw; }
};

// Ring bytes of a BF16 chunk of u units: 16 rows at a stride of 64 bytes modulo 128, so that the
// eight rows of a fragment load fall into different banks.
__host__ __device__ constexpr int bf16_row_stride(int u) { return u * 64 + ((u & 1) ? 0 : 64); }

// Bytes of the largest chunk.
inline int chunk_bytes(const KSplit& s, int unit_bytes_i4 /* 0: BF16 */) {
  int most = 0;
  for (int w = 0; w < kFewWarps; w += s.cw) {
    const int u = s.start(w + s.cw) - s.start(w);
    if (u > most) most = u;
  }
  return unit_bytes_i4 ? most * unit_bytes_i4 : 16 * bf16_row_stride(most);
}

// The fewest chunks a tile that fit in a ring slot.
inline KSplit make_ksplit(int units, int slot_bytes, int unit_bytes_i4) {
  KSplit s{units, kFewWarps};
  while (s.cw > 1 && chunk_bytes(s, unit_bytes_i4) > slot_bytes) s.cw = (s.cw + 1) / 2;
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
  const void* x;           // [T, K], BF16, or FP32 with wide
  const uint8_t* w;        // packed [tiles, K / 128, superblock]
  void* out;               // [T, N] (SwiGLU: FP32 [T, N / 2])
  uint64_t wait_limit_ns;
  int T, N, K, tiles;
  int out_kind;            // Int4Out
  int wide;                // T <= 8
  int cluster;             // CTAs that split K
  int recv;                // receive buffers of partial tiles (cluster > 1)
  int cw;                  // KSplit::cw of the largest K range
  int stages, slot_bytes, stage_bytes;  // the last: of a warp's token buffer
};

// In the status region of a workspace whose last forward was a few-token one: it has the experts' counts
// where every workspace does, and no slot rows.  (Other forwards clear the region.)
constexpr int kFewMarkWord = 8;
constexpr uint32_t kFewMark = 0x77656600u;

struct FewRouterArgs {
  const __nv_bfloat16* h;  // [T, d]
  const float* W;          // [E, d]
  const float* bias;       // [E]
  float2* sc;              // [T, E] out: score, biased score
  uint32_t* status;        // cleared (4 words), and marked
  uint4* unwritten;        // what the layer kernel exchanges, set to all ones
  int64_t unwritten_n;     // in 16-byte units
  uint64_t wait_limit_ns;
  int T, d, E;
};

struct FewLayerArgs {
  const __nv_bfloat16* h;  // [T, d]
  const float2* sc;        // [T, E]
  const void* w_gate;      // BF16 [E, I, d], or packed gate|up
  const void* w_up;        // BF16 [E, I, d], or null
  const void* w_down;      // BF16 [E, d, I], or packed
  float* act;              // [T * k, I], all ones on entry
  float* y;                // [T * k, d], all ones on entry
  __nv_bfloat16* out;      // [T, d]
  int32_t* idx;            // [T, k] out, or null
  float* wts;              // [T, k] out, or null
  int32_t* cnt;            // [E] out, tokens of each expert
  uint32_t* status;
  uint64_t wait_limit_ns;
  KSplit k1, k2;           // gate/up and down K slices
  int T, d, E, G, Gk, k, I;
  float scale;
  int norm;
  int entry_max;           // tokens of an entry at most
  int room;                // a warp's buffer holds all BF16 pieces of an activation row
  int stages, slot_bytes, stage_bytes;  // the last: of a warp's token buffer
};

cudaError_t launch_int4_quantize(const Int4QuantArgs& a, cudaStream_t s);
cudaError_t launch_int4_linear(Int4LinearArgs a, int group, int sms, cudaStream_t s);
cudaError_t launch_few_router(const FewRouterArgs& a, cudaStream_t s);
int few_router_tokens(int d);  // of one launch_few_router at most
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

// The part of a wait that finds its phase open: the hardware parks the thread between checks
// (a waiting warp that polls takes issue slots from the warps it waits for).  A limit of 0 gives
// up at once (a try_wait may park the thread long enough to miss the open phase).
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            uint64_t limit_ns, uint32_t* status, uint32_t where) {
  if (limit_ns != 0) {
    // the timer is read once a wait is long: reading it takes longer than most waits
#pragma unroll 1
    for (int it = 0; it < 16; ++it)
      if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!*abort_flag && globaltimer_ns() - t0 <= limit_ns) {
      if (mbar_try_wait_hint(bar, parity, 4000u)) return true;
    }
  }
  if (!*abort_flag) {
    *abort_flag = 1;
    record_status(status, kDevTimeout, where);
  }
  return false;
}

// Bounded wait of a whole warp; every lane polls (each must see the phase complete before it reads
// what the barrier guards).  False on all lanes when any lane gave up.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, uint64_t limit_ns,
                                               uint32_t* status, uint32_t where) {
  bool ok = mbar_test_wait(bar, parity);
  if (!ok) ok = mbar_wait_slow(bar, parity, abort_flag, limit_ns, status, where);
  return __all_sync(0xffffffffu, ok);
}

// The same, where `seen` is an earlier mbar_test_wait of the phase by each lane.  A test takes about 100
// clocks to answer; asked before the work that precedes the wait, it costs none.
__device__ __forceinline__ bool mbar_wait_seen(bool seen, uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, uint64_t limit_ns,
                                               uint32_t* status, uint32_t where) {
  if (__all_sync(0xffffffffu, seen)) return true;
  return mbar_wait_warp(bar, parity, abort_flag, limit_ns, status, where);
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
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 v = lds128(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ void sts128(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// D (16 x 8, FP32) += A (16 x 16, BF16) * B (16 x 8, BF16).
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with D = A * B.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D (16 x 8, INT32) += A (16 x 32, INT8) * B (32 x 8, INT8).
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with D = c + A * B.
__device__ __forceinline__ void mma_s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, int c) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c));
}

// The MMA sums over k in any order as long as both operands agree: in each run of 32 elements
// lane column c owns elements 8 c .. 8 c + 7 (one 16-byte load of BF16); a BF16 run is two MMAs,
// the first with the first four of each column, an INT8 run is one.

// ---- reading token rows

__device__ __forceinline__ uint4 ld_relaxed(const void* p) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
constexpr float kInfinity = __builtin_huge_valf();

// FP32 rows that other CTAs of the kernel are writing.  Every element was set to kUnwritten32 (a NaN that
// no computation produces) before the kernel, so an element tells by itself whether it is there:
// no flag has to follow the data through a fence and an atomic, which take 2 us together.
constexpr uint32_t kUnwritten32 = 0xffffffffu;
__device__ __forceinline__ bool has_unwritten32(uint4 v) {
  return max(max(v.x, v.y), max(v.z, v.w)) == kUnwritten32;
}

struct TokenSource {
  bool polled = false;  // whether others may still be writing the rows
  volatile int* abort_flag = nullptr;
  uint64_t limit_ns = 0;
  uint32_t* status = nullptr;
  uint32_t where = 0;
  bool ok = true;
  uint32_t looks = 0;
  // Whether to look again; gives up after limit_ns, or when another wait did.  The timer and the status
  // are read every eighth time: that takes as long as a look.
  __device__ bool again(uint64_t& t0) {
    if (looks++ % 8 && limit_ns) return ok;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    uint32_t other;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(other) : "l"(status) : "memory");
    if (*abort_flag || other || now - t0 >= limit_ns) {
      if (!*abort_flag) {
        *abort_flag = 1;
        if (!other) record_status(status, kDevTimeout, where);
      }
      ok = false;
    }
    return ok;
  }
};

// The K slice of a token row is brought in by the whole warp, 16 bytes a lane and load, and staged in
// shared memory, from where each lane picks its fragments.  Everything that runs once per entry
// is kept short and in loops: code that is not in the instruction cache costs about 10 ns an
// instruction, more than its execution.
//
// Rows are BF16, or (wide) FP32: the activations between an expert's two products.  Rounding those to
// BF16 would add an error as large as the rounding of the output.  One copy of the code for both: with
// two, fragments were moved between the registers of either.
constexpr int kRowLoads = kFewMaxK / kFewWarps / 128;
__device__ __forceinline__ void fetch_row(uint4 (&v)[kRowLoads], const void* row, int bytes, int lane) {
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    if (row != nullptr && (i * 32 + lane) * 16 < bytes)
      v[i] = ld_relaxed(static_cast<const uint4*>(row) + i * 32 + lane);
  }
}
// Waits until what fetch_row brought is there; all loads of the row at a time, one round trip.
__device__ __forceinline__ void settle_row(uint4 (&v)[kRowLoads], TokenSource& src, const void* row, int bytes,
                                           int lane) {
  if (!src.polled) return;
  uint64_t t0 = 0;
#pragma unroll 1
  while (true) {
    bool missing = false;
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i)
      missing |= (i * 32 + lane) * 16 < bytes && has_unwritten32(v[i]);
    if (!missing || !src.ok || !src.again(t0)) return;
    fetch_row(v, row, bytes, lane);
  }
}
// Stages a row; returns the largest magnitude bits of the lane's elements, as FP32 (NaN and infinity are
// the largest).
__device__ __forceinline__ uint32_t stage_row(const uint4 (&v)[kRowLoads], bool wide, int bytes, uint8_t* raw,
                                              int lane) {
  uint32_t top = 0;
  const uint32_t mask = wide ? 0x7fffffffu : 0x7fff7fffu;
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    if ((i * 32 + lane) * 16 < bytes) {
      *reinterpret_cast<uint4*>(raw + (i * 32 + lane) * 16) = v[i];
      const uint32_t x = v[i].x & mask, y = v[i].y & mask, z = v[i].z & mask, w = v[i].w & mask;
      if (wide) {
        top = max(top, max(max(x, y), max(z, w)));
      } else {  // magnitudes, two at a time
        const uint32_t m = __vmaxu2(__vmaxu2(x, y), __vmaxu2(z, w));
        top = max(top, max(m << 16, m & 0xffff0000u));
      }
    }
  }
  return top;
}
// Stages the three BF16 pieces of an FP32 row of n elements, each n elements behind the one before; without
// room for the third, keeps it in v's first two words.  Each piece is the rest's rounding to BF16, 8 bits and a sign,
// so that the three hold all 24 bits of an element of at least 2^-110 (smaller ones lose what lies below
// BF16's smallest step, 2^-133); beyond BF16's range the others are zero.
__device__ __forceinline__ void stage_pieces(uint4 (&v)[kRowLoads], int n, bool room, uint8_t* raw, int lane) {
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    if (i * 128 >= n) break;
    const int k = (i * 32 + lane) * 4;
    if (k < n) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t p[3][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = __uint_as_float(w[j * 2]), y = __uint_as_float(w[j * 2 + 1]);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
          p[q][j] = *reinterpret_cast<const uint32_t*>(&h);
          const float hx = bf16_lo(p[q][j]), hy = bf16_hi(p[q][j]);
          x = fabsf(hx) < kInfinity ? x - hx : 0.f;  // exact
          y = fabsf(hy) < kInfinity ? y - hy : 0.f;
        }
      }
      *reinterpret_cast<uint2*>(raw + k * 2) = make_uint2(p[0][0], p[0][1]);
      *reinterpret_cast<uint2*>(raw + (n + k) * 2) = make_uint2(p[1][0], p[1][1]);
      if (room) *reinterpret_cast<uint2*>(raw + (2 * n + k) * 2) = make_uint2(p[2][0], p[2][1]);
      v[i].x = p[2][0];
      v[i].y = p[2][1];
    }
  }
}
__device__ __forceinline__ void stage_third(const uint4 (&v)[kRowLoads], int n, uint8_t* raw, int lane) {
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    if (i * 128 >= n) break;
    const int k = (i * 32 + lane) * 4;
    if (k < n) *reinterpret_cast<uint2*>(raw + k * 2) = make_uint2(v[i].x, v[i].y);
  }
}

// B fragments of the K slices of tokens, n elements each, 4 registers per 32 elements and set of 8 columns.
//   BF16 rows         one set, column t is token t, up to 8
//   FP32 rows (wide)  column 2 p + t % 2 of set t / 2 is piece p of token t; one set for up to 2 tokens,
//                     for up to 4 a second one whose registers are those of runs RUNS / 2 and on
// row(t): the slice's first element of token t, or null (columns of zeros).  room: whether the buffer holds
// all pieces of a row.
template <int RUNS, int REGS, class Row>
__device__ __forceinline__ void load_tokens(uint32_t (&b)[REGS], TokenSource& src, Row row, bool wide, bool room,
                                            int tokens, int n, uint8_t* raw, const uint8_t* zeros, int lane) {
  static_assert(RUNS * 4 <= REGS, "the fragments must fit");
  const int g = lane >> 2, c = lane & 3, bytes = n * (wide ? 4 : 2);
  const bool two = wide && tokens > 2;
  const int passes = wide && !room ? 2 : 1;
  uint4 v[kRowLoads];
  const void* next = row(0);
  fetch_row(v, next, bytes, lane);
#pragma unroll 1
  for (int t = 0; t < tokens; ++t) {
    const void* from = next;
    if (from != nullptr) settle_row(v, src, from, bytes, lane);
    // without room two of the pieces, then in their place the third
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
      if (from != nullptr) {
        if (pass)
          stage_third(v, n, raw, lane);
        else if (wide)
          stage_pieces(v, n, room, raw, lane);
        else
          stage_row(v, false, bytes, raw, lane);
      }
      __syncwarp();
      if (pass + 1 == passes) {
        next = t + 1 < tokens ? row(t + 1) : nullptr;
        fetch_row(v, next, bytes, lane);
      }
      const int piece = g >> 1;
      const bool mine = from != nullptr && (wide ? (g & 1) == (t & 1) && (pass ? piece == 2 : piece < 4 - passes) : g == t);
      const bool clear = t == 0 && pass == 0;  // the first token also clears the other columns
      if (mine || clear) {
        const uint8_t* p = mine ? raw + (wide && !pass ? piece * n * 2 : 0) + c * 16 : zeros;
        const int step = mine ? 64 : 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // two sets: half of the registers each
          const bool other = two && half != t >> 1;  // not the token's set
          const int left = two ? (!other || clear ? n : 0) : n - half * (RUNS / 2) * 32;
          const int first = two ? 0 : half * (RUNS / 2) * step, each = other ? 0 : step;
          const uint8_t* from_half = other ? zeros : p + first;
#pragma unroll
          for (int j = 0; j < RUNS / 2; ++j) {
            if (j * 32 >= left) break;
            const uint4 w = *reinterpret_cast<const uint4*>(from_half + j * each);
            uint32_t* f = b + (half * (RUNS / 2) + j) * 4;
            f[0] = w.x;
            f[1] = w.y;
            f[2] = w.z;
            f[3] = w.w;
          }
        }
      }
      __syncwarp();
    }
  }
}

// acc[s] += 16 BF16 weight rows (`base`: row 0 of the warp's slice, rows `stride` bytes apart) times
// set s of token columns, over `runs` runs of 32 K elements.  The registers of set s begin at those of run
// s RUNS.
template <int RUNS, int SETS, int REGS>
__device__ __forceinline__ void bf16_slice(float (&acc)[SETS][4], const uint32_t (&b)[REGS],
                                           uint32_t base, int stride, int runs, int lane) {
  static_assert(SETS * RUNS * 4 <= REGS, "the fragments must fit");
  const uint32_t lo = base + (lane >> 2) * stride + (lane & 3) * 16;
  const uint32_t hi = lo + 8 * stride;
  float d0[SETS][4] = {}, d1[SETS][4] = {};  // chains of dependent MMAs
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
    if (j < runs) {
      const uint4 r = lds128(lo + j * 64), s = lds128(hi + j * 64);
#pragma unroll
      for (int q = 0; q < SETS; ++q) {
        const uint32_t* f = b + (q * RUNS + j) * 4;
        mma_bf16(d0[q], r.x, s.x, r.y, s.y, f[0], f[1]);
        mma_bf16(d1[q], r.z, s.z, r.w, s.w, f[2], f[3]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < SETS; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[q][i] += d0[q][i] + d1[q][i];
}

// Sum over the three pieces of each token: on every lane, what columns 0 and 1 of the result hold.  The
// columns behind the third piece are zero.
__device__ __forceinline__ float4 sum_pieces(float4 v) {
  float* o = &v.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);  // third piece to the first, zeros to the second
    o[i] += __shfl_xor_sync(0xffffffffu, o[i], 1);
  }
  return v;
}

// Products with 4-bit weights run on INT8 MMAs for up to 8 tokens.  A code block of 16 rows x 64
// columns takes 22 clocks of an SM to arrive (528 bytes at 6.5 TB/s over the GPU), and expanding it
// to BF16 for m16n8k16 measured 20 whatever the number of warps: 28 shifts and masks, 16
// subtractions and 4 MMAs of 2 clocks.  As 8-bit operands the codes take 12 shifts and masks and 2
// MMAs of 4 clocks for each 8 columns of tokens, 9 clocks in all.  (E4M3 MMAs would take the codes
// as they lie, but mma.sync expands E4M3 operands with ALU operations: 18.5 clocks.)
//
// The token is a 23-bit integer per element, in three signed 8-bit digits:
//   x = 2^(E - 21) (65536 d0 + 256 d1 + d2),  2^E <= largest of the warp's K slice < 2^(E + 1)
// which is x exactly for every element within 2^-14 of the slice's largest, and off by at most
// 2^-22 of the largest otherwise -- a quarter step of FP32 in the sum that holds it.  (FP32 activations
// lose up to two bits by it: of a layer's BF16 outputs 7 in 10,000 then differ from the correctly rounded
// ones, with exact activations 3, and the error to three digits does not.)  The digits of a token are columns of their own, in one of three arrangements by the number of tokens (MODE = MMAs
// per run of 32):
//   MODE 1, up to 2 tokens: column 2 p + t holds digit p of token t
//   MODE 2, up to 4: of the first MMA column 4 p + t, p = 0, 1; of the second column t digit 2
//   MODE 3, up to 8: MMA p, column t
// Integer sums are exact.  A group's sum (|16 q d| <= 2^14, at most 128 of them) starts at the bit
// pattern of 1.5 2^23, so that it is read as a float without a conversion.
constexpr int kI4SumStart = 0x4b400000;
constexpr float kI4SumStartF = 12582912.f;
// A warp's buffer for one token of n elements: the row, and for 4-bit weights three bytes of digits.
__host__ __device__ constexpr int stage_bytes(int n, bool i4, bool wide) {
  return n * ((wide ? 4 : 2) + (i4 ? 3 : 0));
}
constexpr int kI4NonFinite = 1 << 20;           // in the place of an exponent

// Runs of 32 of a warp's K slice at most: 64, 80 or 120 registers of fragments.
__host__ __device__ constexpr int i4_mode_runs(int mode) { return mode == 1 ? 32 : 20; }
__host__ __device__ constexpr int i4_mode_regs(int mode) { return i4_mode_runs(mode) * 2 * mode; }

__host__ __device__ constexpr int i4_mode(int tokens) { return tokens <= 2 ? 1 : tokens <= 4 ? 2 : 3; }

// E of a K slice from its largest magnitude's FP32 bits, at least -105 (2^(21 - E) has to be a normal
// number; smaller tokens keep an absolute accuracy of 2^-127), and 2^(21 - E).
struct I4Scale {
  int E;
  float f;
};
__device__ __forceinline__ I4Scale i4_scale(uint32_t top) {
  const int E = max(static_cast<int>(top >> 23) - 127, -105);
  return {E, __uint_as_float(static_cast<uint32_t>(127 + 21 - E) << 23)};
}
// Digits of 4 elements, a byte each: d[p] holds digit p.  The addition of 1.5 2^23 rounds x 2^(21 - E) to
// an integer i, and leaves it in the low bits; the bytes of i + 0x808080 are the balanced digits plus 128.
__device__ __forceinline__ void i4_digits(uint32_t (&d)[3], const float (&e)[4], float f) {
  uint32_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = __float_as_uint(fmaf(e[j], f, kI4SumStartF)) + 0x00408080u;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t at = 0x0040u + 0x0011u * (2 - p);  // byte 2 - p of both
    d[p] = __byte_perm(__byte_perm(x[0], x[1], at), __byte_perm(x[2], x[3], at), 0x5410) ^ 0x80808080u;
  }
}
// The same of two words of BF16 pairs.
__device__ __forceinline__ void i4_digits(uint32_t (&d)[3], uint32_t w0, uint32_t w1, float f) {
  const float e[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
  i4_digits(d, e, f);
}
__device__ __forceinline__ void i4_digits(uint32_t (&d)[3], uint4 w, float f) {  // four FP32
  const float e[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
  i4_digits(d, e, f);
}
// Splits a staged slice (n elements, a multiple of 128) into its digits, n bytes each.
__device__ __forceinline__ void i4_split(const uint8_t* raw, bool wide, uint8_t* digits, int n, float f,
                                         int lane) {
#pragma unroll 1
  for (int k = lane * 4; k < n; k += 128) {
    uint4 w;  // as FP32
    if (wide) {
      w = *reinterpret_cast<const uint4*>(raw + k * 4);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(raw + k * 2);
      w = make_uint4(u.x << 16, u.x & 0xffff0000u, u.y << 16, u.y & 0xffff0000u);
    }
    uint32_t d[3];
    i4_digits(d, w, f);
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<uint32_t*>(digits + p * n + k) = d[p];
  }
}

// What a token's products have to be multiplied with, 2^(E - 9) for sums in units of digit 0 (codes
// count 16 times), in two factors (2^(E - 9) may be out of range); NaN for a non-finite token.
struct I4Factor {
  float a, b;
};
__device__ __forceinline__ I4Factor i4_factor(int E) {
  if (E >= kI4NonFinite / 2) return {__uint_as_float(0x7fc00000u), 1.f};
  const int r = E - 9;
  return {__uint_as_float(static_cast<uint32_t>(127 + r / 2) << 23),
          __uint_as_float(static_cast<uint32_t>(127 + r - r / 2) << 23)};
}

// B fragments of a warp's K slice (`units` superblocks) of `tokens` tokens, 2 MODE registers a run;
// row(t): the slice's first element of token t (BF16, or FP32 with wide), or null.  factor[h]: of the
// token of the lane's result column h.
//
// MODE 1 and 2 split a token at a time with the whole warp, through shared memory: a lane's share of the
// work is 1/32 of the slice, the code is short, and few registers are held beside the fragments.  At 8
// tokens that takes 13 us: with MODE 3 each lane converts the elements of its own column's token, in the
// registers that take the digits.
template <int MODE, int REGS, class Row>
__device__ __forceinline__ void i4_load_tokens(uint32_t (&b)[REGS], I4Factor (&factor)[2], TokenSource& src,
                                               Row row, bool wide, int tokens, int units, uint8_t* raw,
                                               const uint8_t* zeros, int lane) {
  constexpr int kRuns = i4_mode_runs(MODE);
  static_assert(kRuns * 2 * MODE <= REGS, "the fragments must fit");
  const int g = lane >> 2, c = lane & 3, n = units * kI4Unit;
  const int first = MODE == 1 ? 0 : MODE == 2 ? 2 * (c & 1) : 2 * c;  // token of the lane's result column 0
  int E[2] = {0, 0};
  if constexpr (MODE < 3) {
    const int bytes = n * (wide ? 4 : 2);
    uint8_t* const digits = raw + bytes;
    const int token = MODE == 1 ? (g < 6 ? g & 1 : -1) : g & 3;  // of B column g
    uint4 v[kRowLoads];
    const void* next = row(0);
    fetch_row(v, next, bytes, lane);
#pragma unroll 1
    for (int t = 0; t < tokens; ++t) {
      const void* from = next;
      uint32_t top = 0;
      if (from != nullptr) {
        settle_row(v, src, from, bytes, lane);
        top = stage_row(v, wide, bytes, raw, lane);
      }
      __syncwarp();
      top = __reduce_max_sync(0xffffffffu, top);
      next = t + 1 < tokens ? row(t + 1) : nullptr;
      fetch_row(v, next, bytes, lane);
      const I4Scale s = i4_scale(top);
      if (from != nullptr) i4_split(raw, wide, digits, n, s.f, lane);
      __syncwarp();
      const int e = top >= 0x7f800000u ? kI4NonFinite : s.E;
      E[0] = t == first ? e : E[0];
      E[1] = t == first + 1 ? e : E[1];
      const bool mine = token == t && from != nullptr;
      if (mine || t == 0) {  // the first token also clears the other columns
#pragma unroll
        for (int q = 0; q < MODE; ++q) {
          const int digit = MODE == 1 ? g >> 1 : q == 0 ? g >> 2 : 2;  // of column g in MMA q
          const bool any = mine && (q == 0 || g < 4);
          const uint8_t* p = any ? digits + digit * n + c * 8 : zeros;
          const int step = any ? 32 : 0;
#pragma unroll
          for (int j = 0; j < kRuns; ++j) {
            if (j < units * 4) {
              const uint2 w = *reinterpret_cast<const uint2*>(p + j * step);
              b[(j * MODE + q) * 2] = w.x;
              b[(j * MODE + q) * 2 + 1] = w.y;
            }
          }
        }
      }
      __syncwarp();
    }
  } else {
    auto convert = [&](auto is_wide) {
      constexpr bool kWide = decltype(is_wide)::value;
      // a lane's 8 elements of run j; of FP32 rows the second half comes 16 bytes on
      const uint4* p = g < tokens ? reinterpret_cast<const uint4*>(row(g)) + c * (kWide ? 2 : 1) : nullptr;
      auto part = [&](int j, int half) {
        if (p == nullptr || j >= units * 4) return make_uint4(0u, 0u, 0u, 0u);
        return __ldcg(p + j * (kWide ? 8 : 4) + half);
      };
      uint32_t top = 0;
      if constexpr (kWide) {  // read twice: 8 words of a run do not fit where its 6 of digits go
#pragma unroll
        for (int j = 0; j < kRuns * 2; ++j) {
          const uint4 v = part(j / 2, j % 2);
          top = max(top, max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu)));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {  // the elements of a run, where its digits go
          const uint4 v = part(j, 0);
          b[j * 6] = v.x;
          b[j * 6 + 1] = v.y;
          b[j * 6 + 2] = v.z;
          b[j * 6 + 3] = v.w;
        }
        uint32_t w = 0;  // magnitudes, two at a time
#pragma unroll
        for (int j = 0; j < kRuns; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) w = __vmaxu2(w, b[j * 6 + i] & 0x7fff7fffu);
        top = max(w << 16, w & 0xffff0000u);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const I4Scale s = i4_scale(top);
      const int e = top >= 0x7f800000u ? kI4NonFinite : s.E;
      E[0] = __shfl_sync(0xffffffffu, e, first * 4);
      E[1] = __shfl_sync(0xffffffffu, e, first * 4 + 4);
#pragma unroll
      for (int j = 0; j < kRuns; ++j) {
        uint32_t lo[3], hi[3];
        if constexpr (kWide) {
          i4_digits(lo, part(j, 0), s.f);
          i4_digits(hi, part(j, 1), s.f);
        } else {
          i4_digits(lo, b[j * 6], b[j * 6 + 1], s.f);
          i4_digits(hi, b[j * 6 + 2], b[j * 6 + 3], s.f);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          b[j * 6 + q * 2] = lo[q];
          b[j * 6 + q * 2 + 1] = hi[q];
        }
      }
    };
    if (wide)
      convert(std::true_type{});
    else
      convert(std::false_type{});
  }
  factor[0] = i4_factor(E[0]);
  factor[1] = i4_factor(E[1]);
}

// Sums of i4_slice, per MMA of a run.  Digits are kept apart to the end, so that a token's result has
// the same bits in every arrangement (as long as K is cut alike: the linear product of more than 5120
// columns may take fewer CTAs to a tile for up to 2 tokens).
template <int MODE>
struct I4Acc {
  float v[MODE][4] = {};
};

// (a0, a1) += s * ((d0, d1) - kI4SumStartF), each rounded as by single instructions
__device__ __forceinline__ void i4_scale2(float& a0, float& a1, float s, int d0, int d1) {
  constexpr float kNeg = -kI4SumStartF;
  asm("{\n\t.reg .b64 a, s, d, n;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 d, {%3, %4};\n\tmov.b64 n, {%5, %5};\n\t"
      "add.rn.f32x2 d, d, n;\n\tfma.rn.f32x2 a, s, d, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(s), "r"(d0), "r"(d1), "f"(kNeg));
}

// acc[r] += 16 rows of 4-bit weights (`base` + r * apart: the warp's first superblock of tile r) times the
// token digits, over UNITS superblocks.  Each group is summed unscaled; its scale multiplies the sum in
// FP32.
template <int MODE, int GROUP, int UNITS, int R, int REGS>
__device__ __forceinline__ void i4_slice_of(I4Acc<MODE> (&acc)[R], const uint32_t (&b)[REGS], uint32_t base,
                                            uint32_t apart, int lane) {
  constexpr int kUnitBytes = i4_unit_bytes(GROUP);
  constexpr uint32_t kMask = 0xf0f0f0f0u;
  uint32_t codes[R], scales[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    codes[r] = base + r * apart + lane * 16;
    scales[r] = base + r * apart + 1024 + (lane >> 2) * 4;
  }
  int d[R][MODE][4];
  uint4 q[R];
#pragma unroll
  for (int j = 0; j < UNITS * 4; ++j) {  // runs of 32
    const int u = j / 4, run = j % 4;
    constexpr int kRunsPerGroup = GROUP / 32;
    const bool first = j % kRunsPerGroup == 0, last = j % kRunsPerGroup == kRunsPerGroup - 1;
    if (run % 2 == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) q[r] = lds128(codes[r] + u * kUnitBytes + (run / 2) * 512);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t lo = run % 2 ? q[r].z : q[r].x, hi = run % 2 ? q[r].w : q[r].y;
      const uint32_t a0 = lo & kMask, a1 = (lo << 4) & kMask, a2 = hi & kMask, a3 = (hi << 4) & kMask;
#pragma unroll
      for (int nt = 0; nt < MODE; ++nt) {
        const uint32_t b0 = b[(j * MODE + nt) * 2], b1 = b[(j * MODE + nt) * 2 + 1];
        if (first)
          mma_s8_first(d[r][nt], a0, a1, a2, a3, b0, b1, kI4SumStart);
        else
          mma_s8(d[r][nt], a0, a1, a2, a3, b0, b1);
      }
    }
    if (last) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t s = lds32(scales[r] + u * kUnitBytes + (run / kRunsPerGroup) * 32);
#pragma unroll
        for (int nt = 0; nt < MODE; ++nt) {
          float* v = acc[r].v[nt];
          const int* e = d[r][nt];
          i4_scale2(v[0], v[1], bf16_lo(s), e[0], e[1]);
          i4_scale2(v[2], v[3], bf16_hi(s), e[2], e[3]);
        }
      }
    }
  }
}

// One straight run of code for each number of superblocks: with a branch after every superblock
// the loads and products of two of them do not overlap (a fifth slower).
template <int GROUP, int MODE, int R, int REGS>
__device__ __forceinline__ void i4_slice(I4Acc<MODE> (&acc)[R], const uint32_t (&b)[REGS], uint32_t base,
                                         uint32_t apart, int units, int lane) {
  constexpr int kMax = i4_mode_runs(MODE) / 4;
  switch (units) {
    case 1: i4_slice_of<MODE, GROUP, 1>(acc, b, base, apart, lane); break;
    case 2: i4_slice_of<MODE, GROUP, 2>(acc, b, base, apart, lane); break;
    case 3: i4_slice_of<MODE, GROUP, 3>(acc, b, base, apart, lane); break;
    case 4: i4_slice_of<MODE, GROUP, 4>(acc, b, base, apart, lane); break;
    case 5: if constexpr (kMax >= 5) i4_slice_of<MODE, GROUP, 5>(acc, b, base, apart, lane); break;
    case 6: if constexpr (kMax >= 6) i4_slice_of<MODE, GROUP, 6>(acc, b, base, apart, lane); break;
    case 7: if constexpr (kMax >= 7) i4_slice_of<MODE, GROUP, 7>(acc, b, base, apart, lane); break;
    case 8: if constexpr (kMax >= 8) i4_slice_of<MODE, GROUP, 8>(acc, b, base, apart, lane); break;
    default: break;
  }
}

// The warp's partial tile of a slice: rows g, g of tokens 2 c, 2 c + 1, then rows g + 8.  Digits in
// different lanes are added here.
template <int MODE>
__device__ __forceinline__ float4 i4_result(const I4Acc<MODE>& acc, const I4Factor (&factor)[2], int lane) {
  constexpr float k1 = 1.f / 256, k2 = 1.f / 65536;  // digits 1 and 2 in units of digit 0
  const int c = lane & 3;
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (MODE == 1) {  // lanes c hold digit c; lanes 3 zeros
      o[i] = acc.v[0][i] * (c == 0 ? 1.f : c == 1 ? k1 : k2);
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], 1);
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);
    } else if constexpr (MODE == 2) {  // lanes 0, 1 hold digits 0 and 2, lanes 2, 3 digit 1
      o[i] = acc.v[0][i] * (c < 2 ? 1.f : k1);
      o[i] += __shfl_xor_sync(0xffffffffu, o[i], 2);
      o[i] = fmaf(acc.v[1][i], k2, o[i]);
    } else {
      o[i] = fmaf(acc.v[2][i], k2, fmaf(acc.v[1][i], k1, acc.v[0][i]));
    }
    o[i] = o[i] * factor[i & 1].a * factor[i & 1].b;
  }
  return make_float4(o[0], o[1], o[2], o[3]);
}

// ---- 9 to 16 tokens: BF16 MMAs, two sets of 8 columns (six INT8 MMAs of 4 clocks a run are slower:
// 16 x 40960 x 5120 in 55 us, with these 42)

// Two codes (two's complement, bits 0..3 and 16..19 of v) as exact BF16, q 2^-10: with the sign bit
// inverted a code is q + 8, 0x3e00 | (q + 8) is the BF16 value (136 + q) 2^-10.  At 2^-10 a group's unscaled
// sum (128 products with |q| <= 8) is no larger than the largest token element and cannot overflow.
constexpr float kI4PairUnscale = 1024.f;
__device__ __forceinline__ uint32_t i4_pair(uint32_t v) {
  uint32_t u, d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(u) : "r"(v), "r"(0x000f000fu), "r"(0x3e083e08u));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(u), "r"(0x3e083e08u));
  return d;
}

// B fragments, 8 registers a run: per set of 8 tokens, the four registers of load_tokens with the
// elements of each four paired (0, 2), (1, 3) as the codes' bytes are.
template <int RUNS, class Row>
__device__ __forceinline__ void i4_load_tokens16(uint32_t (&b)[RUNS * 8], Row row, int tokens, int units,
                                                 int lane) {
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int t = nt * 8 + (lane >> 2);
    const __nv_bfloat16* p = t < tokens ? row(t) + (lane & 3) * 8 : nullptr;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (p != nullptr && j < units * 4) v = __ldcg(reinterpret_cast<const uint4*>(p + j * 32));
      b[(j * 2 + nt) * 4 + 0] = __byte_perm(v.x, v.y, 0x5410);
      b[(j * 2 + nt) * 4 + 1] = __byte_perm(v.x, v.y, 0x7632);
      b[(j * 2 + nt) * 4 + 2] = __byte_perm(v.z, v.w, 0x5410);
      b[(j * 2 + nt) * 4 + 3] = __byte_perm(v.z, v.w, 0x7632);
    }
  }
}

template <int GROUP, int UNITS, int REGS>
__device__ __forceinline__ void i4_slice16_of(float (&acc)[2][4], const uint32_t (&b)[REGS], uint32_t base, int lane) {
  constexpr int kUnitBytes = i4_unit_bytes(GROUP);
  const uint32_t codes = base + lane * 16, scales = base + 1024 + (lane >> 2) * 4;
  float d[2][4];
  uint4 q;
#pragma unroll
  for (int j = 0; j < UNITS * 4; ++j) {  // runs of 32
    const int u = j / 4, run = j % 4;
    constexpr int kRunsPerGroup = GROUP / 32;
    const bool first = j % kRunsPerGroup == 0, last = j % kRunsPerGroup == kRunsPerGroup - 1;
    if (run % 2 == 0) q = lds128(codes + u * kUnitBytes + (run / 2) * 512);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = run % 2 ? (h ? q.w : q.z) : (h ? q.y : q.x);
      const uint32_t a0 = i4_pair(w >> 4), a1 = i4_pair(w), a2 = i4_pair(w >> 12), a3 = i4_pair(w >> 8);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t b0 = b[(j * 2 + nt) * 4 + h * 2], b1 = b[(j * 2 + nt) * 4 + h * 2 + 1];
        if (first && h == 0)
          mma_bf16_first(d[nt], a0, a1, a2, a3, b0, b1);
        else
          mma_bf16(d[nt], a0, a1, a2, a3, b0, b1);
      }
    }
    if (last) {
      const uint32_t s = lds32(scales + u * kUnitBytes + (run / kRunsPerGroup) * 32);
      const float sc[2] = {bf16_lo(s), bf16_hi(s)};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = fmaf(sc[i >> 1], d[nt][i], acc[nt][i]);
    }
  }
}

// acc[s] += one tile times set s of 8 token columns, in units of 2^-10.
template <int GROUP, int REGS>
__device__ __forceinline__ void i4_slice16(float (&acc)[2][4], const uint32_t (&b)[REGS], uint32_t base, int units,
                                           int lane) {
  static_assert(REGS == 128, "four superblocks");
  switch (units) {
    case 1: i4_slice16_of<GROUP, 1>(acc, b, base, lane); break;
    case 2: i4_slice16_of<GROUP, 2>(acc, b, base, lane); break;
    case 3: i4_slice16_of<GROUP, 3>(acc, b, base, lane); break;
    case 4: i4_slice16_of<GROUP, 4>(acc, b, base, lane); break;
    default: break;
  }
}

// SiLU(g) * u in FP32.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

#endif  // __CUDACC__

}  // namespace beam
