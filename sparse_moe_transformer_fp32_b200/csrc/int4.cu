// 4-bit weights with group scales: conversion of BF16 weights, and y = x W^T for 1 to 16 tokens.
#include "beam_moe_few.cuh"

#include <cstring>

namespace beam {
namespace {

// ------------------------------------------------------------------ conversion

// One warp per superblock (16 output rows x 128 K elements).  s = bf16(amax / 7),
// q = clamp(rne(x / s), -8, 7): lane (g, c) = (lane / 4, lane % 4) reads exactly the elements whose
// codes its 16-byte words hold, so no code moves between lanes; a group's maximum is combined
// over the four lanes that share its rows.  HBM-bound: 2 bytes read and about half a byte written
// per weight, once per model.
__global__ void __launch_bounds__(256) int4_quantize_kernel(const Int4QuantArgs a) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int sbs = a.cols / kI4Unit;
  const int sb = static_cast<int>(unit % sbs);
  const int64_t tile_all = unit / sbs;
  const int tile = static_cast<int>(tile_all % a.tiles);
  const int64_t grp = tile_all / a.tiles;
  // rows of the lane's two fragment rows: 8 of a and 8 of b, or 16 consecutive ones of a
  const __nv_bfloat16* src[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = a.b ? tile * 8 + g : tile * 16 + h * 8 + g;
    const __nv_bfloat16* m = a.b && h ? a.b : a.a;
    src[h] = r < a.rows ? m + (static_cast<size_t>(grp) * a.rows + r) * a.cols +
                              static_cast<size_t>(sb) * kI4Unit + c * 8
                        : nullptr;
  }
  uint4 v[2][4];  // [row half][run of 32]
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[h][j] = src[h] ? __ldg(reinterpret_cast<const uint4*>(src[h] + j * 32))
                       : make_uint4(0u, 0u, 0u, 0u);
  float amax[2][4];  // per run of 32
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      amax[h][j] = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    }
  const int runs = a.group / 32;  // runs of 32 per group: 1, 2 or 4
  if (runs >= 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      amax[h][0] = amax[h][1] = fmaxf(amax[h][0], amax[h][1]);
      amax[h][2] = amax[h][3] = fmaxf(amax[h][2], amax[h][3]);
      if (runs == 4) amax[h][0] = amax[h][1] = amax[h][2] = amax[h][3] = fmaxf(amax[h][0], amax[h][2]);
    }
  }
  uint8_t* dst = a.packed + static_cast<size_t>(unit) * i4_unit_bytes(a.group);
  uint32_t word[8] = {};
  uint32_t scale_bits[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat16 s0 = __float2bfloat16_rn(__fdiv_rn(amax[0][j], 7.f));
    const __nv_bfloat16 s1 = __float2bfloat16_rn(__fdiv_rn(amax[1][j], 7.f));
    scale_bits[j] = static_cast<uint32_t>(__bfloat16_as_ushort(s0)) |
                    (static_cast<uint32_t>(__bfloat16_as_ushort(s1)) << 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s = __bfloat162float(h ? s1 : s0);
      const uint32_t w[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // element k = 32 j + 8 c + i
        const float x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        float q = s > 0.f ? rintf(__fdiv_rn(x, s)) : 0.f;
        q = fminf(fmaxf(q, -8.f), 7.f);
        const uint32_t n = static_cast<uint32_t>(static_cast<int>(q)) & 15u;
        word[j * 2 + (i >> 2)] |= n << (8 * (i & 3) + (h ? 0 : 4));
      }
    }
  }
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(word[0], word[1], word[2], word[3]);
  reinterpret_cast<uint4*>(dst + 512)[lane] = make_uint4(word[4], word[5], word[6], word[7]);
  if (c == 0) {
    uint32_t* sc = reinterpret_cast<uint32_t*>(dst + 1024);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j % runs == 0) sc[(j / runs) * 8 + g] = scale_bits[j];
  }
}

// ------------------------------------------------------------------ linear product

constexpr int kLinRecv = 8;             // receive buffers for a tile's partial results, at most
constexpr int kLinRecvBytes = 16384;    // all of them
constexpr int kLinMaxCluster = 8;
constexpr int kLinSlotBytes = 46080;  // ring slot: a tile of K = 5120, any group

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 16 bytes into another CTA's shared memory, counted by the mbarrier `bar` there.
__device__ __forceinline__ void remote_store(uint32_t a, float4 v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
      "r"(__float_as_uint(v.w)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of a warp for another CTA of the cluster.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             uint64_t limit_ns) {
  bool ok = mbar_try_wait_cluster(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!(ok = mbar_try_wait_cluster(bar, parity))) {
      if (*abort_flag) break;
      if (globaltimer_ns() - t0 > limit_ns) {
        *abort_flag = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// y = x W^T; MODE 1, 2, 3: up to 2, 4, 8 tokens on INT8 MMAs, 4: up to 16 on BF16 MMAs.  A tile is 16
// rows of W; a cluster of C CTAs shares a tile, each taking a K range, and the CTA whose turn it is
// (tile index mod C) receives the partial tiles of all in its shared memory and adds them in rank order.
// One warp sends and another receives, several tiles apart: with one warp for both a tile took the
// exchange's 1.5 us.  C > 1 is for matrices with few tiles (the spread over 148 SMs would be uneven) and
// for K ranges whose token fragments do not fit in registers.
//
// Bound by HBM, N K (1/2 + 2 / group) bytes, for up to 4 tokens (1 x 151936 x 5120, groups of 128: 62 us,
// 6.5 TB/s).  From 5 tokens on by the consumers: at 8 the three MMAs of a run alone take the time in which
// its weights arrive (86 us), at 16 the expansion to BF16 and the waits between (139 us).
//
// Launched with programmatic stream serialisation, so that barriers are set up while the kernel before
// drains.  Every warp that reads or writes global memory, the producer too, does so after
// griddepcontrol.wait: whatever ran before may have let its successor start early and still be writing
// these weights, and an ended kernel's writes are only sure to be seen after the wait.  (Weights copied
// ahead of it gained nothing but on a second product of 55 MB, 1.2 us of 33.)  Since every CTA waits, the end
// of a product is the end of all before it.

// Superblocks per warp at most: 64 to 128 registers of token fragments.
__host__ __device__ constexpr int lin_units(int mode) { return mode == 4 ? 4 : i4_mode_runs(mode) / 4; }
__host__ __device__ constexpr int lin_sets(int mode) { return mode == 4 ? 2 : 1; }  // of 8 tokens

// Buffers of the partial tiles of a step: a finishing warp has to have seen a buffer's last phase, or a
// later tile's, when it waits; three of them in turn, so that the tile before is two steps back at most.
__host__ __device__ constexpr int lin_red(int step) { return 4 / step; }
// Tiles of a CTA from which on a step is two tiles, for up to 4 tokens: half the waits, but twice the code
// to fetch for a first tile (1 x 1280 x 2560 with one tile to a CTA: 3.5 us, with steps of two 4.0; 1 x 40960
// x 5120 with 18: 21.3 and 20.2; 4 x 40960 x 5120: 27.8 and 25.7).  Beyond 4 tokens the products of a tile
// take longer than the waits, and two at a time nothing off.
constexpr int kLinStepTiles = 4;

template <int MODE, int GROUP, int STEP>
__global__ void __launch_bounds__(kFewThreads, 1) int4_linear_kernel(const Int4LinearArgs a) {
  constexpr int kUnits = lin_units(MODE);
  constexpr int kSets = lin_sets(MODE);
  constexpr int kUnitBytes = i4_unit_bytes(GROUP);
  constexpr int kRedBytes = 512 * kSets;   // one partial tile
  constexpr int kRed = lin_red(STEP);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kFewMaxStages], empty_bar[kFewMaxStages];
  __shared__ __align__(8) uint64_t red_full[kRed], red_empty[kRed];
  __shared__ __align__(8) uint64_t recv_full[kLinRecv], recv_free[kLinMaxCluster][kLinRecv];
  __shared__ int abort_sh;
  __shared__ __align__(16) uint8_t zeros_sh[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t C = a.cluster, rank = C > 1 ? cluster_rank() : 0;
  const uint32_t ring = smem_u32(smem);
  const uint32_t red = ring + a.stages * a.slot_bytes;
  const uint32_t recv = red + kRed * kFewWarps * STEP * kRedBytes;
  [[maybe_unused]] uint8_t* const split = smem + a.stages * a.slot_bytes + kRed * kFewWarps * STEP * kRedBytes +
                         (a.cluster > 1 ? a.recv * a.cluster * kRedBytes : 0) + (threadIdx.x >> 5) * a.stage_bytes;
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), kFewWarps);
    }
    for (int i = 0; i < kRed; ++i) {
      mbar_init(smem_u32(&red_full[i]), kFewWarps);
      mbar_init(smem_u32(&red_empty[i]), STEP);
    }
    for (int i = 0; i < kLinRecv; ++i) {
      mbar_init(smem_u32(&recv_full[i]), 2);  // the receiver, and this CTA's own part
      for (int r = 0; r < kLinMaxCluster; ++r) mbar_init(smem_u32(&recv_free[r][i]), 1);
    }
    abort_sh = 0;
    *reinterpret_cast<uint4*>(zeros_sh) = make_uint4(0u, 0u, 0u, 0u);
    fence_mbarrier_init();
  }
  pdl_launch();
  if (C > 1)
    cluster_sync_all();
  else
    __syncthreads();

  const int nclus = gridDim.x / C, q = blockIdx.x / C;
  const int tile0 = static_cast<int>(static_cast<int64_t>(q) * a.tiles / nclus);
  const int tile1 = static_cast<int>(static_cast<int64_t>(q + 1) * a.tiles / nclus);
  const int units_all = a.K / kI4Unit;
  const int u0 = rank * units_all / C, u1 = (rank + 1) * units_all / C;
  // the chunk size is chosen on the host for the largest K range
  const KSplit ks{u1 - u0, a.cw};

  if (warp < kFewWarps) {
    more_registers<kFewRegsConsumer>();
    // ---- consumers
    const int units = ks.count(warp), mine = warp / ks.cw, chunks = ks.chunks();
    const int cstart = ks.start(mine * ks.cw);
    const uint32_t off = (ks.start(warp) - cstart) * kUnitBytes;
    [[maybe_unused]] const uint32_t apart = (ks.start((mine + 1) * ks.cw) - cstart) * kUnitBytes;  // tiles in a slot
    uint32_t b[kUnits * 8 * MODE];
    [[maybe_unused]] I4Factor factor[2];
    pdl_wait();
    const size_t k0 = static_cast<size_t>(u0 + ks.start(warp)) * kI4Unit;
    auto row = [&](int t) -> const void* {
      const size_t k = static_cast<size_t>(t) * a.K + k0;
      return static_cast<const uint8_t*>(a.x) + (a.wide ? k * 4 : k * 2);
    };
    [[maybe_unused]] TokenSource src;
    if constexpr (MODE == 4)
      i4_load_tokens16<kUnits * 4>(
          b, [&](int t) { return static_cast<const __nv_bfloat16*>(a.x) + static_cast<size_t>(t) * a.K + k0; },
          a.T, units, lane);
    else
      i4_load_tokens<MODE>(b, factor, src, row, a.wide, a.T, units, split, zeros_sh, lane);
    int slot = 0, rb = 0;
    uint32_t par = 0, rpar = 1;
    bool ok = true;
    bool seen = false;  // of the current slot's phase
    for (int tile = tile0; tile < tile1; tile += STEP) {
      float4 part[STEP * kSets] = {};
      bool red_seen = false;
      // every warp passes every chunk in order: a phase may only be waited for by who has seen the
      // slot's phase before
#pragma unroll 1
      for (int ch = 0; ch < chunks; ++ch) {
        ok = mbar_wait_seen(seen, smem_u32(&full_bar[slot]), par, abort_flag, a.wait_limit_ns, nullptr, 0);
        if (!ok) break;
        const int next = slot + 1 == a.stages ? 0 : slot + 1;
        if (next == 0) par ^= 1;
        // Steps of two tiles: the tests of barriers come after the slice's loads from shared memory, which
        // wait for the answer of a test ahead of them.  With one tile that is 4 % slower.
        auto test = [&] {
          seen = mbar_test_wait(smem_u32(&full_bar[next]), par);
          if (ch + 1 == chunks) red_seen = mbar_test_wait(smem_u32(&red_empty[rb]), rpar);
        };
        if (STEP == 1 || ch != mine) test();
        if (ch == mine) {
          // Every tile of a step is multiplied even where the last step has fewer: the others are then
          // what the slot held before, and their sums are not stored.
          const uint32_t base = ring + slot * a.slot_bytes + off;
          if constexpr (MODE == 4) {
            static_assert(MODE < 4 || STEP == 1, "one tile to a step");
            float acc[2][4] = {};
            i4_slice16<GROUP>(acc, b, base, units, lane);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* v = acc[i];
              part[i] = make_float4(v[0] * kI4PairUnscale, v[1] * kI4PairUnscale, v[2] * kI4PairUnscale,
                                    v[3] * kI4PairUnscale);
            }
          } else {
            I4Acc<MODE> acc[STEP] = {};
            i4_slice<GROUP>(acc, b, base, apart, units, lane);
            if (STEP > 1) test();
#pragma unroll
            for (int r = 0; r < STEP; ++r) part[r] = i4_result(acc[r], factor, lane);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty_bar[slot]));
        slot = next;
      }
      if (!ok) break;
      if (!mbar_wait_seen(red_seen, smem_u32(&red_empty[rb]), rpar, abort_flag, a.wait_limit_ns, nullptr, 0))
        break;
      if (units > 0) {
#pragma unroll
        for (int i = 0; i < STEP * kSets; ++i)
          sts128(red + (rb * kFewWarps + warp) * STEP * kRedBytes + i * 512 + lane * 16, part[i]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&red_full[rb]));
      if (++rb == kRed) {
        rb = 0;
        rpar ^= 1;
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
    pdl_wait();
    for (int tile = tile0; tile < tile1 && ok; tile += STEP) {
      const int len = tile1 - tile < STEP ? tile1 - tile : STEP;
      const uint8_t* src = a.w + (static_cast<size_t>(tile) * units_all + u0) * kUnitBytes;
      for (int w = 0; w < kFewWarps; w += ks.cw) {
        ok = mbar_wait_warp(smem_u32(&empty_bar[slot]), par, abort_flag, a.wait_limit_ns, nullptr, 0);
        if (!ok) break;
        const int s = ks.start(w), n = ks.start(w + ks.cw) - s;
        const uint32_t bar = smem_u32(&full_bar[slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, len * n * kUnitBytes);
        __syncwarp();
        if (lane < len)  // lane r copies the chunk of tile r
          bulk_load(ring + slot * a.slot_bytes + lane * n * kUnitBytes,
                    src + static_cast<size_t>(lane * units_all + s) * kUnitBytes, n * kUnitBytes, bar);
        ++issued;
        if (++slot == a.stages) {
          slot = 0;
          par ^= 1;
        }
      }
    }
    if (!ok) {  // copies in flight must land before this CTA's shared memory is given up
      volatile int never = 0;
      const uint32_t back = issued < static_cast<uint32_t>(a.stages) ? issued : a.stages;
      for (uint32_t i = issued - back; i < issued; ++i)
        mbar_wait_bounded(smem_u32(&full_bar[i % a.stages]), (i / a.stages) & 1, &never,
                          2000000000ull, nullptr, 0);
    }
  } else {
    // ---- finishing warps (one alone took 0.7 us a tile).  Three in turn add the consumers' partial
    // tiles and store the result of a tile that is whole (C = 1); or two in turn add them and send them
    // to the tile's owner, and the third adds what an owner got
    const int active = ks.n < kFewWarps ? ks.n : kFewWarps;
    const int g = lane >> 2, c = lane & 3;
    const bool receiver = warp == kFewWarps + 3 && C > 1;
    const int finishers = C > 1 ? 2 : 3, mine = warp - kFewWarps - 1;
    bool ok = true;
    pdl_wait();
    for (int i = receiver ? rank : mine; i < tile1 - tile0; i += receiver ? C : finishers) {
      float4 v[kSets];  // rows g, g of tokens 2 c, 2 c + 1, then rows g + 8
#pragma unroll
      for (int s = 0; s < kSets; ++s) v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      // of an owner's n-th tile: its buffer, and how often that was used before
      const int n = i / C, slot = n % a.recv, use = n / a.recv;
      const uint32_t owner = i % C, buffer = recv + slot * C * kRedBytes + lane * 16;
      if (receiver) {
        if (ok) {
          if (lane == 0) mbar_arrive_expect_tx(smem_u32(&recv_full[slot]), (C - 1) * kRedBytes);
          ok = wait_cluster(smem_u32(&recv_full[slot]), use & 1, abort_flag, a.wait_limit_ns);
        }
        if (ok) {
          for (uint32_t r = 0; r < C; ++r)
#pragma unroll
            for (int s = 0; s < kSets; ++s) v[s] = add4(v[s], lds_f4(buffer + r * kRedBytes + s * 512));
          __syncwarp();
          if (lane < static_cast<int>(C)) remote_arrive(map_rank(smem_u32(&recv_free[rank][slot]), lane));
        }
      } else {
        const int rb = i / STEP % kRed;
        if (ok)
          ok = mbar_wait_warp(smem_u32(&red_full[rb]), (i / (STEP * kRed)) & 1, abort_flag, a.wait_limit_ns,
                              nullptr, 0);
        if (ok) {
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) {
            if (w >= active) break;
#pragma unroll
            for (int s = 0; s < kSets; ++s)
              v[s] = add4(v[s], lds_f4(red + ((rb * kFewWarps + w) * STEP + i % STEP) * kRedBytes +
                                         s * 512 + lane * 16));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&red_empty[rb]));
        }
        if (C > 1) {
          if (ok && use > 0)
            ok = wait_cluster(smem_u32(&recv_free[owner][slot]), (use - 1) & 1, abort_flag,
                              a.wait_limit_ns);
          if (!ok) break;
          const uint32_t full = smem_u32(&recv_full[slot]);
#pragma unroll
          for (int s = 0; s < kSets; ++s) {
            const uint32_t dst = buffer + rank * kRedBytes + s * 512;
            if (owner == rank)
              sts128(dst, v[s]);
            else
              remote_store(map_rank(dst, owner), v[s], map_rank(full, owner));
          }
          __syncwarp();
          if (owner == rank && lane == 0) mbar_arrive(full);
          continue;
        }
      }
      if (!ok) {  // a wait ran out: the tile's outputs say so
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int s = 0; s < kSets; ++s) v[s] = make_float4(nan, nan, nan, nan);
      }
      const int tile = tile0 + i;
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        const float lo[2] = {v[s].x, v[s].y}, hi[2] = {v[s].z, v[s].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = s * kFewCols + c * 2 + h;
          if (t >= a.T) continue;
          if (a.out_kind == kI4OutSwiglu) {  // row g: gate, row g + 8: up
            const int n = tile * 8 + g;
            if (n < a.N / 2)
              static_cast<float*>(a.out)[static_cast<size_t>(t) * (a.N / 2) + n] = swiglu(lo[h], hi[h]);
          } else {
            const int n = tile * 16 + g;
            const size_t o = static_cast<size_t>(t) * a.N + n;
            if (a.out_kind == kI4OutF32) {
              if (n < a.N) static_cast<float*>(a.out)[o] = lo[h];
              if (n + 8 < a.N) static_cast<float*>(a.out)[o + 8] = hi[h];
            } else {
              if (n < a.N) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(lo[h]);
              if (n + 8 < a.N) static_cast<__nv_bfloat16*>(a.out)[o + 8] = __float2bfloat16_rn(hi[h]);
            }
          }
        }
      }
    }
  }
    __syncwarp();
  }
  if (C > 1) {  // no CTA leaves while another may still write its shared memory
    if (*abort_flag) {  // stores that nobody waited for
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 20000) {
      }
    }
    __syncwarp();
    cluster_sync_all();
  }
}

using LinearKernel = void (*)(Int4LinearArgs);
template <int MODE, int STEP>
LinearKernel linear_kernel_of(int group) {
  return group == 32   ? int4_linear_kernel<MODE, 32, STEP>
         : group == 64 ? int4_linear_kernel<MODE, 64, STEP>
                       : int4_linear_kernel<MODE, 128, STEP>;
}
LinearKernel linear_kernel(int mode, int group, int step) {
  return mode == 1   ? (step == 2 ? linear_kernel_of<1, 2>(group) : linear_kernel_of<1, 1>(group))
         : mode == 2 ? (step == 2 ? linear_kernel_of<2, 2>(group) : linear_kernel_of<2, 1>(group))
         : mode == 3 ? linear_kernel_of<3, 1>(group)
                     : linear_kernel_of<4, 1>(group);
}

// Co-resident clusters of C CTAs on this device, by log2 C (filled by prepare_int4_kernels; one
// kind of device per process).
int g_max_clusters[4] = {0, 0, 0, 0};

cudaLaunchConfig_t linear_config(int grid, size_t smem, cudaStream_t s, int cluster,
                                 cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

constexpr size_t kLinDynamicSmem = kFewSmemMax - 1024;  // the rest: barriers

}  // namespace

cudaError_t launch_int4_quantize(const Int4QuantArgs& a, cudaStream_t s) {
  const int64_t blocks = (a.units + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  int4_quantize_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_int4_linear(Int4LinearArgs a, int group, int sms, cudaStream_t s) {
  const int mode = a.T > kFewCols ? 4 : i4_mode(a.T);
  const int units = a.K / kI4Unit, unit_bytes = i4_unit_bytes(group);
  const int max_units = kFewWarps * lin_units(mode);  // K range of a CTA
  // The cluster size that finishes soonest: the largest share of bytes of one CTA at its share of
  // the HBM rate, and about 1 us for the exchange between the CTAs of a cluster.
  int best = 0, best_clus = 0;
  double best_t = 0.;
  for (int lc = 0; lc < 4; ++lc) {
    const int C = 1 << lc;
    const int per = (units + C - 1) / C;
    if (per > max_units || C > units) continue;
    int clus = lc == 0 ? sms : g_max_clusters[lc];
    if (clus > a.tiles) clus = a.tiles;
    if (clus <= 0) continue;
    const double t = static_cast<double>((a.tiles + clus - 1) / clus) * per * unit_bytes / 44.0 +
                     (C > 1 ? 1000.0 : 0.0);
    if (!best || t < best_t) {
      best = C;
      best_clus = clus;
      best_t = t;
    }
  }
  if (!best) return cudaErrorInvalidConfiguration;
  a.cluster = best;
  const int per = (units + best - 1) / best;
  a.stage_bytes = mode > 2 ? 0 : stage_bytes((per + kFewWarps - 1) / kFewWarps * kI4Unit, true, a.wide);
  a.recv = kLinRecvBytes / (best * 512 * lin_sets(mode));
  if (a.recv > kLinRecv) a.recv = kLinRecv;
  const int step = mode <= 2 && (a.tiles + best_clus - 1) / best_clus >= kLinStepTiles ? 2 : 1;
  const size_t rest = static_cast<size_t>(lin_red(step)) * kFewWarps * step * 512 * lin_sets(mode) +
                      (best > 1 ? static_cast<size_t>(a.recv) * best * 512 * lin_sets(mode) : 0) +
                      static_cast<size_t>(kFewWarps) * a.stage_bytes;
  const KSplit ks = make_ksplit(per, kLinSlotBytes, step * unit_bytes);
  a.cw = ks.cw;
  a.slot_bytes = chunk_bytes(ks, step * unit_bytes);
  a.stages = static_cast<int>((kLinDynamicSmem - rest) / a.slot_bytes);
  if (a.stages > kFewMaxStages) a.stages = kFewMaxStages;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      linear_config(best * best_clus, a.stages * static_cast<size_t>(a.slot_bytes) + rest, s, best, attr);
  return cudaLaunchKernelEx(&cfg, linear_kernel(mode, group, step), a);
}

cudaError_t prepare_int4_kernels() {
  for (int mode : {1, 2, 3, 4})
    for (int group : {32, 64, 128})
      for (int step : {1, 2}) {
        const cudaError_t e = cudaFuncSetAttribute(linear_kernel(mode, group, step),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kLinDynamicSmem));
        if (e != cudaSuccess) return e;
      }
  for (int lc = 1; lc < 4; ++lc) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = linear_config(1 << lc, kLinDynamicSmem, nullptr, 1 << lc, attr);
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, linear_kernel(1, 128, 1), &cfg);
    if (e != cudaSuccess) return e;
    g_max_clusters[lc] = n;
  }
  return cudaSuccess;
}

}  // namespace beam
