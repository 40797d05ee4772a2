// Gradients of causal attention with a sliding window and sinks, for sm_100a (bf16, D = 64
// or 128).
//
// Mathematics: the chain rule through the definition, with the forward's lse, on the pairs
// that see each other:
//     P = exp(scale q k^T - lse),  dV = P^T dO,  dP = dO V^T,  Delta = rowsum(dO * O),
//     dS = P * (dP - Delta),  dQ = scale dS K,  dK = scale dS^T Q
// (dK, dV summed over the query heads of a group). P and dS are rounded to bf16 for the
// products that give dV and dK; sums and statistics are fp32. For dQ, dS enters as two bf16
// terms, its rounding and what that left: a row of dS sums to about zero, so that dQ is small
// against its terms and their rounding would show (1.5 to 1.6 times the error of rounding
// the result alone; with two terms 1.0).
//
// Kernels, on one stream:
//   prep    -Delta and -lse log2 e per row, padded to whole 128-row tiles (0 / -inf)
//   grads   CTAs of two kinds, in one launch: the short ones fill the SMs that the last of
//           the long ones leave idle.
//           dkdv: a 128-key tile and part of its queries, 64 query rows at a time,
//           S^T = K Q^T and dP^T = V dO^T into tensor memory, P^T and dS^T by eight warps,
//           then dV += P^T dO and dK += dS^T Q with the packed operand in tensor memory
//           dq: 128 query rows, 64 keys at a time: S, dP, dS, dQ += dS K
//   reduce  sums the parts of tiles that have more than one, in a fixed order
// as in the ring's backward kernels (bwd_sm100.cu), from which the tensor-memory layout,
// the double buffering and the one-slot-per-step rings are taken over. No atomics: the
// same call gives the same bits.
//
// The work is uneven where that form is not: a tile with sinks is seen by every later
// query, S / 64 steps instead of window / 64 + 3. Such a tile's queries are cut into parts
// of a plain tile's length that run as CTAs of their own, and where the tiles alone do not
// fill the GPU the heads of a group are divided among CTAs too.
//
// What bounds it: the products. At D = 128 a step of dkdv is 1280 clocks of them (the score
// products read both operands from shared memory: 48 clocks each at N = 64, of 32 for the
// multiplications) and takes 1500 to 1570, a step of dq 1024 and takes 1190; a CTA's start and
// end, which nothing overlaps, take 6000 to 8000. 32k tokens, window 2048, 16 query heads over
// 4: 2.11 to 2.12 ms, 665 to 669 TFLOP/s at 10 D flops a pair.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ringattn_internal.h"
#include "sm100_ptx.cuh"
#include "softmax_rows.cuh"
#include "window_geom.h"
#include "window_store.cuh"

namespace ringattn {
namespace winbwd {

constexpr int BT = 128;                    // rows of a stationary tile (keys or queries)
constexpr int TS = 64;                     // rows of a streamed step
constexpr int BOXW = 64;
constexpr int kSmemLimit = 232448;
constexpr int kThreads = 384;              // 8 elementwise warps, producer, MMA, 2 idle
constexpr int kEwWarps = 8;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kProducerSleepNs = 64;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColAcc = 256;
constexpr uint32_t kColQ = 384;
constexpr uint32_t kColDO = 448;
constexpr uint32_t kIdescSS = idesc_bf16_f32(BT, TS, 0, 0);
constexpr int kBoxBytes = BT * BOXW * 2;
constexpr int kStepBoxBytes = TS * BOXW * 2;
constexpr int kStepStatBytes = TS * 4;

// Columns of double buffer b: the score tile (transposed in dkdv) and the dP tile.
__device__ __forceinline__ uint32_t col_s(int b) { return (uint32_t)(64 * b); }
__device__ __forceinline__ uint32_t col_dp(int b) { return (uint32_t)(128 + 64 * b); }
// K step k (16 columns) of a K-major operand staged as 64-column boxes.
template <int kBox>
__device__ __forceinline__ uint64_t kmajor_step(uint64_t base, int k) {
  return base + (uint64_t)((((k / 4) * kBox) + (k % 4) * 32) >> 4);
}
// K step k (16 rows) of an operand whose rows run along K.
__device__ __forceinline__ uint64_t mnmajor_step(uint64_t base, int k) {
  return base + (uint64_t)((k * 16 * 128) >> 4);
}
// K step k of a packed bf16 operand over 64 K rows written by the two column halves.
__device__ __forceinline__ uint32_t packed_step_col(int k) { return (uint32_t)((k / 2) * 32 + (k % 2) * 8); }

template <int D>
struct CfgA {  // dkdv
  static constexpr int kTileBytes = BT * D * 2;
  static constexpr int kStepTileBytes = TS * D * 2;
  static constexpr int kOffV = kTileBytes;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kSlotDO = kStepTileBytes;
  static constexpr int kSlotLse = 2 * kStepTileBytes;
  static constexpr int kSlotDelta = kSlotLse + kStepStatBytes;
  static constexpr int kSlotFill = 2 * kStepTileBytes + 2 * kStepStatBytes;
  static constexpr int kSlotBytes = ((kSlotFill + 1023) / 1024) * 1024;
  static constexpr int kSlots = 4;
  static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
  static constexpr int kNumBars = 7 + 2 * kSlots;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  static_assert(kSlots >= 3, "steps n, n + 1 and n + 2 are held at once");
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
  static constexpr uint32_t kIdescTS = idesc_bf16_f32(BT, D, 0, 1);
};
enum BarA { kA_KVFull = 0, kA_STFull = 1, kA_PReady = 3, kA_Done = 5, kA_Drain = 6, kA_Ring = 7 };

template <int D>
struct CfgB {  // dq
  static constexpr int kStepTileBytes = TS * D * 2;
  static constexpr int kSlotBytes = 2 * kStepTileBytes;
  static constexpr int kSlots = 6;
  static constexpr int kOffBar = kSlots * kSlotBytes;
  static constexpr int kNumBars = 8 + 2 * kSlots;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  static_assert(kSlots >= 3, "steps n, n + 1 and n + 2 are held at once");
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
  static constexpr uint32_t kIdescTS = idesc_bf16_f32(BT, D, 0, 1);
  // Q and dO wait in the ring's last two slots for the warps that take them to tensor memory
  static constexpr int kSlotQ = kSlots - 2, kSlotDO = kSlots - 1;
  static constexpr int kTileBytes = BT * D * 2;
  static_assert(kTileBytes <= kSlotBytes, "a tile of queries fits a slot");
};
enum BarB { kB_QReady = 0, kB_SFull = 1, kB_PReady = 3, kB_Done = 5, kB_Drain = 6, kB_QFull = 7, kB_Ring = 8 };

// How the key tiles are divided. Tiles [0, sink_tiles) are seen by every later query: their
// query steps are cut into `segs` runs. Every tile's query heads are cut into `splits`
// groups. A tile with more than one part keeps fp32 partial sums.
struct Plan {
  int64_t tiles;       // key tiles of a sequence
  int64_t sink_tiles;
  int segs, splits;
  int64_t sink_units;  // units of all (b, kv head) that belong to sink tiles: launched first
  int64_t units;
};

struct Params {
  WinGeom g;
  Plan plan;
  const float* nlse2;  // [B*Hq][s_pad]: -lse log2 e
  const float* ndelta; // -Delta
  int64_t s_pad;
  void* dq;
  void* dk;
  void* dv;
  float* parts;        // [part][dV, dK][128][D]
  float scale, scale_log2;
  int* status;
  uint64_t watchdog_ns;
};

struct KeyUnit {
  int64_t bh;           // b * Hkv + kv head
  int64_t kt;           // key tile
  int h0, h1;           // query heads of the group
  int64_t s0, s1;       // query steps of 64 rows
  int64_t part;         // slot of its partial sums, -1: alone
};

// Query steps that meet key tile kt.
__host__ __device__ __forceinline__ void tile_steps(const WinGeom& g, int64_t kt, int64_t& s0, int64_t& s1) {
  s0 = kt * (BT / TS);
  int64_t last = kt * BT + BT - 1 + g.window - 1;
  if (kt * BT < g.sinks || last > g.S - 1) last = g.S - 1;
  s1 = last / TS + 1;
}

__host__ __device__ __forceinline__ KeyUnit key_unit(const WinGeom& g, const Plan& pl, int64_t u) {
  const int rep = g.Hq / g.Hkv;
  KeyUnit x;
  int64_t seg = 0, segs = 1, split;
  if (u < pl.sink_units) {
    split = u % pl.splits;
    u /= pl.splits;
    seg = u % pl.segs;
    segs = pl.segs;
    u /= pl.segs;
    x.kt = u % pl.sink_tiles;
    x.bh = u / pl.sink_tiles;
    x.part = pl.segs * pl.splits > 1 ? ((x.bh * pl.sink_tiles + x.kt) * pl.segs + seg) * pl.splits + split : -1;
  } else {
    u -= pl.sink_units;
    split = u % pl.splits;
    u /= pl.splits;
    const int64_t rest = pl.tiles - pl.sink_tiles;
    x.kt = pl.sink_tiles + u % rest;
    x.bh = u / rest;
    x.part = pl.splits > 1 ? (pl.segs * pl.splits > 1 ? pl.sink_units : 0) +
                                 (x.bh * rest + x.kt - pl.sink_tiles) * pl.splits + split
                           : -1;
  }
  x.h0 = (int)(rep * split / pl.splits);
  x.h1 = (int)(rep * (split + 1) / pl.splits);
  int64_t s0, s1;
  tile_steps(g, x.kt, s0, s1);
  x.s0 = s0 + (s1 - s0) * seg / segs;
  x.s1 = s0 + (s1 - s0) * (seg + 1) / segs;
  return x;
}

// Slot and phase of a ring's step, counted along (a division per step would stand in the
// issuing thread's way).
template <int kSlots>
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

// Bits c of [lo, hi) in 0..31, for a chunk that starts at column c0.
__host__ __device__ __forceinline__ uint32_t range_bits(int lo, int hi, int c0) {
  lo = lo - c0 > 0 ? lo - c0 : 0;
  hi = hi - c0 < 32 ? hi - c0 : 32;
  if (hi <= lo) return 0u;
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Queries [u, key_past) see key u.
__host__ __device__ __forceinline__ int64_t key_past(const WinGeom& g, int64_t u) {
  return u < g.sinks || u + g.window > g.S ? g.S : u + g.window;
}
// Steps whose every query sees every key of tile kt: [in0, in1), most of a tile's.
__host__ __device__ __forceinline__ void inner_steps(const WinGeom& g, int64_t kt, int64_t& in0, int64_t& in1) {
  in0 = (kt + 1) * (BT / TS);
  in1 = ((kt + 1) * BT <= g.sinks ? g.S : key_past(g, kt * BT < g.sinks ? g.sinks : kt * BT)) / TS;
}
// Queries of 32 columns of step s that see key u.
__host__ __device__ __forceinline__ uint32_t key_sees(int64_t u, int64_t past, int64_t s, int c0, int64_t in0,
                                                      int64_t in1) {
  if (s >= in0 && s < in1) return 0xffffffffu;
  return range_bits(win_clip(u - s * TS, TS), win_clip(past - s * TS, TS), c0);
}
// Keys of 32 columns of the step that starts at key `first` that query a of the block at a0 sees.
__host__ __device__ __forceinline__ uint32_t query_sees(const WinGeom& g, int64_t a0, int64_t a, int64_t first, int c0) {
  if (first + TS - 1 <= a0 && first > a0 + BT - 1 - g.window) return 0xffffffffu;
  const WinCut cut = win_cut(g, a, first, TS);
  return range_bits(cut.lo, cut.hi, c0) | range_bits(0, cut.sk < cut.hi ? cut.sk : cut.hi, c0);
}

// Raw scores and dP of two neighbouring columns to P and dS: P = 2^x with x = s scale_log2 -
// lse2, dS = P (dP - Delta); the statistics come negated.
__device__ __forceinline__ void p_ds_pair(uint32_t s0, uint32_t s1, uint32_t dp0, uint32_t dp1, uint64_t c2, uint64_t nl,
                                          uint64_t nd, float& p0, float& p1, float& d0, float& d1) {
  float x0, x1;
  f2_unpack(f2_fma(f2_pack(s0, s1), c2, nl), x0, x1);
  p0 = ex2_approx(x0);
  p1 = ex2_approx(x1);
  f2_unpack(f2_mul(f2_pack(__float_as_uint(p0), __float_as_uint(p1)), f2_add(f2_pack(dp0, dp1), nd)), d0, d1);
}

// dkdv: 32 keys x 32 queries of a warp as two fragments of 16 keys (tmem_ld_frag16), so that a
// thread needs the statistics of 8 queries for its 32 pairs and not of 32: they come from
// shared memory, whose reads by the products bound the step (with a key per thread, 64 values
// read by each, a step took 1780 cycles; 1280 are the products'). nlse2c, ndeltac: those of
// the thread's first query. see[2 t + j]: the queries from there on that see its key of
// fragment t, row j; zeros for the others whatever they held.
template <bool kWhole>
__device__ __forceinline__ void p_ds_keys(const uint32_t (&s)[32], const uint32_t (&dp)[32], const float* nlse2c,
                                          const float* ndeltac, float scale_log2, const uint32_t (&see)[4],
                                          uint32_t (&pp)[16], uint32_t (&pds)[16]) {
  const uint64_t c2 = f2_splat(scale_log2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lv = *reinterpret_cast<const float2*>(nlse2c + 8 * i);
    const float2 dv = *reinterpret_cast<const float2*>(ndeltac + 8 * i);
    const uint64_t nl = f2_pack(__float_as_uint(lv.x), __float_as_uint(lv.y));
    const uint64_t nd = f2_pack(__float_as_uint(dv.x), __float_as_uint(dv.y));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int e = (x / 2) * 16 + 4 * i + 2 * (x % 2), o = (x / 2) * 8 + 2 * i + x % 2;
      float p0, p1, d0, d1;
      p_ds_pair(s[e], s[e + 1], dp[e], dp[e + 1], c2, nl, nd, p0, p1, d0, d1);
      if (!kWhole) {
        if (!(see[x] >> (8 * i) & 1)) p0 = d0 = 0.f;
        if (!(see[x] >> (8 * i + 1) & 1)) p1 = d1 = 0.f;
      }
      pp[o] = pack_bf16x2(p0, p1);
      pds[o] = pack_bf16x2(d0, d1);
    }
  }
}

// dq: 32 columns of a query, its statistics in registers; pds receives dS, rest what its
// rounding left (exact in fp32, rounded to bf16).
template <bool kWhole>
__device__ __forceinline__ void ds_query(const uint32_t (&s)[32], const uint32_t (&dp)[32], float nlse2, float ndelta,
                                         float scale_log2, uint32_t see, uint32_t (&pds)[16], uint32_t (&rest)[16]) {
  const uint64_t c2 = f2_splat(scale_log2), nl = f2_splat(nlse2), nd = f2_splat(ndelta);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float p0, p1, d0, d1;
    p_ds_pair(s[e], s[e + 1], dp[e], dp[e + 1], c2, nl, nd, p0, p1, d0, d1);
    if (!kWhole) {
      if (!(see >> e & 1)) d0 = 0.f;
      if (!(see >> (e + 1) & 1)) d1 = 0.f;
    }
    const uint32_t r = pack_bf16x2(d0, d1);
    pds[e / 2] = r;
    rest[e / 2] = pack_bf16x2(d0 - __uint_as_float(r << 16), d1 - __uint_as_float(r & 0xffff0000u));
  }
}

// ------------------------------------------------------------------------------ prep
// D / 8 lanes per row, 16 bytes of dO and of O each.
template <int D>
__global__ void __launch_bounds__(256) window_prep_kernel(const uint16_t* __restrict__ out,
                                                          const uint16_t* __restrict__ dout,
                                                          const float* __restrict__ lse, float* __restrict__ nlse2,
                                                          float* __restrict__ ndelta, int64_t S, int64_t s_pad,
                                                          int64_t rows, int* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = RING_ATTN_OK;
  grid_let_next();
  constexpr int kTpr = D / 8;
  const int64_t row = (int64_t)blockIdx.x * (256 / kTpr) + threadIdx.x / kTpr;
  const int sub = threadIdx.x % kTpr;
  const bool in = row < rows;
  const int64_t bh = in ? row / s_pad : 0, a = in ? row % s_pad : 0;
  const bool real = in && a < S;
  float acc = 0.f;
  if (real) {
    const int64_t base = (bh * S + a) * D + sub * 8;
    const uint4 o = *reinterpret_cast<const uint4*>(out + base);
    const uint4 x = *reinterpret_cast<const uint4*>(dout + base);
    const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = fmaf(__uint_as_float(ow[i] << 16), __uint_as_float(xw[i] << 16), acc);
      acc = fmaf(__uint_as_float(ow[i] & 0xffff0000u), __uint_as_float(xw[i] & 0xffff0000u), acc);
    }
  }
#pragma unroll
  for (int off = kTpr / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (in && sub == 0) {
    nlse2[row] = real ? lse[bh * S + a] * -1.4426950408889634f : -INFINITY;
    ndelta[row] = -acc;
  }
}

// ------------------------------------------------------------------------------ dK, dV
template <int D>
__device__ __forceinline__ void dkdv_unit(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                          const CUtensorMap& tm_v, const Params& p, uint8_t* smem, int64_t unit) {
  using C = CfgA<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  uint64_t* full = &bars[kA_Ring];
  uint64_t* empty = &bars[kA_Ring + C::kSlots];
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const WinGeom& g = p.g;

  if (threadIdx.x == 0) {
    mbar_init(&bars[kA_KVFull], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kA_STFull + b], 1);
      mbar_init(&bars[kA_PReady + b], kEwWarps);
    }
    mbar_init(&bars[kA_Done], 1);
    mbar_init(&bars[kA_Drain], 1);
    for (int s = 0; s < 2 * C::kSlots; ++s) mbar_init(&bars[kA_Ring + s], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  const Watchdog wd{abort_flag, p.status, p.watchdog_ns};
  const KeyUnit U = key_unit(g, p.plan, unit);
  const int rep = g.Hq / g.Hkv;
  const int per_head = (int)(U.s1 - U.s0);
  const int N = (U.h1 - U.h0) * per_head;  // steps
  auto slot_of = [&](int m) { return m % C::kSlots; };
  auto phase_of = [&](int m) { return (uint32_t)(m / C::kSlots) & 1; };

  if (warp == kProducerWarp) {
    if (lane == 0 && N > 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      mbar_arrive_expect_tx(&bars[kA_KVFull], 2 * C::kTileBytes);
      for (int bx = 0; bx < D / BOXW; ++bx) {
        tma_load_4d(smem + bx * kBoxBytes, &tm_k, &bars[kA_KVFull], bx * BOXW, (int)(U.kt * BT), 0, (int)U.bh);
        tma_load_4d(smem + C::kOffV + bx * kBoxBytes, &tm_v, &bars[kA_KVFull], bx * BOXW, (int)(U.kt * BT), 0,
                    (int)U.bh);
      }
      int m = 0;
      bool ok = true;
      for (int h = U.h0; h < U.h1 && ok; ++h) {
        const int bh_q = (int)U.bh * rep + h;
        for (int64_t s = U.s0; s < U.s1; ++s, ++m) {
          const int slot = slot_of(m);
          if (!(ok = mbar_wait_backoff<false>(&empty[slot], phase_of(m) ^ 1, wd, kProducerSleepNs))) break;
          uint8_t* dst = smem + C::kOffRing + slot * C::kSlotBytes;
          mbar_arrive_expect_tx(&full[slot], C::kSlotFill);
          for (int bx = 0; bx < D / BOXW; ++bx)
            tma_load_4d(dst + bx * kStepBoxBytes, &tm_q, &full[slot], bx * BOXW, (int)(s * TS), 0, bh_q);
          for (int bx = 0; bx < D / BOXW; ++bx)
            tma_load_4d(dst + C::kSlotDO + bx * kStepBoxBytes, &tm_do, &full[slot], bx * BOXW, (int)(s * TS), 0, bh_q);
          const int64_t stat = (int64_t)bh_q * p.s_pad + s * TS;
          bulk_load(dst + C::kSlotLse, p.nlse2 + stat, kStepStatBytes, &full[slot]);
          bulk_load(dst + C::kSlotDelta, p.ndelta + stat, kStepStatBytes, &full[slot]);
        }
      }
      if (!ok) {
        // wind down: this CTA's own copies must land before its shared memory goes away
        drain_wait(&bars[kA_KVFull], 0, p.watchdog_ns);
        for (int x = (m > C::kSlots ? m - C::kSlots : 0); x < m; ++x)
          drain_wait(&full[slot_of(x)], phase_of(x), p.watchdog_ns);
      }
    }
  } else if (warp == kMmaWarp) {
    // one thread waits and issues: the tensor pipe holds two or three products ahead, so what
    // passes between a step's last and the next one's first is time that it idles
    if (elect_one_sync()) {
      const uint32_t sbase = smem_u32(smem);
      const uint64_t dK = smem_desc_sw128(sbase, 0, 1024);
      const uint64_t dV = smem_desc_sw128(sbase + C::kOffV, 0, 1024);
      RingPos<C::kSlots> in, use;  // steps of the next S^T and of the next dV
      auto issue_st = [&](int b) -> bool {
        if (!mbar_wait(&full[in.slot], in.phase, wd)) return false;
        tc_fence_after();
        const uint32_t at = sbase + C::kOffRing + in.slot * C::kSlotBytes;
        const uint64_t bq = smem_desc_sw128(at, 0, 1024);
        const uint64_t bd = smem_desc_sw128(at + C::kSlotDO, 0, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + col_s(b), kmajor_step<kBoxBytes>(dK, k), kmajor_step<kStepBoxBytes>(bq, k), kIdescSS, k > 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + col_dp(b), kmajor_step<kBoxBytes>(dV, k), kmajor_step<kStepBoxBytes>(bd, k), kIdescSS, k > 0);
        mma_commit(&bars[kA_STFull + b]);
        in.next();
        return true;
      };
      bool ok = N > 0 && mbar_wait(&bars[kA_KVFull], 0, wd);
      if (ok) ok = issue_st(0);
      if (ok && N > 1) ok = issue_st(1);
      for (int n = 0; ok && n < N; ++n, use.next()) {
        const int b = n & 1;
        const uint32_t at = sbase + C::kOffRing + use.slot * C::kSlotBytes;
        const uint64_t mq = smem_desc_sw128(at, kStepBoxBytes, 1024);
        const uint64_t md = smem_desc_sw128(at + C::kSlotDO, kStepBoxBytes, 1024);
        if (!(ok = mbar_wait(&bars[kA_PReady + b], (uint32_t)((n >> 1) & 1), wd))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TS / 16; ++k)  // dV += P^T dO
          mma_ts(tmem + kColAcc, tmem + col_s(b) + packed_step_col(k), mnmajor_step(md, k), C::kIdescTS,
                 !(n == 0 && k == 0));
#pragma unroll
        for (int k = 0; k < TS / 16; ++k)  // dK += dS^T Q
          mma_ts(tmem + kColAcc + D, tmem + col_dp(b) + packed_step_col(k), mnmajor_step(mq, k), C::kIdescTS,
                 !(n == 0 && k == 0));
        mma_commit(&empty[use.slot]);
        // buffer b is free for step n + 2 once these products have read its P and dS
        if (n + 2 < N && !(ok = issue_st(b))) break;
      }
      mma_commit(&bars[kA_Done]);
      mma_commit(&bars[kA_Drain]);
      drain_wait(&bars[kA_Drain], 0, p.watchdog_ns);
    }
    __syncwarp();
  } else if (warp < kEwWarps) {
    // warp = 4 hh + wq: TMEM lanes 32 wq (key rows), query columns 32 hh .. 32 hh + 31 of a step
    const int wq = warp % 4, hh = warp / 4;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const int fr = lane / 4, fc = 2 * (lane % 4);  // fragment row, first column
    int64_t in0, in1;
    inner_steps(g, U.kt, in0, in1);
    bool ok = true;
    int n = 0;
    for (int h = U.h0; h < U.h1 && ok; ++h) {
      for (int64_t s = U.s0; s < U.s1; ++s, ++n) {
        const int b = n & 1;
        const int sl = slot_of(n);
        if (!(ok = mbar_wait(&bars[kA_STFull + b], (uint32_t)((n >> 1) & 1), wd))) break;
        // the statistics came with the tiles: wait on their barrier too (already complete)
        if (!(ok = mbar_wait(&full[sl], phase_of(n), wd))) break;
        tc_fence_after();
        const float* nlse2c = reinterpret_cast<const float*>(smem + C::kOffRing + sl * C::kSlotBytes + C::kSlotLse);
        const float* ndeltac = reinterpret_cast<const float*>(smem + C::kOffRing + sl * C::kSlotBytes + C::kSlotDelta);
        nlse2c += 32 * hh + fc;
        ndeltac += 32 * hh + fc;
        uint32_t sv[32], dpv[32], pp[16], pds[16], see[4];
        const uint32_t tS = tmem + lane_off + col_s(b) + 32 * hh, tDP = tmem + lane_off + col_dp(b) + 32 * hh;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          tmem_ld_frag16(tS + (t << 20), sv + 16 * t);
          tmem_ld_frag16(tDP + (t << 20), dpv + 16 * t);
        }
        const bool whole = s >= in0 && s < in1;
        if (__builtin_expect(!whole, 0)) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int64_t key = U.kt * BT + wq * 32 + 8 * x + fr;
            see[x] = key_sees(key, key_past(g, key), s, 32 * hh, in0, in1) >> fc;
          }
        }
        tmem_wait_ld();
        if (__builtin_expect(whole, 1))
          p_ds_keys<true>(sv, dpv, nlse2c, ndeltac, p.scale_log2, see, pp, pds);
        else
          p_ds_keys<false>(sv, dpv, nlse2c, ndeltac, p.scale_log2, see, pp, pds);
        // the packed columns overlap only this warp's own, already loaded fp32 columns
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          tmem_st_frag16(tS + (t << 20), pp + 8 * t);
          tmem_st_frag16(tDP + (t << 20), pds + 8 * t);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kA_PReady + b]);
      }
    }
    const bool have = N > 0 && ok && mbar_wait(&bars[kA_Done], 0, wd);
    if (have || N == 0) {
      tc_fence_after();
      const uint32_t tAcc = tmem + lane_off + kColAcc + hh * (D / 2);
      // (every copy into the ring has been used: it is free)
      uint8_t* stage = smem + C::kOffRing + warp * kStageBytesF32;
      if (U.part < 0) {
        const int64_t first = U.kt * BT + wq * 32;
        store_rows_staged<D / 2, false>(tAcc, N > 0, 1.f, stage, p.dv, U.bh * g.S + first, g.S - first, D, hh * (D / 2));
        store_rows_staged<D / 2, false>(tAcc + D, N > 0, p.scale, stage, p.dk, U.bh * g.S + first, g.S - first, D,
                                        hh * (D / 2));
      } else {
        const int64_t first = U.part * 2 * BT + wq * 32;
        store_rows_staged<D / 2, true>(tAcc, N > 0, 1.f, stage, p.parts, first, 32, D, hh * (D / 2));
        store_rows_staged<D / 2, true>(tAcc + D, N > 0, p.scale, stage, p.parts, first + BT, 32, D, hh * (D / 2));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Sums a tile's parts, first to last. One thread per 8 columns of a key row of dV or dK; the
// first `sink_items` threads take the sink tiles, the others the tiles behind them.
template <int D>
__global__ void __launch_bounds__(256) window_reduce_kernel(const __grid_constant__ Params p, int64_t sink_items,
                                                            int64_t items) {
  grid_wait();
  int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  const Plan& pl = p.plan;
  const bool sink = it < sink_items;
  if (!sink) it -= sink_items;
  constexpr int kTpr = D / 8;
  const int c = (int)(it % kTpr) * 8;
  int64_t x = it / kTpr;
  const int r = (int)(x % BT);
  x /= BT;
  const int which = (int)(x % 2);  // 0 dV, 1 dK
  x /= 2;
  const int64_t tiles = sink ? pl.sink_tiles : pl.tiles - pl.sink_tiles;
  const int64_t t = x % tiles, bh = x / tiles;
  const int64_t u = (t + (sink ? 0 : pl.sink_tiles)) * BT + r;
  if (u >= p.g.S) return;
  const int n = sink ? pl.segs * pl.splits : pl.splits;
  const int64_t first = (sink ? 0 : (pl.segs * pl.splits > 1 ? pl.sink_units : 0)) + (bh * tiles + t) * n;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  const float* src = p.parts + ((first * 2 + which) * BT + r) * D + c;
#pragma unroll 4
  for (int i = 0; i < n; ++i, src += 2 * BT * D) {
    const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  uint16_t* dst = static_cast<uint16_t*>(which ? p.dk : p.dv) + (bh * p.g.S + u) * D + c;
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                              pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

// ---------------------------------------------------------------------------------- dQ
template <int D>
__device__ __forceinline__ void dq_unit(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                        const CUtensorMap& tm_v, const Params& p, uint8_t* smem, int64_t u) {
  using C = CfgB<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  uint64_t* full = &bars[kB_Ring];
  uint64_t* empty = &bars[kB_Ring + C::kSlots];
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const WinGeom& g = p.g;

  // units: the heads of a group innermost (shared K and V), then the row blocks
  const int rep = g.Hq / g.Hkv;
  const int64_t blocks = p.s_pad / BT;
  const int hr = (int)(u % rep);
  u /= rep;
  const int64_t a0 = (u % blocks) * BT;
  const int bh_kv = (int)(u / blocks);
  const int bh_q = bh_kv * rep + hr;
  const WinTiles wt = win_tiles(g, a0, a0 + BT - 1, TS);
  const int N = win_count(wt);
  if (threadIdx.x == 0) {
    mbar_init(&bars[kB_QReady], kEwWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kB_SFull + b], 1);
      mbar_init(&bars[kB_PReady + b], kEwWarps);
    }
    mbar_init(&bars[kB_Done], 1);
    mbar_init(&bars[kB_Drain], 1);
    mbar_init(&bars[kB_QFull], 1);
    for (int s = 0; s < 2 * C::kSlots; ++s) mbar_init(&bars[kB_Ring + s], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.status, p.watchdog_ns};
  auto slot_of = [&](int m) { return m % C::kSlots; };
  auto phase_of = [&](int m) { return (uint32_t)(m / C::kSlots) & 1; };

  if (warp == kProducerWarp) {
    if (lane == 0 && N > 0) {
      mbar_arrive_expect_tx(&bars[kB_QFull], 2 * C::kTileBytes);
      for (int t = 0; t < 2; ++t) {
        uint8_t* dst = smem + (t == 0 ? C::kSlotQ : C::kSlotDO) * C::kSlotBytes;
        for (int bx = 0; bx < D / BOXW; ++bx)
          for (int r = 0; r < BT; r += TS)
            tma_load_4d(dst + bx * kBoxBytes + r * 128, t == 0 ? &tm_q : &tm_do, &bars[kB_QFull], bx * BOXW, (int)a0 + r, 0,
                        bh_q);
      }
      int m = 0;
      bool ok = true;
      for (; m < N; ++m) {
        const int slot = slot_of(m);
        const int row = win_tile(wt, m) * TS;
        if (m == C::kSlotQ && !(ok = mbar_wait_backoff<false>(&bars[kB_QReady], 0, wd, kProducerSleepNs))) break;
        if (!(ok = mbar_wait_backoff<false>(&empty[slot], phase_of(m) ^ 1, wd, kProducerSleepNs))) break;
        uint8_t* dst = smem + slot * C::kSlotBytes;
        mbar_arrive_expect_tx(&full[slot], C::kSlotBytes);
        for (int bx = 0; bx < D / BOXW; ++bx)
          tma_load_4d(dst + bx * kStepBoxBytes, &tm_k, &full[slot], bx * BOXW, row, 0, bh_kv);
        for (int bx = 0; bx < D / BOXW; ++bx)
          tma_load_4d(dst + C::kStepTileBytes + bx * kStepBoxBytes, &tm_v, &full[slot], bx * BOXW, row, 0, bh_kv);
      }
      if (!ok) {
        drain_wait(&bars[kB_QFull], 0, p.watchdog_ns);
        for (int x = (m > C::kSlots ? m - C::kSlots : 0); x < m; ++x)
          drain_wait(&full[slot_of(x)], phase_of(x), p.watchdog_ns);
      }
    }
  } else if (warp == kMmaWarp) {
    if (elect_one_sync()) {
      const uint32_t sbase = smem_u32(smem);
      RingPos<C::kSlots> in, use;  // steps of the next S and of the next dQ
      auto issue_sd = [&](int b) -> bool {
        if (!mbar_wait(&full[in.slot], in.phase, wd)) return false;
        tc_fence_after();
        const uint32_t at = sbase + in.slot * C::kSlotBytes;
        const uint64_t bk = smem_desc_sw128(at, 0, 1024);
        const uint64_t bv = smem_desc_sw128(at + C::kStepTileBytes, 0, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)  // K step k: dims 16k..16k+15 = packed columns 8k..8k+7
          mma_ts(tmem + col_s(b), tmem + kColQ + 8 * k, kmajor_step<kStepBoxBytes>(bk, k), kIdescSS, k > 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(tmem + col_dp(b), tmem + kColDO + 8 * k, kmajor_step<kStepBoxBytes>(bv, k), kIdescSS, k > 0);
        mma_commit(&bars[kB_SFull + b]);
        in.next();
        return true;
      };
      bool ok = N > 0 && mbar_wait(&bars[kB_QReady], 0, wd);
      if (ok) {
        tc_fence_after();
        ok = issue_sd(0);
      }
      if (ok && N > 1) ok = issue_sd(1);
      for (int n = 0; ok && n < N; ++n, use.next()) {
        const int b = n & 1;
        const uint64_t mk = smem_desc_sw128(sbase + use.slot * C::kSlotBytes, kStepBoxBytes, 1024);
        if (!(ok = mbar_wait(&bars[kB_PReady + b], (uint32_t)((n >> 1) & 1), wd))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < TS / 16; ++k) {  // dQ += dS K, both terms of dS
          mma_ts(tmem + kColAcc, tmem + col_s(b) + packed_step_col(k), mnmajor_step(mk, k), C::kIdescTS,
                 !(n == 0 && k == 0));
          mma_ts(tmem + kColAcc, tmem + col_dp(b) + packed_step_col(k), mnmajor_step(mk, k), C::kIdescTS, 1);
        }
        mma_commit(&empty[use.slot]);
        if (n + 2 < N && !(ok = issue_sd(b))) break;
      }
      mma_commit(&bars[kB_Done]);
      mma_commit(&bars[kB_Drain]);
      drain_wait(&bars[kB_Drain], 0, p.watchdog_ns);
    }
    __syncwarp();
  } else if (warp < kEwWarps) {
    // warp = 4 hh + wq: TMEM lanes 32 wq (query rows), keys 32 hh .. 32 hh + 31 of a step
    const int wq = warp % 4, hh = warp / 4;
    const int64_t a = a0 + wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    grid_wait();
    const int64_t stat = (int64_t)bh_q * p.s_pad + a;  // a < s_pad always
    const float row_nlse2 = p.nlse2[stat];
    const float row_ndelta = p.ndelta[stat];
    bool ok = N > 0 && mbar_wait(&bars[kB_QFull], 0, wd);
    if (ok) {
      // this thread's row of Q and dO, dims (D/2) hh .., as bf16 pairs (the memory order; rows
      // past the sequence are zeros), from the swizzled tiles: row by row from global memory the
      // 16-byte loads of 32 rows each took 4000 clocks
      const int r = wq * 32 + lane;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint8_t* row = smem + (t == 0 ? C::kSlotQ : C::kSlotDO) * C::kSlotBytes + (D == 128 ? hh * kBoxBytes : 0) + r * 128;
        uint32_t x[D / 4];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const int ch = D == 128 ? c : 4 * hh + c;
          const uint4 v4 = *reinterpret_cast<const uint4*>(row + ((ch ^ (r & 7)) * 16));
          x[4 * c] = v4.x;
          x[4 * c + 1] = v4.y;
          x[4 * c + 2] = v4.z;
          x[4 * c + 3] = v4.w;
        }
        const uint32_t dst = tmem + lane_off + (t == 0 ? kColQ : kColDO) + (D / 4) * hh;
        if constexpr (D == 128)
          tmem_st32(dst, x);
        else
          tmem_st16(dst, x);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kB_QReady]);
    }
    for (int n = 0; ok && n < N; ++n) {
      const int b = n & 1;
      if (!(ok = mbar_wait(&bars[kB_SFull + b], (uint32_t)((n >> 1) & 1), wd))) break;
      tc_fence_after();
      const uint32_t see = query_sees(g, a0, a, (int64_t)win_tile(wt, n) * TS, 32 * hh);
      uint32_t sv[32], dpv[32], pds[16], rest[16];
      tmem_ld32(tmem + lane_off + col_s(b) + 32 * hh, sv);
      tmem_ld32(tmem + lane_off + col_dp(b) + 32 * hh, dpv);
      tmem_wait_ld();
      // only dS feeds the dQ product: its rounding to bf16 and the rounding of the rest
      if (__builtin_expect(see == 0xffffffffu, 1))
        ds_query<true>(sv, dpv, row_nlse2, row_ndelta, p.scale_log2, see, pds, rest);
      else
        ds_query<false>(sv, dpv, row_nlse2, row_ndelta, p.scale_log2, see, pds, rest);
      tmem_st16(tmem + lane_off + col_s(b) + 32 * hh, pds);
      tmem_st16(tmem + lane_off + col_dp(b) + 32 * hh, rest);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kB_PReady + b]);
    }
    if (N > 0 && ok && mbar_wait(&bars[kB_Done], 0, wd)) {
      tc_fence_after();
      const int64_t first = a0 + wq * 32;
      store_rows_staged<D / 2, false>(tmem + lane_off + kColAcc + hh * (D / 2), true, p.scale,
                                      smem + warp * kStageBytesF32, p.dq, (int64_t)bh_q * g.S + first, g.S - first, D,
                                      hh * (D / 2));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_grads_kernel(const __grid_constant__ CUtensorMap tm_q64, const __grid_constant__ CUtensorMap tm_do64,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k64, const __grid_constant__ CUtensorMap tm_v64,
                        const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  grid_let_next();
  if (blockIdx.x < p.plan.units)
    dkdv_unit<D>(tm_q64, tm_do64, tm_k, tm_v, p, smem, blockIdx.x);
  else
    dq_unit<D>(tm_q64, tm_do64, tm_k64, tm_v64, p, smem, blockIdx.x - p.plan.units);
}

Plan make_plan(const WinGeom& g) {
  Plan pl;
  const int rep = g.Hq / g.Hkv;
  const int64_t bh = (int64_t)g.B * g.Hkv;
  pl.tiles = (g.S + BT - 1) / BT;
  pl.sink_tiles = (g.sinks + BT - 1) / BT;
  // two units per SM keep the GPU busy to the end; fewer tiles than that are divided by heads
  pl.splits = 1;
  while (pl.splits < rep && bh * pl.tiles * pl.splits < 2 * 148) pl.splits = pl.splits * 2 < rep ? pl.splits * 2 : rep;
  // a sink tile's queries: runs of a plain tile's length, but no more runs than it takes to
  // give every SM four (many sink tiles are parallel by themselves)
  pl.segs = 1;
  if (pl.sink_tiles > 0) {
    int64_t s0, s1;
    tile_steps(g, 0, s0, s1);
    const int64_t plain = (g.window + BT) / TS + 1;
    const int64_t want = (s1 - s0 + plain - 1) / plain;
    const int64_t units = bh * pl.sink_tiles * pl.splits;
    const int64_t most = (4 * 148 + units - 1) / units;
    pl.segs = (int)(want < most ? want : most);
  }
  pl.sink_units = bh * pl.sink_tiles * pl.segs * pl.splits;
  pl.units = pl.sink_units + bh * (pl.tiles - pl.sink_tiles) * pl.splits;
  return pl;
}

int64_t plan_parts(const Plan& pl) {
  return (pl.segs * pl.splits > 1 ? pl.sink_units : 0) + (pl.splits > 1 ? pl.units - pl.sink_units : 0);
}

int64_t stat_rows(const WinGeom& g) { return (int64_t)g.B * g.Hq * ((g.S + BT - 1) / BT * BT); }

template <int D>
int launch(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout, void* dq,
           void* dk, void* dv, const WinGeom& g, float scale, float* scratch, int* status, uint64_t watchdog_ns,
           cudaStream_t stream) {
  const int64_t rows = stat_rows(g);
  Params p;
  p.g = g;
  p.plan = make_plan(g);
  p.nlse2 = scratch;
  p.ndelta = scratch + rows;
  p.s_pad = (g.S + BT - 1) / BT * BT;
  p.parts = scratch + 2 * rows;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.status = status;
  p.watchdog_ns = watchdog_ns;
  const int64_t prep_blocks = (rows + 256 / (D / 8) - 1) / (256 / (D / 8));
  const int64_t q_units = (int64_t)g.B * g.Hq * (p.s_pad / BT);
  if (prep_blocks > 0x7fffffff || p.plan.units + q_units > 0x7fffffff) return RING_ATTN_EINVAL;
  CUtensorMap mq, mdo, mk, mv, mk64, mv64;
  int rc;
  const int64_t bhq = (int64_t)g.B * g.Hq, bhk = (int64_t)g.B * g.Hkv;
  if ((rc = encode_rows_map(&mq, q, bhq, g.S, D, TS)) != 0) return rc;
  if ((rc = encode_rows_map(&mdo, dout, bhq, g.S, D, TS)) != 0) return rc;
  if ((rc = encode_rows_map(&mk, k, bhk, g.S, D, BT)) != 0) return rc;
  if ((rc = encode_rows_map(&mv, v, bhk, g.S, D, BT)) != 0) return rc;
  if ((rc = encode_rows_map(&mk64, k, bhk, g.S, D, TS)) != 0) return rc;
  if ((rc = encode_rows_map(&mv64, v, bhk, g.S, D, TS)) != 0) return rc;
  constexpr int smem = CfgA<D>::kSmemBytes > CfgB<D>::kSmemBytes ? CfgA<D>::kSmemBytes : CfgB<D>::kSmemBytes;
  if (cudaFuncSetAttribute(window_grads_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return RING_ATTN_ECUDA;
  window_prep_kernel<D><<<(unsigned)prep_blocks, 256, 0, stream>>>(
      static_cast<const uint16_t*>(out), static_cast<const uint16_t*>(dout), lse, scratch, scratch + rows, g.S, p.s_pad,
      rows, status);
  if (cudaGetLastError() != cudaSuccess) return RING_ATTN_ECUDA;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  if (launch_early(window_grads_kernel<D>, (unsigned)(p.plan.units + q_units), kThreads, smem, stream, mq, mdo, mk, mv,
                   mk64, mv64, p) != cudaSuccess)
    return RING_ATTN_ECUDA;
  const int64_t per_tile = bhk * 2 * BT * (D / 8);
  const int64_t sink_items = p.plan.segs * p.plan.splits > 1 ? per_tile * p.plan.sink_tiles : 0;
  const int64_t items = sink_items + (p.plan.splits > 1 ? per_tile * (p.plan.tiles - p.plan.sink_tiles) : 0);
  if (items == 0) return RING_ATTN_OK;
  if ((items + 255) / 256 > 0x7fffffff) return RING_ATTN_EINVAL;
  return launch_early(window_reduce_kernel<D>, (unsigned)((items + 255) / 256), 256, 0, stream, p, sink_items, items) ==
                 cudaSuccess
             ? RING_ATTN_OK
             : RING_ATTN_ECUDA;
}

}  // namespace winbwd

size_t window_bwd_scratch_bytes(const WinGeom& g) {
  return sizeof(float) * (2 * (size_t)winbwd::stat_rows(g) +
                          (size_t)winbwd::plan_parts(winbwd::make_plan(g)) * 2 * winbwd::BT * g.D);
}

// The backward kernels' walks on the host, for batch 0's first kv head: pass 0 every key
// unit with its query steps and column masks (a pair counts once per query head of the
// group), pass 1 the dQ kernel's.
int64_t window_bwd_visits(const WinGeom& g, int pass, int32_t* counts) {
  using namespace winbwd;
  int64_t visits = 0;
  if (pass == 0) {
    const Plan pl = make_plan(g);
    for (int64_t i = 0; i < pl.units; ++i) {
      const KeyUnit U = key_unit(g, pl, i);
      if (U.bh != 0) continue;
      for (int h = U.h0; h < U.h1; ++h)
        for (int64_t s = U.s0; s < U.s1; ++s, ++visits)
          for (int64_t u = U.kt * BT; u < (U.kt + 1) * BT; ++u) {
            int64_t in0, in1;
            inner_steps(g, U.kt, in0, in1);
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t see = key_sees(u, key_past(g, u), s, 32 * hh, in0, in1);
              for (int e = 0; e < 32; ++e)
                if (see >> e & 1) {
                  const int64_t t = s * TS + 32 * hh + e;
                  if (u >= g.S || t >= g.S) return -1;
                  counts[t * g.S + u] += 1;
                }
            }
          }
    }
    return visits;
  }
  for (int64_t a0 = 0; a0 < g.S; a0 += BT) {
    const WinTiles wt = win_tiles(g, a0, a0 + BT - 1, TS);
    for (int n = 0; n < win_count(wt); ++n, ++visits)
      for (int64_t a = a0; a < a0 + BT && a < g.S; ++a) {
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t see = query_sees(g, a0, a, (int64_t)win_tile(wt, n) * TS, 32 * hh);
          for (int e = 0; e < 32; ++e)
            if (see >> e & 1) counts[a * g.S + (int64_t)win_tile(wt, n) * TS + 32 * hh + e] += 1;
        }
      }
  }
  return visits;
}

int launch_window_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse, const void* dout,
                      void* dq, void* dk, void* dv, const WinGeom& g, float scale, float* scratch, int* status,
                      uint64_t watchdog_ns, cudaStream_t stream) {
  if (g.D == 64)
    return winbwd::launch<64>(q, k, v, out, lse, dout, dq, dk, dv, g, scale, scratch, status, watchdog_ns, stream);
  return winbwd::launch<128>(q, k, v, out, lse, dout, dq, dk, dv, g, scale, scratch, status, watchdog_ns, stream);
}

}  // namespace ringattn
