// Causal attention with a sliding window and sinks, forward, for sm_100a (bf16; D = 128 on
// CTA pairs, D = 64 and small problems on single CTAs).
//
// Mathematics: the blockwise online softmax of the ring kernels (softmax_rows.cuh) over the
// keys that win_tiles lists; lse = m + ln l. Exponentials come from the special-function
// unit alone, so lse is good to a few units in its last place.
//
// What bounds it: the tensor cores (4 D flops per visible pair). Keys and values come from L2, a
// unit's window and its own rows once: at D = 128 and a window of 4096 a unit of 512 queries
// reads 2.4 MB for 1.07 GFLOP, 2.2 TB/s at the rate below. P is rounded to bf16, the type of the V
// that it multiplies (l sums it unrounded): out is off from 64 bits by 1.2 to 1.4 times what
// rounding the result alone would cost. A unit is one or two query tiles of 128 * CTAS rows: in a pair one
// M = 256 product covers a tile of both CTAs and each CTA stages half of every K and V
// tile, which is what lets shared memory feed the products. Each query tile walks only the
// key tiles that its own rows see: of a unit's two tiles the first skips the key tiles past
// its diagonal, the second those that only the first one's window holds. That makes a
// row's overhead at most the two key tiles that its window and its diagonal cut. As built, the
// chain of a query tile (scores ready, exponentials, P, products) bounds it: tensor pipe 54 %
// busy, exponentials 54 %. 128k tokens, window 4096, 8 heads, D = 128: 2.22 to 2.26 ms, 973 to 992 TFLOP/s.
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
namespace winfwd {

constexpr int BM = 128;   // query rows of a tile in one CTA (TMEM lanes)
constexpr int BN = 128;   // keys per tile
constexpr int BOXW = 64;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr int kRegsSoftmax = 208;
constexpr int kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kLaunchRegs, "register split exceeds the launch pool");
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kProducerSleepNs = 64;
constexpr uint64_t kCopyGraceNs = 2000000;  // after a watchdog abort, see the producer
constexpr float kSpecMaxSum = 1048576.0f;   // 2^20, see the softmax
constexpr int kSmemLimit = 232448;
constexpr uint32_t kTmemCols = 512;

template <int D, int CTAS, int NQ>  // NQ: query tiles per unit, 1 or 2
struct Cfg {
  static constexpr int kQTileBytes = BM * D * 2;
  static constexpr int kQBoxBytes = BM * BOXW * 2;
  // what one CTA stages of a K or V tile: K keys [64 r, 64 r + 64) and V head-dim columns
  // [64 r, 64 r + 64) in a pair, the whole tile alone
  static constexpr int kPartBytes = BN * D * 2 / CTAS;
  static constexpr int kKRows = BN / CTAS;
  static constexpr int kKBoxBytes = kKRows * BOXW * 2;
  static constexpr int kVBoxBytes = BN * BOXW * 2;
  static constexpr int kVBoxes = D / BOXW / CTAS;
  static constexpr int kOffKV = NQ * kQTileBytes;
  static constexpr int kSlotsFit = (kSmemLimit - 1024 - 512 - kOffKV) / kPartBytes;
  static constexpr int kSlots = kSlotsFit < 10 ? kSlotsFit : 10;
  static constexpr int kOffBar = kOffKV + kSlots * kPartBytes;
  static constexpr int kNumBars = 8 + 2 * kSlots;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  static_assert(kSlots >= 4, "tiles n and n + 1 are held at once");
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
  static constexpr uint32_t kColS = 0;
  static constexpr uint32_t kColO = 2 * BN;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(CTAS * BM, BN, 0, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(CTAS * BM, D, 0, 1);
  static constexpr int kUnitRows = NQ * CTAS * BM;
};
enum Bar { kQFull = 0, kSFull = 1, kPReady = 3, kODone = 5, kDrain = 7, kRing = 8 };

struct Params {
  WinGeom g;
  void* out;
  float* lse;
  int* status;
  float scale_log2;
  int64_t blocks;  // units per head
  uint64_t watchdog_ns;
};

// The 32 query rows from a_warp see the whole key tile at k0: most tiles, which need no mask.
RA_HD bool warp_sees_all(const WinGeom& g, int64_t a_warp, int64_t k0) {
  return k0 + BN - 1 <= a_warp && (k0 > a_warp + 31 - g.window || k0 + BN <= g.sinks);
}
RA_HD uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
// Columns c0 .. c0 + 31 that a row with this cut sees.
RA_HD uint32_t cut_bits(const WinCut& cut, int c0) {
  return low_bits(cut.hi - c0) & (~low_bits(cut.lo - c0) | low_bits(cut.sk - c0));
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

template <int D, int CTAS, int NQ>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<D, CTAS, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  uint64_t* full = &bars[kRing];
  uint64_t* empty = &bars[kRing + C::kSlots];

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const WinGeom& g = p.g;

  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *p.status = RING_ATTN_OK;  // (no wait can have run out yet)
    mbar_init(&bars[kQFull], 1);
    for (int q = 0; q < NQ; ++q) {
      mbar_init(&bars[kSFull + q], 1);
      mbar_init(&bars[kPReady + q], CTAS * BM / 32);  // one arrival per softmax warp of each CTA
      mbar_init(&bars[kODone + q], 1);
    }
    mbar_init(&bars[kDrain], 1);
    for (int s = 0; s < 2 * C::kSlots; ++s) mbar_init(&bars[kRing + s], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    if (CTAS == 2) {
      tmem_alloc_2sm(tmem_slot, kTmemCols);
      tmem_relinquish_2sm();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  if (CTAS == 2) cluster_sync(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.status, p.watchdog_ns};

  // units: the heads of a GQA group innermost (they read the same K and V), then the row
  // blocks, then (b, kv head)
  int64_t u = blockIdx.x / CTAS;
  const int rep = g.Hq / g.Hkv;
  const int hr = (int)(u % rep);
  u /= rep;
  const int64_t tb = u % p.blocks;
  const int bh_kv = (int)(u / p.blocks);
  const int bh_q = bh_kv * rep + hr;  // b * Hq + kvh * rep + hr, as Hq = Hkv * rep
  const int64_t a0 = tb * C::kUnitRows;
  constexpr int kRowsQ = CTAS * BM;
  const WinTiles all = win_tiles(g, a0, a0 + C::kUnitRows - 1, BN);
  const int N = win_count(all);
  WinTiles tq[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) tq[q] = win_tiles(g, a0 + q * kRowsQ, a0 + (q + 1) * kRowsQ - 1, BN);

  if (warp >= 8) {
    regs_decrease<kRegsOther>();
    if (warp == kProducerWarp && lane == 0) {
      // ---------------------------------------------------------------- producer (every CTA)
      auto bar_addr = [&](uint64_t* bar) { return CTAS == 2 ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar); };
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int c0, int64_t row, int bh) {
        if (CTAS == 2)
          tma_load_4d_2sm(dst, tm, bar_addr(bar), c0, (int)row, 0, bh);
        else
          tma_load_4d(dst, tm, bar, c0, (int)row, 0, bh);
      };
      int n = 0;
      bool ok = N > 0;
      if (ok) {
        if (leader) mbar_arrive_expect_tx(&bars[kQFull], CTAS * NQ * C::kQTileBytes);
        for (int q = 0; q < NQ; ++q)
          for (int bx = 0; bx < D / BOXW; ++bx)
            load(smem + q * C::kQTileBytes + bx * C::kQBoxBytes, &tm_q, &bars[kQFull], bx * BOXW,
                 a0 + kRowsQ * q + BM * (int)rank, bh_q);
      }
      for (int i = 0; i < N && ok; ++i) {
        const int64_t k0 = (int64_t)win_tile(all, i) * BN;
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int slot = n % C::kSlots;
          const uint32_t ph = (uint32_t)(n / C::kSlots) & 1;
          if (!(ok = mbar_wait_backoff<CTAS == 2>(&empty[slot], ph ^ 1, wd, kProducerSleepNs))) break;
          if (leader) mbar_arrive_expect_tx(&full[slot], CTAS * C::kPartBytes);
          uint8_t* dst = smem + C::kOffKV + slot * C::kPartBytes;
          if (kv == 0) {
            for (int bx = 0; bx < D / BOXW; ++bx)
              load(dst + bx * C::kKBoxBytes, &tm_k, &full[slot], bx * BOXW, k0 + C::kKRows * (int)rank, bh_kv);
          } else {
            for (int bx = 0; bx < C::kVBoxes; ++bx)
              load(dst + bx * C::kVBoxBytes, &tm_v, &full[slot], (C::kVBoxes * (int)rank + bx) * BOXW, k0, bh_kv);
          }
        }
      }
      if (!ok && N > 0) {
        // wind down: this CTA's own copies must land before its shared memory goes away. In a
        // pair their bytes are counted on the leader's barriers, which the other CTA cannot
        // wait on, so both give them a fixed grace period (about 1000 times a tile copy's time).
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kCopyGraceNs) {
        }
      }
    } else if (warp == kMmaWarp && leader) {
      // ---------------------------------------------------------------- MMA issuer
      // (one thread: what passes between two products is time that the tensor pipe idles)
      if (elect_one_sync()) {
        const uint32_t sbase = smem_u32(smem);
        const uint64_t dq0 = smem_desc_sw128(sbase, 0, 1024);
        const uint64_t dk0 = smem_desc_sw128(sbase + C::kOffKV, 0, 1024);
        const uint64_t dv0 = smem_desc_sw128(sbase + C::kOffKV, C::kVBoxBytes, 1024);
        auto issue_s = [&](int q, int slot) {
          const uint64_t dq = dq0 + (uint64_t)((q * C::kQTileBytes) >> 4);
          const uint64_t dk = dk0 + (uint64_t)((slot * C::kPartBytes) >> 4);
          const uint32_t d = tmem + C::kColS + q * BN;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t da = dq + (((k / 4) * C::kQBoxBytes + (k % 4) * 32) >> 4);
            const uint64_t db = dk + (((k / 4) * C::kKBoxBytes + (k % 4) * 32) >> 4);
            if (CTAS == 2)
              mma_ss_2sm(d, da, db, C::kIdescQK, k > 0);
            else
              mma_ss(d, da, db, C::kIdescQK, k > 0);
          }
        };
        auto issue_pv = [&](int q, int slot, bool first) {
          const uint64_t dv = dv0 + (uint64_t)((slot * C::kPartBytes) >> 4);
          const uint32_t d = tmem + C::kColO + q * D;
          const uint32_t pa = tmem + C::kColS + q * BN;
#pragma unroll
          for (int k = 0; k < BN / 16; ++k) {
            if (CTAS == 2)
              mma_ts_2sm(d, pa + k * 8, dv + ((k * 16 * 128) >> 4), C::kIdescPV, !(first && k == 0));
            else
              mma_ts(d, pa + k * 8, dv + ((k * 16 * 128) >> 4), C::kIdescPV, !(first && k == 0));
          }
        };
        auto commit = [&](uint64_t* bar) {
          if (CTAS == 2)
            mma_commit_2sm(bar, 0x3);
          else
            mma_commit(bar);
        };
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
          return mbar_wait_cluster(bar, parity, wd);
        };
        auto kslot = [&](int n) { return (2 * n) % C::kSlots; };
        auto kphase = [&](int n) { return (uint32_t)((2 * n) / C::kSlots) & 1; };
        auto vslot = [&](int n) { return (2 * n + 1) % C::kSlots; };
        auto vphase = [&](int n) { return (uint32_t)((2 * n + 1) / C::kSlots) & 1; };
        int done[NQ], total[NQ];  // key tiles of query tile q: finished, all
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          done[q] = 0;
          total[q] = win_count(tq[q]);
        }
        bool ok = N > 0 && wait_all(&bars[kQFull], 0);
        if (ok) ok = wait_all(&full[kslot(0)], kphase(0));
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < NQ; ++q)
            if (win_has(tq[q], win_tile(all, 0))) {
              issue_s(q, kslot(0));
              commit(&bars[kSFull + q]);
            }
          commit(&empty[kslot(0)]);
        }
        // per key tile n: PV0(n), S0(n+1), PV1(n), S1(n+1), each only where the query tile meets
        // the key tile. The commit that reports S_q covers the query tile's last PV.
        for (int n = 0; ok && n < N; ++n) {
          const int tile = win_tile(all, n);
          const bool more = n + 1 < N;
          const int next = more ? win_tile(all, n + 1) : 0;
          if (!(ok = wait_all(&full[vslot(n)], vphase(n)))) break;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (win_has(tq[q], tile)) {
              if (!(ok = wait_all(&bars[kPReady + q], (uint32_t)(done[q] & 1)))) break;
              tc_fence_after();
              issue_pv(q, vslot(n), done[q] == 0);
              if (++done[q] == total[q]) commit(&bars[kODone + q]);
            }
            if (more && q == 0) {
              if (!(ok = wait_all(&full[kslot(n + 1)], kphase(n + 1)))) break;
              tc_fence_after();
            }
            if (more && win_has(tq[q], next)) {
              issue_s(q, kslot(n + 1));
              commit(&bars[kSFull + q]);
            }
          }
          if (!ok) break;
          commit(&empty[vslot(n)]);
          if (more) commit(&empty[kslot(n + 1)]);
        }
        commit(&bars[kDrain]);
        drain_wait(&bars[kDrain], 0, p.watchdog_ns);
      }
      __syncwarp();
    } else if (warp == kMmaWarp && lane == 0) {
      drain_wait(&bars[kDrain], 0, p.watchdog_ns);
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // -------------------------------------------------------------------- softmax (every CTA)
    const int q = warp / 4;
    const int wq = warp % 4;
    const int64_t a_warp = a0 + kRowsQ * q + BM * (int64_t)rank + wq * 32, a = a_warp + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::kColS + q * BN;
    const uint32_t tO = tmem + lane_off + C::kColO + q * D;
    const uint32_t leader_p = CTAS == 2 ? mapa_shared(smem_u32(&bars[kPReady + q]), 0) : 0;
    const float NEG_INF = -INFINITY;
    const WinTiles mine = q == 0 ? tq[0] : tq[NQ - 1];
    const int n_mine = q < NQ ? win_count(mine) : 0;
    float m_ref = NEG_INF;
    float l = 0.f;
    bool ok = true;
    for (int n = 0; n < n_mine; ++n) {
      const int64_t k0 = (int64_t)win_tile(mine, n) * BN;
      const bool whole = warp_sees_all(g, a_warp, k0);
      if (!(ok = mbar_wait_cluster(&bars[kSFull + q], (uint32_t)(n & 1), wd))) break;
      tc_fence_after();
      if (__builtin_expect(!whole, 0)) {
        // hidden scores are overwritten in place, by a loop: the straight path below stays short
        const WinCut cut = win_cut(g, a, k0, BN);
#pragma unroll 1
        for (int c0 = 0; c0 < BN; c0 += 32) {
          uint32_t x[32];
          tmem_ld32(tS + c0, x);
          const uint32_t see = cut_bits(cut, c0);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(see >> e & 1)) x[e] = 0xff800000u;  // -inf
          tmem_st32(tS + c0, x);
        }
        tmem_wait_st();
      }
      // Exponentials against the current reference maximum first: O / l and lse do not
      // depend on it, so a block whose row sums stay <= kSpecMaxSum (every P <= 2^20) is
      // kept as is. Otherwise, and for a row's first block, the warp takes the block maximum
      // and moves the reference where that exceeds it by more than kRescaleLog2.
      uint32_t pk[BN / 2];
      float lb;
      bool fast = __all_sync(0xffffffffu, m_ref != NEG_INF);
#pragma unroll 1
      while (true) {
        uint32_t sr[BN];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
        tmem_wait_ld();
        if (!fast) {
          const float mblk = raw_rowmax<BN>(sr) * p.scale_log2;
          float alpha = 1.f;
          bool resc = false;
          if (mblk > m_ref + kRescaleLog2) {
            alpha = (m_ref == NEG_INF) ? 0.f : ex2_approx(m_ref - mblk);
            l *= alpha;
            m_ref = mblk;
            resc = true;
          }
          // S ready for this tile implies that this query tile's last PV completed: O is
          // stable (and not yet written before its first PV, which overwrites it)
          if (n > 0 && __any_sync(0xffffffffu, resc)) rescale_o<D>(tO, alpha);
        }
        lb = exp_pack_phased<BN, 0>(sr, p.scale_log2, (m_ref == NEG_INF) ? 0.f : m_ref, pk);
        if (!fast || __all_sync(0xffffffffu, lb <= kSpecMaxSum)) break;
        fast = false;
      }
      l += lb;
#pragma unroll
      for (int c = 0; c < BN / 64; ++c) tmem_st32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[c * 32]));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 2)
          mbar_arrive_cluster(leader_p);
        else
          mbar_arrive(&bars[kPReady + q]);
      }
    }
    if (n_mine > 0 && ok && mbar_wait_cluster(&bars[kODone + q], 0, wd)) {
      tc_fence_after();
      const bool row_ok = a < g.S;
      const float inv_l = l > 0.f ? 1.f / l : 0.f;
      const int64_t row = (int64_t)bh_q * g.S + a;
      // (this query tile's products are done: its Q is not needed any more)
      store_rows_staged<D, false>(tO, true, inv_l, smem + q * C::kQTileBytes + wq * kStageBytesBf16, p.out,
                                  (int64_t)bh_q * g.S + a_warp, g.S - a_warp, D, 0);
      if (row_ok) p.lse[row] = (m_ref + log2f(l)) * 0.69314718055994530942f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();  // the leader's MMAs read this CTA's shared and tensor memory until here
  if (warp == kMmaWarp) {
    tc_fence_after();
    if (CTAS == 2)
      tmem_dealloc_2sm(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int CTAS, int NQ>
int launch(const void* q, const void* k, const void* v, void* out, float* lse, const WinGeom& g, float scale,
           int* status, uint64_t watchdog_ns, cudaStream_t stream) {
  using C = Cfg<D, CTAS, NQ>;
  CUtensorMap mq, mk, mv;
  int rc;
  if ((rc = encode_rows_map(&mq, q, (int64_t)g.B * g.Hq, g.S, D, BM)) != 0) return rc;
  if ((rc = encode_rows_map(&mk, k, (int64_t)g.B * g.Hkv, g.S, D, C::kKRows)) != 0) return rc;
  if ((rc = encode_rows_map(&mv, v, (int64_t)g.B * g.Hkv, g.S, D, BN)) != 0) return rc;
  Params p;
  p.g = g;
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.blocks = (g.S + C::kUnitRows - 1) / C::kUnitRows;
  p.watchdog_ns = watchdog_ns;
  auto kern = window_fwd_kernel<D, CTAS, NQ>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
    return RING_ATTN_ECUDA;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return RING_ATTN_ECUDA;
  if (fa.numRegs * kThreads < 128 * (2 * kRegsSoftmax + kRegsOther)) return RING_ATTN_EUNSUPPORTED;
  const int64_t ctas = (int64_t)g.B * g.Hq * p.blocks * CTAS;
  if (ctas > 0x7fffffff) return RING_ATTN_EINVAL;
  kern<<<(unsigned)ctas, kThreads, C::kSmemBytes, stream>>>(mq, mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

// CTAs of a unit and its query tiles. Where one CTA per query tile of 128 rows still runs in
// one wave, that is the shorter chain: a tile's softmax has the special-function unit to
// itself (window 256, 4 heads, us, alone / in units: D = 64, S 1024 12.7 / 17.5 and 4096 14.8 /
// 19.4; D = 128 14.5 / 26.7 and 15.0 / 27.2). Past one wave the units' shared key tiles win
// (D = 64, S 8192: 24.5 / 19.4; D = 128, window 2048, S 8192: 75.8 / 54.4).
struct Shape {
  int ctas, nq;
};
Shape shape_of(const WinGeom& g) {
  if ((int64_t)g.B * g.Hq * ((g.S + BM - 1) / BM) <= 148) return {1, 1};
  return {g.D == 64 ? 1 : 2, 2};
}

}  // namespace winfwd

int launch_window_fwd(const void* q, const void* k, const void* v, void* out, float* lse, const WinGeom& g,
                      float scale, int* status, uint64_t watchdog_ns, cudaStream_t stream) {
  const winfwd::Shape x = winfwd::shape_of(g);
  if (g.D == 64)
    return x.nq == 1 ? winfwd::launch<64, 1, 1>(q, k, v, out, lse, g, scale, status, watchdog_ns, stream)
                     : winfwd::launch<64, 1, 2>(q, k, v, out, lse, g, scale, status, watchdog_ns, stream);
  return x.nq == 1 ? winfwd::launch<128, 1, 1>(q, k, v, out, lse, g, scale, status, watchdog_ns, stream)
                   : winfwd::launch<128, 2, 2>(q, k, v, out, lse, g, scale, status, watchdog_ns, stream);
}

// The forward kernel's walk on the host: per unit the union of tiles in order, each query
// tile taking those that win_has lists for it, the masks as the softmax applies them.
int64_t window_fwd_visits(const WinGeom& g, int32_t* counts) {
  const winfwd::Shape x = winfwd::shape_of(g);
  const int rows_q = x.ctas * winfwd::BM;
  int64_t visits = 0;
  for (int64_t a0 = 0; a0 < g.S; a0 += x.nq * rows_q) {
    const WinTiles all = win_tiles(g, a0, a0 + x.nq * rows_q - 1, winfwd::BN);
    for (int q = 0; q < x.nq; ++q) {
      const WinTiles t = win_tiles(g, a0 + q * rows_q, a0 + (q + 1) * rows_q - 1, winfwd::BN);
      int n = 0;
      for (int i = 0; i < win_count(all); ++i) {
        const int tile = win_tile(all, i);
        if (!win_has(t, tile)) continue;
        if (win_tile(t, n) != tile) return -1;  // the query tile's own order
        ++n;
        ++visits;
        for (int64_t a = a0 + q * rows_q; a < a0 + (q + 1) * rows_q && a < g.S; ++a) {
          const int64_t k0 = (int64_t)tile * winfwd::BN;
          const bool whole = winfwd::warp_sees_all(g, a - (a - a0) % 32, k0);
          const WinCut cut = win_cut(g, a, k0, winfwd::BN);
          for (int c0 = 0; c0 < winfwd::BN; c0 += 32) {
            const uint32_t see = whole ? 0xffffffffu : winfwd::cut_bits(cut, c0);
            for (int e = 0; e < 32; ++e)
              if (see >> e & 1) counts[a * g.S + k0 + c0 + e] += 1;
          }
        }
      }
      if (n != win_count(t)) return -1;
    }
  }
  return visits;
}

}  // namespace ringattn
