// Attention of drafted tokens over a cache, for many query rows per kv head (more than one
// warp tile's 16), on tcgen05 (bf16, mxfp8 or mxfp4 cache; D = 64 or 128).
//
// Mathematics: as in tree_rows.cu. A group is 128 query rows, the rows of one M = 128
// product: S = Q K^T with Q in tensor memory, O += P V with P in tensor memory, 128 cache
// rows at a time.
//
// What bounds it: the tensor cores (4 * 128 * 128 * D flops per tile of 128 rows, whatever
// part of the group's rows is real) once a cache row is used by more rows than its bytes pay
// for; before that the conversion of codes, 2.3 instructions per element on 7 warps. The
// cache's rows come in as they are (each converting thread copies and later reads its own 16
// bytes, so the ring of raw tiles needs no barrier), are converted to bf16 in registers and
// written once into the swizzled K and V tiles that the products read. bf16 rows are copied
// straight into those tiles.
//
// Roles (512 threads): warps 0-7 softmax (warp w: rows 32 (w % 4) .., keys 64 (w / 4) .. of a
// tile; the two warps of a row agree on its maximum through shared memory), warp 8 issues the
// products, warps 9-15 fill the tiles. Tensor memory: S double-buffered [0,128) and
// [128,256), O [256,384), Q [384,448). Every role walks the CTA's share of the work by itself
// (tree_common.cuh), so tiles of the next unit are filled while the last one is finished.
//
// Codes to bf16: the bits of tree_rows.cu's bf16 form, one multiplication. To keep its factor
// inside bf16's range, K and V are held 2^40 too small and Q and P 2^40 too large (exact);
// blocks whose scale byte is above 160 take two multiplications. Elements are written in the
// order that the bit operations give (4 codes: 0 2 1 3, 8 codes: 0 4 1 5 2 6 3 7); Q is
// stored in the same order and the output put back.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sm100_ptx.cuh"
#include "softmax_rows.cuh"
#include "tree_common.cuh"

namespace ringattn {
namespace tree {
namespace tiles {

constexpr int TK = 128;   // cache rows per tile
constexpr int TM = 128;   // query rows per group
constexpr int kThreads = 512;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 8;
constexpr int kFillWarp = 9;  // first of the filling warps
constexpr int kFillWarps = 7;
constexpr int kFill = 32 * kFillWarps;
constexpr int kBoxBytes = TK * 128;  // 128 rows x 64 elements
constexpr int kSmemLimit = 232448;
constexpr uint32_t kTmemCols = 512, kColO = 256, kColQ = 384;
constexpr float kRescale = 8.f;

template <int FMT, int D>
struct Cfg {
  static constexpr bool kMx = FMT != RING_ATTN_CACHE_BF16;
  static constexpr int kRowBytes = cache_row_bytes<FMT>(D);
  static constexpr int kChunks = kRowBytes / 16;       // per row
  static constexpr int kTileChunks = TK * kChunks;
  static constexpr int kPer = (kTileChunks + kFill - 1) / kFill;  // chunks per filling thread and tile
  static constexpr int kTileBytes = TK * D * 2;        // a bf16 tile
  static constexpr int kOffV = 2 * kTileBytes;
  static constexpr int kOffRaw = 4 * kTileBytes;
  static constexpr int kRawBytes = kMx ? 2 * kPer * kFill * 20 : 0;  // codes and scale words of K and V
  static constexpr int kRawFit = kMx ? (kSmemLimit - 1024 - 2048 - kOffRaw - 512) / kRawBytes : 0;
  static constexpr int kRaw = kRawFit < 4 ? kRawFit : 4;
  static_assert(!kMx || kRaw >= 2, "a tile is fetched while another is converted");
  static constexpr int kOffMax = kOffRaw + kRaw * kRawBytes;  // [2][2][128] floats
  static constexpr int kOffBar = kOffMax + 2048;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
  static constexpr float kLift = kMx ? 40.f : 0.f;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(TM, TK, 0, 0);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(TM, D, 0, 1);
};
enum Bar { kKFull = 0, kVFull = 2, kKFree = 4, kVFree = 6, kSFull = 8, kPReady = 10, kPvDone = 12, kQReady = 13,
           kODone = 14, kDrain = 15, kPair = 16, kNumBars = 20 };

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void store16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src));
  return v;
}
__device__ __forceinline__ uint32_t load4(uint32_t src) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src));
  return v;
}

// Bits c of [lo, hi) in 0..31 for a chunk of columns that starts at c0.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int c0) {
  lo = max(lo - c0, 0);
  hi = min(hi - c0, 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - (hi - lo))) << lo;
}
__device__ __forceinline__ int clip(int64_t x) { return x <= 0 ? 0 : (x >= TK ? TK : (int)x); }

// The CTA's tiles one by one (of all its parts).
struct TileIter {
  Walk walk;
  Part part;
  int i;
  bool valid;
  __device__ __forceinline__ void begin(const Params& p, const Walk& w) {
    walk = w;
    valid = next_part(p, walk, part);
    i = valid ? part.q0 : 0;
  }
  __device__ __forceinline__ void next(const Params& p) {
    if (++i < part.q1) return;
    valid = next_part(p, walk, part);
    i = valid ? part.q0 : 0;
  }
};

template <int FMT, int D>
struct Fill {
  using C = Cfg<FMT, D>;

  // Raw copies of one tile into this thread's ring slot.
  static __device__ __forceinline__ void fetch(const Params& p, const TileIter& it, uint32_t slot, int ct) {
    const int kb = step_key(p, it.part.ks, it.i);
    const int64_t first = it.part.head_row + kb;
    constexpr int kScaleRow = D / kMxBlock;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* rows = static_cast<const uint8_t*>(kv ? p.c.v : p.c.k) + first * C::kRowBytes;
      const uint8_t* sc = static_cast<const uint8_t*>(kv ? p.c.v_scale : p.c.k_scale);
#pragma unroll
      for (int i = 0; i < C::kPer; ++i) {
        const int idx = ct + i * kFill;
        if (idx < C::kTileChunks) {
          const int row = idx / C::kChunks;
          const bool live = key_live(p, it.part.ks, kb + row);
          copy16(slot + ((kv * C::kPer + i) * kFill + ct) * 16, rows + (live ? idx * 16 : 0), live);
          // the word that holds the row's scale bytes (with D = 64 its pair's too)
          const int64_t at = ((first + (live ? row : 0)) * kScaleRow) & ~(int64_t)3;
          copy4(slot + 2 * C::kPer * kFill * 16 + ((kv * C::kPer + i) * kFill + ct) * 4, sc + at, live);
        }
      }
    }
  }

  // This thread's chunks of K (kv = 0) or V to bf16, into the swizzled tile at `dst`.
  static __device__ __forceinline__ void convert(uint32_t slot, int kv, uint32_t dst, int ct) {
#pragma unroll
    for (int i = 0; i < C::kPer; ++i) {
      const int idx = ct + i * kFill;
      if (idx >= C::kTileChunks) break;
      const int row = idx / C::kChunks, ch = idx % C::kChunks;
      const uint4 w4 = load16(slot + ((kv * C::kPer + i) * kFill + ct) * 16);
      const uint32_t sw = load4(slot + 2 * C::kPer * kFill * 16 + ((kv * C::kPer + i) * kFill + ct) * 4);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      const int blk = FMT == RING_ATTN_CACHE_MXFP8 ? ch / 2 : ch;
      const uint32_t byte = sw >> (8 * (D == 64 ? 2 * (row & 1) + blk : blk)) & 255u;
      // held value = raw * 2^120 (or 126) * 2^(byte - 127) * 2^-40
      constexpr int kUp = (FMT == RING_ATTN_CACHE_MXFP8 ? 120 : 126) - 40;
      const bool far = byte > 160u;
      uint32_t f = ((far ? byte - 100u : byte) + kUp) << 7;
      if (byte == 255u) f = 0x7fc0u;
      f *= 0x10001u;
      const uint32_t row_at = dst + row * 128;
      auto put = [&](uint32_t (&v)[4], int c16) {  // 16-byte chunk c16 of the row's D elements
        if (far) {
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = mul2(v[x], 0x71807180u);  // 2^100
        }
        store16(row_at + (c16 / 8) * kBoxBytes + (((c16 % 8) ^ (row & 7)) * 16), v[0], v[1], v[2], v[3]);
      };
      if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
        // lanes of the row's two halves write their two chunks in opposite order (bank conflicts)
        const int flip = ch / 4 & 1;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int y = x ^ flip;
          const uint32_t a = y ? w[2] : w[0], b = y ? w[3] : w[1];
          const uint32_t a8 = a << 8, b8 = b << 8;
          uint32_t v[4] = {mul2(((a8 >> 4) & 0x07f007f0u) | (a8 & 0x80008000u), f),
                           mul2(((a >> 4) & 0x07f007f0u) | (a & 0x80008000u), f),
                           mul2(((b8 >> 4) & 0x07f007f0u) | (b8 & 0x80008000u), f),
                           mul2(((b >> 4) & 0x07f007f0u) | (b & 0x80008000u), f)};
          put(v, 2 * ch + y);
        }
      } else {
        // chunk ch: elements 32 ch .., one output chunk per word
        const int flip = ch >> 1 << 1;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int y = x ^ flip;
          const uint32_t a = y == 0 ? w[0] : (y == 1 ? w[1] : (y == 2 ? w[2] : w[3]));
          const uint32_t a0 = a << 12, a1 = a << 8, a2 = a << 4;
          uint32_t v[4] = {mul2(((a0 >> 6) & 0x01c001c0u) | (a0 & 0x80008000u), f),
                           mul2(((a1 >> 6) & 0x01c001c0u) | (a1 & 0x80008000u), f),
                           mul2(((a2 >> 6) & 0x01c001c0u) | (a2 & 0x80008000u), f),
                           mul2(((a >> 6) & 0x01c001c0u) | (a & 0x80008000u), f)};
          put(v, 4 * ch + y);
        }
      }
    }
  }

  // bf16 rows straight into the swizzled tile.
  static __device__ __forceinline__ void copy_tile(const Params& p, const TileIter& it, const void* base, uint32_t dst,
                                                   int ct) {
    const int kb = step_key(p, it.part.ks, it.i);
    const uint8_t* rows = static_cast<const uint8_t*>(base) + (it.part.head_row + kb) * C::kRowBytes;
#pragma unroll 4
    for (int idx = ct; idx < C::kTileChunks; idx += kFill) {
      const int row = idx / C::kChunks, ch = idx % C::kChunks;
      const bool live = key_live(p, it.part.ks, kb + row);
      copy16(dst + (ch / 8) * kBoxBytes + row * 128 + (((ch % 8) ^ (row & 7)) * 16), rows + (live ? idx * 16 : 0), live);
    }
  }
};

// Query elements 8 at a time (16 bytes, memory order) in the order of the tiles' elements.
template <int FMT>
__device__ __forceinline__ void order8(uint4 v, uint32_t (&x)[4]) {
  if (FMT == RING_ATTN_CACHE_BF16) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else if (FMT == RING_ATTN_CACHE_MXFP8) {
    x[0] = __byte_perm(v.x, v.y, 0x5410); x[1] = __byte_perm(v.x, v.y, 0x7632);
    x[2] = __byte_perm(v.z, v.w, 0x5410); x[3] = __byte_perm(v.z, v.w, 0x7632);
  } else {
    x[0] = __byte_perm(v.x, v.z, 0x5410); x[1] = __byte_perm(v.x, v.z, 0x7632);
    x[2] = __byte_perm(v.y, v.w, 0x5410); x[3] = __byte_perm(v.y, v.w, 0x7632);
  }
}
// Place of head dimension e (of 8) among the tiles' elements.
template <int FMT>
__host__ __device__ constexpr int place8(int e) {
  return FMT == RING_ATTN_CACHE_BF16 ? e
         : FMT == RING_ATTN_CACHE_MXFP8 ? (e & 4) + (e % 4 == 1 ? 2 : (e % 4 == 2 ? 1 : e % 4))
                                        : (e < 4 ? 2 * e : 2 * (e - 4) + 1);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_tiles_kernel(const Params p) {
  using C = Cfg<FMT, D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Walk s_walk;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + kNumBars * 8 + 8);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *p.status = RING_ATTN_OK;
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kKFull + b], kFillWarps);
      mbar_init(&bars[kVFull + b], kFillWarps);
      mbar_init(&bars[kKFree + b], 1);
      mbar_init(&bars[kVFree + b], 1);
      mbar_init(&bars[kSFull + b], 1);
      mbar_init(&bars[kPReady + b], kSoftmaxWarps);
    }
    mbar_init(&bars[kPvDone], 1);
    mbar_init(&bars[kQReady], kSoftmaxWarps);
    mbar_init(&bars[kODone], 1);
    mbar_init(&bars[kDrain], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[kPair + i], 2);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0) warp_begin_walk(p, &s_walk);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{abort_flag, p.status, p.watchdog_ns};
  const uint32_t sbase = smem_u32(smem);

  if (warp >= kFillWarp) {
    // ------------------------------------------------------------------ fill the tiles
    const int ct = threadIdx.x - 32 * kFillWarp;
    using F = Fill<FMT, D>;
    TileIter it;
    it.begin(p, s_walk);
    auto all = [&](bool r) { return __all_sync(0xffffffffu, r) != 0; };
    auto ready = [&](uint64_t* bar) {  // this warp's part is written: visible to the products
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if constexpr (C::kMx) {
      const uint32_t raw = sbase + C::kOffRaw;
      int fetched = 0;
      auto fetch = [&]() {
        if (it.valid) {
          F::fetch(p, it, raw + (fetched % C::kRaw) * C::kRawBytes, ct);
          it.next(p);
          ++fetched;
        }
        copy_commit();
      };
#pragma unroll 1
      for (int i = 0; i < C::kRaw - 1; ++i) fetch();
#pragma unroll 1
      for (int t = 0;; ++t) {
        fetch();
        if (t >= fetched) break;
        copy_wait<C::kRaw - 1>();
        const uint32_t slot = raw + (t % C::kRaw) * C::kRawBytes;
        const uint32_t par = (uint32_t)(t >> 1 & 1) ^ 1;
        if (!all(mbar_wait(&bars[kKFree + (t & 1)], par, wd))) break;
        F::convert(slot, 0, sbase + (t & 1) * C::kTileBytes, ct);
        ready(&bars[kKFull + (t & 1)]);
        if (!all(mbar_wait(&bars[kVFree + (t & 1)], par, wd))) break;
        F::convert(slot, 1, sbase + C::kOffV + (t & 1) * C::kTileBytes, ct);
        ready(&bars[kVFull + (t & 1)]);
      }
      copy_wait<0>();
    } else {
      int t = 0;
      bool ok = true;
      for (; it.valid; ++t) {
        const uint32_t par = (uint32_t)(t >> 1 & 1) ^ 1;
        if (!(ok = all(mbar_wait(&bars[kKFree + (t & 1)], par, wd)))) break;
        F::copy_tile(p, it, p.c.k, sbase + (t & 1) * C::kTileBytes, ct);
        copy_commit();
        if (t > 0) {  // the tile before: its K and V have landed once only this K is in flight
          copy_wait<1>();
          ready(&bars[kKFull + (t - 1 & 1)]);
          ready(&bars[kVFull + (t - 1 & 1)]);
        }
        if (!(ok = all(mbar_wait(&bars[kVFree + (t & 1)], par, wd)))) break;
        F::copy_tile(p, it, p.c.v, sbase + C::kOffV + (t & 1) * C::kTileBytes, ct);
        copy_commit();
        it.next(p);
      }
      copy_wait<0>();
      if (ok && t > 0) {
        ready(&bars[kKFull + (t - 1 & 1)]);
        ready(&bars[kVFull + (t - 1 & 1)]);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ products
    const bool issuer = elect_one_sync();
    auto all = [&](bool r) { return __all_sync(0xffffffffu, r) != 0; };
    Walk walk = s_walk;
    Part part;
    int t0 = 0, parts = 0;
    bool ok = true;
    while (ok && next_part(p, walk, part)) {
      const int n_tiles = part.q1 - part.q0;
      auto issue_s = [&](int t) -> bool {
        if (!all(mbar_wait(&bars[kKFull + (t & 1)], (uint32_t)(t >> 1 & 1), wd))) return false;
        tc_fence_after();
        const uint64_t dk = smem_desc_sw128(sbase + (t & 1) * C::kTileBytes, 0, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          if (issuer)
            mma_ts(tmem + 128 * (t & 1), tmem + kColQ + 8 * k, dk + (uint64_t)(((k / 4) * kBoxBytes + (k % 4) * 32) >> 4),
                   C::kIdescS, k > 0);
        if (issuer) {
          mma_commit(&bars[kSFull + (t & 1)]);
          mma_commit(&bars[kKFree + (t & 1)]);
        }
        return true;
      };
      if (!(ok = all(mbar_wait(&bars[kQReady], (uint32_t)(parts & 1), wd)))) break;
      tc_fence_after();
      ok = issue_s(t0);
      if (ok && n_tiles > 1) ok = issue_s(t0 + 1);
      for (int n = 0; ok && n < n_tiles; ++n) {
        const int t = t0 + n;
        if (!(ok = all(mbar_wait(&bars[kVFull + (t & 1)], (uint32_t)(t >> 1 & 1), wd)))) break;
        if (!(ok = all(mbar_wait(&bars[kPReady + (t & 1)], (uint32_t)(t >> 1 & 1), wd)))) break;
        tc_fence_after();
        const uint64_t dv = smem_desc_sw128(sbase + C::kOffV + (t & 1) * C::kTileBytes, kBoxBytes, 1024);
#pragma unroll
        for (int k = 0; k < TK / 16; ++k)
          if (issuer)
            mma_ts(tmem + kColO, tmem + 128 * (t & 1) + 8 * k, dv + (uint64_t)((k * 16 * 128) >> 4), C::kIdescO,
                   !(n == 0 && k == 0));
        if (issuer) {
          mma_commit(&bars[kPvDone]);
          mma_commit(&bars[kVFree + (t & 1)]);
          if (n + 1 == n_tiles) mma_commit(&bars[kODone]);
        }
        if (n + 2 < n_tiles && !(ok = issue_s(t + 2))) break;
      }
      t0 += n_tiles;
      ++parts;
    }
    // every product this thread issued must finish before tensor memory is released
    if (issuer) mma_commit(&bars[kDrain]);
    const uint64_t since = global_timer_ns();
    while (!mbar_try_wait(&bars[kDrain], 0)) {
      if (global_timer_ns() - since > p.watchdog_ns) break;
    }
  } else {
    // ------------------------------------------------------------------ softmax and epilogue
    const int wq = warp % 4, hh = warp / 4;
    const int r = 32 * wq + lane;  // row of the group
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    float* s_x = reinterpret_cast<float*>(smem + C::kOffMax);  // [use & 1][half][row]
    int uses = 0;                                              // of the pair's exchange
    // hands this row's value to the warp with the other half of its keys and takes that one's
    auto exchange = [&](float mine, float& other) -> bool {
      float* at = s_x + (uses & 1) * 256;
      at[hh * 128 + r] = mine;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kPair + wq]);
      if (!mbar_wait(&bars[kPair + wq], (uint32_t)(uses & 1), wd)) return false;
      tc_fence_after();
      other = at[(hh ^ 1) * 128 + r];
      ++uses;
      return true;
    };
    Walk walk = s_walk;
    Part part;
    int t0 = 0, parts = 0;
    bool ok = true;
    while (ok && next_part(p, walk, part)) {
      const Keys& ks = part.ks;
      const int n_tiles = part.q1 - part.q0;
      const int row = part.grp * TM + r;
      const bool live = row < ks.cnt * p.rep;
      const int node = live ? row / p.rep : 0;
      {
        // half a query row into tensor memory
        const uint16_t* src = p.q + part.b * p.qs_b + (int64_t)(part.kvh * p.rep + (live ? row % p.rep : 0)) * p.qs_h +
                              node * p.qs_t + hh * (D / 2);
        uint32_t x[D / 4];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0, 0, 0, 0);
          uint32_t y[4];
          order8<FMT>(v, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * c + e] = C::kMx ? mul2(y[e], 0x53805380u) : y[e];  // 2^40
        }
        if constexpr (D == 128)
          tmem_st32(tmem + lane_off + kColQ + 32 * hh, x);
        else
          tmem_st16(tmem + lane_off + kColQ + 16 * hh, x);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kQReady]);
      }
      const Nodes nodes = warp_nodes(p, part.b, ks);
      uint64_t seen;
      int depth;
      node_of(nodes, node, seen, depth);
      const int lo_key = p.window > 0 ? ks.n + depth - p.window + 1 : 0;
      float m = -INFINITY, l = 0.f;  // reference (a whole number), sum of this half
      for (int n = 0; n < n_tiles; ++n) {
        const int t = t0 + n;
        const int kb = step_key(p, ks, part.q0 + n);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[kSFull + (t & 1)], (uint32_t)(t >> 1 & 1), wd)) != 0)) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + 128 * (t & 1);
        uint32_t sr[64];
        tmem_ld32(tS + 64 * hh, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(tS + 64 * hh + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_wait_ld();
        // every row sees the whole tile
        const bool whole = kb + TK <= ks.n &&
                           (p.window <= 0 || kb + TK <= p.sinks || (int64_t)kb >= (int64_t)ks.n + p.T - p.window);
        if (!whole) {
          const int hi = clip((int64_t)ks.n - kb), lo = clip((int64_t)lo_key - kb), sk = min(clip((int64_t)p.sinks - kb), hi);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int c0 = 64 * hh + 32 * c;
            const int64_t j0 = (int64_t)kb + c0 - ks.n;  // drafted node of the chunk's first column
            const uint32_t drafts = j0 >= 64 || j0 <= -32 ? 0u : (uint32_t)(j0 >= 0 ? seen >> j0 : seen << -j0);
            const uint32_t see = span_bits(lo, hi, c0) | span_bits(0, sk, c0) | drafts;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see >> e & 1)) sr[32 * c + e] = 0xff800000u;  // -inf
          }
        }
        const float mine = raw_rowmax<64>(sr) * p.scale_log2;
        float other;
        if (!(ok = __all_sync(0xffffffffu, exchange(mine, other)) != 0)) break;
        const float top = fmaxf(mine, other);
        bool moved = false;
        float alpha = 1.f;
        if (top > m + kRescale || (m == -INFINITY && top != -INFINITY)) {
          const float to = ceilf(top);
          alpha = m == -INFINITY ? 0.f : ex2_approx(m - to);
          l *= alpha;
          m = to;
          moved = true;
        }
        if (n > 0 && __any_sync(0xffffffffu, moved)) {
          // S of this tile was issued before the last P V: O must hold every product so far
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[kPvDone], (uint32_t)((t - 1) & 1), wd)) != 0)) break;
          tc_fence_after();
          rescale_o<D / 2>(tmem + lane_off + kColO + hh * (D / 2), alpha);
        }
        uint32_t pk[32];
        l += exp_pack<64, 0>(sr, p.scale_log2, m == -INFINITY ? 0.f : m - C::kLift, pk);
        // packed P takes the columns of keys that both halves have loaded (see exchange)
        tmem_st32(tS + 32 * hh, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPReady + (t & 1)]);
      }
      if (!ok) break;
      float l_other;
      if (!(ok = __all_sync(0xffffffffu, exchange(l, l_other)) != 0)) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[kODone], (uint32_t)(parts & 1), wd)) != 0)) break;
      tc_fence_after();
      const float down = C::kMx ? 0x1p-40f : 1.f;  // l carries 2^40
      const float L = (hh == 0 ? l + l_other : l_other + l) * down;
      const bool none = m == -INFINITY;
      const float inv = none ? 0.f : 1.f / L;
      const float lse2 = none ? -INFINITY : m + log2f(L);
      const int64_t slot = (int64_t)blockIdx.x + part.unit;
      const int64_t orow = live ? out_row(p, part.b, part.kvh, row) : 0;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_off + kColO + hh * (D / 2) + 32 * c, o);
        tmem_wait_ld();
        if (live) {
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[(e & ~7) + place8<FMT>(e & 7)]) * inv;
          const int d0 = hh * (D / 2) + 32 * c;
          if (part.alone) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + d0);
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              dst[e / 8] = make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                                      pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
          } else {
            float* dst = p.o_parts + (slot * TM + r) * D + d0;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
      }
      if (live && hh == 0) {
        if (part.alone)
          p.lse[orow] = lse2 * 0.69314718055994530942f;
        else
          p.lse_parts[slot * TM + r] = lse2;
      }
      tc_fence_before();  // O is read before the next part's products (issued after its queries arrive)
      t0 += n_tiles;
      ++parts;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int FMT, int D>
int launch(const Params& p, cudaStream_t stream) {
  constexpr int smem = Cfg<FMT, D>::kSmemBytes;
  auto kern = tree_tiles_kernel<FMT, D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return RING_ATTN_ECUDA;
  kern<<<p.ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

template <int FMT>
int launch_d(const Params& p, cudaStream_t stream) {
  return p.c.D == 64 ? launch<FMT, 64>(p, stream) : launch<FMT, 128>(p, stream);
}

}  // namespace tiles

int launch_tiles(const Params& p, cudaStream_t stream) {
  switch (p.c.format) {
    case RING_ATTN_CACHE_BF16: return tiles::launch_d<RING_ATTN_CACHE_BF16>(p, stream);
    case RING_ATTN_CACHE_MXFP8: return tiles::launch_d<RING_ATTN_CACHE_MXFP8>(p, stream);
    default: return tiles::launch_d<RING_ATTN_CACHE_MXFP4>(p, stream);
  }
}

}  // namespace tree
}  // namespace ringattn
