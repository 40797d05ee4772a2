// Attention of drafted tokens over a cache, for many query rows per kv head (more than one
// warp tile's 16), on tcgen05 (bf16, mxfp8 or mxfp4 cache; D = 64 or 128).
//
// Mathematics: as in tree_rows.cu. A group is 128 query rows, the rows of one M = 128
// product: S = Q K^T with Q in tensor memory, O += P V with P in tensor memory, 128 cache
// rows at a time.
//
// Floors: the tensor cores (4 * 128 * 128 * D flops per tile of 128 rows, whatever part of
// the group's rows is real), the exponentials (128 x 128 per tile at 16 a clock: as long as
// the products at D = 128) and, with codes, their conversion. What bounds it as built is the
// chain of one softmax warp (scores ready, maxima, reference, exponentials, P), 4400 clocks a
// tile, of which two run at a time: 148 CTAs take 50 us for 12 groups of 116 rows and 50k keys
// of e2m1 (D = 128, 17 us of products), 86 us for 128 full groups and 8k keys of e4m3 (D = 64,
// 21 us). The cache's rows are contiguous and come in as they are, by bulk copies into a ring of
// raw tiles; eight warps convert them, 8 elements at a time, into the swizzled K and V tiles
// that the products read. bf16 rows are copied straight into those tiles.
//
// Roles (640 threads): warps 0-3 softmax of the even tiles, warps 4-7 of the odd ones (warp w:
// rows 32 (w % 4) ..), warps 8-11 fill K tiles, warps 12-15 V tiles, warp 16 issues the
// products, warp 17 fetches raw tiles, warps 18 and 19 look at their scales. A softmax warp first
// takes its tile's row maxima and hands the row's reference maximum to the warp of the next
// tile, then exponentiates while that one is already at its maxima: the chain from tile to
// tile is the short first half only. (Both warps on one tile, 64 columns each: 5000 clocks a
// tile, as every step of the chain waited for the one before. Sixteen softmax warps of 64
// columns, or the reference taken on trust and checked by the sums: within 3 % of this.)
// Tensor memory: S of three tiles at D = 64, of two at D = 128, then O, Q and its bf16 form;
// with the third the scores of a set's next tile are there when it ends one (D = 64: 100 ->
// 92 us). Every role walks the CTA's share of the work by itself (tree_common.cuh), so tiles
// of the next unit are filled while the last one is finished.
//
// Codes become fp16 operands as in tree_rows.cu, two per conversion instruction, times their
// block's scale and 2^6 (e4m3) or 2^8 (e2m1): fp16 then holds every value of a block exactly
// when its scale 2^k has -20 <= k <= 1 or -22 <= k <= 5 (largest magnitudes of 2^-12 to 896, or
// 2^-20 to 192). The weights p = 2^(s - m) <= 2^6 enter as p 2^9, so that fp16 rounds them to
// 11 bits down to 2^-23 and below that by at most 2^-34; a query row with its largest element
// in [2^14, 2^15). A K or V tile with a scale outside that range is converted to bf16 instead,
// and its product taken with the bf16 form of Q or P: the code's sign, exponent and mantissa
// bits are moved to bf16's (times 2^-120 or 2^-126 of the value), and two exact
// multiplications bring in the rest. The weights of such a V tile, and of a bf16 cache, round to 8
// bits (see tree_rows.cu, also on blocks of zeros, which count as outside the range).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "sm100_ptx.cuh"
#include "softmax_rows.cuh"
#define TREE_INLINE
#include "tree_common.cuh"

namespace ringattn {
namespace tree {
namespace tiles {

constexpr int TK = 128;   // cache rows per tile
constexpr int TM = 128;   // query rows per group
constexpr int kThreads = 640;
constexpr int kSoftmaxWarps = 8;
constexpr int kFillWarp = 8;  // four warps for K, four for V
constexpr int kFillWarps = 4;
constexpr int kFill = 32 * kFillWarps;
constexpr int kMmaWarp = 16;
constexpr int kFetchWarp = 17;
constexpr int kScaleWarp = 18;  // two: K's and V's scales
constexpr int kLaunchRegs = 96;  // 65536 / 640, rounded down to a multiple of 8
constexpr int kRegsSoftmax = 144, kRegsFill = 72, kRegsOther = 48;
static_assert(2 * kRegsSoftmax + 2 * kRegsFill + kRegsOther <= 5 * kLaunchRegs, "register split exceeds the launch pool");
constexpr int kBoxBytes = TK * 128;  // 128 rows x 64 elements
constexpr int kSmemLimit = 232448;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxRaw = 4;
constexpr int kFlags = 16;  // tiles whose form is remembered (more than are ever in flight)

enum Bar { kKFull = 0, kVFull = 2, kKFree = 4, kVFree = 6, kPReady = 8, kQReady = 11, kODone = 12, kDrain = 13,
           kPair = 14, kMax = 18, kSFull = 26, kRawFull = 29, kRawFree = kRawFull + kMaxRaw,
           kRawSeen = kRawFree + kMaxRaw, kNumBars = kRawSeen + 2 * kMaxRaw };

// Which of a kind's barriers tile t uses, and the phase of it that the tile completes.
struct Turn {
  int at;
  uint32_t phase;
};
RA_HD Turn turn(int t, int n) { return {t % n, (uint32_t)(t / n & 1)}; }

template <int FMT, int D>
struct Cfg {
  static constexpr bool kMx = FMT != RING_ATTN_CACHE_BF16;
  static constexpr int kRowBytes = cache_row_bytes<FMT>(D);
  // tensor memory: scores of kBufs tiles, O, Q and its bf16 form
  static constexpr int kBufs = D == 64 ? 3 : 2;
  static constexpr uint32_t kColO = 128 * kBufs, kColQ = kColO + D, kColQb = kColQ + D / 2;
  static_assert(kColQb + D / 2 <= kTmemCols, "tensor memory");
  // "Scores of tile t are there" and "its weights are": a barrier each per score buffer. Scores of
  // tile t + kBufs are asked for only once the weights of tile t were waited for, so no barrier
  // completes a second phase before the first was seen. (With two for the weights of three
  // buffers a set of softmax warps could finish tiles t and t + 2 while the products still
  // waited for V of tile t, and these then waited for a phase that nothing completes.)
  static RA_HD Turn s_full(int t) { return turn(t, kBufs); }
  static RA_HD Turn p_ready(int t) { return turn(t, kBufs); }
  static_assert(kPReady + kBufs <= kQReady && kSFull + kBufs <= kRawFull, "barriers per score buffer");
  static constexpr int kChunks = kRowBytes / 16;       // per row
  static constexpr int kTileChunks = TK * kChunks;     // 16-byte chunks of a tile of bf16 rows
  static constexpr int kTileBytes = TK * D * 2;        // a bf16 tile
  static constexpr int kOffV = 2 * kTileBytes;
  static constexpr int kOffRaw = 4 * kTileBytes;
  // a raw tile: K codes, V codes, K scales, V scales
  static constexpr int kScaleRow = kMx ? D / kMxBlock : 0;
  static constexpr int kRawScale = 2 * TK * kRowBytes;
  static constexpr int kRawBytes = 2 * TK * (kRowBytes + kScaleRow);
  static constexpr int kRawFit = kMx ? (kSmemLimit - 1024 - 2560 - kOffRaw - 512) / kRawBytes : 0;
  static constexpr int kRaw = kRawFit < kMaxRaw ? kRawFit : kMaxRaw;
  static_assert(!kMx || kRaw >= 2, "a tile is fetched while another is converted");
  // Converting: a task is 16 elements of one row, two 16-byte chunks out. Four lanes take the
  // four tasks of a 64-element box, the next four those of the next row: their 8 stores of one
  // instruction fall on different chunk positions, as the swizzle of neighbouring rows differs
  // in the lowest bit. A thread's rows lie a multiple of 8 apart, so its positions stay.
  static constexpr int kBoxes = D / 64;
  static constexpr int kRowStep = kFill / (4 * kBoxes);
  static constexpr int kPasses = TK / kRowStep;
  static_assert(kRowStep % 8 == 0 && TK % kRowStep == 0, "one swizzled position per thread");
  static constexpr int kOffMax = kOffRaw + kRaw * kRawBytes;  // [5][128] floats
  static constexpr int kOffBar = kOffMax + 2560;
  static constexpr int kSmemBytes = kOffBar + 512 + 1024;  // barriers, flags, alignment
  static_assert(kNumBars * 8 + 16 + 2 * kFlags <= 512, "barriers and flags");
  static_assert(kSmemBytes <= kSmemLimit, "shared memory budget");
  // p's factor in the operand, how far a score may pass the reference before it moves, and the
  // codes' factor
  static constexpr float kLift = kMx ? 9.f : 0.f;
  static constexpr float kRescale = kMx ? 6.f : 8.f;
  static constexpr int kBias = !kMx ? 0 : (FMT == RING_ATTN_CACHE_MXFP8 ? 6 : 8);
  // smallest and largest scale byte whose blocks fp16 holds exactly with that factor
  static constexpr uint32_t kLeast = 127 - 14 - kBias;
  static constexpr uint32_t kMost = 127 + (FMT == RING_ATTN_CACHE_MXFP8 ? 7 : 13) - kBias;
  static constexpr uint32_t kBf16Types = (1u << 7) | (1u << 10);  // operand types of the instruction descriptor
  static constexpr uint32_t kIdescS = idesc_bf16_f32(TM, TK, 0, 0);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(TM, D, 0, 1);
};

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
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
__device__ __forceinline__ uint32_t mul2h(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair_f16(uint32_t codes16) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)codes16));
  return d;
}
// The four pairs of a word of e2m1 codes.
__device__ __forceinline__ void e2m1_pairs_f16(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void store16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Bits c of [lo, hi) in 0..31 for a chunk of columns that starts at c0.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int c0) {
  lo = max(lo - c0, 0);
  hi = min(hi - c0, 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - (hi - lo))) << lo;
}
__device__ __forceinline__ int clip(int x) { return x <= 0 ? 0 : (x >= TK ? TK : x); }

// exp_pack of softmax_rows.cuh, the weights packed to fp16 or bf16.
__device__ __forceinline__ float exp_pack_as(uint32_t (&sr)[64], float scale_log2, float m_sub, bool half,
                                             uint32_t (&pk)[32]) {
  const uint64_t c2 = f2_splat(scale_log2), negm = f2_splat(-m_sub);
  uint64_t acc[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(sr[c], sr[c + 1]), c2, negm), x0, x1);
    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    acc[c / 2 % 2] = f2_add(acc[c / 2 % 2], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
    sr[c] = __float_as_uint(p0);
    sr[c + 1] = __float_as_uint(p1);
  }
  if (half) {
#pragma unroll
    for (int c = 0; c < 32; ++c) pk[c] = pack_f16x2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1]));
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1]));
  }
  float t0, t1;
  f2_unpack(f2_add(acc[0], acc[1]), t0, t1);
  return t0 + t1;
}

// The CTA's tiles one by one (of all its parts): for (it.start(w); it.next(p);) ...
struct TileIter {
  Walk walk;
  Part part;
  int i;
  __device__ __forceinline__ void start(const Walk& w) {
    walk = w;
    part.q1 = 0;
    i = -1;
  }
  __device__ __forceinline__ bool next(const Params& p) {
    if (++i < part.q1) return true;
    if (!next_part(p, walk, part)) return false;
    i = part.q0;
    return true;
  }
};

// mbar_wait of sm100_ptx.cuh in less code: the whole warp polls; the clock and the abort flag
// are looked at every 32 polls.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (n % 32 == 31) {
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      bool stop = watchdog_aborted(wd);
      if (now - since > wd.limit_ns) {
        watchdog_trip(wd);
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

template <int FMT, int D>
struct Fill {
  using C = Cfg<FMT, D>;

  // One thread: the rows of a tile as they are, up to the cache's end (rows past it are dead).
  static __device__ __forceinline__ void fetch(const Params& p, const TileIter& it, uint8_t* slot, uint64_t* full) {
    const int kb = step_key(p, it.part.ks, it.i);
    const int64_t first = it.part.head_row + kb;
    const uint32_t rows = (uint32_t)(p.c.capacity - kb < TK ? p.c.capacity - kb : TK);  // a multiple of 16
    mbar_arrive_expect_tx(full, 2 * rows * (C::kRowBytes + C::kScaleRow));
    bulk_load(slot, static_cast<const uint8_t*>(p.c.k) + first * C::kRowBytes, rows * C::kRowBytes, full);
    bulk_load(slot + TK * C::kRowBytes, static_cast<const uint8_t*>(p.c.v) + first * C::kRowBytes, rows * C::kRowBytes,
              full);
    uint8_t* sc = slot + C::kRawScale;
    bulk_load(sc, static_cast<const uint8_t*>(p.c.k_scale) + first * C::kScaleRow, rows * C::kScaleRow, full);
    bulk_load(sc + TK * C::kScaleRow, static_cast<const uint8_t*>(p.c.v_scale) + first * C::kScaleRow,
              rows * C::kScaleRow, full);
  }

  // Rows of a raw tile that lie past the cache's end or that no query row sees hold anything.
  static __device__ __forceinline__ bool whole(const Params& p, const TileIter& it, int kb) {
    return kb + TK <= it.part.ks.n + it.part.ks.cnt &&
           (p.window <= 0 || kb + TK <= p.sinks || kb > it.part.ks.n - p.window);
  }

  // One warp: whether K's (kv = 0) or V's scales leave fp16's range.
  static __device__ __forceinline__ bool wide(const Params& p, const TileIter& it, const uint8_t* slot, int kv) {
    using Word = typename std::conditional<C::kScaleRow == 4, uint32_t, uint16_t>::type;
    const int lane = threadIdx.x % 32;
    const int kb = step_key(p, it.part.ks, it.i);
    const bool all = whole(p, it, kb);
    const Word* sc = reinterpret_cast<const Word*>(slot + C::kRawScale + kv * TK * C::kScaleRow) + lane;
    uint32_t top = 0, low = 0x00ff00ffu;
#pragma unroll
    for (int i = 0; i < TK / 32; ++i) {
      const uint32_t w = all || key_live(p, it.part.ks, kb + lane + 32 * i) ? sc[32 * i] : 0x7f7f7f7fu;
      const uint32_t a = w & 0x00ff00ffu, b = w >> 8 & 0x00ff00ffu;
      if (C::kScaleRow == 4) {
        top = __vmaxu2(top, __vmaxu2(a, b));
        low = __vminu2(low, __vminu2(a, b));
      } else {  // two bytes: one in the low half of a and of b
        top = max(top, max(a & 255u, b & 255u));
        low = min(low & 255u, min(a & 255u, b & 255u));
      }
    }
    const uint32_t hi = max(top & 0xffffu, top >> 16);
    const uint32_t lo = C::kScaleRow == 4 ? min(low & 0xffffu, low >> 16) : low & 255u;
    return __any_sync(0xffffffffu, hi > C::kMost || lo < C::kLeast) != 0;
  }

  // K (kv = 0) or V of a raw tile into the swizzled tile at `dst`, in fp16 or (wide) bf16.
  static __device__ __forceinline__ void convert(const Params& p, const TileIter& it, const uint8_t* slot, int kv,
                                                 bool wide, uint32_t dst, int ct) {
    const int kb = step_key(p, it.part.ks, it.i);
    const int j = ct % 4, box = ct / 8 % C::kBoxes;                       // task of the box; box
    const int row0 = ct / (8 * C::kBoxes) * 2 + (ct / 4 & 1);
    constexpr int kWords = FMT == RING_ATTN_CACHE_MXFP8 ? 4 : 2;          // of codes per task
    const uint8_t* from = slot + kv * TK * C::kRowBytes + row0 * C::kRowBytes + (box * 4 + j) * 4 * kWords;
    const uint8_t* sc = slot + C::kRawScale + kv * TK * C::kScaleRow + row0 * C::kScaleRow + box * 2 + j / 2;
    const uint32_t to0 = dst + box * kBoxBytes + row0 * 128 + (((2 * j) ^ (row0 & 7)) * 16);
    const uint32_t to1 = dst + box * kBoxBytes + row0 * 128 + (((2 * j + 1) ^ (row0 & 7)) * 16);
    const bool all = whole(p, it, kb);
    // the loads of a batch of passes before its first store: loads may not pass the stores
    constexpr int kBatch = C::kPasses < 4 ? C::kPasses : 4;
#pragma unroll 1
    for (int i0 = 0; i0 < C::kPasses; i0 += kBatch) {
      uint32_t words[kBatch][kWords], bytes[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = (i0 + i) * C::kRowStep;
        bytes[i] = sc[row * C::kScaleRow];
        if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
          const uint4 x = *reinterpret_cast<const uint4*>(from + row * C::kRowBytes);
          words[i][0] = x.x; words[i][1] = x.y; words[i][2] = x.z; words[i][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(from + row * C::kRowBytes);
          words[i][0] = x.x; words[i][1] = x.y;
        }
        if (__builtin_expect(!all, 0) && !key_live(p, it.part.ks, kb + row0 + row)) {
          bytes[i] = 127u;
#pragma unroll
          for (int x = 0; x < kWords; ++x) words[i][x] = 0u;
        }
      }
      const uint32_t off = i0 * C::kRowStep * 128;
      if (__builtin_expect(!wide, 1)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          // 2^(byte - 127 + kBias) in both halves, fields (byte - 112 + kBias) << 10
          const uint32_t f = bytes[i] * 0x4000400u + (uint32_t)(C::kBias - 112) * 0x4000400u;
          uint32_t v[8];
          if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = e4m3_pair_f16(words[i][x / 2] >> (16 * (x % 2)));
          } else {
            uint32_t a[4], b[4];
            e2m1_pairs_f16(words[i][0], a);
            e2m1_pairs_f16(words[i][1], b);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              v[x] = a[x];
              v[4 + x] = b[x];
            }
          }
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = mul2h(v[x], f);
          store16(to0 + off + i * C::kRowStep * 128, v[0], v[1], v[2], v[3]);
          store16(to1 + off + i * C::kRowStep * 128, v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          // raw * 2^120 (or 126) * 2^(byte - 127 + kBias), as 2^(byte - 127 + 20 or 26 + kBias), 2^100
          constexpr uint32_t kUp = (FMT == RING_ATTN_CACHE_MXFP8 ? 20 : 26) + C::kBias;
          const uint32_t e = bytes[i] + kUp;  // the factor's exponent field; past its end (2^93 and more) infinity
          const uint32_t f = bytes[i] == 255u ? 0x7fc07fc0u : (e < 255u ? e * 0x800080u : 0x7f807f80u);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[4];
            if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
              const uint32_t w0 = h ? words[i][2] : words[i][0], w1 = h ? words[i][3] : words[i][1];
              const uint32_t e0 = ((w0 << 4) & 0x07f007f0u) | ((w0 << 8) & 0x80008000u);
              const uint32_t o0 = ((w0 >> 4) & 0x07f007f0u) | (w0 & 0x80008000u);
              const uint32_t e1 = ((w1 << 4) & 0x07f007f0u) | ((w1 << 8) & 0x80008000u);
              const uint32_t o1 = ((w1 >> 4) & 0x07f007f0u) | (w1 & 0x80008000u);
              v[0] = __byte_perm(e0, o0, 0x5410);
              v[1] = __byte_perm(e0, o0, 0x7632);
              v[2] = __byte_perm(e1, o1, 0x5410);
              v[3] = __byte_perm(e1, o1, 0x7632);
            } else {
              constexpr uint32_t M = 0x01c001c0u, S = 0x80008000u;
              const uint32_t w0 = h ? words[i][1] : words[i][0];
              const uint32_t r0 = ((w0 << 6) & M) | ((w0 << 12) & S), r1 = ((w0 << 2) & M) | ((w0 << 8) & S);
              const uint32_t r2 = ((w0 >> 2) & M) | ((w0 << 4) & S), r3 = ((w0 >> 6) & M) | (w0 & S);
              v[0] = __byte_perm(r0, r1, 0x5410);
              v[1] = __byte_perm(r2, r3, 0x5410);
              v[2] = __byte_perm(r0, r1, 0x7632);
              v[3] = __byte_perm(r2, r3, 0x7632);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = mul2(mul2(v[x], f), 0x71807180u);  // 2^100
            store16((h ? to1 : to0) + off + i * C::kRowStep * 128, v[0], v[1], v[2], v[3]);
          }
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

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_tiles_kernel(const __grid_constant__ Params p) {
  using C = Cfg<FMT, D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Walk s_walk;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + kNumBars * 8 + 8);
  volatile uint8_t* s_wide = reinterpret_cast<volatile uint8_t*>(smem + C::kOffBar + kNumBars * 8 + 16);  // [2][kFlags]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *p.status = RING_ATTN_OK;
    grid_let_next();
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kKFull + b], kFillWarps);
      mbar_init(&bars[kVFull + b], kFillWarps);
      mbar_init(&bars[kKFree + b], 1);
      mbar_init(&bars[kVFree + b], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&bars[kSFull + b], 1);
      mbar_init(&bars[kPReady + b], kSoftmaxWarps / 2);
    }
    mbar_init(&bars[kQReady], kSoftmaxWarps);
    mbar_init(&bars[kODone], 1);
    mbar_init(&bars[kDrain], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[kPair + i], 2);
    for (int i = 0; i < 8; ++i) mbar_init(&bars[kMax + i], 1);
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(&bars[kRawFull + i], 1);
      mbar_init(&bars[kRawFree + i], 2 * kFillWarps);
      mbar_init(&bars[kRawSeen + i], 1);
      mbar_init(&bars[kRawSeen + kMaxRaw + i], 1);
    }
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

  auto all = [&](bool r) { return __all_sync(0xffffffffu, r) != 0; };
  // every warp of a warpgroup takes the same branch up to its setmaxnreg
  if (warp >= kMmaWarp) {
    regs_decrease<kRegsOther>();
    if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ products
      const bool issuer = elect_one_sync();
      Walk walk = s_walk;
      Part part;
      int t0 = 0, parts = 0;
      bool ok = true;
      while (ok && next_part(p, walk, part)) {
        const int n_tiles = part.q1 - part.q0;
        auto issue_s = [&](int t) -> bool {
          if (!(wait_bar(&bars[kKFull + (t & 1)], (uint32_t)(t >> 1 & 1), wd))) return false;
          tc_fence_after();
          const uint64_t dk = smem_desc_sw128(sbase + (t & 1) * C::kTileBytes, 0, 1024);
          const bool half = C::kMx && !s_wide[t % kFlags];
          const uint32_t qa = tmem + (half || !C::kMx ? C::kColQ : C::kColQb);
          const uint32_t desc = half ? C::kIdescS & ~C::kBf16Types : C::kIdescS;
  #pragma unroll
          for (int k = 0; k < D / 16; ++k)
            if (issuer)
              mma_ts(tmem + 128 * (t % C::kBufs), qa + 8 * k, dk + (uint64_t)(((k / 4) * kBoxBytes + (k % 4) * 32) >> 4), desc, k > 0);
          if (issuer) {
            mma_commit(&bars[kSFull + C::s_full(t).at]);
            mma_commit(&bars[kKFree + (t & 1)]);
          }
          return true;
        };
        if (!(ok = (wait_bar(&bars[kQReady], (uint32_t)(parts & 1), wd)))) break;
        tc_fence_after();
        ok = issue_s(t0);
        for (int n = 1; ok && n < C::kBufs && n < n_tiles; ++n) ok = issue_s(t0 + n);
        for (int n = 0; ok && n < n_tiles; ++n) {
          const int t = t0 + n;
          if (!(ok = (wait_bar(&bars[kVFull + (t & 1)], (uint32_t)(t >> 1 & 1), wd)))) break;
          if (!(ok = (wait_bar(&bars[kPReady + C::p_ready(t).at], C::p_ready(t).phase, wd)))) break;
          tc_fence_after();
          const uint64_t dv = smem_desc_sw128(sbase + C::kOffV + (t & 1) * C::kTileBytes, kBoxBytes, 1024);
          const uint32_t desc = C::kMx && !s_wide[kFlags + t % kFlags] ? C::kIdescO & ~C::kBf16Types : C::kIdescO;
  #pragma unroll
          for (int k = 0; k < TK / 16; ++k)
            if (issuer)
              mma_ts(tmem + C::kColO, tmem + 128 * (t % C::kBufs) + 64 * (k / 4) + 8 * (k % 4), dv + (uint64_t)((k * 16 * 128) >> 4),
                     desc, !(n == 0 && k == 0));
          if (issuer) {
            mma_commit(&bars[kVFree + (t & 1)]);
            if (n + 1 == n_tiles) mma_commit(&bars[kODone]);
          }
          if (n + C::kBufs < n_tiles && !(ok = issue_s(t + C::kBufs))) break;
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
    } else if (warp == kFetchWarp) {
      // ------------------------------------------------------------------ fetch raw tiles
      if constexpr (C::kMx) {
        TileIter it;
        it.start(s_walk);
        int t = 0;
        bool ok = true;
#pragma unroll 1
        for (; it.next(p); ++t) {
          const int slot = t % C::kRaw;
          if (!(ok = wait_bar(&bars[kRawFree + slot], (uint32_t)(t / C::kRaw & 1) ^ 1, wd))) break;
          if (lane == 0) Fill<FMT, D>::fetch(p, it, smem + C::kOffRaw + slot * C::kRawBytes, &bars[kRawFull + slot]);
        }
        if (!ok) {
          // wind down: this CTA's own copies must land before its shared memory goes away
          const uint64_t since = global_timer_ns();
          for (int x = t > C::kRaw ? t - C::kRaw : 0; x < t; ++x)
            while (!mbar_try_wait(&bars[kRawFull + x % C::kRaw], (uint32_t)(x / C::kRaw & 1)) &&
                   global_timer_ns() - since <= p.watchdog_ns) {
            }
        }
      }
    } else {
      if constexpr (C::kMx) {
        // ------------------------------------------------------------------ their scales
        const int kv = warp - kScaleWarp;
        TileIter it;
        it.start(s_walk);
  #pragma unroll 1
        for (int t = 0; it.next(p); ++t) {
          const int slot = t % C::kRaw;
          if (!wait_bar(&bars[kRawFull + slot], (uint32_t)(t / C::kRaw & 1), wd)) break;
          const bool out = Fill<FMT, D>::wide(p, it, smem + C::kOffRaw + slot * C::kRawBytes, kv);
          if (lane == 0) {
            s_wide[kv * kFlags + t % kFlags] = out;
            mbar_arrive(&bars[kRawSeen + kv * kMaxRaw + slot]);
          }
          __syncwarp();
        }
      }
    }
  } else if (warp >= kFillWarp) {
    regs_decrease<kRegsFill>();
    // ------------------------------------------------------------------ fill the tiles
    using F = Fill<FMT, D>;
    const int kv = warp >= kFillWarp + kFillWarps ? 1 : 0;
    const int ct = (threadIdx.x - 32 * kFillWarp) % kFill;
    const uint32_t tile0 = sbase + kv * C::kOffV;
    uint64_t* full = &bars[kv ? kVFull : kKFull];
    uint64_t* free = &bars[kv ? kVFree : kKFree];
    TileIter it;
    it.start(s_walk);
    auto ready = [&](uint64_t* bar) {  // this warp's part is written: visible to the products
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if constexpr (C::kMx) {
#pragma unroll 1
      for (int t = 0; it.next(p); ++t) {
        const int slot = t % C::kRaw;
        // (both: V's form is also what the softmax of this tile packs to, and it starts after K)
        if (!(wait_bar(&bars[kRawSeen + slot], (uint32_t)(t / C::kRaw & 1), wd))) break;
        if (!(wait_bar(&bars[kRawSeen + kMaxRaw + slot], (uint32_t)(t / C::kRaw & 1), wd))) break;
        // the bulk copies' own barrier: their bytes are visible to those who wait on it
        if (!(wait_bar(&bars[kRawFull + slot], (uint32_t)(t / C::kRaw & 1), wd))) break;
        if (!(wait_bar(&free[t & 1], (uint32_t)(t >> 1 & 1) ^ 1, wd))) break;
        F::convert(p, it, smem + C::kOffRaw + slot * C::kRawBytes, kv, s_wide[kv * kFlags + t % kFlags] != 0,
                   tile0 + (t & 1) * C::kTileBytes, ct);
        ready(&full[t & 1]);
        if (lane == 0) mbar_arrive(&bars[kRawFree + slot]);
      }
    } else {
      int t = 0;
      bool ok = true;
#pragma unroll 1
      for (; it.next(p); ++t) {
        if (!(ok = (wait_bar(&free[t & 1], (uint32_t)(t >> 1 & 1) ^ 1, wd)))) break;
        F::copy_tile(p, it, kv ? p.c.v : p.c.k, tile0 + (t & 1) * C::kTileBytes, ct);
        copy_commit();
        if (t > 0) {  // the tile before has landed once only this one is in flight
          copy_wait<1>();
          ready(&full[(t - 1) & 1]);
        }
      }
      copy_wait<0>();
      if (ok && t > 0) ready(&full[(t - 1) & 1]);
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax and epilogue
    const int wq = warp % 4, hh = warp / 4;  // hh: this warp's tiles are those with t % 2 == hh
    const int r = 32 * wq + lane;            // row of the group
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    float* s_m = reinterpret_cast<float*>(smem + C::kOffMax);  // [t % 2][row]: the row's reference after tile t
    float* s_x = s_m + 256;                                    // [half][row]
    float* s_scale = s_m + 512;                                // [row]: scores to the base-2 domain
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
        // Sixteen query rows into tensor memory, as fragments (four lanes side by side on a row: with
        // a row per lane the loads' 32 lines each took 5000 clocks a part). With codes: in fp16,
        // times 2^(14 - exponent of the row's largest element), and the same in bf16.
        const int r16 = 32 * wq + 16 * hh;  // first of them
        uint32_t x[D / 4], top[2] = {0, 0};  // registers as in tmem_ld_frag16, 32 words of a row after 32
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int mine = part.grp * TM + r16 + lane / 4 + 8 * j;
          const bool in = mine < ks.cnt * p.rep;
          const uint16_t* src = p.q + part.b * p.qs_b + (int64_t)(part.kvh * p.rep + (in ? mine % p.rep : 0)) * p.qs_h +
                                (in ? mine / p.rep : 0) * p.qs_t + 4 * (lane % 4);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint2 v = in ? *reinterpret_cast<const uint2*>(src + 16 * i) : make_uint2(0u, 0u);
            x[4 * i + 2 * j] = v.x;
            x[4 * i + 2 * j + 1] = v.y;
            top[j] = max(max(top[j], max(v.x & 0x7fffu, v.x >> 16 & 0x7fffu)), max(v.y & 0x7fffu, v.y >> 16 & 0x7fffu));
          }
        }
        auto put = [&](uint32_t col) {
#pragma unroll
          for (int w = 0; w < D / 64; ++w)
            tmem_st_frag16_wide(tmem + ((uint32_t)r16 << 16) + col + 32 * w, x + 16 * w);
        };
        if (C::kMx) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
            top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
            const int e = max((int)(top[j] >> 7), 15) - 127;  // not below 2^-112
            const float up = pow2i(14 - e);
            if (lane % 4 == 0) s_scale[r16 + lane / 4 + 8 * j] = p.scale_log2 * exp2f((float)(e - 14 - C::kBias));
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int w = 4 * i + 2 * j; w < 4 * i + 2 * j + 2; ++w)
                x[w] = pack_f16x2(__uint_as_float(x[w] << 16) * up, __uint_as_float(x[w] & 0xffff0000u) * up);
          }
          put(C::kColQ);
#pragma unroll
          for (int w = 0; w < D / 4; ++w) {  // (exact: 8 significant bits)
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[w]));
            x[w] = pack_bf16x2(f.x, f.y);
          }
          put(C::kColQb);
        } else {
          put(C::kColQ);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[kQReady]);
          mbar_arrive(&bars[kPair + wq]);
        }
      }
      const Nodes nodes = warp_nodes(p, part.b, ks);
      uint64_t seen;
      int depth;
      node_of(nodes, node, seen, depth);
      const int lo_key = p.window > 0 ? ks.n + depth - p.window + 1 : 0;
      // (the pair's barrier passes twice a part)
      if (!(ok = (wait_bar(&bars[kPair + wq], 0, wd)))) break;
      const float score_scale = C::kMx ? s_scale[r] : p.scale_log2;
      // this warp's part of the row's sum, relative to the reference m (a whole number) of its
      // last tile
      float m = -INFINITY, l = 0.f;
      for (int n = 0; n < n_tiles; ++n) {
        const int t = t0 + n;
        if ((t & 1) != hh) continue;
        const int kb = step_key(p, ks, part.q0 + n);
        // every row sees the whole tile
        const bool whole = kb + TK <= ks.n &&
                           (p.window <= 0 || kb + TK <= p.sinks || kb >= ks.n + p.T - p.window);
        if (!(ok = (wait_bar(&bars[kSFull + C::s_full(t).at], C::s_full(t).phase, wd)))) break;
        tc_fence_after();
        const uint32_t tS = tmem + lane_off + 128 * (t % C::kBufs);
        if (__builtin_expect(!whole, 0)) {
          // hidden scores are overwritten in place, by a loop: the straight path below stays
          // short (what the roles share is the instruction caches)
          const int hi = clip(ks.n - kb), lo = clip(lo_key - kb), sk = min(clip(p.sinks - kb), hi);
#pragma unroll 1
          for (int c0 = 0; c0 < TK; c0 += 32) {
            uint32_t x[32];
            tmem_ld32(tS + c0, x);
            const int j0 = kb + c0 - ks.n;  // drafted node of the chunk's first column
            const uint32_t drafts = j0 >= 64 || j0 <= -32 ? 0u : (uint32_t)(j0 >= 0 ? seen >> j0 : seen << -j0);
            const uint32_t see = span_bits(lo, hi, c0) | span_bits(0, sk, c0) | drafts;
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see >> e & 1)) x[e] = 0xff800000u;  // -inf
            tmem_st32(tS + c0, x);
          }
          tmem_wait_st();
        }
        uint32_t sr[64];
        auto load = [&](int c0) {  // columns c0 .. c0 + 63
          tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(tS + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_wait_ld();
        };
        float top = -INFINITY;
#pragma unroll 1  // (one copy of the code each: the roles share the instruction caches)
        for (int c0 = 0; c0 < TK; c0 += 64) {
          load(c0);
          top = fmaxf(top, raw_rowmax<64>(sr));
        }
        top *= score_scale;
        // the reference after the tile before, from the other warp of these rows
        float before = -INFINITY;
        if (n > 0) {
          if (!(ok = (wait_bar(&bars[kMax + 2 * wq + (hh ^ 1)], (uint32_t)((t - 1) >> 1 & 1), wd)))) break;
          before = s_m[(hh ^ 1) * 128 + r];
        }
        const bool moved = top > before + C::kRescale || (before == -INFINITY && top != -INFINITY);
        const float now = moved ? ceilf(top) : before;
        s_m[hh * 128 + r] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kMax + 2 * wq + hh]);
        if (m != now) {
          // (before the first finite score l is 0, or NaN, which the row keeps)
          if (m != -INFINITY) l *= ex2_approx(m - now);
          m = now;
        }
        const float alpha = !moved ? 1.f : (before == -INFINITY ? 0.f : ex2_approx(before - now));
        const float sub = m == -INFINITY ? 0.f : m - C::kLift;
        // (the last columns are still in registers: they go first)
        const bool half = C::kMx && !s_wide[kFlags + t % kFlags];
#pragma unroll 1
        for (int c0 = 64; c0 >= 0; c0 -= 64) {
          if (c0 == 0) load(0);
          uint32_t pk[32];
          l += exp_pack_as(sr, score_scale, sub, half, pk);
          tmem_st32(tS + c0, pk);  // P of columns c0 .. takes the first half of their place
        }
        if (n > 0 && __any_sync(0xffffffffu, moved)) {
          // O must hold every product so far (V's slot is free when they are done; those three
          // tiles back are, or S would not be here). The last one waits for the other set's
          // weights: 3000 clocks where this came before the exponentials.
          if (!(ok = (wait_bar(&bars[kVFree + ((t - 1) & 1)], (uint32_t)((t - 1) >> 1 & 1), wd)))) break;
          tc_fence_after();
          rescale_o<D>(tmem + lane_off + C::kColO, alpha);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPReady + C::p_ready(t).at]);
      }
      if (!ok) break;
      // the two warps of the rows join their sums (m never falls: the larger one is the row's)
      s_x[hh * 128 + r] = l;
      s_m[hh * 128 + r] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kPair + wq]);
      if (!(ok = (wait_bar(&bars[kPair + wq], 1, wd)))) break;
      const float m_other = s_m[(hh ^ 1) * 128 + r], l_other = s_x[(hh ^ 1) * 128 + r];
      const float m_row = fmaxf(m, m_other);
      if (m != -INFINITY) l *= ex2_approx(m - m_row);
      const float lo2 = m_other == -INFINITY ? l_other : l_other * ex2_approx(m_other - m_row);
      m = m_row;
      if (!(ok = (wait_bar(&bars[kODone], (uint32_t)(parts & 1), wd)))) break;
      tc_fence_after();
      // l carries the same 2^kLift as O
      const float L = hh == 0 ? l + lo2 : lo2 + l;  // the same sum in both
      const bool none = L == 0.f;  // a row of keys that are not finite has L = NaN and m = -inf
      const float inv = none ? 0.f : pow2i(-C::kBias) / L;  // O carries V's factor as well
      const float lse2 = none ? -INFINITY : m + log2f(L * (C::kMx ? 0x1p-9f : 1.f));
      const int64_t slot = (int64_t)blockIdx.x + part.unit;
      // columns hh D/2 .. of this warp's rows, as fragments: four lanes side by side on a row
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          const int d0 = hh * (D / 2) + 32 * c;
          uint32_t o[16];
          tmem_ld_frag16(tmem + lane_off + ((uint32_t)t << 20) + C::kColO + d0, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int rr = 16 * t + 8 * j + lane / 4, at = part.grp * TM + 32 * wq + rr;
            const float f = __shfl_sync(0xffffffffu, inv, rr);
            if (at >= ks.cnt * p.rep) continue;
            if (part.alone) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + out_row(p, part.b, part.kvh, at) * D + d0) + lane % 4;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[4 * i] = pack_bf16x2(__uint_as_float(o[4 * i + 2 * j]) * f, __uint_as_float(o[4 * i + 2 * j + 1]) * f);
            } else {
              float* dst = p.o_parts + (slot * TM + 32 * wq + rr) * D + d0 + 2 * (lane % 4);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(__uint_as_float(o[4 * i + 2 * j]) * f,
                                                                      __uint_as_float(o[4 * i + 2 * j + 1]) * f);
            }
          }
        }
      }
      if (live && hh == 0) {
        if (part.alone)
          p.lse[out_row(p, part.b, part.kvh, row)] = lse2 * 0.69314718055994530942f;
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
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return RING_ATTN_ECUDA;
  if (fa.numRegs * kThreads < 128 * (2 * kRegsSoftmax + 2 * kRegsFill + kRegsOther)) return RING_ATTN_EUNSUPPORTED;
  kern<<<p.ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

template <int FMT, int D>
int barriers(int t, int32_t* out) {
  using C = Cfg<FMT, D>;
  const int32_t x[6] = {C::kBufs, C::kRaw, C::s_full(t).at, (int32_t)C::s_full(t).phase,
                        C::p_ready(t).at, (int32_t)C::p_ready(t).phase};
  for (int i = 0; i < 6; ++i) out[i] = x[i];
  return RING_ATTN_OK;
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

int tree_tile_barriers(int format, int D, int t, int32_t* out) {
  using namespace tree::tiles;
  switch (format) {
    case RING_ATTN_CACHE_BF16: return D == 64 ? barriers<RING_ATTN_CACHE_BF16, 64>(t, out) : barriers<RING_ATTN_CACHE_BF16, 128>(t, out);
    case RING_ATTN_CACHE_MXFP8: return D == 64 ? barriers<RING_ATTN_CACHE_MXFP8, 64>(t, out) : barriers<RING_ATTN_CACHE_MXFP8, 128>(t, out);
    default: return D == 64 ? barriers<RING_ATTN_CACHE_MXFP4, 64>(t, out) : barriers<RING_ATTN_CACHE_MXFP4, 128>(t, out);
  }
}

}  // namespace ringattn
