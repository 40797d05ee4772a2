// Attention of drafted tokens over a cache, for few query rows per kv head (bf16, mxfp8 or
// mxfp4 cache; D = 64 or 128), and the merge of split results.
//
// Mathematics: online softmax over the visible keys in base 2, m = reference maximum,
// p = 2^(s scale log2 e - m), l = sum p, O = sum p v, result O / l and m + log2 l.
//
// What bounds it: reading the cache once; then the instructions that turn codes into
// operands. Every warp works alone on kStep keys at a time: it keeps its own ring of cache
// rows in shared memory (16-byte asynchronous copies, no block barrier in the loop),
// converts codes in registers straight into the operand fragments, and holds the group's
// queries, running state and output in registers. Nothing that was dequantised is written
// anywhere. The tensor work is small here, which is why this form uses the warp-level matrix
// instructions: their operands come from registers, whereas tcgen05 reads them from shared
// memory, where the dequantised tile would have to be written and read again.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and head
// dimensions fill the 16 rows of an m16n8k16 tile and 8 query rows its columns: a decode
// step's 1 to 8 rows per kv head then cost half the instructions and registers of a 16-row
// tile. P^T changes sides between the products by one 8x8 transpose per 8 keys.
//
// Microscaled codes become fp16 operands: two codes per conversion instruction, one packed
// multiplication by the block's scale. fp16 holds every code exactly; its small exponent
// range is met by references that are powers of two, so nothing but the far end of the
// range is ever rounded:
//   * a step's K (and V) scales are taken relative to the largest one in the step, R;
//   * a query row is scaled so that its largest element lies in [2^14, 2^15);
//   * the weights p = 2^(s - m) <= 2^2 enter as p 2^(R - E + 13), where E is the largest R of
//     V so far (O is rescaled in the rare step that raises it) and R >= E - 3: fp16 then
//     rounds p to 11 bits down to 2^-24, and below that by at most 2^-35 (half its smallest
//     step, 2^-25, over 2^10), 2^-15 in all for the weights of 2^20 keys.
// A step that does not fit (scales more than 2^15 apart, R more than 2^3 below E, a block
// that is not finite) takes the same products in bf16, whose range they always fit: the
// code's sign, exponent and mantissa bits are moved to bf16's, which gives its value times
// 2^-120 (e4m3) or 2^-126 (e2m1), and the multiplication by the scale makes up for that. Its
// weights round to 8 bits. So they do over a bf16 cache, whose V they must match in type (l sums
// them unrounded): out is then off from 64 bits by 1.2 to 1.3 times what rounding the result
// alone costs, where fp16 weights cost 1.01 times. A block of zeros has the smallest scale of all,
// 2^-127, so a step that holds one takes the bf16 form too.
//
// Four contexts of up to 128k, 4 query rows per kv head, e4m3, D = 128: 168 to 172 us a call,
// 4.9 to 5.1 TB/s of the cache.
//
// Which head dimension or key meets which k index of a matrix instruction is free as long
// as both operands agree, so lanes load 16 contiguous bytes and use them in memory order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "sm100_ptx.cuh"
#include "tree_common.cuh"

namespace ringattn {
namespace tree {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
static_assert(kWarps == 4, "a quad of steps is one step for each warp");
constexpr int kLiftP = 13;   // log2 of the factor that p carries into fp16 (see above)
constexpr int kSpread = 15;  // scales of a step may lie 2^kSpread apart in the fp16 form
constexpr int kBelow = 3;    // and R this far below E
// The reference maximum moves when a score passes it by this (base 2): the room that p needs
// at the top of fp16's range, and more than bf16 has use for.
template <int FMT>
__host__ __device__ constexpr float rescale_log2() {
  return FMT == RING_ATTN_CACHE_BF16 ? 8.f : 2.f;
}

template <int FMT, int D>
struct Fmt {
  static constexpr int kRowBytes = cache_row_bytes<FMT>(D);
  static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks per row
  static constexpr bool kMx = FMT != RING_ATTN_CACHE_BF16;
  static constexpr int kStep = kMx || D == 64 ? 32 : 16;     // keys per warp and step
  static constexpr int kSubs = kStep / 16;
  static constexpr int kScaleRow = kMx ? D / kMxBlock : 0;   // scale bytes per row
  static constexpr int kTileBytes = kStep * kRowBytes;       // K or V of one step
  static constexpr int kScaleBytes = kStep * kScaleRow;      // K or V scales of one step
  static constexpr int kStageBytes = 2 * kTileBytes + 2 * kScaleBytes;
  // ring stages: two steps ahead of 12 warps per SM, as far as shared memory goes
  static constexpr int kStagesFit = (232448 / 3 - 4096) / (kWarps * kStageBytes);
  static constexpr int kStages = kStagesFit < 4 ? kStagesFit : 4;
  static_assert(kStages >= 2, "a step is loaded while another is worked on");
  static constexpr int kKSteps = D / 16;                     // k16 steps of the score product
  // resident CTAs: 168 registers a thread, or 255 for the tile that needs them
  static constexpr int per_sm(int nt) { return D == 128 && nt == 2 ? 2 : 3; }
  static constexpr int smem(int rows) {
    const int ring = kWarps * kStages * kStageBytes, merge = kWarps * rows * (D + 4) * 4;
    return ring > merge ? ring : merge;
  }
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e, 0 below 2^-126 (e <= 127).
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(e + 127) << 23); }
// An fp16 pair as bf16 (exact for what a query holds, see the head of the file).
__device__ __forceinline__ uint32_t bf16_of_f16(uint32_t a) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
  return pack_bf16x2(f.x, f.y);
}
// Two e4m3 codes (the low or high half of a word) to fp16.
template <int H>
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t w) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)(H ? w >> 16 : w)));
  return d;
}
// Two e2m1 codes (byte I of a word) to fp16.
template <int I>
__device__ __forceinline__ uint32_t e2m1_f16x2(uint32_t w) {
  uint32_t d;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(d) : "r"(w));
  return d;
}

// bf16 with the code's bits in place (times 2^-120 or 2^-126, see the head of the file):
// e4m3 bytes 0 and 2 (Odd = false) or 1 and 3; e2m1 nibbles I and I + 4.
template <bool Odd>
__device__ __forceinline__ uint32_t e4m3_raw(uint32_t w) {
  if (!Odd) w <<= 8;
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
template <int I>
__device__ __forceinline__ uint32_t e2m1_raw(uint32_t w) {
  const uint32_t x = w << (12 - 4 * I);
  return ((x >> 6) & 0x01c001c0u) | (x & 0x80008000u);
}

// Pairs of adjacent elements of a word of codes, times the factors f: fp16 or bf16.
template <int FMT, bool kHalf>
__device__ __forceinline__ void word_pairs(uint32_t w, uint32_t f, uint32_t* out) {
  if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
    if constexpr (kHalf) {
      out[0] = mul_f16x2(e4m3_f16x2<0>(w), f);
      out[1] = mul_f16x2(e4m3_f16x2<1>(w), f);
    } else {
      const uint32_t e = mul_bf16x2(e4m3_raw<false>(w), f), o = mul_bf16x2(e4m3_raw<true>(w), f);
      out[0] = __byte_perm(e, o, 0x5410);
      out[1] = __byte_perm(e, o, 0x7632);
    }
  } else {
    if constexpr (kHalf) {
      out[0] = mul_f16x2(e2m1_f16x2<0>(w), f);
      out[1] = mul_f16x2(e2m1_f16x2<1>(w), f);
      out[2] = mul_f16x2(e2m1_f16x2<2>(w), f);
      out[3] = mul_f16x2(e2m1_f16x2<3>(w), f);
    } else {
      const uint32_t r0 = mul_bf16x2(e2m1_raw<0>(w), f), r1 = mul_bf16x2(e2m1_raw<1>(w), f);
      const uint32_t r2 = mul_bf16x2(e2m1_raw<2>(w), f), r3 = mul_bf16x2(e2m1_raw<3>(w), f);
      out[0] = __byte_perm(r0, r1, 0x5410);
      out[1] = __byte_perm(r2, r3, 0x5410);
      out[2] = __byte_perm(r0, r1, 0x7632);
      out[3] = __byte_perm(r2, r3, 0x7632);
    }
  }
}

// Pairs (key a, key b) of every element of two words of codes, times the factors f (low
// half a's, high half b's), in element order.
template <int FMT, bool kHalf>
__device__ __forceinline__ void key_pairs(uint32_t a, uint32_t b, uint32_t f, uint32_t* out) {
  if constexpr (FMT == RING_ATTN_CACHE_BF16) {
    out[0] = __byte_perm(a, b, 0x5410);
    out[1] = __byte_perm(a, b, 0x7632);
  } else if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
    if constexpr (kHalf) {
      const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
      out[0] = mul_f16x2(e4m3_f16x2<0>(x), f);
      out[1] = mul_f16x2(e4m3_f16x2<1>(x), f);
      out[2] = mul_f16x2(e4m3_f16x2<0>(y), f);
      out[3] = mul_f16x2(e4m3_f16x2<1>(y), f);
    } else {
      const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
      out[0] = mul_bf16x2(e4m3_raw<false>(x), f);
      out[1] = mul_bf16x2(e4m3_raw<true>(x), f);
      out[2] = mul_bf16x2(e4m3_raw<false>(y), f);
      out[3] = mul_bf16x2(e4m3_raw<true>(y), f);
    }
  } else {
    if constexpr (kHalf) {
      const uint32_t x = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);  // elements 0, 2, 4, 6
      const uint32_t y = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);  // elements 1, 3, 5, 7
      out[0] = mul_f16x2(e2m1_f16x2<0>(x), f);
      out[1] = mul_f16x2(e2m1_f16x2<0>(y), f);
      out[2] = mul_f16x2(e2m1_f16x2<1>(x), f);
      out[3] = mul_f16x2(e2m1_f16x2<1>(y), f);
      out[4] = mul_f16x2(e2m1_f16x2<2>(x), f);
      out[5] = mul_f16x2(e2m1_f16x2<2>(y), f);
      out[6] = mul_f16x2(e2m1_f16x2<3>(x), f);
      out[7] = mul_f16x2(e2m1_f16x2<3>(y), f);
    } else {
      const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
      out[0] = mul_bf16x2(e2m1_raw<0>(x), f);
      out[1] = mul_bf16x2(e2m1_raw<1>(x), f);
      out[2] = mul_bf16x2(e2m1_raw<2>(x), f);
      out[3] = mul_bf16x2(e2m1_raw<3>(x), f);
      out[4] = mul_bf16x2(e2m1_raw<0>(y), f);
      out[5] = mul_bf16x2(e2m1_raw<1>(y), f);
      out[6] = mul_bf16x2(e2m1_raw<2>(y), f);
      out[7] = mul_bf16x2(e2m1_raw<3>(y), f);
    }
  }
}

// log2 of the factor that operands carry beside the scale: keeps the smallest codes well
// inside fp16 and the bf16 form's factor within 2^127.
template <int FMT>
__host__ __device__ constexpr int lift_code() {
  return FMT == RING_ATTN_CACHE_MXFP8 ? 7 : 1;
}

// The factor 2^(byte - ref + lift) of two codes, `lo` and `hi` their blocks' scale bytes: as
// two fp16 (fields (byte - ref + lift + 15) << 10, built by one multiply-add per byte), or
// times 2^120 or 2^126 as two bf16 for the bf16 form (NaN for a block that is not finite, 0
// far below the reference).
template <int FMT, bool kHalf>
__device__ __forceinline__ uint32_t code_factors(uint32_t lo, uint32_t hi, int ref) {
  if (kHalf) return lo * 0x400u + hi * 0x4000000u + (uint32_t)(lift_code<FMT>() + 15 - ref) * 0x4000400u;
  auto one = [&](int byte) {
    const int e = byte - ref + lift_code<FMT>() + (FMT == RING_ATTN_CACHE_MXFP8 ? 120 : 126) + 127;
    return byte == 255 ? 0x7fc0u : (e <= 0 ? 0u : (uint32_t)e << 7);
  };
  return one((int)lo) | (one((int)hi) << 16);
}
template <int FMT, bool kHalf>
__device__ __forceinline__ uint32_t code_factor(uint32_t byte, int ref) {
  if (kHalf) return byte * 0x4000400u + (uint32_t)(lift_code<FMT>() + 15 - ref) * 0x4000400u;
  return code_factors<FMT, false>(byte, byte, ref);
}

// Chunk positions inside a row of the ring (16-byte units) that keep the fragment loads
// free of bank conflicts: K is read by 8 rows x 4 chunks, V by 4 even rows x 8 chunks.
template <int NC>
__device__ __forceinline__ int k_pos(int row, int ch) {
  return NC >= 8 ? ch ^ ((row & 1) << 2) : ch;
}
template <int NC>
__device__ __forceinline__ int v_slot(int row) {  // row's place in the step (16 rows stay together)
  return NC <= 4 ? (row & 16) | (row >> 1 & 7) | ((row & 1) << 3) : row;
}
template <int NC>
__device__ __forceinline__ int v_pos(int row, int ch) {
  if (NC == 16) return ch ^ (((row >> 1) & 1) | (row & 4));
  if (NC == 8) return ch ^ (row & 6);
  if (NC == 4) return ch ^ ((row >> 2 & 1) << 1);
  return ch;
}

// Head dimension at (k16 step s, lane quad position c, register half h, element e) of the
// score product.
template <int FMT, int D>
__device__ __forceinline__ int score_dim(int s, int c, int h, int e) {
  if (FMT == RING_ATTN_CACHE_BF16) return (4 * (s / 2) + c) * 8 + (s % 2) * 4 + h * 2 + e;
  if (FMT == RING_ATTN_CACHE_MXFP8) return (c + 4 * (s / 4)) * 16 + (s % 4) * 4 + h * 2 + e;
  return c * (D / 4) + s * 4 + h * 2 + e;
}

// 8x8 transpose of 16-bit elements held two per lane (lane 4 r + c: row r, columns 2c, 2c+1).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int FMT, int D, int NT>
struct Warp {
  using F = Fmt<FMT, D>;

  // Copies of the step whose first key is kb into ring stage `st`. The step's rows are
  // contiguous: lane l copies bytes 16 l + 512 x.
  static __device__ __forceinline__ void load(const Params& p, const Keys& ks, int64_t head_row, int kb, uint8_t* st) {
    const int lane = threadIdx.x % 32;
    const int64_t first = head_row + kb;
    const uint8_t* k = static_cast<const uint8_t*>(p.c.k) + first * F::kRowBytes + lane * 16;
    const uint8_t* v = static_cast<const uint8_t*>(p.c.v) + first * F::kRowBytes + lane * 16;
    constexpr int kCopies = F::kStep * F::kChunks;
    const bool all = whole_live(p, ks, kb);
#pragma unroll
    for (int e0 = 0; e0 < kCopies; e0 += 32) {
      const int e = e0 + lane;
      const int row = e / F::kChunks, ch = e % F::kChunks;
      // a dead row's copy is a zero fill that reads nothing
      const bool live = all || key_live(p, ks, kb + row);
      const int off = live ? e0 * 16 : -lane * 16;
      cp_async16(st + row * F::kRowBytes + k_pos<F::kChunks>(row, ch) * 16, k + off, live);
      cp_async16(st + F::kTileBytes + v_slot<F::kChunks>(row) * F::kRowBytes + v_pos<F::kChunks>(row, ch) * 16,
                 v + off, live);
    }
    if (F::kMx) {
      // scale bytes of 16 rows that start inside the cache lie inside it (capacity and kb are
      // multiples of 16); the second 16 may lie past its end
      constexpr int kWords = F::kScaleBytes / 4;  // 32 or 16 per tensor
      const bool in = lane < kWords / 2 || kb + 16 < p.c.capacity;
      if (lane < kWords && in) {
        cp_async4(st + 2 * F::kTileBytes + lane * 4,
                  static_cast<const uint8_t*>(p.c.k_scale) + first * F::kScaleRow + lane * 4);
        cp_async4(st + 2 * F::kTileBytes + F::kScaleBytes + lane * 4,
                  static_cast<const uint8_t*>(p.c.v_scale) + first * F::kScaleRow + lane * 4);
      }
    }
  }

  // All rows of the step that starts at kb can be seen by some query row.
  static __device__ __forceinline__ bool whole_live(const Params& p, const Keys& ks, int kb) {
    return kb + F::kStep <= ks.n + ks.cnt &&
           (p.window <= 0 || kb + F::kStep <= p.sinks || kb > ks.n - p.window);
  }

  // The largest and smallest scale bytes of the step's live K rows (ref[0], low[0]) and V rows
  // (ref[1], low[1]); false if one of them is 255. Such a block, which is not finite, is no part
  // of the reference: under 2^127 the step's other blocks, which rows that do not see that one
  // still need, would lose their bits. Dead rows hold zero codes under scale bytes that may be
  // anything: theirs become the reference, so that no factor is out of range.
  static __device__ __forceinline__ bool scale_range(uint8_t* st, bool all_live, uint32_t live_rows, int (&ref)[2],
                                                     int (&low)[2]) {
    bool finite = true;
    using Word = typename std::conditional<F::kScaleRow == 4, uint32_t, uint16_t>::type;
    const int lane = threadIdx.x % 32;
    const bool mine = all_live || (live_rows >> lane & 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Word* sc = reinterpret_cast<Word*>(st + 2 * F::kTileBytes + i * F::kScaleBytes) + lane;
      const uint32_t w = *sc;
      uint32_t hi, lo;
      if (F::kScaleRow == 4) {
        const uint32_t a = w & 0x00ff00ffu, b = w >> 8 & 0x00ff00ffu;
        const uint32_t mx = __vmaxu2(a, b), mn = __vminu2(a, b);
        hi = max(mx & 0xffffu, mx >> 16);
        lo = min(mn & 0xffffu, mn >> 16);
      } else {
        hi = max(w & 255u, w >> 8);
        lo = min(w & 255u, w >> 8);
      }
      ref[i] = (int)__reduce_max_sync(0xffffffffu, mine ? hi : 0u);
      low[i] = (int)__reduce_min_sync(0xffffffffu, mine ? lo : 255u);
      if (__builtin_expect(ref[i] == 255, 0)) {
        finite = false;
        hi = 0;
#pragma unroll 1
        for (uint32_t x = w; x != 0; x >>= 8)
          if ((x & 255u) != 255u) hi = max(hi, x & 255u);
        ref[i] = (int)__reduce_max_sync(0xffffffffu, mine ? hi : 0u);
      }
      if (!all_live) {
        if (!mine) *sc = (Word)(ref[i] * 0x01010101u);
        __syncwarp();
      }
    }
    return finite;
  }

  // d += a b with the query fragment in fp16 and a in fp16 or bf16.
  template <bool kHalf>
  static __device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&q)[2]) {
    if constexpr (kHalf || !F::kMx)
      mma16816<kHalf>(d, a, q[0], q[1]);
    else
      mma16816<false>(d, a, bf16_of_f16(q[0]), bf16_of_f16(q[1]));
  }

  // Scores of 16 keys (16 sub .. 16 sub + 15 of the step): s[x] the m16n8 tile of query rows
  // 8x .. 8x+7.
  template <bool kHalf>
  static __device__ __forceinline__ void scores(const uint8_t* st, int sub, const uint32_t (&q)[NT][F::kKSteps][2],
                                                float (&s)[NT][4], int ref) {
    const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const int row0 = 16 * sub + g, row1 = row0 + 8;
    const uint8_t* k0 = st + row0 * F::kRowBytes;
    const uint8_t* k1 = st + row1 * F::kRowBytes;
    const uint8_t* sc = st + 2 * F::kTileBytes;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] = 0.f;
    auto factor = [&](int row, int blk) { return code_factor<FMT, kHalf>(sc[row * F::kScaleRow + blk], ref); };
    if constexpr (FMT == RING_ATTN_CACHE_BF16) {
#pragma unroll
      for (int i = 0; i < F::kKSteps / 2; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(k0 + k_pos<F::kChunks>(row0, 4 * i + c) * 16);
        const uint4 z = *reinterpret_cast<const uint4*>(k1 + k_pos<F::kChunks>(row1, 4 * i + c) * 16);
        const uint32_t a[4] = {w.x, z.x, w.y, z.y}, b[4] = {w.z, z.z, w.w, z.w};
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          product<false>(s[x], a, q[x][2 * i]);
          product<false>(s[x], b, q[x][2 * i + 1]);
        }
      }
    } else if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
#pragma unroll
      for (int i = 0; i < F::kKSteps / 4; ++i) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(k0 + k_pos<F::kChunks>(row0, c + 4 * i) * 16);
        const uint4 z4 = *reinterpret_cast<const uint4*>(k1 + k_pos<F::kChunks>(row1, c + 4 * i) * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w}, z[4] = {z4.x, z4.y, z4.z, z4.w};
        const uint32_t f0 = factor(row0, (c + 4 * i) / 2), f1 = factor(row1, (c + 4 * i) / 2);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t b0[2], b1[2];
          word_pairs<FMT, kHalf>(w[y], f0, b0);
          word_pairs<FMT, kHalf>(z[y], f1, b1);
          const uint32_t a[4] = {b0[0], b1[0], b0[1], b1[1]};
#pragma unroll
          for (int x = 0; x < NT; ++x) product<kHalf>(s[x], a, q[x][4 * i + y]);
        }
      }
    } else {
      constexpr int kWords = D / 32;  // words of 8 codes per lane and row
      uint32_t w[kWords], z[kWords];
      if constexpr (D == 128) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(k0 + c * 16), z4 = *reinterpret_cast<const uint4*>(k1 + c * 16);
        w[0] = w4.x; w[1] = w4.y; w[2] = w4.z; w[3] = w4.w;
        z[0] = z4.x; z[1] = z4.y; z[2] = z4.z; z[3] = z4.w;
      } else {
        const uint2 w2 = *reinterpret_cast<const uint2*>(k0 + c * 8), z2 = *reinterpret_cast<const uint2*>(k1 + c * 8);
        w[0] = w2.x; w[1] = w2.y;
        z[0] = z2.x; z[1] = z2.y;
      }
      const uint32_t f0 = factor(row0, c * (D / 4) / kMxBlock), f1 = factor(row1, c * (D / 4) / kMxBlock);
#pragma unroll
      for (int y = 0; y < kWords; ++y) {
        uint32_t b0[4], b1[4];
        word_pairs<FMT, kHalf>(w[y], f0, b0);
        word_pairs<FMT, kHalf>(z[y], f1, b1);
        const uint32_t a[4] = {b0[0], b1[0], b0[1], b1[1]}, b[4] = {b0[2], b1[2], b0[3], b1[3]};
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          product<kHalf>(s[x], a, q[x][2 * y]);
          product<kHalf>(s[x], b, q[x][2 * y + 1]);
        }
      }
    }
  }

  // O^T += V^T P^T over 16 keys; pb[x] the P^T fragment of query rows 8x .. 8x+7. Lane row g of
  // o[x][i] is head dimension g * (D / 8) + 2i, lane row g + 8 the next one.
  template <bool kHalf>
  static __device__ __forceinline__ void values(const uint8_t* st, int sub, const uint32_t (&pb)[NT][2],
                                                float (&o)[NT][D / 16][4], int ref) {
    const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const uint8_t* vt = st + F::kTileBytes;
    const uint8_t* sc = st + 2 * F::kTileBytes + F::kScaleBytes;
    const int r0 = 16 * sub + 2 * c;
    const int rows[4] = {r0, r0 + 1, r0 + 8, r0 + 9};
    constexpr int kBytes = F::kRowBytes / 8;  // this lane's bytes of a row
    constexpr int kW = kBytes / 4;
    constexpr int kPer = D / 8 / kW;          // elements per word
    uint32_t w[4][kW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* vr = vt + v_slot<F::kChunks>(rows[r]) * F::kRowBytes;
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int x = 0; x < kBytes / 16; ++x) {
          const uint4 a =
              *reinterpret_cast<const uint4*>(vr + v_pos<F::kChunks>(rows[r], g * (kBytes / 16) + x) * 16);
          w[r][4 * x] = a.x; w[r][4 * x + 1] = a.y; w[r][4 * x + 2] = a.z; w[r][4 * x + 3] = a.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 a = *reinterpret_cast<const uint2*>(vr + v_pos<F::kChunks>(rows[r], g / 2) * 16 + (g % 2) * 8);
        w[r][0] = a.x; w[r][1] = a.y;
      } else {
        w[r][0] = *reinterpret_cast<const uint32_t*>(vr + v_pos<F::kChunks>(rows[r], g / 4) * 16 + (g % 4) * 4);
      }
    }
    uint32_t f01 = 0, f23 = 0;
    if (F::kMx) {
      const int blk = g * (D / 8) / kMxBlock;
      uint32_t f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = sc[rows[r] * F::kScaleRow + blk];
      f01 = code_factors<FMT, kHalf>(f[0], f[1], ref);
      f23 = code_factors<FMT, kHalf>(f[2], f[3], ref);
    }
#pragma unroll
    for (int y = 0; y < kW; ++y) {
      uint32_t b0[kPer], b1[kPer];
      key_pairs<FMT, kHalf>(w[0][y], w[1][y], f01, b0);
      key_pairs<FMT, kHalf>(w[2][y], w[3][y], f23, b1);
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const uint32_t a[4] = {b0[e], b0[e + 1], b1[e], b1[e + 1]};
#pragma unroll
        for (int x = 0; x < NT; ++x) mma16816<kHalf>(o[x][(kPer * y + e) / 2], a, pb[x][0], pb[x][1]);
      }
    }
  }
};

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, Fmt<FMT, D>::per_sm(NT)) tree_rows_kernel(const __grid_constant__ Params p) {
  using F = Fmt<FMT, D>;
  using W = Warp<FMT, D, NT>;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Walk s_walk;
  __shared__ float s_ml[kWarps][kRows][3];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;

  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = RING_ATTN_OK;  // the merge kernel reports
  grid_let_next();
  if (warp == 0) warp_begin_walk(p, &s_walk);
  __syncthreads();
  Walk walk = s_walk;
  Part part;
  uint8_t* ring = smem + warp * F::kStages * F::kStageBytes;
  while (next_part(p, walk, part)) {
    const Keys& ks = part.ks;
    const int b = part.b, grp = part.grp, kvh = part.kvh, q0 = part.q0, q1 = part.q1;
    const int64_t head_row = part.head_row;
    const int live_rows = ks.cnt * p.rep;

    // this warp's steps: one of every quad (the last quad of a unit may be short of some)
    const int quads = q1 - q0;
    auto step_of = [&](int j) { return kWarps * (q0 + j) + warp; };
    auto prefetch = [&](int j) {
      if (j < quads && step_of(j) < ks.steps)
        W::load(p, ks, head_row, step_key(p, ks, step_of(j)), ring + (j % F::kStages) * F::kStageBytes);
      cp_commit();
    };
#pragma unroll 1
    for (int j = 0; j < F::kStages - 1; ++j) prefetch(j);
    const Nodes nodes = warp_nodes(p, b, ks);

    // queries in the score product's order of head dimensions (lane column g: query row g of
    // the tile); fp16 ones times 2^(14 - exponent of the row's largest)
    uint32_t q[NT][F::kKSteps][2];
    float own_scale[NT];  // scores of query row 8x + g to the base-2 domain, K's step reference apart
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int row = grp * kRows + 8 * i + g;
      const bool in = row < live_rows;
      const uint16_t* src = p.q + b * p.qs_b + (int64_t)(kvh * p.rep + (in ? row % p.rep : 0)) * p.qs_h +
                            (in ? row / p.rep : 0) * p.qs_t;
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < F::kKSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t v = in ? *reinterpret_cast<const uint32_t*>(src + score_dim<FMT, D>(s, c, h, 0)) : 0u;
          q[i][s][h] = v;
          top = max(top, max(v & 0x7fffu, v >> 16 & 0x7fffu));
        }
      own_scale[i] = p.scale_log2;
      if (F::kMx) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(top >> 7), 15) - 127;  // exponent of the largest (not below 2^-112)
        const float up = pow2(14 - e);
#pragma unroll
        for (int s = 0; s < F::kKSteps; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v = q[i][s][h];
            q[i][s][h] = pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
          }
        own_scale[i] = p.scale_log2 * exp2f((float)(e - 14 - lift_code<FMT>()));
      }
    }
    // this lane's query rows in a score tile: 8i + 2c and the next one
    float row_scale[NT][2];
    int lo_key[NT][2];      // first key of the row's window
    uint64_t vis[NT][2];    // drafted nodes it sees
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        row_scale[i][r] = __shfl_sync(0xffffffffu, own_scale[i], 4 * (2 * c + r));
        const int row = grp * kRows + 8 * i + 2 * c + r;
        int depth;
        node_of(nodes, row < live_rows ? row / p.rep : 0, vis[i][r], depth);
        lo_key[i][r] = p.window > 0 ? ks.n + depth - p.window + 1 : 0;
      }

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][d][e] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
    int v_ref = 0;  // E, see the head of the file

#pragma unroll 1
    for (int j = 0; j < quads; ++j) {
      prefetch(j + F::kStages - 1);
      cp_wait<F::kStages - 1>();
      __syncwarp();
      const int i_step = step_of(j);
      if (i_step < ks.steps) {
        uint8_t* st = ring + (j % F::kStages) * F::kStageBytes;
        const int kb = step_key(p, ks, i_step);
        // every row sees all keys of the step
        const bool whole =
            kb + F::kStep <= ks.n &&
            (p.window <= 0 || kb + F::kStep <= p.sinks || kb >= ks.n + p.T - p.window);
        uint32_t live = 0xffffffffu;
        int ref[2] = {0, 0};
        bool half = true;
        float p_up = 1.f, k_up = 1.f;
        if (F::kMx) {
          if (!whole) live = __ballot_sync(0xffffffffu, key_live(p, ks, kb + lane));
          int low[2];
          half = W::scale_range(st, whole, live, ref, low);
          half = half && ref[0] - low[0] <= kSpread && ref[1] - low[1] <= kSpread;
          if (ref[1] > v_ref) {  // raise E: O carries 2^-E
            const float a = pow2(v_ref - ref[1]);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][d][e] *= a;
            v_ref = ref[1];
          }
          half = half && v_ref - ref[1] <= kBelow;
          p_up = pow2(ref[1] - v_ref + kLiftP);
          k_up = pow2(ref[0] - 127);
        }
#pragma unroll 1
        for (int sub = 0; sub < F::kSubs; ++sub) {
          float s[NT][4];  // (key g, rows 2c, 2c+1), (key g + 8, the same rows)
          if (!F::kMx || __builtin_expect(half, 1))
            W::template scores<F::kMx>(st, sub, q, s, ref[0]);
          else
            W::template scores<false>(st, sub, q, s, ref[0]);
          bool rise = false;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] *= k_up * row_scale[i][e & 1];
            if (!whole) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = e & 1, u = kb + 16 * sub + g + 8 * (e >> 1);
                const bool see = u < ks.n ? (u < p.sinks || u >= lo_key[i][r])
                                          : (u < ks.n + ks.cnt && (vis[i][r] >> (u - ks.n) & 1));
                if (!see) s[i][e] = -INFINITY;
              }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) rise |= fmaxf(s[i][r], s[i][r + 2]) > m[i][r] + rescale_log2<FMT>();
          }
          // the reference maximum moves only when a score passes it by rescale_log2 (or is the first)
          if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float top = fmaxf(s[i][r], s[i][r + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                if (top > m[i][r]) {
                  const float a = m[i][r] == -INFINITY ? 0.f : ex2_approx(m[i][r] - top);
                  m[i][r] = top;
                  l[i][r] *= a;
#pragma unroll
                  for (int d = 0; d < D / 16; ++d) {
                    o[i][d][r] *= a;
                    o[i][d][r + 2] *= a;
                  }
                }
              }
          }
          uint32_t pb[NT][2];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const float z0 = m[i][0] == -INFINITY ? 0.f : m[i][0], z1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
            const float p0 = ex2_approx(s[i][0] - z0), p1 = ex2_approx(s[i][1] - z1);
            const float p2 = ex2_approx(s[i][2] - z0), p3 = ex2_approx(s[i][3] - z1);
            l[i][0] += p0 + p2;
            l[i][1] += p1 + p3;
            uint32_t a, d;
            if (F::kMx && half) {
              a = pack_f16x2(p0 * p_up, p1 * p_up);
              d = pack_f16x2(p2 * p_up, p3 * p_up);
            } else {
              a = pack_bf16x2(p0 * p_up, p1 * p_up);
              d = pack_bf16x2(p2 * p_up, p3 * p_up);
            }
            pb[i][0] = transpose8(a);  // (keys 2c, 2c + 1, query row g)
            pb[i][1] = transpose8(d);
          }
          if (!F::kMx || __builtin_expect(half, 1))
            W::template values<F::kMx>(st, sub, pb, o, ref[1]);
          else
            W::template values<false>(st, sub, pb, o, ref[1]);
        }
      }
      __syncwarp();
    }
    cp_wait<0>();

    // Join the four warps' states: weights 2^(m_w - M), and 2^E_w on what carries it, then O / l.
    // A state that saw no key is known by its sum, which is 0: scores that are NaN leave the
    // reference at -inf too (no maximum takes them up), but make the sum NaN, and with it the row.
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float y = l[i][r];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (g == 0) {
          s_ml[warp][8 * i + 2 * c + r][0] = m[i][r];
          s_ml[warp][8 * i + 2 * c + r][1] = y;
          s_ml[warp][8 * i + 2 * c + r][2] = F::kMx ? (float)(v_ref - 127 - kLiftP - lift_code<FMT>()) : 0.f;
        }
      }
    __syncthreads();  // every warp has left its ring: the O tiles take its place
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float* dst = so + (warp * kRows + 8 * i + 2 * c + r) * (D + 4) + g * (D / 8);
#pragma unroll
        for (int d = 0; d < D / 16; d += 2)
          *reinterpret_cast<float4*>(dst + 2 * d) =
              make_float4(o[i][d][r], o[i][d][r + 2], o[i][d + 1][r], o[i][d + 1][r + 2]);
      }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + part.unit;
    {
      constexpr int kTpr = kThreads / kRows, kPer = D / kTpr;  // threads and dimensions per row
      const int r = threadIdx.x / kTpr, d0 = (threadIdx.x % kTpr) * kPer;
      const int row = grp * kRows + r;
      if (row < live_rows) {
        float M = -INFINITY, E = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          M = fmaxf(M, s_ml[w][r][0]);
          E = fmaxf(E, s_ml[w][r][2]);
        }
        float L = 0.f, acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float lw = s_ml[w][r][1];
          if (lw == 0.f) continue;
          const float a = ex2_approx(s_ml[w][r][0] - M);
          L += a * lw;
          const float av = a * exp2f(s_ml[w][r][2] - E);
          const float* src = so + (w * kRows + r) * (D + 4) + d0;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(av, src[e], acc[e]);
        }
        const bool none = L == 0.f;
        const float inv = none ? 0.f : 1.f / L;
        const float up = exp2f(E);  // applied apart from 1 / L: the two together may leave fp32's range
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * inv * up;
        const float lse2 = none ? -INFINITY : M + log2f(L);
        if (part.alone) {
          const int64_t orow = out_row(p, b, kvh, row);
#pragma unroll
          for (int e = 0; e < kPer; e += 4)
            *reinterpret_cast<uint2*>(p.out + orow * D + d0 + e) =
                make_uint2(pack_bf16x2(acc[e], acc[e + 1]), pack_bf16x2(acc[e + 2], acc[e + 3]));
          if (d0 == 0) p.lse[orow] = lse2 * 0.69314718055994530942f;
        } else {
          float* dst = p.o_parts + (slot * kRows + r) * D + d0;
#pragma unroll
          for (int e = 0; e < kPer; e += 4)
            *reinterpret_cast<float4*>(dst + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
          if (d0 == 0) p.lse_parts[slot * kRows + r] = lse2;
        }
      }
    }
    __syncthreads();  // s_ml and the O tiles are read before the ring is filled again
  }
}

// Block 0 of a merge: lengths, counts and parents out of range go to the status word.
__device__ __noinline__ void report_bad(const Params& p) {
  int bad = 0;
#pragma unroll 1
  for (int i = threadIdx.x; i < p.c.B * p.T; i += 128) {
    const int x = i / p.T, t = i - x * p.T;
    int n, cnt;
    if (bad_sequence(p, x, n, cnt)) {
      bad = 1;
    } else if (p.parents && t < cnt) {
      const int par = p.parents[i];
      if (par < -1 || par >= t) bad = 1;
    }
  }
  if (bad) atomicExch(p.status, RING_ATTN_EINVAL);
}

// One block per unit and row: the row's partials (in the order of the CTAs that made them)
// are joined with weights 2^(lse_i - max); rows that no key reaches and rows of dead nodes
// get out = 0 and lse = -inf. A unit that one CTA did alone is only completed by its dead
// rows. Block 0 writes the status word.
template <int D>
__global__ void __launch_bounds__(128) tree_merge_kernel(const __grid_constant__ Params p) {
  constexpr int kTpr = D / 4;              // threads per partial row (float4 each)
  constexpr int kPar = 128 / kTpr;         // partials in flight
  __shared__ Parts s_parts;
  __shared__ float s_max[4];
  __shared__ float s_sum[kPar];
  __shared__ float4 s_acc[kPar][kTpr];
  const int unit = blockIdx.x / p.rows_per_group;
  const int r = blockIdx.x - unit * p.rows_per_group;
  const int head = unit / p.groups, b = head / p.c.Hkv, kvh = head - b * p.c.Hkv;
  const int row = (unit - head * p.groups) * p.rows_per_group + r;
  const Keys ks = sequence_keys(p, b);
  const uint32_t per = unit_quads(p, ks);
  const int d4 = threadIdx.x % kTpr, part = threadIdx.x / kTpr;
  if (per != 0 && threadIdx.x < 32) {
    const Parts x = warp_parts(p, b, unit - b * p.c.Hkv * p.groups, per);
    if (threadIdx.x == 0) s_parts = x;
  }
  grid_wait();
  if (blockIdx.x == 0) report_bad(p);
  if (row >= p.T * p.rep) return;
  const int64_t orow = out_row(p, b, kvh, row);
  if (row >= ks.cnt * p.rep || per == 0) {
    if (threadIdx.x < D / 8) reinterpret_cast<uint4*>(p.out + orow * D)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) p.lse[orow] = -INFINITY;
    return;
  }
  __syncthreads();
  const int parts = (int)s_parts.count;
  if (parts == 1) return;
  const int64_t slot = (int64_t)s_parts.first + unit;
  const float* lse = p.lse_parts + slot * p.rows_per_group + r;
  const float* src = p.o_parts + (slot * p.rows_per_group + r) * D + 4 * d4;
  const int64_t stride = (int64_t)p.rows_per_group * D;
  float M = -INFINITY;
#pragma unroll 1
  for (int i = threadIdx.x; i < parts; i += 128) M = fmaxf(M, lse[i * p.rows_per_group]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  if (M == -INFINITY) M = 0.f;  // no part is finite: a NaN among them still reaches the sum
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int i = part; i < parts; i += kPar) {
    const float w = ex2_approx(lse[i * p.rows_per_group] - M);
    const float4 v = *reinterpret_cast<const float4*>(src + i * stride);
    sum += w;  // an empty part's row is 0 and so is its weight
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  s_acc[part][d4] = acc;
  if (d4 == 0) s_sum[part] = sum;
  __syncthreads();
  if (part != 0) return;
  float tot = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPar; ++i) {
    tot += s_sum[i];
    a.x += s_acc[i][d4].x;
    a.y += s_acc[i][d4].y;
    a.z += s_acc[i][d4].z;
    a.w += s_acc[i][d4].w;
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  reinterpret_cast<uint2*>(p.out + orow * D)[d4] =
      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (d4 == 0) p.lse[orow] = (M + log2f(tot)) * 0.69314718055994530942f;  // (log2 0 = -inf)
}

// The same for units of many rows, whose parts are fewer. The unit's parts are found once for
// 16 / G rows; G groups of 8 lanes share a row's parts: 4 where the rows alone leave SMs idle,
// else 1 (12 units of 128 rows, D = 128, 13 parts: 4 groups 7 us, 1 group 13, a warp per row 10; 128 units, D = 64,
// 2 parts: a warp per row 13 us, 1 group 6.5).
template <int D, int G>
__global__ void __launch_bounds__(128) tree_merge_rows_kernel(const __grid_constant__ Params p) {
  constexpr int kRows = 16 / G;  // per block
  const int lane = threadIdx.x % 32, sub = lane % 8, grp = lane / 8 % G;
  const int per_unit = p.rows_per_group / kRows;
  const int unit = blockIdx.x / per_unit;
  const int r = (blockIdx.x - unit * per_unit) * kRows + threadIdx.x / (8 * G);
  const int head = unit / p.groups, b = head / p.c.Hkv, kvh = head - b * p.c.Hkv;
  const int row = (unit - head * p.groups) * p.rows_per_group + r;
  const Keys ks = sequence_keys(p, b);
  const uint32_t per = unit_quads(p, ks);
  Parts x{0u, 1u};
  if (per != 0) x = warp_parts(p, b, unit - b * p.c.Hkv * p.groups, per);
  grid_wait();
  if (blockIdx.x == 0) report_bad(p);
  if (row >= p.T * p.rep) return;
  const int64_t orow = out_row(p, b, kvh, row);
  constexpr int kVec = D / 32;  // four neighbouring dimensions each, 32 apart
  uint16_t* dst = p.out + orow * D + 4 * sub;
  if (row >= ks.cnt * p.rep || per == 0) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) *reinterpret_cast<uint2*>(dst + 32 * e) = make_uint2(0u, 0u);
    if (sub + grp == 0) p.lse[orow] = -INFINITY;
    return;
  }
  const int parts = (int)x.count;
  if (parts == 1) return;
  const int64_t slot = (int64_t)x.first + unit;
  const float* lse = p.lse_parts + slot * p.rows_per_group + r;
  const float* src = p.o_parts + (slot * p.rows_per_group + r) * D + 4 * sub;
  const int64_t stride = (int64_t)p.rows_per_group * D;
  const uint32_t row_lanes = G == 4 ? 0xffffffffu : 0xffu << (lane & 24);
  float M = -INFINITY;
#pragma unroll 1
  for (int i = sub + 8 * grp; i < parts; i += 8 * G) M = fmaxf(M, lse[(int64_t)i * p.rows_per_group]);
#pragma unroll
  for (int o = 4 * G; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(row_lanes, M, o));
  if (M == -INFINITY) M = 0.f;  // as above
  float sum = 0.f;
  float4 acc[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < parts; i += G) {
    const float w = ex2_approx(lse[(int64_t)i * p.rows_per_group] - M);
    sum += w;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {  // an empty part's row is 0 and so is its weight
      const float4 v = *reinterpret_cast<const float4*>(src + i * stride + 32 * e);
      acc[e].x = fmaf(w, v.x, acc[e].x);
      acc[e].y = fmaf(w, v.y, acc[e].y);
      acc[e].z = fmaf(w, v.z, acc[e].z);
      acc[e].w = fmaf(w, v.w, acc[e].w);
    }
  }
#pragma unroll
  for (int o = 8; o < 8 * G; o *= 2) {
    sum += __shfl_xor_sync(row_lanes, sum, o);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      acc[e].x += __shfl_xor_sync(row_lanes, acc[e].x, o);
      acc[e].y += __shfl_xor_sync(row_lanes, acc[e].y, o);
      acc[e].z += __shfl_xor_sync(row_lanes, acc[e].z, o);
      acc[e].w += __shfl_xor_sync(row_lanes, acc[e].w, o);
    }
  }
  if (grp != 0) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < kVec; ++e)
    *reinterpret_cast<uint2*>(dst + 32 * e) =
        make_uint2(pack_bf16x2(acc[e].x * inv, acc[e].y * inv), pack_bf16x2(acc[e].z * inv, acc[e].w * inv));
  if (sub == 0) p.lse[orow] = (M + log2f(sum)) * 0.69314718055994530942f;
}

template <int FMT, int D, int NT>
int launch_rows_t(const Params& p, cudaStream_t stream) {
  constexpr int smem = Fmt<FMT, D>::smem(8 * NT);
  auto kern = tree_rows_kernel<FMT, D, NT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return RING_ATTN_ECUDA;
  kern<<<p.ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

template <int FMT, int D>
int launch_rows(const Params& p, cudaStream_t stream) {
  return p.rows_per_group == 8 ? launch_rows_t<FMT, D, 1>(p, stream) : launch_rows_t<FMT, D, 2>(p, stream);
}

template <int FMT>
int launch_rows_d(const Params& p, cudaStream_t stream) {
  return p.c.D == 64 ? launch_rows<FMT, 64>(p, stream) : launch_rows<FMT, 128>(p, stream);
}

int launch_merge(void (*kern)(Params), int64_t blocks, const Params& p, cudaStream_t stream) {
  return launch_early(kern, (unsigned)blocks, 128, 0, stream, p) == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

inline int step_keys(int format, int D) { return format == RING_ATTN_CACHE_BF16 && D == 128 ? 16 : 32; }

}  // namespace tree

namespace {

// Shape of a launch: row groups, the division's grain and the partial slots.
struct TreePlan {
  int rows_per_group, groups, step, quad_log2, ctas, min_quads;
  int64_t units, slots;
};

// More than 16 query rows per kv head go to the tcgen05 form, whose tile is 128 rows whatever
// part of them is real; up to 16 the warp form, which takes the cache once per 16 rows. 32
// (sequence, head) pairs of 32k keys, us, warps / tiles, at 8, 16, 20 and 64 rows: e4m3, D = 128
// 66 / 106, 91 / 107, 154 / 108, 291 / 113; e2m1, D = 64 43 / 80, 55 / 81, 90 / 81, 167 / 83;
// bf16, D = 128 95 / 93, 92 / 94, 166 / 95, 293 / 99.
TreePlan tree_plan(const CacheView& c, int Hq, int T) {
  TreePlan t;
  const int rows = T * (Hq / c.Hkv);
  if (rows > 16) {
    t.rows_per_group = 128;
    t.step = 128;
    t.quad_log2 = 0;
    t.ctas = 148;
    t.min_quads = 1;
  } else {
    t.rows_per_group = rows <= 8 ? 8 : 16;
    t.step = tree::step_keys(c.format, c.D);
    t.quad_log2 = 2;
    t.ctas = 148 * (c.D == 128 && t.rows_per_group == 16 ? 2 : 3);
    t.min_quads = 2;
  }
  t.groups = (rows + t.rows_per_group - 1) / t.rows_per_group;
  t.units = (int64_t)c.B * c.Hkv * t.groups;
  t.slots = t.ctas + t.units;
  return t;
}

}  // namespace

size_t tree_workspace_bytes(const CacheView& c, int Hq, int T) {
  const TreePlan t = tree_plan(c, Hq, T);
  return kWorkspaceHeaderBytes + sizeof(float) * (size_t)t.slots * t.rows_per_group * (size_t)(c.D + 1);
}

int launch_tree(const CacheView& c, const void* q, const int64_t* qs, void* out, float* lse, const int32_t* lengths,
                const int32_t* parents, const int32_t* counts, int Hq, int T, int window, int sinks, float scale,
                void* workspace, uint64_t watchdog_ns, cudaStream_t stream) {
  const TreePlan t = tree_plan(c, Hq, T);
  tree::Params p;
  p.c = c;
  p.q = static_cast<const uint16_t*>(q);
  p.qs_b = qs[0];
  p.qs_h = qs[1];
  p.qs_t = qs[2];
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.lengths = lengths;
  p.parents = parents;
  p.counts = counts;
  p.Hq = Hq;
  p.T = T;
  p.rep = Hq / c.Hkv;
  p.window = window;
  p.sinks = sinks;
  p.groups = t.groups;
  p.rows_per_group = t.rows_per_group;
  p.step = t.step;
  p.step_log2 = t.step == 128 ? 7 : (t.step == 32 ? 5 : 4);
  p.quad_log2 = t.quad_log2;
  p.ctas = t.ctas;
  p.min_quads = t.min_quads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o_parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeaderBytes);
  p.lse_parts = p.o_parts + (size_t)t.slots * t.rows_per_group * c.D;
  p.status = static_cast<int*>(workspace);
  p.watchdog_ns = watchdog_ns;
  // the device's arithmetic on units and their quads is in 32 bits
  const int64_t quads = t.units * ((c.capacity / t.step + 2) / (1 << t.quad_log2) + 1);
  if (t.units * t.rows_per_group > 0x7fffffff || quads > 0x7fffffff || (int64_t)c.B * T > 0x7fffffff)
    return RING_ATTN_EINVAL;
  int rc;
  if (t.rows_per_group == 128) {
    rc = tree::launch_tiles(p, stream);
  } else {
    switch (c.format) {
      case RING_ATTN_CACHE_BF16: rc = tree::launch_rows_d<RING_ATTN_CACHE_BF16>(p, stream); break;
      case RING_ATTN_CACHE_MXFP8: rc = tree::launch_rows_d<RING_ATTN_CACHE_MXFP8>(p, stream); break;
      default: rc = tree::launch_rows_d<RING_ATTN_CACHE_MXFP4>(p, stream); break;
    }
  }
  if (rc) return rc;
  if (t.rows_per_group == 128) {
    const int64_t rows = t.units * t.rows_per_group;
    if (rows < 16 * 4 * 148)
      return tree::launch_merge(c.D == 64 ? tree::tree_merge_rows_kernel<64, 4> : tree::tree_merge_rows_kernel<128, 4>,
                                rows / 4, p, stream);
    return tree::launch_merge(c.D == 64 ? tree::tree_merge_rows_kernel<64, 1> : tree::tree_merge_rows_kernel<128, 1>,
                              rows / 16, p, stream);
  }
  return tree::launch_merge(c.D == 64 ? tree::tree_merge_kernel<64> : tree::tree_merge_kernel<128>,
                            t.units * t.rows_per_group, p, stream);
}

}  // namespace ringattn
