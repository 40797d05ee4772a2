// Attention of drafted tokens over a cache, for few query rows per kv head (bf16, mxfp8 or
// mxfp4 cache; D = 64 or 128), and the merge of split results.
//
// Mathematics: online softmax over the visible keys in base 2, m = reference maximum,
// p = 2^(s scale log2 e - m), l = sum p, O = sum p v, result O / l and m + log2 l.
//
// What bounds it: reading the cache once. A group of 16 query rows is one m16n8k16 tile,
// and every warp works alone on 16 keys at a time: it keeps its own ring of cache rows in
// shared memory (16-byte asynchronous copies, no block barrier in the loop), converts
// codes to bf16 in registers straight into the operand fragments, and holds the group's
// queries, running state and output in registers. Nothing that was dequantised is written
// anywhere. The tensor work is small here (one row tile), which is why this form uses the
// warp-level matrix instructions: their operands come from registers, whereas tcgen05
// reads them from shared memory, where the dequantised tile would have to be written and
// read again (1536 of 1460 clocks that HBM needs for 128 mxfp8 keys).
//
// Codes to bf16 without a conversion instruction: the code's sign goes to the sign bit,
// its exponent and mantissa to the low exponent and high mantissa bits. That bf16 value is
// the code's value times 2^-120 (e4m3) or 2^-126 (e2m1), subnormal codes included, and one
// exact multiplication by a power of two brings in the block's scale. To keep that factor
// inside bf16's range for every scale up to 2^63, K and V are held 2^62 too small and Q and
// P 2^62 too large; the products are those of the true values. A block whose scale is
// larger reads as NaN. Which head dimension or key meets which k index of a matrix
// instruction is free as long as both operands agree, so the pairs are those that a word
// of codes yields by shifts: (0,2),(1,3) of four 8-bit codes, (i, i+4) of eight 4-bit ones.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sm100_ptx.cuh"
#include "tree_common.cuh"

namespace ringattn {
namespace tree {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;    // query rows per group
constexpr int kStep = 16;    // keys per warp and step
constexpr float kLift = 62.f;            // log2 of the factor between held and true K, V (see above)
constexpr float kRescale = 8.f;          // the reference maximum moves when a score passes it by this

template <int FMT, int D>
struct Fmt {
  static constexpr int kRowBytes = cache_row_bytes<FMT>(D);
  static constexpr int kChunks = kRowBytes / 16;             // 16-byte chunks per row
  static constexpr bool kMx = FMT != RING_ATTN_CACHE_BF16;
  static constexpr int kScaleRow = kMx ? D / kMxBlock : 0;   // scale bytes per row
  static constexpr int kTileBytes = kStep * kRowBytes;       // K or V of one step
  static constexpr int kScaleBytes = kStep * kScaleRow;
  static constexpr int kStageBytes = 2 * kTileBytes + (kMx ? 128 : 0);
  static constexpr int kStages = FMT == RING_ATTN_CACHE_BF16 ? (D == 128 ? 3 : 4) : (FMT == RING_ATTN_CACHE_MXFP8 ? 4 : 6);
  static constexpr int kMerge = kWarps * kRows * (D + 4) * 4;  // end of unit: O of every warp
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static constexpr int kKSteps = D / 16;                     // k16 steps of the score product
  // resident CTAs per SM: what registers allow (168 or 128 a thread), less where the rings fill shared memory
  static constexpr int kFit = 232448 / (kSmem + 4096);
  static constexpr int kPerSm = kFit < (D == 128 ? 3 : 4) ? kFit : (D == 128 ? 3 : 4);
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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// bf16 (exponent field shifted, see the head of the file) pairs from a word of codes:
// e4m3 bytes 0 and 2 (Odd = false) or 1 and 3.
template <bool Odd>
__device__ __forceinline__ uint32_t e4m3_raw(uint32_t w) {
  if (!Odd) w <<= 8;
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
// e2m1 nibbles I and I + 4.
template <int I>
__device__ __forceinline__ uint32_t e2m1_raw(uint32_t w) {
  const uint32_t x = w << (12 - 4 * I);
  return ((x >> 6) & 0x01c001c0u) | (x & 0x80008000u);
}

// 2^(byte - 127 + lift of the raw form - 62) as bf16 bits; NaN above a scale of 2^63.
template <int FMT>
__device__ __forceinline__ uint32_t raw_factor(uint32_t byte) {
  constexpr uint32_t up = FMT == RING_ATTN_CACHE_MXFP8 ? 58u : 64u;  // 120 - 62, 126 - 62
  return byte > 190u ? 0x7fc0u : (byte + up) << 7;
}

// Chunk positions inside a row of the ring (16-byte units) that keep the fragment loads
// free of bank conflicts: K is read by 8 rows x 4 chunks, V by 4 even rows x 8 chunks.
template <int NC>
__device__ __forceinline__ int k_pos(int row, int ch) {
  return NC >= 8 ? ch ^ ((row & 1) << 2) : ch;
}
template <int NC>
__device__ __forceinline__ int v_slot(int row) {  // row's place among the 16
  return NC <= 4 ? (row >> 1) | ((row & 1) << 3) : row;
}
template <int NC>
__device__ __forceinline__ int v_pos(int row, int ch) {
  if (NC == 16) return ch ^ (((row >> 1) & 1) | (row & 4));
  if (NC == 8) return ch ^ (row & 6);
  if (NC == 4) return ch ^ (((v_slot<NC>(row) >> 1) & 1) << 1);
  return ch;
}

// Head dimension at (k16 step s, lane quad position c, register half h, element e) of the
// score product.
template <int FMT, int D>
__device__ __forceinline__ int score_dim(int s, int c, int h, int e) {
  if (FMT == RING_ATTN_CACHE_BF16) return (4 * (s / 2) + c) * 8 + (s % 2) * 4 + h * 2 + e;
  if (FMT == RING_ATTN_CACHE_MXFP8) return (c + 4 * (s / 4)) * 16 + (s % 4) * 4 + h + 2 * e;
  return c * (D / 4) + (s / 2) * 8 + (s % 2) * 2 + h + 4 * e;
}

template <int FMT, int D>
struct Warp {
  using F = Fmt<FMT, D>;

  // Copies of step `i` into ring stage `st` (one commit group, empty when i is out of range).
  static __device__ __forceinline__ void load(const Params& p, const Keys& ks, int64_t head_row, int i, bool in,
                                              uint8_t* st) {
    const int lane = threadIdx.x % 32;
    if (in) {
      const int kb = step_key(p, ks, i);
      const uint8_t* k = static_cast<const uint8_t*>(p.c.k) + (head_row + kb) * F::kRowBytes;
      const uint8_t* v = static_cast<const uint8_t*>(p.c.v) + (head_row + kb) * F::kRowBytes;
      constexpr int kCopies = kStep * F::kChunks;
#pragma unroll
      for (int e0 = 0; e0 < kCopies; e0 += 32) {
        const int e = e0 + lane;
        const int row = e / F::kChunks, ch = e % F::kChunks;
        // a dead row's copy is a zero fill that reads nothing
        const bool live = key_live(p, ks, kb + row);
        const int64_t off = live ? (int64_t)row * F::kRowBytes + ch * 16 : 0;
        cp_async16(st + row * F::kRowBytes + k_pos<F::kChunks>(row, ch) * 16, k + off, live);
        cp_async16(st + F::kTileBytes + v_slot<F::kChunks>(row) * F::kRowBytes + v_pos<F::kChunks>(row, ch) * 16,
                   v + off, live);
      }
      if (F::kMx) {
        // the step's scale bytes are contiguous: capacity and kb are multiples of 16 rows
        constexpr int kWords = F::kScaleBytes / 4;
        if (lane < kWords)
          cp_async4(st + 2 * F::kTileBytes + lane * 4,
                    static_cast<const uint8_t*>(p.c.k_scale) + (head_row + kb) * F::kScaleRow + lane * 4);
        else if (lane >= 16 && lane < 16 + kWords)
          cp_async4(st + 2 * F::kTileBytes + 64 + (lane - 16) * 4,
                    static_cast<const uint8_t*>(p.c.v_scale) + (head_row + kb) * F::kScaleRow + (lane - 16) * 4);
      }
    }
    cp_commit();
  }

  // Scale byte j of cache row `row` of the step (sc: the step's K or V scale bytes).
  static __device__ __forceinline__ uint32_t scale_byte(const uint8_t* sc, int row, int j) {
    return sc[row * F::kScaleRow + j];
  }

  // Scores of 16 keys: s[t] the m16n8 tile of keys 8t .. 8t+7.
  static __device__ __forceinline__ void scores(const uint8_t* st, const uint32_t (&q)[F::kKSteps][4],
                                                float (&s)[2][4], const bool (&key_ok)[2]) {
    const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int row = 8 * t + g;
      const uint8_t* kr = st + row * F::kRowBytes;
      const uint8_t* sc = st + 2 * F::kTileBytes;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
      if constexpr (FMT == RING_ATTN_CACHE_BF16) {
#pragma unroll
        for (int i = 0; i < F::kKSteps / 2; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(kr + k_pos<F::kChunks>(row, 4 * i + c) * 16);
          mma16816(s[t], q[2 * i], w.x, w.y);
          mma16816(s[t], q[2 * i + 1], w.z, w.w);
        }
      } else if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
#pragma unroll
        for (int i = 0; i < F::kKSteps / 4; ++i) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(kr + k_pos<F::kChunks>(row, c + 4 * i) * 16);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          const uint32_t f = key_ok[t] ? raw_factor<FMT>(scale_byte(sc, row, (c + 4 * i) / 2)) * 0x10001u : 0u;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma16816(s[t], q[4 * i + x], mul_bf16x2(e4m3_raw<false>(w[x]), f), mul_bf16x2(e4m3_raw<true>(w[x]), f));
        }
      } else {
        constexpr int kWords = D / 32;  // words of 8 codes per lane
        uint32_t w[kWords];
        if constexpr (D == 128) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(kr + c * 16);
          w[0] = w4.x; w[1] = w4.y; w[2] = w4.z; w[3] = w4.w;
        } else {
          const uint2 w2 = *reinterpret_cast<const uint2*>(kr + c * 8);
          w[0] = w2.x; w[1] = w2.y;
        }
        const uint32_t f = key_ok[t] ? raw_factor<FMT>(scale_byte(sc, row, c * (D / 4) / kMxBlock)) * 0x10001u : 0u;
#pragma unroll
        for (int x = 0; x < kWords; ++x) {
          mma16816(s[t], q[2 * x], mul_bf16x2(e2m1_raw<0>(w[x]), f), mul_bf16x2(e2m1_raw<1>(w[x]), f));
          mma16816(s[t], q[2 * x + 1], mul_bf16x2(e2m1_raw<2>(w[x]), f), mul_bf16x2(e2m1_raw<3>(w[x]), f));
        }
      }
    }
  }

  // O += P V over the 16 keys. o[j] is the m16n8 tile whose column x is head dimension
  // x * (D / 8) + j.
  static __device__ __forceinline__ void values(const uint8_t* st, const uint32_t (&pa)[4], float (&o)[D / 8][4],
                                                const bool (&v_ok)[4]) {
    const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const uint8_t* vt = st + F::kTileBytes;
    const uint8_t* sc = st + 2 * F::kTileBytes + 64;
    const int rows[4] = {2 * c, 2 * c + 1, 2 * c + 8, 2 * c + 9};
    constexpr int kBytes = F::kRowBytes / 8;  // this lane's bytes of a row
    constexpr int kW = kBytes / 4;
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
      for (int r = 0; r < 4; ++r) f[r] = v_ok[r] ? raw_factor<FMT>(scale_byte(sc, rows[r], blk)) : 0u;
      f01 = f[0] | (f[1] << 16);
      f23 = f[2] | (f[3] << 16);
    }
#pragma unroll
    for (int x = 0; x < kW; ++x) {
      // the low and high halves of the word, of two keys side by side
      const uint32_t a0 = __byte_perm(w[0][x], w[1][x], 0x5410), a1 = __byte_perm(w[0][x], w[1][x], 0x7632);
      const uint32_t b0 = __byte_perm(w[2][x], w[3][x], 0x5410), b1 = __byte_perm(w[2][x], w[3][x], 0x7632);
      if constexpr (FMT == RING_ATTN_CACHE_BF16) {
        mma16816(o[2 * x], pa, a0, b0);
        mma16816(o[2 * x + 1], pa, a1, b1);
      } else if constexpr (FMT == RING_ATTN_CACHE_MXFP8) {
        mma16816(o[4 * x], pa, mul_bf16x2(e4m3_raw<false>(a0), f01), mul_bf16x2(e4m3_raw<false>(b0), f23));
        mma16816(o[4 * x + 1], pa, mul_bf16x2(e4m3_raw<true>(a0), f01), mul_bf16x2(e4m3_raw<true>(b0), f23));
        mma16816(o[4 * x + 2], pa, mul_bf16x2(e4m3_raw<false>(a1), f01), mul_bf16x2(e4m3_raw<false>(b1), f23));
        mma16816(o[4 * x + 3], pa, mul_bf16x2(e4m3_raw<true>(a1), f01), mul_bf16x2(e4m3_raw<true>(b1), f23));
      } else {
        mma16816(o[8 * x], pa, mul_bf16x2(e2m1_raw<0>(a0), f01), mul_bf16x2(e2m1_raw<0>(b0), f23));
        mma16816(o[8 * x + 1], pa, mul_bf16x2(e2m1_raw<1>(a0), f01), mul_bf16x2(e2m1_raw<1>(b0), f23));
        mma16816(o[8 * x + 2], pa, mul_bf16x2(e2m1_raw<2>(a0), f01), mul_bf16x2(e2m1_raw<2>(b0), f23));
        mma16816(o[8 * x + 3], pa, mul_bf16x2(e2m1_raw<3>(a0), f01), mul_bf16x2(e2m1_raw<3>(b0), f23));
        mma16816(o[8 * x + 4], pa, mul_bf16x2(e2m1_raw<0>(a1), f01), mul_bf16x2(e2m1_raw<0>(b1), f23));
        mma16816(o[8 * x + 5], pa, mul_bf16x2(e2m1_raw<1>(a1), f01), mul_bf16x2(e2m1_raw<1>(b1), f23));
        mma16816(o[8 * x + 6], pa, mul_bf16x2(e2m1_raw<2>(a1), f01), mul_bf16x2(e2m1_raw<2>(b1), f23));
        mma16816(o[8 * x + 7], pa, mul_bf16x2(e2m1_raw<3>(a1), f01), mul_bf16x2(e2m1_raw<3>(b1), f23));
      }
    }
  }
};

template <int FMT, int D>
__global__ void __launch_bounds__(kThreads, Fmt<FMT, D>::kPerSm) tree_rows_kernel(const Params p) {
  using F = Fmt<FMT, D>;
  using W = Warp<FMT, D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_anc[kMaxNodes], s_vis[kMaxNodes];
  __shared__ int s_depth[kMaxNodes], s_jump[kMaxNodes];
  __shared__ int64_t s_plan[4];
  __shared__ float s_ml[kWarps][kRows][2];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  const float lift = F::kMx ? kLift : 0.f;

  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = RING_ATTN_OK;  // the merge kernel reports
  if (warp == 0) {
    int64_t total, before = 0, none;
    warp_totals(p, 0, total, none);
    const int64_t act = active_ctas(p, total);
    const int64_t cta = blockIdx.x;
    const int64_t x0 = cta < act ? share_begin(total, act, cta) : 0;
    const int64_t x1 = cta < act ? share_begin(total, act, cta + 1) : 0;
    const int b = x0 < x1 ? warp_find_sequence(p, x0, before) : p.c.B;
    if (lane == 0) {
      s_plan[0] = x0;
      s_plan[1] = x1;
      s_plan[2] = b;
      s_plan[3] = before;
    }
  }
  __syncthreads();
  int64_t x = s_plan[0];
  const int64_t x_end = s_plan[1];
  int b = (int)s_plan[2];
  int64_t before = s_plan[3];

  uint8_t* ring = smem + warp * F::kStages * F::kStageBytes;
  bool fresh = true;  // masks of sequence b are still to be made
  while (x < x_end) {
    const Keys ks = sequence_keys(p, b);
    const int64_t per = (ks.steps + p.quad - 1) / p.quad;
    const int64_t here = per * p.c.Hkv * p.groups;
    if (x >= before + here) {
      before += here;
      ++b;
      fresh = true;
      continue;
    }
    if (fresh) {
      tree_masks(p, b, ks, s_anc, s_vis, s_depth, s_jump);
      fresh = false;
    }
    const int64_t local = x - before;
    const int64_t u_local = local / per;
    const int grp = (int)(u_local % p.groups), kvh = (int)(u_local / p.groups);
    const int q0 = (int)(local % per);
    const int q1 = (int)(per - q0 < x_end - x ? per : q0 + (x_end - x));
    const int64_t unit = (int64_t)b * p.c.Hkv * p.groups + u_local;
    const int64_t head_row = ((int64_t)b * p.c.Hkv + kvh) * p.c.capacity;
    const int live_rows = ks.cnt * p.rep;

    // queries of rows g and g + 8 in the score product's order of head dimensions
    uint32_t q[F::kKSteps][4];
    int row_t[2];
    bool row_live[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = grp * kRows + g + 8 * r;
      row_live[r] = row < live_rows;
      row_t[r] = row_live[r] ? row / p.rep : 0;
      const uint16_t* src = p.q + b * p.qs_b + (int64_t)(kvh * p.rep + (row_live[r] ? row % p.rep : 0)) * p.qs_h +
                            row_t[r] * p.qs_t;
#pragma unroll
      for (int s = 0; s < F::kKSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = row_live[r] ? src[score_dim<FMT, D>(s, c, h, 0)] : 0;
          const uint32_t hi = row_live[r] ? src[score_dim<FMT, D>(s, c, h, 1)] : 0;
          const uint32_t v = lo | (hi << 16);
          q[s][2 * h + r] = F::kMx ? mul_bf16x2(v, 0x5e805e80u) : v;  // 2^62
        }
    }
    // first key of each row's window and the drafted nodes it sees
    int lo_key[2];
    uint64_t vis[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      lo_key[r] = p.window > 0 ? ks.n + s_depth[row_t[r]] - p.window + 1 : 0;
      vis[r] = s_vis[row_t[r]];
    }

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const int quads = q1 - q0;
    auto step_of = [&](int j) { return p.quad * (q0 + j) + warp; };
#pragma unroll 1
    for (int j = 0; j < F::kStages - 1; ++j)
      W::load(p, ks, head_row, step_of(j), j < quads && step_of(j) < ks.steps, ring + j * F::kStageBytes);
#pragma unroll 1
    for (int j = 0; j < quads; ++j) {
      {
        const int a = j + F::kStages - 1;
        W::load(p, ks, head_row, step_of(a), a < quads && step_of(a) < ks.steps,
                ring + (a % F::kStages) * F::kStageBytes);
      }
      cp_wait<F::kStages - 1>();
      __syncwarp();
      const int i = step_of(j);
      if (i < ks.steps) {
        const uint8_t* st = ring + (j % F::kStages) * F::kStageBytes;
        const int kb = step_key(p, ks, i);
        // every row sees all 16 keys
        const bool whole = kb + kStep <= ks.n &&
                           (p.window <= 0 || kb + kStep <= p.sinks || (int64_t)kb >= (int64_t)ks.n + p.T - p.window);
        bool k_ok[2] = {true, true}, v_ok[4] = {true, true, true, true};
        if (F::kMx && !whole) {
#pragma unroll
          for (int t = 0; t < 2; ++t) k_ok[t] = key_live(p, ks, kb + 8 * t + g);
#pragma unroll
          for (int t = 0; t < 4; ++t) v_ok[t] = key_live(p, ks, kb + 2 * c + (t & 1) + 8 * (t >> 1));
        }
        float s[2][4];
        W::scores(st, q, s, k_ok);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][e] *= p.scale_log2;
        if (!whole) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = e / 2;
              const int u = kb + 8 * t + 2 * c + (e & 1);
              const bool see = u < ks.n ? (u < p.sinks || u >= lo_key[r])
                                        : (u < ks.n + ks.cnt && (vis[r] >> (u - ks.n) & 1));
              if (!see) s[t][e] = -INFINITY;
            }
        }
        // the reference maximum moves only when a score passes it by kRescale (or is the first)
        const float m0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        const float m1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        if (__any_sync(0xffffffffu, m0 > m[0] + kRescale || m1 > m[1] + kRescale)) {
          float top[2] = {m0, m1};
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            if (top[r] > m[r]) {
              const float a = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - top[r]);
              m[r] = top[r];
              l[r] *= a;
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                o[d][2 * r] *= a;
                o[d][2 * r + 1] *= a;
              }
            }
          }
        }
        uint32_t pa[4];
        const float z0 = m[0] == -INFINITY ? 0.f : m[0] - lift, z1 = m[1] == -INFINITY ? 0.f : m[1] - lift;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2_approx(s[t][0] - z0), p1 = ex2_approx(s[t][1] - z0);
          const float p2 = ex2_approx(s[t][2] - z1), p3 = ex2_approx(s[t][3] - z1);
          l[0] += p0 + p1;
          l[1] += p2 + p3;
          pa[2 * t] = pack_bf16x2(p0, p1);
          pa[2 * t + 1] = pack_bf16x2(p2, p3);
        }
        W::values(st, pa, o, v_ok);
      }
      __syncwarp();
    }
    cp_wait<0>();

    // join the four warps' states: weights 2^(m_w - M), then O / l
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        s_ml[warp][g + 8 * r][0] = m[r];
        s_ml[warp][g + 8 * r][1] = l[r];
      }
    }
    __syncthreads();  // every warp has left its ring: the O tiles take its place
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* dst = so + (warp * kRows + g + 8 * r) * (D + 4) + (2 * c + e) * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 8; j += 4)
          *reinterpret_cast<float4*>(dst + j) =
              make_float4(o[j][2 * r + e], o[j + 1][2 * r + e], o[j + 2][2 * r + e], o[j + 3][2 * r + e]);
      }
    __syncthreads();
    const bool alone = q0 == 0 && q1 == per;  // the unit's only part
    const int64_t slot = (int64_t)blockIdx.x + unit;
    {
      const int r = threadIdx.x / 8, d0 = (threadIdx.x % 8) * (D / 8);
      const int row = grp * kRows + r;
      if (row < live_rows) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][r][0]);
        float L = 0.f, acc[D / 8];
#pragma unroll
        for (int e = 0; e < D / 8; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = s_ml[w][r][0];
          if (mw == -INFINITY) continue;
          const float a = ex2_approx(mw - M);
          L += a * s_ml[w][r][1];
          const float* src = so + (w * kRows + r) * (D + 4) + d0;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) acc[e] = fmaf(a, src[e], acc[e]);
        }
        // held values are 2^-lift of the true ones, l is 2^lift of its own
        const bool none = M == -INFINITY;
        const float inv = none ? 0.f : exp2f(lift) / L;
        const float lse2 = none ? -INFINITY : M + log2f(L) - lift;
        if (alone) {
          const int64_t orow = out_row(p, b, kvh, row);
          uint32_t pk[D / 16];
#pragma unroll
          for (int e = 0; e < D / 16; ++e) pk[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + d0);
#pragma unroll
          for (int e = 0; e < D / 64; ++e)
            dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          if (d0 == 0) p.lse[orow] = lse2 * 0.69314718055994530942f;
        } else {
          float* dst = p.o_parts + (slot * kRows + r) * D + d0;
#pragma unroll
          for (int e = 0; e < D / 8; e += 4)
            *reinterpret_cast<float4*>(dst + e) =
                make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
          if (d0 == 0) p.lse_parts[slot * kRows + r] = lse2;
        }
      }
    }
    __syncthreads();  // s_ml and the O tiles are read before the ring is filled again
    x += q1 - q0;
  }
}

// One block per unit and row: the row's partials (in the order of the CTAs that made them)
// are joined with weights 2^(lse_i - max); rows that no key reaches and rows of dead nodes
// get out = 0 and lse = -inf. A unit that one CTA did alone is only completed by its dead
// rows. Block 0 writes the status word.
template <int D>
__global__ void __launch_bounds__(128) tree_merge_kernel(const Params p) {
  constexpr int kTpr = D / 4;              // threads per partial row (float4 each)
  constexpr int kPar = 128 / kTpr;         // partials in flight
  __shared__ int64_t s_plan[2];
  __shared__ float s_max[4];
  __shared__ float s_sum[kPar];
  __shared__ float4 s_acc[kPar][kTpr];
  const int rows = p.T * p.rep;
  const int64_t ub = (int64_t)p.c.Hkv * p.groups;
  const int64_t unit = blockIdx.x / p.rows_per_group;
  const int r = blockIdx.x % p.rows_per_group;
  const int b = (int)(unit / ub);
  const int64_t u_local = unit % ub;
  const int kvh = (int)(u_local / p.groups), grp = (int)(u_local % p.groups);
  const int row = grp * p.rows_per_group + r;
  if (threadIdx.x < 32) {
    int64_t total, before;
    warp_totals(p, b, total, before);
    if (threadIdx.x == 0) {
      s_plan[0] = total;
      s_plan[1] = before;
    }
  }
  if (blockIdx.x == 0) {
    int bad = 0;
    for (int x = threadIdx.x; x < p.c.B; x += 128) {
      int n, cnt;
      if (bad_sequence(p, x, n, cnt)) {
        bad = 1;
        continue;
      }
      for (int t = 0; p.parents && t < cnt; ++t) {
        const int par = p.parents[(int64_t)x * p.T + t];
        if (par < -1 || par >= t) bad = 1;
      }
    }
    if (bad) atomicExch(p.status, RING_ATTN_EINVAL);
  }
  __syncthreads();
  if (row >= rows) return;
  const Keys ks = sequence_keys(p, b);
  const int64_t orow = out_row(p, b, kvh, row);
  const int64_t per = (ks.steps + p.quad - 1) / p.quad;
  const int64_t total = s_plan[0];
  const int d4 = threadIdx.x % kTpr, part = threadIdx.x / kTpr;
  if (row >= ks.cnt * p.rep || per == 0) {
    if (threadIdx.x < D / 8) reinterpret_cast<uint4*>(p.out + orow * D)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) p.lse[orow] = -INFINITY;
    return;
  }
  const int64_t act = active_ctas(p, total);
  const int64_t first = s_plan[1] + u_local * per;
  const int64_t c0 = share_of(total, act, first), c1 = share_of(total, act, first + per - 1);
  if (c0 == c1) return;
  const float* lse = p.lse_parts + (c0 + unit) * p.rows_per_group + r;
  const int parts = (int)(c1 - c0 + 1);
  float M = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += 128) M = fmaxf(M, lse[(int64_t)i * p.rows_per_group]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (M != -INFINITY) {
    for (int i = part; i < parts; i += kPar) {
      const float w = exp2f(lse[(int64_t)i * p.rows_per_group] - M);
      const float4 v = *reinterpret_cast<const float4*>(
          p.o_parts + ((c0 + unit + i) * p.rows_per_group + r) * D + 4 * d4);
      if (w == 0.f) continue;  // nothing of this part's (possibly empty) row
      sum += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
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
  const float inv = M == -INFINITY ? 0.f : 1.f / tot;
  reinterpret_cast<uint2*>(p.out + orow * D)[d4] =
      make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (d4 == 0) p.lse[orow] = M == -INFINITY ? -INFINITY : (M + log2f(tot)) * 0.69314718055994530942f;
}

template <int FMT, int D>
int launch_rows(const Params& p, cudaStream_t stream) {
  constexpr int smem = Fmt<FMT, D>::kSmem;
  if (cudaFuncSetAttribute(tree_rows_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return RING_ATTN_ECUDA;
  tree_rows_kernel<FMT, D><<<p.ctas, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

inline int ctas_per_sm(int format, int D) {
  switch (format) {
    case RING_ATTN_CACHE_BF16:
      return D == 64 ? Fmt<RING_ATTN_CACHE_BF16, 64>::kPerSm : Fmt<RING_ATTN_CACHE_BF16, 128>::kPerSm;
    case RING_ATTN_CACHE_MXFP8:
      return D == 64 ? Fmt<RING_ATTN_CACHE_MXFP8, 64>::kPerSm : Fmt<RING_ATTN_CACHE_MXFP8, 128>::kPerSm;
    default: return D == 64 ? Fmt<RING_ATTN_CACHE_MXFP4, 64>::kPerSm : Fmt<RING_ATTN_CACHE_MXFP4, 128>::kPerSm;
  }
}

template <int FMT>
int launch_rows_d(const Params& p, cudaStream_t stream) {
  return p.c.D == 64 ? launch_rows<FMT, 64>(p, stream) : launch_rows<FMT, 128>(p, stream);
}

}  // namespace tree

namespace {

// Shape of a launch: row groups, the division's grain and the partial slots.
struct TreePlan {
  int rows_per_group, groups, step, quad, ctas, min_quads;
  int64_t units, slots;
};

TreePlan tree_plan(const CacheView& c, int Hq, int T) {
  TreePlan t;
  t.rows_per_group = tree::kRows;
  t.groups = (T * (Hq / c.Hkv) + t.rows_per_group - 1) / t.rows_per_group;
  t.step = tree::kStep;
  t.quad = tree::kWarps;
  t.ctas = 148 * tree::ctas_per_sm(c.format, c.D);
  t.min_quads = 2;
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
  p.quad = t.quad;
  p.ctas = t.ctas;
  p.min_quads = t.min_quads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o_parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeaderBytes);
  p.lse_parts = p.o_parts + (size_t)t.slots * t.rows_per_group * c.D;
  p.status = static_cast<int*>(workspace);
  p.watchdog_ns = watchdog_ns;
  if (t.units * t.rows_per_group > 0x7fffffff) return RING_ATTN_EINVAL;
  int rc;
  switch (c.format) {
    case RING_ATTN_CACHE_BF16: rc = tree::launch_rows_d<RING_ATTN_CACHE_BF16>(p, stream); break;
    case RING_ATTN_CACHE_MXFP8: rc = tree::launch_rows_d<RING_ATTN_CACHE_MXFP8>(p, stream); break;
    default: rc = tree::launch_rows_d<RING_ATTN_CACHE_MXFP4>(p, stream); break;
  }
  if (rc) return rc;
  const unsigned blocks = (unsigned)(t.units * t.rows_per_group);
  if (c.D == 64)
    tree::tree_merge_kernel<64><<<blocks, 128, 0, stream>>>(p);
  else
    tree::tree_merge_kernel<128><<<blocks, 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

}  // namespace ringattn
