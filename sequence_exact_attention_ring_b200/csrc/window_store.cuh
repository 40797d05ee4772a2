// The end of a window kernel's tile: accumulator rows from tensor memory to global memory.
//
// A warp holds one row per lane. Stored from there, every 16-byte store of the warp falls
// on 32 lines, and a tile of 128 rows takes the memory unit 4000 clocks; so 32 columns at a time
// go through shared memory and leave with 4 (bf16) or 8 (fp32) lanes side by side on a row.
#pragma once

#include <stdint.h>

#include "sm100_ptx.cuh"

namespace ringattn {

constexpr int kStageBytesF32 = 32 * 144;  // per warp: 32 rows of 128 bytes, 16 apart from a bank's multiple
constexpr int kStageBytesBf16 = 32 * 80;

// Columns [col0, col0 + kCols) of rows row0 .. row0 + rows - 1 (lane l: row l, times its
// `scale`) of an array of `stride` elements a row; all lanes call it, rows <= 0 stores none.
template <int kCols, bool kF32>
__device__ __forceinline__ void store_rows_staged(uint32_t tAcc, bool have, float scale, uint8_t* stage, void* out,
                                                  int64_t row0, int64_t rows, int stride, int col0) {
  constexpr int kPitch = kF32 ? 144 : 80, kBytes = kF32 ? 4 : 2, kLanes = kF32 ? 8 : 4, kRows = 32 / kLanes;
  const int lane = threadIdx.x % 32, r0 = lane / kLanes, piece = lane % kLanes;
  uint8_t* mine = stage + lane * kPitch;
  const uint8_t* from = stage + r0 * kPitch + piece * 16;
  uint8_t* to = static_cast<uint8_t*>(out) + ((row0 + r0) * stride + col0) * kBytes + piece * 16;
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    uint32_t o[32];
    if (have) {
      tmem_ld32(tAcc + c, o);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0u;
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
#pragma unroll
    for (int e = 0; e < 32; e += kF32 ? 4 : 8) {
      uint4 v;
      if (kF32) {
        v = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {
        auto pair = [&](int x) { return pack_bf16x2(__uint_as_float(o[x]), __uint_as_float(o[x + 1])); };
        v = make_uint4(pair(e), pair(e + 2), pair(e + 4), pair(e + 6));
      }
      *reinterpret_cast<uint4*>(mine + e * kBytes) = v;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLanes; ++i)
      if (i * kRows + r0 < rows)
        *reinterpret_cast<uint4*>(to + (int64_t)i * kRows * stride * kBytes) =
            *reinterpret_cast<const uint4*>(from + i * kRows * kPitch);
    to += 32 * kBytes;
    __syncwarp();
  }
}

}  // namespace ringattn
