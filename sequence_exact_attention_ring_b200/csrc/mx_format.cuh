// Microscaled cache formats: blocks of 32 values along the head dimension share one
// power of two 2^k, kept as the byte k + 127 (255: the block holds a value that is not
// finite and reads as NaN). k is the smallest integer with max|x| <= M 2^k, so no value
// saturates; the elements are x 2^-k rounded to nearest even:
//   mxfp8  e4m3, M = 448, one byte per element
//   mxfp4  e2m1, M = 6, element 2i in the low half of byte i
// Scaling by a power of two is exact, so an element's only rounding is to the element
// format, and every stored value is exact in bf16 (3 or 1 mantissa bits) down to bf16's
// own subnormals.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ringattn.h"

namespace ringattn {

constexpr int kMxBlock = 32;

template <int FMT>
__host__ __device__ constexpr int cache_row_bytes(int D) {
  return FMT == RING_ATTN_CACHE_BF16 ? 2 * D : (FMT == RING_ATTN_CACHE_MXFP8 ? D : D / 2);
}

// Scale byte of a block from the largest |x| in it, as fp32 bits (NaN and infinity have
// exponent field 255 and compare above every finite value). With amax = f 2^e,
// 1 <= f < 2: k = e - 8 (+1 if f > 1.75) for e4m3, e - 2 (+1 if f > 1.5) for e2m1.
// Subnormal amax and zero end at the smallest scale, 2^-127.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  if (e == 255) return 255u;
  const uint32_t frac = amax_bits & 0x7fffffu;
  const int up = FMT == RING_ATTN_CACHE_MXFP8 ? (frac > 0x600000u) : (frac > 0x400000u);
  const int b = e - (FMT == RING_ATTN_CACHE_MXFP8 ? 8 : 2) + up;  // (e - 127 - 8 + up) + 127
  return b < 0 ? 0u : (uint32_t)b;
}

// 2^(127 - byte), the factor of the encoder (byte 255 never reaches it with finite data;
// byte 254 needs the subnormal 2^-127).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) {
  return byte >= 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); NaN for a block that is not finite.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : (byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23));
}

// Four values to four e4m3 codes, eight to eight e2m1 codes, the first value lowest; to
// nearest even, larger magnitudes to the largest code.
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ uint32_t e2m1_eight(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
  const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3));
  return __half22float2(h);
}
__device__ __forceinline__ float2 e2m1_values(uint32_t codes) {
  const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(codes & 0xffu), __NV_E2M1));
  return __half22float2(h);
}

}  // namespace ringattn
