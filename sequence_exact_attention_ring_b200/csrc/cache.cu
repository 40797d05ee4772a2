// Writing rows of K and V into a cache in its format, and reading them back.
//
// Both are bound by HBM: a write reads the new rows once and writes codes and scales
// once, a read the other way round. A thread owns 8 consecutive elements of a row on the
// write side (one 16-byte load of bf16, 8 or 4 bytes of codes out), so the 32 values of
// a scale block sit in 4 neighbouring lanes and their maximum takes two shuffles; on the
// read side it owns the elements of one 16-byte store. A block takes a run of rows of one
// (K or V, sequence, head), so that the divisions that find it are made once per block and
// not per row (made per row they were most of a read's instructions: 2 x 65536 tokens of 8
// heads took 209 us). K and V rows go through one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mx_format.cuh"
#include "ringattn_internal.h"

namespace ringattn {
namespace cache {

constexpr int kThreads = 256;

struct WriteParams {
  const void* src[2];      // k_new, v_new
  int64_t stride[2][3];    // (b, h, t) in elements
  uint8_t* codes[2];
  uint8_t* scale[2];
  const int32_t* start;    // [B]
  const int32_t* count;    // [B] or null
  const int32_t* index;    // [B, T] or null
  int B, Hkv, T, T_src;
  int64_t capacity;
  int* status;             // or null
};

struct ReadParams {
  const uint8_t* codes[2];
  const uint8_t* scale[2];
  void* out[2];            // [B, Hkv, T, D]
  const int32_t* start;
  const int32_t* count;
  int B, Hkv, T;
  int64_t capacity;
};

// Eight consecutive elements of a row as they were loaded; `amax` gives the largest
// magnitude as fp32 bits (an unsigned maximum, so a NaN is kept), `scaled` the values times
// a power of two. bf16 is worked on in pairs: its exponents are fp32's, so the product by a
// power of two is exact but for values that end below every code's half step.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ uint32_t amax() const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void scaled(float f, float (&y)[8]) const {
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * f;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ void scaled(float f, float (&y)[8]) const {
    const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), f2);
      const uint32_t v = *reinterpret_cast<const uint32_t*>(&h);
      y[2 * i] = __uint_as_float(v << 16);
      y[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The run of rows that a block takes: K or V (which), head bh = b * Hkv + h, rows from `first`.
struct Run {
  int which;
  uint32_t b, h, first;
};
__device__ __forceinline__ Run block_run(int B, int Hkv, uint32_t rows) {
  // heads run fastest: the rows of a token of a fused projection lie side by side
  Run r;
  const uint32_t heads = 2u * B * Hkv, c = blockIdx.x / heads;
  const uint32_t x = blockIdx.x - c * heads;
  r.first = c * rows;
  r.which = x >= (uint32_t)(B * Hkv);
  const uint32_t bh = r.which ? x - (uint32_t)(B * Hkv) : x;
  r.b = bh / (uint32_t)Hkv;
  r.h = bh - r.b * (uint32_t)Hkv;
  return r;
}

// kRows rows per thread, their loads issued before any of them is encoded.
template <int FMT, int D, typename T, int kRows>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kTpr = D / 8;                   // threads per row
  const uint32_t rpb = blockDim.x / kTpr;       // rows per block and step
  const Run run = block_run(p.B, p.Hkv, rpb * kRows);
  const int sub = threadIdx.x % kTpr;
  const int32_t n = p.count ? p.count[run.b] : p.T;
  const int64_t start = p.start[run.b];
  const bool w = run.which != 0;
  const T* src = static_cast<const T*>(w ? p.src[1] : p.src[0]) + run.b * (w ? p.stride[1][0] : p.stride[0][0]) +
                 run.h * (w ? p.stride[1][1] : p.stride[0][1]) + sub * 8;
  const int64_t stride = w ? p.stride[1][2] : p.stride[0][2];
  // the new rows whose place is inside the cache: [lo, hi)
  const int64_t rows = n < p.T ? n : p.T;
  const int64_t lo = start < 0 ? -start : 0, hi = rows < p.capacity - start ? rows : p.capacity - start;
  if (p.status && threadIdx.x == 0 && (n > p.T || (rows > 0 && (lo > 0 || hi < rows)))) atomicExch(p.status, RING_ATTN_EINVAL);
  const uint32_t i0 = run.first + threadIdx.x / kTpr;
  const int64_t row0 = ((int64_t)run.b * p.Hkv + run.h) * p.capacity + start + i0;
  uint8_t* codes = (w ? p.codes[1] : p.codes[0]) + row0 * cache_row_bytes<FMT>(D) + sub * (cache_row_bytes<FMT>(D) / kTpr);
  uint8_t* scale = (w ? p.scale[1] : p.scale[0]) + row0 * (D / kMxBlock) + sub / 4;
  Eight<T> x[kRows];
  bool live[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const uint32_t i = i0 + u * rpb;
    x[u].clear();
    live[u] = i >= lo && i < hi;
    if (!live[u]) continue;
    int64_t from = i;
    if (p.index) {
      from = p.index[(int64_t)run.b * p.T + i];
      if (from < 0 || from >= p.T_src) {
        if (p.status && sub == 0) atomicExch(p.status, RING_ATTN_EINVAL);
        live[u] = false;
        continue;
      }
    }
    x[u].load(src + from * stride);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    float y[8];
    if (FMT == RING_ATTN_CACHE_BF16) {
      if (!live[u]) continue;
      uint4 o;
      if constexpr (sizeof(T) == 2) {
        o = x[u].w;
      } else {
        x[u].scaled(1.f, y);
        o = make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7]));
      }
      *reinterpret_cast<uint4*>(codes + u * rpb * (2 * D)) = o;
      continue;
    }
    uint32_t m = x[u].amax();
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (!live[u]) continue;
    const uint32_t byte = mx_scale_byte<FMT>(m);
    const bool finite = byte != 255u;  // the codes of a block that is not finite are zeros
    x[u].scaled(mx_inverse_scale(byte), y);
    if (FMT == RING_ATTN_CACHE_MXFP8) {
      const uint2 o = make_uint2(e4m3_quad(y[0], y[1], y[2], y[3]), e4m3_quad(y[4], y[5], y[6], y[7]));
      *reinterpret_cast<uint2*>(codes + u * rpb * D) = finite ? o : make_uint2(0u, 0u);
    } else {
      *reinterpret_cast<uint32_t*>(codes + u * rpb * (D / 2)) = finite ? e2m1_eight(y) : 0u;
    }
    if (sub % 4 == 0) scale[u * rpb * (D / kMxBlock)] = (uint8_t)byte;
  }
}

template <int FMT, int D, typename T, int kRows>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kEl = 16 / (int)sizeof(T);      // elements per thread: one 16-byte store
  constexpr int kTpr = D / kEl;
  constexpr int kBytes = FMT == RING_ATTN_CACHE_BF16 ? 2 * kEl : (FMT == RING_ATTN_CACHE_MXFP8 ? kEl : kEl / 2);
  constexpr int kWords = (kBytes + 3) / 4;
  const uint32_t rpb = blockDim.x / kTpr;
  const Run run = block_run(p.B, p.Hkv, rpb * kRows);
  const int sub = threadIdx.x % kTpr;
  const int32_t n = p.count ? p.count[run.b] : p.T;
  const int64_t start = p.start[run.b];
  const int64_t head = (int64_t)run.b * p.Hkv + run.h;
  const uint8_t* codes = (run.which ? p.codes[1] : p.codes[0]) + head * p.capacity * cache_row_bytes<FMT>(D) + sub * kBytes;
  const uint8_t* scale = (run.which ? p.scale[1] : p.scale[0]) + head * p.capacity * (D / kMxBlock) + sub * kEl / kMxBlock;
  T* out = static_cast<T*>(run.which ? p.out[1] : p.out[0]) + head * p.T * D + sub * kEl;
  uint32_t c[kRows][kWords], s[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const uint32_t i = run.first + u * rpb + threadIdx.x / kTpr;
    const int64_t pos = start + i;
    s[u] = 127u;
#pragma unroll
    for (int e = 0; e < kWords; ++e) c[u][e] = 0u;
    // rows past the count, or outside the cache, read as zeros
    if (i >= (uint32_t)p.T || (int32_t)i >= n || pos < 0 || pos >= p.capacity) continue;
    const uint8_t* q = codes + pos * cache_row_bytes<FMT>(D);
    if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(q);
      c[u][0] = v.x; c[u][1] = v.y; c[u][2] = v.z; c[u][3] = v.w;
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      c[u][0] = v.x; c[u][1] = v.y;
    } else if constexpr (kBytes == 4) {
      c[u][0] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      c[u][0] = *reinterpret_cast<const uint16_t*>(q);
    }
    if (FMT != RING_ATTN_CACHE_BF16) s[u] = scale[pos * (D / kMxBlock)];
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const uint32_t i = run.first + u * rpb + threadIdx.x / kTpr;
    if (i >= (uint32_t)p.T) continue;
    float x[kEl];
    const float f = FMT == RING_ATTN_CACHE_BF16 ? 1.f : mx_scale(s[u]);
#pragma unroll
    for (int e = 0; e < kEl; e += 2) {
      float2 v;
      if (FMT == RING_ATTN_CACHE_BF16) {
        v = make_float2(__uint_as_float(c[u][e / 2] << 16), __uint_as_float(c[u][e / 2] & 0xffff0000u));
      } else if (FMT == RING_ATTN_CACHE_MXFP8) {
        v = e4m3_values(c[u][e / 4] >> (8 * (e % 4)));
      } else {
        v = e2m1_values(c[u][e / 8] >> (4 * (e % 8)));
      }
      x[e] = FMT == RING_ATTN_CACHE_BF16 ? v.x : v.x * f;
      x[e + 1] = FMT == RING_ATTN_CACHE_BF16 ? v.y : v.y * f;
    }
    uint4 o;
    if constexpr (sizeof(T) == 2) {
      o = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    } else {
      o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    *reinterpret_cast<uint4*>(out + (int64_t)i * D) = o;
  }
}

// A launch: `heads` = 2 B Hkv runs of T rows, `tpr` threads per row. Four rows per thread
// where that still leaves every SM its 8 resident blocks, else one; blocks no larger than
// their rows need (a single token's append is one small block per head either way).
struct Launch {
  int rows_per_thread;
  unsigned threads, blocks;
};
inline Launch plan_launch(uint32_t heads, int T, int tpr) {
  Launch l;
  const uint64_t rows = (uint64_t)heads * T;
  const int64_t need = ((int64_t)T * tpr + 31) / 32 * 32;  // threads that one head's rows take
  l.rows_per_thread = rows * tpr >= 4ull * 8 * 148 * kThreads && need >= 4 * kThreads ? 4 : 1;
  l.threads = need < kThreads ? (unsigned)need : kThreads;
  const uint32_t per = l.threads / tpr * l.rows_per_thread;
  l.blocks = heads * (((uint32_t)T + per - 1) / per);  // at most the number of rows, below 2^31
  return l;
}

template <int FMT, int D, typename T>
int write_t(WriteParams p, cudaStream_t stream) {
  const Launch l = plan_launch(2u * p.B * p.Hkv, p.T, D / 8);
  if (l.rows_per_thread == 4)
    cache_write_kernel<FMT, D, T, 4><<<l.blocks, l.threads, 0, stream>>>(p);
  else
    cache_write_kernel<FMT, D, T, 1><<<l.blocks, l.threads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

template <int FMT, int D, typename T>
int read_t(ReadParams p, cudaStream_t stream) {
  const Launch l = plan_launch(2u * p.B * p.Hkv, p.T, D * (int)sizeof(T) / 16);
  if (l.rows_per_thread == 4)
    cache_read_kernel<FMT, D, T, 4><<<l.blocks, l.threads, 0, stream>>>(p);
  else
    cache_read_kernel<FMT, D, T, 1><<<l.blocks, l.threads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ECUDA;
}

template <int FMT>
int write_f(const WriteParams& p, int D, int dtype, cudaStream_t s) {
  if (dtype == RING_ATTN_DTYPE_BF16)
    return D == 64 ? write_t<FMT, 64, __nv_bfloat16>(p, s) : write_t<FMT, 128, __nv_bfloat16>(p, s);
  return D == 64 ? write_t<FMT, 64, float>(p, s) : write_t<FMT, 128, float>(p, s);
}

template <int FMT>
int read_f(const ReadParams& p, int D, int dtype, cudaStream_t s) {
  if (dtype == RING_ATTN_DTYPE_BF16)
    return D == 64 ? read_t<FMT, 64, __nv_bfloat16>(p, s) : read_t<FMT, 128, __nv_bfloat16>(p, s);
  return D == 64 ? read_t<FMT, 64, float>(p, s) : read_t<FMT, 128, float>(p, s);
}

}  // namespace cache

int launch_cache_write(const CacheView& c, const void* k_new, const void* v_new, const int64_t* strides, int dtype,
                       int T, int T_src, const int32_t* start, const int32_t* count, const int32_t* index,
                       int* status, cudaStream_t stream) {
  cache::WriteParams p;
  p.src[0] = k_new;
  p.src[1] = v_new;
  for (int i = 0; i < 2; ++i) {
    for (int x = 0; x < 3; ++x) p.stride[i][x] = strides[3 * i + x];
    p.codes[i] = static_cast<uint8_t*>(i == 0 ? c.k : c.v);
    p.scale[i] = static_cast<uint8_t*>(i == 0 ? c.k_scale : c.v_scale);
  }
  p.start = start;
  p.count = count;
  p.index = index;
  p.B = c.B;
  p.Hkv = c.Hkv;
  p.T = T;
  p.T_src = T_src;
  p.capacity = c.capacity;
  p.status = status;
  switch (c.format) {
    case RING_ATTN_CACHE_BF16: return cache::write_f<RING_ATTN_CACHE_BF16>(p, c.D, dtype, stream);
    case RING_ATTN_CACHE_MXFP8: return cache::write_f<RING_ATTN_CACHE_MXFP8>(p, c.D, dtype, stream);
    default: return cache::write_f<RING_ATTN_CACHE_MXFP4>(p, c.D, dtype, stream);
  }
}

int launch_cache_read(const CacheView& c, int T, const int32_t* start, const int32_t* count, void* k_out, void* v_out,
                      int dtype, cudaStream_t stream) {
  cache::ReadParams p;
  for (int i = 0; i < 2; ++i) {
    p.codes[i] = static_cast<const uint8_t*>(i == 0 ? c.k : c.v);
    p.scale[i] = static_cast<const uint8_t*>(i == 0 ? c.k_scale : c.v_scale);
    p.out[i] = i == 0 ? k_out : v_out;
  }
  p.start = start;
  p.count = count;
  p.B = c.B;
  p.Hkv = c.Hkv;
  p.T = T;
  p.capacity = c.capacity;
  switch (c.format) {
    case RING_ATTN_CACHE_BF16: return cache::read_f<RING_ATTN_CACHE_BF16>(p, c.D, dtype, stream);
    case RING_ATTN_CACHE_MXFP8: return cache::read_f<RING_ATTN_CACHE_MXFP8>(p, c.D, dtype, stream);
    default: return cache::read_f<RING_ATTN_CACHE_MXFP4>(p, c.D, dtype, stream);
  }
}

}  // namespace ringattn
