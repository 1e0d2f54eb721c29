// The 8-bit format with a scale per 128 values: E4M3 codes (largest value 448) and one fp32 scale
// per row and 128 columns of a matrix of rows, or per 128 x 128 block of a weight matrix.
//   scale = max(amax * (1 / 448), 2^-126) (the reciprocal and the product in fp32), 1 for zeros, NaN for
//           one that holds an infinity or a NaN (its codes are zeros, so every value of it reads back as
//           NaN)
//   code  = the E4M3 number nearest to x * (1 / scale), ties to the even mantissa
// 1 / scale is rounded to fp32 once per block, and the product once per value: a code is the nearest
// one of a number that is off by at most 2 units of 2^-24, against the format's half step of 2^-4.
// A row of C values takes fp8_cols(C) bytes (zero codes past C).
//
// Rows are handled in segments of 256 values, one per warp and step.  Where rows start on 16 bytes
// lane l holds the values 8 l .. 8 l + 7, so a half warp holds a block; elsewhere lane l holds the
// values 32 j + l, j = 0 .. 7, so that neighbouring lanes access neighbouring values whatever the
// alignment.
#pragma once

#include "elem.cuh"

namespace moe {

constexpr int kSeg = 256;

__host__ __device__ inline int64_t fp8_cols(int64_t cols) { return (cols + 127) / 128 * 128; }

__device__ __forceinline__ float f8_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return amax == 0u ? 1.0f : fmaxf(__uint_as_float(amax) * (1.0f / 448.0f), 1.17549435e-38f);
}
// 1 / scale, 0 for a NaN scale
__device__ __forceinline__ float f8_inverse(float scale) { return scale == scale ? 1.0f / scale : 0.0f; }

// The largest magnitude among eight values, as bits; a NaN if one is.
__device__ __forceinline__ uint32_t amax8(const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(y[j]), "f"(y[j + 1]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}
// Codes of eight values times inv, the earlier ones in the low bytes; inv = 0 gives zeros whatever
// the values are.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
  mul2(a, b, inv, inv);
  mul2(c, d, inv, inv);
  const uint32_t w = e4m3x2(a, b) | (e4m3x2(c, d) << 16);
  return inv == 0.0f ? 0u : w;
}
// Values of two codes
__device__ __forceinline__ float2 e4m3x2_f32(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight values of a segment that begins at `seg` (its first of n values; n may exceed 256 or be
// negative), zeros past n.  Not the read-only path: callers may write the same place later.
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> load_seg(const T* seg, int n, int lane) {
  Raw8<T> r;
  if constexpr (VEC) {
    if (8 * lane + 8 <= n) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) {
        uint4& v = reinterpret_cast<uint4*>(&r)[i];
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(reinterpret_cast<const char*>(seg + 8 * lane) + 16 * i));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[j] = 8 * lane + j < n ? seg[8 * lane + j] : T(0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = 32 * j + lane < n ? seg[32 * j + lane] : T(0);
  }
  return r;
}
// (STREAM: written once and not read again soon)
template <bool VEC, bool STREAM = false, typename T>
__device__ __forceinline__ void store_seg(T* seg, int n, int lane, const Raw8<T>& r) {
  if constexpr (VEC) {
    if (8 * lane + 8 <= n) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i)
        if constexpr (STREAM)
          __stcs(reinterpret_cast<uint4*>(seg + 8 * lane) + i, reinterpret_cast<const uint4*>(&r)[i]);
        else
          st_v4(reinterpret_cast<char*>(seg + 8 * lane) + 16 * i, reinterpret_cast<const uint4*>(&r)[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * lane + j < n) seg[8 * lane + j] = r.v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j + lane < n) seg[32 * j + lane] = r.v[j];
  }
}

// The largest magnitudes of V blocks at a time (as bits; m[i]: this lane's part of block i of its half
// warp) and their scales.  A step of 8 lanes, and with four blocks one of 4, leaves each lane with one
// block, so that a scale and its reciprocal are computed once for V blocks: the scale of block
// which(lane), and every block's reciprocal.
template <int V>
struct Scales {
  float scale, inv[V];
  static __device__ __forceinline__ int which(int lane) {
    return V == 1 ? 0 : V == 2 ? (lane >> 3) & 1 : (lane >> 2) & 3;
  }
  // one lane per block
  static __device__ __forceinline__ bool stores(int lane) {
    return (lane & (V == 1 ? 15 : V == 2 ? 7 : 3)) == 0;
  }
  __device__ __forceinline__ Scales(const uint32_t (&m)[V], int lane) {
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    uint32_t a = m[0];
    if constexpr (V == 1) {
      a = max(a, __shfl_xor_sync(kAll, a, 8));
      a = max(a, __shfl_xor_sync(kAll, a, 4));
    } else if constexpr (V == 2) {
      const bool h = lane & 8;
      a = max(h ? m[1] : m[0], __shfl_xor_sync(kAll, h ? m[0] : m[1], 8));
      a = max(a, __shfl_xor_sync(kAll, a, 4));
    } else {
      const bool h = lane & 8, g = lane & 4;
      const uint32_t b = max(h ? m[2] : m[0], __shfl_xor_sync(kAll, h ? m[0] : m[2], 8));
      const uint32_t c = max(h ? m[3] : m[1], __shfl_xor_sync(kAll, h ? m[1] : m[3], 8));
      a = max(g ? c : b, __shfl_xor_sync(kAll, g ? b : c, 4));
    }
    a = max(a, __shfl_xor_sync(kAll, a, 2));
    a = max(a, __shfl_xor_sync(kAll, a, 1));
    scale = f8_scale(a);
    const float own = f8_inverse(scale);
    if constexpr (V == 1) {
      inv[0] = own;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) inv[i] = __shfl_sync(kAll, own, (lane & 16) | (i * (16 / V)));
    }
  }
};
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
  return make_uint2(e4m3x4(y[0], y[1], y[2], y[3], inv), e4m3x4(y[4], y[5], y[6], y[7], inv));
}

// The 8-bit form of a warp's segment (two blocks; the values past the row's end are zeros), neighbouring
// lanes holding neighbouring values: codes to q, np of them (a multiple of 128, up to 256), and scales
// to s.
__device__ __forceinline__ void quantize_seg(const float (&y)[8], uint8_t* q, float* s, int np, int lane) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t amax = 0;  // magnitudes order like their bits
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(y[4 * b + j]) & 0x7FFFFFFFu);
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    const float scale = f8_scale(amax), inv = f8_inverse(scale);
    if (128 * b < np) {
      const uint32_t c = e4m3x4(y[4 * b], y[4 * b + 1], y[4 * b + 2], y[4 * b + 3], inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[32 * (4 * b + j) + lane] = static_cast<uint8_t>(c >> (8 * j));
      if (lane == 0) s[b] = scale;
    }
  }
}

}  // namespace moe
