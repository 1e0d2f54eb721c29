// Element types of the row kernels (MOE_DTYPE_*), and eight values of a row at a time.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// A value in fp32 and back (rounded to nearest, ties to even).
template <int DT>
struct In;
template <>
struct In<MOE_DTYPE_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float f32(T v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
  static __device__ __forceinline__ T of(float v) { return bf16_bits(v); }
};
template <>
struct In<MOE_DTYPE_F16> {
  using T = uint16_t;
  static __device__ __forceinline__ float f32(T v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ T of(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};
template <>
struct In<MOE_DTYPE_F32> {
  using T = float;
  static __device__ __forceinline__ float f32(T v) { return v; }
  static __device__ __forceinline__ T of(float v) { return v; }
};

// Two values an instruction, each rounded as by itself: the pipe takes as long, but an issue slot less.
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {  // x *= a, y *= b
  asm("{\n\t.reg .b64 v, m;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 m, {%2, %3};\n\t"
      "mul.rn.f32x2 v, v, m;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {  // x += a, y += b
  asm("{\n\t.reg .b64 v, m;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 m, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, m;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// x = a c + x, y = b d + y
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 v, m, n;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 m, {%2, %3};\n\t"
      "mov.b64 n, {%4, %5};\n\tfma.rn.f32x2 v, m, n, v;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}

// Values 8 l .. 8 l + 7 of a tile that has n of its 128 (zeros past them), raw: converting waits
// for the loads, so it is left for later.
template <typename T>
struct alignas(16) Raw8 {
  T v[8];
};
// Values j and j + 1 (j even) in fp32 and back, a 16-bit pair as one word.
template <int DT>
__device__ __forceinline__ float2 get2(const Raw8<typename In<DT>::T>& r, int j) {
  if constexpr (DT == MOE_DTYPE_F32) {
    return make_float2(r.v[j], r.v[j + 1]);
  } else {
    const uint32_t w = reinterpret_cast<const uint32_t*>(r.v)[j / 2];
    if constexpr (DT == MOE_DTYPE_BF16)
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}
template <int DT>
__device__ __forceinline__ void set2(Raw8<typename In<DT>::T>& r, int j, float x, float y) {
  if constexpr (DT == MOE_DTYPE_F32) {
    r.v[j] = x;
    r.v[j + 1] = y;
  } else if constexpr (DT == MOE_DTYPE_BF16) {
    reinterpret_cast<uint32_t*>(r.v)[j / 2] = pack_bf16x2(x, y);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    reinterpret_cast<uint32_t*>(r.v)[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* tile, int n, int l) {
  Raw8<T> r;
  const int c = 8 * l;
  if (c + 8 <= n) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i)
      reinterpret_cast<uint4*>(&r)[i] = ld_nc_v4(reinterpret_cast<const char*>(tile + c) + 16 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = c + i < n ? __ldg(tile + c + i) : T(0);
  }
  return r;
}

}  // namespace moe
