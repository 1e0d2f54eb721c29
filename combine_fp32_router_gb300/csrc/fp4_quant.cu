// MXFP4 quantisation and its inverse (format: fp4.cuh).
//
// quantize: s = floor(log2(max |x|)) - 2 + 127 of each block of 32, codes
// rne_e2m1(x 2^(127 - s)); every step but the final rounding is exact, so the result is a
// function of the block alone, whatever the launch.  Rows are read once (2 or 4 bytes a value)
// and 17/32 bytes a value are written: bound by HBM.
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

namespace {

// One value of a row in fp32, and eight of them with the widest loads that VEC allows.
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

// Eight values from column c on of a row of `cols` (zeros past its end).  VEC: the row's first
// value and the row stride are multiples of 16 bytes, and so is c's byte offset (c is a
// multiple of 8).
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const typename In<DT>::T* row, int c, int cols,
                                      float (&v)[8]) {
  using T = typename In<DT>::T;
  if (VEC && c + 8 <= cols) {
    constexpr int NV = sizeof(T) * 8 / 16;
    uint4 u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) u[i] = ld_nc_v4(reinterpret_cast<const char*>(row + c) + 16 * i);
    const T* t = reinterpret_cast<const T*>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = In<DT>::f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? In<DT>::f32(__ldg(row + c + i)) : 0.0f;
  }
}

constexpr int kQuantWarps = 8;
constexpr int kQuantSeg = 1024;  // values of a row per warp: 4 x 32 lanes x 8

// A warp quantises 1024 consecutive values of one row: lane l takes values 8 l .. 8 l + 7 of
// each 256, so four lanes hold a block and sixteen the four blocks of a scale tile's word.
// All four loads of a lane are in flight before the first is used.
template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_rows_kernel(const typename In<DT>::T* __restrict__ x, int64_t rows, int cols,
                         int64_t stride, uint32_t segs, uint8_t* __restrict__ q,
                         uint8_t* __restrict__ scales) {
  griddep_wait();
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = w / segs;
  if (row >= rows) return;
  const int c0 = static_cast<int>(w % segs) * kQuantSeg;
  const int kp = static_cast<int>(mx_cols(cols));
  const typename In<DT>::T* xr = x + row * stride;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) load8<DT, VEC>(xr, c0 + i * 256 + lane * 8, cols, v[i]);
  uint8_t* qo = q + row * static_cast<int64_t>(kp / 2) + (c0 + lane * 8) / 2;
  uint8_t* so = scales + mx_scale_at(row, (c0 + lane * 8) / 32, kp / 128);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + i * 256 + lane * 8;
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const uint32_t s = mx_scale_byte(amax);
    const float inv = mx_inverse_scale(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= inv;
    const uint32_t code = s == 255u ? 0u : e2m1x8(v[i]);
    // the four scale bytes of sixteen lanes in one word
    uint32_t sw = s << (8 * ((lane >> 2) & 3));
    sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 4);
    sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 8);
    if (c < kp) {
      *reinterpret_cast<uint32_t*>(qo + i * 128) = code;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(so + i * 2 * kMxTileBytes) = sw;
    }
  }
  // the rows that the last scale tile has and the matrix has not: scale bytes of zero, from
  // the last row's warps (1024 values are 8 words of each)
  if (row == rows - 1) {
    const int missing = static_cast<int>(127 - row % 128), kt = kp / 128, t0 = c0 / 128;
    for (int i = lane; i < missing * 8; i += 32)
      if (t0 + i % 8 < kt)
        *reinterpret_cast<uint32_t*>(scales + mx_scale_at(row + 1 + i / 8, 4 * (t0 + i % 8), kt)) =
            0u;
  }
}

// The inverse: value = code * 2^(s - 127), rounded once to the output type (exact in bf16 and
// fp32 wherever the type reaches).  Eight values per lane as above.
template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kQuantWarps)
    dequantize_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                           int64_t rows, int64_t rows_all, int cols, uint32_t segs,
                           typename In<DT>::T* __restrict__ out) {
  using T = typename In<DT>::T;
  griddep_wait();
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row_all = w / segs;
  if (row_all >= rows_all) return;
  const int64_t g = row_all / rows, row = row_all % rows;
  const int c0 = static_cast<int>(w % segs) * kQuantSeg;
  const int kp = static_cast<int>(mx_cols(cols));
  const uint8_t* qr = q + row_all * static_cast<int64_t>(kp / 2);
  const uint8_t* sg = scales + g * mx_scale_bytes(rows, cols);
  T* o = out + row_all * static_cast<int64_t>(cols);
  const uint8_t* qi = qr + (c0 + lane * 8) / 2;
  const uint8_t* si = sg + mx_scale_at(row, (c0 + lane * 8) / 32, kp / 128);
  uint32_t code[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    code[i] = 0;
    s[i] = 0;
    if (c0 + i * 256 + lane * 8 < cols) {
      code[i] = __ldg(reinterpret_cast<const uint32_t*>(qi + i * 128));
      s[i] = __ldg(si + i * 2 * kMxTileBytes);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + i * 256 + lane * 8;
    if (c >= cols) continue;
    uint32_t h[4];
    e2m1x8_to_half(code[i], h);
    const float f = mx_scale(s[i]);
    alignas(16) T t[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      t[2 * j] = In<DT>::of(p.x * f);
      t[2 * j + 1] = In<DT>::of(p.y * f);
    }
    if (VEC && c + 8 <= cols) {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(t) / 16); ++j)
        // written once and larger than the codes: not kept in L2 in their place
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<char*>(o + c) + 16 * j),
               reinterpret_cast<const uint4*>(t)[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) o[c + j] = t[j];
    }
  }
}

// Weights [E, K, N] bf16 -> [E, N, Kp / 2], blocks along K: a CTA transposes 256 K x 64 N
// through shared memory.  Thread (n pair, block) quantises one block of two neighbouring
// columns; codes and scale words leave through shared memory in 16-byte and 4-byte pieces of
// whole rows.
constexpr int kWtK = 256, kWtN = 64;
__global__ void __launch_bounds__(256)
    quantize_weights_fp4_kernel(const uint16_t* __restrict__ W, int K, int N, int n_tiles,
                                uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  griddep_wait();
  __shared__ uint32_t tile[kWtK][kWtN / 2 + 1];
  __shared__ uint4 codes[kWtN][9];  // 8 x 16 bytes per row, padded against bank conflicts
  __shared__ uint32_t sw[2][kWtN];
  const int tid = threadIdx.x;
  const int64_t e = blockIdx.y;
  const int n0 = static_cast<int>(blockIdx.x % n_tiles) * kWtN;
  const int k0 = static_cast<int>(blockIdx.x / n_tiles) * kWtK;
  const int kp = static_cast<int>(mx_cols(K));
  const uint16_t* We = W + e * K * static_cast<int64_t>(N);
  if (N % 8 == 0) {
    uint4 u[8];
    const int c = tid & 7, r = tid >> 3;  // 8 lanes read 128 bytes of a K row
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + r + 32 * i, n = n0 + 8 * c;
      u[i] = make_uint4(0, 0, 0, 0);
      if (k < K && n < N) u[i] = ld_nc_v4(We + k * static_cast<int64_t>(N) + n);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t* t = &tile[r + 32 * i][4 * c];
      t[0] = u[i].x;
      t[1] = u[i].y;
      t[2] = u[i].z;
      t[3] = u[i].w;
    }
  } else {
    for (int i = tid; i < kWtK * kWtN / 2; i += 256) {
      const int k = k0 + i / (kWtN / 2), n = n0 + 2 * (i % (kWtN / 2));
      const uint16_t* p = We + k * static_cast<int64_t>(N) + n;
      const uint32_t lo = k < K && n < N ? __ldg(p) : 0, hi = k < K && n + 1 < N ? __ldg(p + 1) : 0;
      tile[i / (kWtN / 2)][i % (kWtN / 2)] = lo | (hi << 16);
    }
  }
  __syncthreads();
  const int np = tid & 31, b = tid >> 5;
  uint32_t a0 = 0, a1 = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t t = tile[32 * b + i][np];
    a0 = max(a0, (t << 16) & 0x7FFFFFFFu);
    a1 = max(a1, t & 0x7FFF0000u);
  }
  const uint32_t s0 = mx_scale_byte(a0), s1 = mx_scale_byte(a1);
  const float i0 = mx_inverse_scale(s0), i1 = mx_inverse_scale(s1);
  uint32_t w0[4], w1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v0[8], v1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t t = tile[32 * b + 8 * i + j][np];
      v0[j] = s0 == 255u ? 0.0f : bf16lo(t) * i0;
      v1[j] = s1 == 255u ? 0.0f : bf16hi(t) * i1;
    }
    w0[i] = e2m1x8(v0);
    w1[i] = e2m1x8(v1);
  }
  codes[2 * np][b] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
  codes[2 * np + 1][b] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  reinterpret_cast<uint8_t*>(&sw[b >> 2][2 * np])[b & 3] = static_cast<uint8_t>(s0);
  reinterpret_cast<uint8_t*>(&sw[b >> 2][2 * np + 1])[b & 3] = static_cast<uint8_t>(s1);
  __syncthreads();
  uint8_t* qe = q + e * N * static_cast<int64_t>(kp / 2);
  for (int i = tid; i < kWtN * 8; i += 256) {
    const int n = n0 + i / 8, k = k0 + 32 * (i % 8);
    if (n < N && k < kp)
      st_v4(qe + n * static_cast<int64_t>(kp / 2) + k / 2, codes[i / 8][i % 8]);
  }
  if (tid < 128) {
    const int n = n0 + (tid & 63), k = k0 + 128 * (tid >> 6);
    if (k < kp)  // n < N rounded up to 128, by the grid
      *reinterpret_cast<uint32_t*>(scales + e * mx_scale_bytes(N, K) +
                                   mx_scale_at(n, k / 32, kp / 128)) = sw[tid >> 6][tid & 63];
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Warps of a launch over `rows` rows of `cols` values; 0 when they pass what a grid's 32-bit
// warp index holds.
uint32_t quant_segs(int64_t rows, int cols, uint32_t* blocks) {
  const int64_t segs = (mx_cols(cols) + kQuantSeg - 1) / kQuantSeg;
  const int64_t warps = rows * segs;
  if (rows > INT32_MAX || warps > INT32_MAX) return 0;
  *blocks = static_cast<uint32_t>((warps + kQuantWarps - 1) / kQuantWarps);
  return static_cast<uint32_t>(segs);
}

template <int DT>
cudaError_t launch_quantize(const void* x, int64_t rows, int cols, int64_t stride, uint32_t segs,
                            uint32_t blocks, uint8_t* q, uint8_t* scales, cudaStream_t s) {
  using T = typename In<DT>::T;
  const bool vec = aligned16(x) && stride * sizeof(T) % 16 == 0;
  return launch_pdl(vec ? quantize_rows_kernel<DT, true> : quantize_rows_kernel<DT, false>,
                    dim3(blocks), dim3(32 * kQuantWarps), 0, s, static_cast<const T*>(x), rows,
                    cols, stride, segs, q, scales);
}
template <int DT>
cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows,
                              int64_t rows_all, int cols, uint32_t segs, uint32_t blocks,
                              void* out, cudaStream_t s) {
  using T = typename In<DT>::T;
  const bool vec = cols * sizeof(T) % 16 == 0;  // `out` itself is 16-byte aligned
  return launch_pdl(vec ? dequantize_rows_kernel<DT, true> : dequantize_rows_kernel<DT, false>,
                    dim3(blocks), dim3(32 * kQuantWarps), 0, s, q, scales, rows, rows_all, cols,
                    segs, static_cast<T*>(out));
}

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool known_dtype(int dt) {
  return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16 || dt == MOE_DTYPE_F32;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_fp4_row_bytes(int cols) { return cols < 0 ? 0 : mx_cols(cols) / 2; }

size_t moe_fp4_scale_bytes(int64_t rows, int cols) {
  return rows < 0 || cols < 0 ? 0 : static_cast<size_t>(mx_scale_bytes(rows, cols));
}

moe_status_t moe_quantize_rows_fp4(const void* x, int dtype, int64_t rows, int cols,
                                   int64_t row_stride, uint8_t* q, uint8_t* scales,
                                   cudaStream_t stream) {
  if (!known_dtype(dtype) || rows < 0 || cols < 1 || row_stride < 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales || !aligned16(q) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  if (rows > 1 && row_stride < cols) return MOE_ERR_INVALID_ARG;
  const uintptr_t unit = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % unit != 0) return MOE_ERR_INVALID_ARG;
  uint32_t blocks = 0;
  if (cols > kMaxFp4Cols) return MOE_ERR_UNSUPPORTED;
  const uint32_t segs = quant_segs(rows, cols, &blocks);
  if (segs == 0) return MOE_ERR_UNSUPPORTED;
  const cudaError_t e =
      dtype == MOE_DTYPE_BF16
          ? launch_quantize<MOE_DTYPE_BF16>(x, rows, cols, row_stride, segs, blocks, q, scales, stream)
      : dtype == MOE_DTYPE_F16
          ? launch_quantize<MOE_DTYPE_F16>(x, rows, cols, row_stride, segs, blocks, q, scales, stream)
          : launch_quantize<MOE_DTYPE_F32>(x, rows, cols, row_stride, segs, blocks, q, scales, stream);
  return cuda_status(e);
}

moe_status_t moe_dequantize_rows_fp4(const uint8_t* q, const uint8_t* scales, int groups,
                                     int64_t rows, int cols, int dtype, void* out,
                                     cudaStream_t stream) {
  if (!known_dtype(dtype) || groups < 0 || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (groups == 0 || rows == 0) return MOE_OK;
  if (!q || !scales || !out || !aligned16(q) || !aligned16(scales) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxFp4Cols || rows > INT32_MAX / groups) return MOE_ERR_UNSUPPORTED;
  uint32_t blocks = 0;
  const uint32_t segs = quant_segs(rows * groups, cols, &blocks);
  if (segs == 0) return MOE_ERR_UNSUPPORTED;
  const int64_t all = rows * groups;
  return cuda_status(
      dtype == MOE_DTYPE_BF16
          ? launch_dequantize<MOE_DTYPE_BF16>(q, scales, rows, all, cols, segs, blocks, out, stream)
      : dtype == MOE_DTYPE_F16
          ? launch_dequantize<MOE_DTYPE_F16>(q, scales, rows, all, cols, segs, blocks, out, stream)
          : launch_dequantize<MOE_DTYPE_F32>(q, scales, rows, all, cols, segs, blocks, out, stream));
}

moe_status_t moe_quantize_weights_fp4(const moe_bf16_t* W, int E, int K, int N, uint8_t* Wq,
                                      uint8_t* scales, cudaStream_t stream) {
  if (E < 1 || K < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (!W || !Wq || !scales || !aligned16(W) || !aligned16(Wq) || !aligned16(scales))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || K > kMaxFp4Cols || N > kMaxFp4Cols) return MOE_ERR_UNSUPPORTED;
  // N is covered to the end of its last scale tile (two CTA tiles), whose missing rows get
  // scale bytes of zero
  const int n_tiles = (N + 127) / 128 * 2, k_tiles = (K + kWtK - 1) / kWtK;
  return cuda_status(launch_pdl(quantize_weights_fp4_kernel, dim3(n_tiles * k_tiles, E), dim3(256),
                                0, stream, W, K, N, n_tiles, Wq, scales));
}

}  // extern "C"
