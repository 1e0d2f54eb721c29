// 8-bit rows and weights with a scale per 128 values (format: fp8.cuh): quantisation of rows, of
// silu(a) b of rows [a | b], its inverse, and quantisation of weights in 128 x 128 blocks.
//
// All of it reads each value once and writes each code once: bound by HBM (2 + 1 + 4/128 bytes a
// value for bf16 rows, 4 + 1 + 4/128 for SwiGLU).  16384 x 7168 bf16: 55 us there, 6.4 TB/s, and 53
// back, 6.7 TB/s; SwiGLU of 65536 x 2048: 115 us, 5.9 TB/s, bound by issuing (71 % of all slots at 34 of
// 64 warps); weights 32 x 2048 x 1024: 33 us, 6.1 TB/s.  Where rows do not start on 16 bytes every
// value is an instruction: 16384 x 1925 bf16 29 us, 3.4 TB/s, weights 32 x 2048 x 1001 58 us.
#include "fp8.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr int kTiles = 4;  // tiles of 128 values per half warp, all loaded before the first is used

// silu(a) b.  The fast exponential and reciprocal keep the value to (6 + |a|) 2^-23, against the
// 2^-4 of a code; with expf and an IEEE division the kernel would be bound by issuing them.  Both
// flush subnormals: silu(a) is 0 below a = -87.3, where it is less than 1.1e-36 in magnitude.
template <int DT>
__device__ __forceinline__ void swiglu8(const Raw8<typename In<DT>::T>& ar, const Raw8<typename In<DT>::T>& br,
                                        float (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 a = get2<DT>(ar, j), b = get2<DT>(br, j);
    float e = a.x, f = a.y;
    mul2(e, f, -1.44269504088896340736f, -1.44269504088896340736f);  // -log2 e
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f));
    add2(e, f, 1.0f, 1.0f);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f));
    // a = -infinity gives 0 as its neighbours do, not -infinity * 0 (a NaN stays in e)
    mul2(e, f, fmaxf(a.x, -3.402823466e38f), fmaxf(a.y, -3.402823466e38f));
    mul2(e, f, b.x, b.y);
    y[j] = e;
    y[j + 1] = f;
  }
}

// ---- rows that start on 16 bytes: the matrix as tiles of 128 values, row-major; a warp takes
// 2 kTiles that follow one another, its halves every second one.  No lane idles on narrow rows.
struct Place {
  uint32_t row;
  int t;
  __device__ __forceinline__ Place(uint32_t tile, uint32_t kt) : row(tile / kt), t(static_cast<int>(tile % kt)) {}
  __device__ __forceinline__ void step(int kt) {
    for (t += 2; t >= kt; t -= kt) ++row;
  }
};

template <int DT, bool GLU>
__global__ void __launch_bounds__(32 * kWarps)
    quantize_tiles_kernel(const typename In<DT>::T* __restrict__ x, int64_t rows, int cols,
                          int64_t stride, const int32_t* __restrict__ perm, uint8_t* __restrict__ q,
                          float* __restrict__ scales) {
  using T = typename In<DT>::T;
  griddep_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int kt = static_cast<int>(fp8_cols(cols) / 128);
  const uint32_t tile = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * 2 * kTiles + (lane >> 4);
  Place at(tile, kt);
  Raw8<T> a[kTiles], b[GLU ? kTiles : 1];
  bool live[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    live[i] = at.row < rows && (!perm || perm[at.row] >= 0);
    const T* v = x + at.row * stride + at.t * 128;
    const int n = live[i] ? cols - at.t * 128 : 0;
    a[i] = load8(v, n, l);
    if constexpr (GLU) b[i] = load8(v + cols, n, l);
    at.step(kt);
  }
  float y[kTiles][8];
  uint32_t m[kTiles], alive = 0;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    if constexpr (GLU) {
      swiglu8<DT>(a[i], b[i], y[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 v = get2<DT>(a[i], j);
        y[i][j] = v.x;
        y[i][j + 1] = v.y;
      }
    }
    m[i] = amax8(y[i]);
    alive |= static_cast<uint32_t>(live[i]) << i;
  }
  const Scales<kTiles> s(m, lane);
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    if (live[i])
      *reinterpret_cast<uint2*>(q + (static_cast<int64_t>(tile) + 2 * i) * 128 + 8 * l) = codes8(y[i], s.inv[i]);
  const int own = s.which(lane);
  if (s.stores(lane) && (alive >> own & 1)) scales[static_cast<int64_t>(tile) + 2 * own] = s.scale;
}

// A value = code * scale, rounded once.
template <int DT>
__device__ __forceinline__ Raw8<typename In<DT>::T> dequantize8(uint2 c, float s) {
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
  Raw8<typename In<DT>::T> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = e4m3x2_f32(static_cast<uint16_t>(w[j]));
    set2<DT>(r, 2 * j, v.x * s, v.y * s);
  }
  return r;
}

template <int DT>
__global__ void __launch_bounds__(32 * kWarps)
    dequantize_tiles_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scales,
                            int64_t rows, int cols, typename In<DT>::T* __restrict__ out) {
  using T = typename In<DT>::T;
  griddep_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int kt = static_cast<int>(fp8_cols(cols) / 128);
  const uint32_t tile = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * 2 * kTiles + (lane >> 4);
  Place at(tile, kt);
  uint2 c[kTiles];
  float s[kTiles];
  int n[kTiles];
  T* to[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int64_t o = static_cast<int64_t>(tile) + 2 * i;
    n[i] = at.row < rows ? cols - at.t * 128 - 8 * l : 0;
    to[i] = out + at.row * static_cast<int64_t>(cols) + at.t * 128 + 8 * l;
    c[i] = make_uint2(0, 0);
    s[i] = 0.0f;
    if (n[i] > 0) {
      c[i] = __ldg(reinterpret_cast<const uint2*>(q + o * 128 + 8 * l));
      s[i] = __ldg(scales + o);
    }
    at.step(kt);
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const Raw8<T> r = dequantize8<DT>(c[i], s[i]);
    if (n[i] >= 8) {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(r) / 16); ++j)
        __stcs(reinterpret_cast<uint4*>(to[i]) + j, reinterpret_cast<const uint4*>(&r)[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n[i]) to[i][j] = r.v[j];
    }
  }
}

// ---- other rows: a warp takes a segment of 256 values of one row, neighbouring lanes neighbouring
// values.
template <int DT, bool GLU>
__global__ void __launch_bounds__(32 * kWarps)
    quantize_any_kernel(const typename In<DT>::T* __restrict__ x, int64_t rows, int cols,
                        int64_t stride, uint32_t segs, const int32_t* __restrict__ perm,
                        uint8_t* __restrict__ q, float* __restrict__ scales) {
  using T = typename In<DT>::T;
  griddep_wait();
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = w / segs;
  if (row >= rows || (perm && perm[row] < 0)) return;
  const int c0 = static_cast<int>(w % segs) * kSeg;
  const int64_t kp = fp8_cols(cols);
  const T* v = x + row * stride + c0;
  const Raw8<T> a = load_seg<false>(v, cols - c0, lane);
  float y[8];
  if constexpr (GLU) {
    swiglu8<DT>(a, load_seg<false>(v + cols, cols - c0, lane), y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = In<DT>::f32(a.v[j]);
  }
  quantize_seg(y, q + row * kp + c0, scales + row * (kp / 128) + c0 / 128,
               static_cast<int>(kp - c0 < kSeg ? kp - c0 : kSeg), lane);
}
template <int DT>
__global__ void __launch_bounds__(32 * kWarps)
    dequantize_any_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scales,
                          int64_t rows, int cols, uint32_t segs,
                          typename In<DT>::T* __restrict__ out) {
  using T = typename In<DT>::T;
  griddep_wait();
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = w / segs;
  if (row >= rows) return;
  const int c0 = static_cast<int>(w % segs) * kSeg;
  const int64_t kp = fp8_cols(cols);
  const Raw8<uint8_t> c = load_seg<false>(q + row * kp + c0, cols - c0, lane);
  const float* s = scales + row * (kp / 128) + c0 / 128;
  Raw8<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    r.v[j] = 32 * j + lane < cols - c0 ? In<DT>::of(e4m3x2_f32(c.v[j]).x * __ldg(s + j / 4)) : T(0);
  store_seg<false>(out + row * static_cast<int64_t>(cols) + c0, cols - c0, lane, r);
}

// ---- weights [E, K, N] bf16 in 128 x 128 blocks, one block per CTA: a thread holds two groups of
// four K rows x 8 columns.  Codes go as [E, N, Kp] (through shared memory), or in the weights' own
// order as [E, K, Np].
template <bool TRANSPOSE>
__global__ void __launch_bounds__(256)
    quantize_blocks_kernel(const uint16_t* __restrict__ W, int K, int N, int n_tiles, int vec,
                           uint8_t* __restrict__ q, float* __restrict__ scales) {
  // Word kg (K rows 4 kg .. 4 kg + 3) of column n = 8 c + j at
  //   4 ((kg / 4) xor c % 8) + (kg % 4 xor 2 (c / 8)):
  // neither a warp's words (16 c, two kg that follow each other) nor its 16-byte reads of whole rows
  // meet in a bank.
  __shared__ uint32_t codes[TRANSPOSE ? 128 : 1][32];
  __shared__ uint32_t tops[8];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t e = blockIdx.y;
  const int nb = static_cast<int>(blockIdx.x % n_tiles), kb = static_cast<int>(blockIdx.x / n_tiles);
  const int n0 = nb * 128, k0 = kb * 128;
  const int c = lane & 15;  // columns 8 c .. 8 c + 7
  const uint16_t* We = W + e * K * static_cast<int64_t>(N);
  Raw8<uint16_t> v[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 4 * (2 * (8 * h + warp) + (lane >> 4)) + i;
      const uint16_t* p = We + static_cast<int64_t>(k) * N + n0;
      const int n = k < K ? N - n0 : 0;
      if (vec) {
        v[h][i] = load8(p, n, c);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[h][i].v[j] = 8 * c + j < n ? __ldg(p + 8 * c + j) : uint16_t(0);
      }
    }
  uint32_t top = 0;  // magnitudes order like their bits: two at a time
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(&v[h][i]);
      constexpr uint32_t m = 0x7FFF7FFFu;
      top = __vimax3_u16x2(top, __vimax3_u16x2(u.x & m, u.y & m, u.z & m), u.w & m);
    }
  uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
  if (lane == 0) tops[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, tops[i]);
  const float scale = f8_scale(amax << 16), inv = f8_inverse(scale);
  const int64_t kp = fp8_cols(K), np = fp8_cols(N);
  if (tid == 0)
    scales[TRANSPOSE ? (e * n_tiles + nb) * (kp / 128) + kb : (e * (kp / 128) + kb) * n_tiles + nb] = scale;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int kg = 2 * (8 * h + warp) + (lane >> 4);
    float f[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = In<MOE_DTYPE_BF16>::f32(v[h][i].v[j]);
    if constexpr (TRANSPOSE) {
      const int w = 4 * ((kg >> 2) ^ (c & 7)) + ((kg & 3) ^ (2 * (c >> 3)));
#pragma unroll
      for (int j = 0; j < 8; ++j) codes[8 * c + j][w] = e4m3x4(f[0][j], f[1][j], f[2][j], f[3][j], inv);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 4 * kg + i;
        if (k < K)
          *reinterpret_cast<uint2*>(q + (e * K + k) * np + n0 + 8 * c) =
              make_uint2(e4m3x4(f[i][0], f[i][1], f[i][2], f[i][3], inv),
                         e4m3x4(f[i][4], f[i][5], f[i][6], f[i][7], inv));
      }
    }
  }
  if constexpr (TRANSPOSE) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * i + (tid >> 3), g = tid & 7;  // 16 bytes of a row of 128
      uint4 u = *reinterpret_cast<const uint4*>(&codes[n][4 * (g ^ ((n >> 3) & 7))]);
      if (i >= 2) u = make_uint4(u.z, u.w, u.x, u.y);  // n / 8 / 8 = 1
      if (n0 + n < N) st_v4(q + (e * N + n0 + n) * kp + k0 + 16 * g, u);
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool known_dtype(int dt) {
  return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16 || dt == MOE_DTYPE_F32;
}
int64_t dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

uint32_t tile_blocks(int64_t rows, int cols) {
  return static_cast<uint32_t>((rows * (fp8_cols(cols) / 128) + 2 * kTiles * kWarps - 1) / (2 * kTiles * kWarps));
}
uint32_t segs_of(int cols) { return static_cast<uint32_t>((cols + kSeg - 1) / kSeg); }
uint32_t seg_blocks(int64_t rows, int cols) {
  return static_cast<uint32_t>((rows * segs_of(cols) + kWarps - 1) / kWarps);
}

template <int DT, bool GLU>
cudaError_t launch_quantize(const void* x, int64_t rows, int cols, int64_t stride, bool vec,
                            const int32_t* perm, uint8_t* q, float* scales, cudaStream_t s) {
  const auto* xt = static_cast<const typename In<DT>::T*>(x);
  return vec ? launch_pdl(quantize_tiles_kernel<DT, GLU>, dim3(tile_blocks(rows, cols)),
                          dim3(32 * kWarps), 0, s, xt, rows, cols, stride, perm, q, scales)
             : launch_pdl(quantize_any_kernel<DT, GLU>, dim3(seg_blocks(rows, cols)),
                          dim3(32 * kWarps), 0, s, xt, rows, cols, stride, segs_of(cols), perm, q, scales);
}
template <int DT>
cudaError_t launch_dequantize(const uint8_t* q, const float* scales, int64_t rows, int cols, bool vec,
                              void* out, cudaStream_t s) {
  auto* ot = static_cast<typename In<DT>::T*>(out);
  return vec ? launch_pdl(dequantize_tiles_kernel<DT>, dim3(tile_blocks(rows, cols)), dim3(32 * kWarps),
                          0, s, q, scales, rows, cols, ot)
             : launch_pdl(dequantize_any_kernel<DT>, dim3(seg_blocks(rows, cols)), dim3(32 * kWarps), 0,
                          s, q, scales, rows, cols, segs_of(cols), ot);
}

bool too_large(int64_t rows, int cols) {
  return cols > kMaxFp8Cols || rows > (INT32_MAX - 64) / (fp8_cols(cols) / 128);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_fp8_row_bytes(int cols) { return cols < 0 ? 0 : fp8_cols(cols); }

moe_status_t moe_quantize_rows_fp8(const void* x, int dtype, int64_t rows, int cols,
                                   int64_t row_stride, int swiglu, const int32_t* perm, uint8_t* q,
                                   float* scales, cudaStream_t stream) {
  if (!known_dtype(dtype) || rows < 0 || cols < 1 || row_stride < 0 || (swiglu != 0 && swiglu != 1))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales || !aligned16(q) || !aligned4(scales) || !aligned4(perm))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxFp8Cols) return MOE_ERR_UNSUPPORTED;
  if (rows > 1 && row_stride < (swiglu ? 2 * static_cast<int64_t>(cols) : cols)) return MOE_ERR_INVALID_ARG;
  const int64_t size = dtype_bytes(dtype);
  if (reinterpret_cast<uintptr_t>(x) % size != 0) return MOE_ERR_INVALID_ARG;
  if (too_large(rows, cols)) return MOE_ERR_UNSUPPORTED;
  const bool vec = aligned16(x) && row_stride * size % 16 == 0 && (!swiglu || cols * size % 16 == 0);
  const auto run = dtype == MOE_DTYPE_BF16
                       ? (swiglu ? launch_quantize<MOE_DTYPE_BF16, true> : launch_quantize<MOE_DTYPE_BF16, false>)
                   : dtype == MOE_DTYPE_F16
                       ? (swiglu ? launch_quantize<MOE_DTYPE_F16, true> : launch_quantize<MOE_DTYPE_F16, false>)
                       : (swiglu ? launch_quantize<MOE_DTYPE_F32, true> : launch_quantize<MOE_DTYPE_F32, false>);
  return cuda_status(run(x, rows, cols, row_stride, vec, perm, q, scales, stream));
}

moe_status_t moe_dequantize_rows_fp8(const uint8_t* q, const float* scales, int64_t rows, int cols,
                                     int dtype, void* out, cudaStream_t stream) {
  if (!known_dtype(dtype) || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!q || !scales || !out || !aligned16(q) || !aligned4(scales) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  if (too_large(rows, cols)) return MOE_ERR_UNSUPPORTED;
  const bool vec = cols * dtype_bytes(dtype) % 16 == 0;  // `out` itself is aligned
  const auto run = dtype == MOE_DTYPE_BF16  ? launch_dequantize<MOE_DTYPE_BF16>
                   : dtype == MOE_DTYPE_F16 ? launch_dequantize<MOE_DTYPE_F16>
                                            : launch_dequantize<MOE_DTYPE_F32>;
  return cuda_status(run(q, scales, rows, cols, vec, out, stream));
}

moe_status_t moe_quantize_blocks_fp8(const moe_bf16_t* W, int E, int K, int N, int transpose,
                                     uint8_t* Wq, float* scales, cudaStream_t stream) {
  if (E < 1 || K < 1 || N < 1 || (transpose != 0 && transpose != 1)) return MOE_ERR_INVALID_ARG;
  if (!W || !Wq || !scales || !aligned16(W) || !aligned16(Wq) || !aligned4(scales))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || K > kMaxFp8Cols || N > kMaxFp8Cols) return MOE_ERR_UNSUPPORTED;
  const int n_tiles = (N + 127) / 128, k_tiles = (K + 127) / 128;
  return cuda_status(launch_pdl(transpose ? quantize_blocks_kernel<true> : quantize_blocks_kernel<false>,
                                dim3(n_tiles * k_tiles, E), dim3(256), 0, stream, W, K, N, n_tiles,
                                static_cast<int>(N % 8 == 0), Wq, scales));
}

}  // extern "C"
