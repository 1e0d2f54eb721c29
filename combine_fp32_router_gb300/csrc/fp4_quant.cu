// MXFP4 quantisation and its inverse (format: fp4.cuh).
//
// quantize: s = floor(log2(max |x|)) - 2 + 127 of each block of 32, codes
// rne_e2m1(x 2^(127 - s)); every step but the final rounding is exact, so the result is a
// function of the block alone, whatever the launch.  Rows are read once (2 or 4 bytes a value)
// and 17/32 bytes a value are written: bound by HBM.
#include "elem.cuh"
#include "fp4.cuh"
#include "internal.h"

namespace moe {

namespace {

// Warps of a CTA.  Four leave an SM's places sooner than eight: 16384 x 7168 bf16 values 50.9 and
// 45.3 us (quantise and back) against 51.4 and 46.0; two are no faster.
constexpr int kQuantWarps = 4;

// ---- rows that start on 16 bytes.  The matrix is cut into tiles of 128 values of a row, rows x kt
// of them in row-major order, and each warp takes eight that follow one another: half a warp every
// second one, lane l of it the values 8 l .. 8 l + 7.  Four lanes then hold a block and sixteen
// the four blocks of a scale word, whatever the width: no lane idles on narrow rows (25894 rows of
// 328 bf16 values: 7.4 us to quantise, 10.1 us with whole rows per warp).
constexpr int kHalfTiles = 4;  // tiles per half warp, all loaded before the first is used

// A half warp's walk over its tiles: row and tile, the tile's first value in a matrix with rows
// `stride` apart, and its place among the scales.  A step inside a row is three additions.
template <typename T>
struct Walk {
  uint32_t row;
  int t;
  T* value;
  int64_t scale;
  __device__ __forceinline__ Walk(uint32_t tile, int kt, T* base, int64_t stride)
      : row(tile / static_cast<uint32_t>(kt)), t(static_cast<int>(tile % static_cast<uint32_t>(kt))) {
    value = base + row * stride + t * 128;
    scale = mx_scale_at(row, 4 * t, kt);
  }
  __device__ __forceinline__ void step(int kt, T* base, int64_t stride) {
    t += 2;
    value += 256;
    scale += 2 * kMxTileBytes;
    if (t >= kt) {
      for (; t >= kt; t -= kt) ++row;
      value = base + row * stride + t * 128;
      scale = mx_scale_at(row, 4 * t, kt);
    }
  }
};

// A lane's part of its block's largest magnitude, as fp32 bits: of eight values, or of eight raw
// 16-bit ones two at a time (all formats order like their bits).
__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return amax;
}
template <int DT>
__device__ __forceinline__ uint32_t largest(const Raw8<uint16_t>& r) {
  const uint4 u = *reinterpret_cast<const uint4*>(&r);
  constexpr uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vimax3_u16x2(__vimax3_u16x2(u.x & m, u.y & m, u.z & m), u.w & m, 0u);
  const uint32_t top = max(t & 0xFFFFu, t >> 16);
  return DT == MOE_DTYPE_BF16 ? top << 16 : __float_as_uint(In<DT>::f32(static_cast<uint16_t>(top)));
}
// The scale byte of the block that four lanes hold; `sw`: those of sixteen lanes' four blocks.
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, int l, uint32_t* sw) {
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const uint32_t s = mx_scale_byte(amax);
  *sw = s << (8 * ((l >> 2) & 3));
  *sw |= __shfl_xor_sync(0xFFFFFFFFu, *sw, 4);
  *sw |= __shfl_xor_sync(0xFFFFFFFFu, *sw, 8);
  return s;
}
__device__ __forceinline__ uint32_t codes8(float (&v)[8], uint32_t s) {
  const float inv = mx_inverse_scale(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= inv;
  return s == 255u ? 0u : e2m1x8(v);
}
// The same from raw values.  A bf16 times a power of two is exact in bf16 (or far below the
// smallest code), two at a time.
template <int DT>
__device__ __forceinline__ uint32_t quantize8(const Raw8<typename In<DT>::T>& r, int l, uint32_t* sw) {
  float v[8];
  if constexpr (DT == MOE_DTYPE_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.v[j];
    const uint32_t s = block_scale(largest(v), l, sw);
    return codes8(v, s);
  } else {
    const uint32_t s = block_scale(largest<DT>(r), l, sw);
    if constexpr (DT == MOE_DTYPE_F16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = In<DT>::f32(r.v[j]);
      return codes8(v, s);
    } else {
      const uint32_t i2 = (__float_as_uint(mx_inverse_scale(s)) >> 16) * 0x10001u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 t = __hmul2(reinterpret_cast<const __nv_bfloat162*>(&r)[j],
                                         *reinterpret_cast<const __nv_bfloat162*>(&i2));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&t);
        v[2 * j] = bf16lo(w);
        v[2 * j + 1] = bf16hi(w);
      }
      return s == 255u ? 0u : e2m1x8(v);
    }
  }
}
// The rows that the last scale tile has and the matrix has not: scale bytes of zero, by the
// sixteen lanes of the last row's tile.
__device__ __forceinline__ void pad_tile(uint8_t* scales, int64_t place, uint32_t row, int l) {
  uint8_t* tile0 = scales + place / kMxTileBytes * kMxTileBytes;
  for (int r = static_cast<int>(row % 128) + 1 + l; r < 128; r += 16)
    *reinterpret_cast<uint32_t*>(tile0 + mx_scale_at(r, 0, 1)) = 0u;
}

template <int DT>
__global__ void __launch_bounds__(32 * kQuantWarps, DT == MOE_DTYPE_F32 ? 8 : 12)
    quantize_rows_kernel(const typename In<DT>::T* __restrict__ x, int64_t rows, int cols,
                         int64_t stride, uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  using T = typename In<DT>::T;
  griddep_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int kt = static_cast<int>(mx_cols(cols) / 128);
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const uint32_t tile = w * 2 * kHalfTiles + (lane >> 4);
  Walk<const T> at(tile, kt, x, stride);
  Raw8<T> raw[kHalfTiles];
  uint32_t row[kHalfTiles];
  int64_t so[kHalfTiles];
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i) {
    row[i] = at.row;
    so[i] = at.scale;
    // lanes past the last row stay in step and load nothing
    raw[i] = load8(at.value, at.row < rows ? cols - at.t * 128 : 0, l);
    at.step(kt, x, stride);
  }
  uint8_t* qo = q + static_cast<int64_t>(tile) * 64 + 4 * l;
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i) {
    uint32_t sw;
    const uint32_t code = quantize8<DT>(raw[i], l, &sw);
    if (row[i] < rows) {
      *reinterpret_cast<uint32_t*>(qo + i * 128) = code;
      if (l == 0) *reinterpret_cast<uint32_t*>(scales + so[i]) = sw;
      if (row[i] == rows - 1) pad_tile(scales, so[i], row[i], l);
    }
  }
}

// The inverse: value = code * 2^(s - 127), rounded once to the output type (exact in bf16 and
// fp32 wherever the type reaches).
template <int DT>
__device__ __forceinline__ Raw8<typename In<DT>::T> dequantize8(uint32_t code, uint32_t s) {
  uint32_t h[4];
  e2m1x8_to_half(code, h);
  const float f = mx_scale(s);
  Raw8<typename In<DT>::T> t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    t.v[2 * j] = In<DT>::of(p.x * f);
    t.v[2 * j + 1] = In<DT>::of(p.y * f);
  }
  return t;
}

template <int DT>
__global__ void __launch_bounds__(32 * kQuantWarps)
    dequantize_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                           int64_t rows, int64_t rows_all, int cols,
                           typename In<DT>::T* __restrict__ out) {
  using T = typename In<DT>::T;
  griddep_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int kt = static_cast<int>(mx_cols(cols) / 128);
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int64_t per = mx_scale_bytes(rows, cols);
  const uint32_t tile = w * 2 * kHalfTiles + (lane >> 4);
  Walk<T> at(tile, kt, out, cols);
  uint32_t code[kHalfTiles], s[kHalfTiles];
  T* to[kHalfTiles];
  int n[kHalfTiles];
  const uint8_t* qi = q + static_cast<int64_t>(tile) * 64 + 4 * l;
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i) {
    code[i] = 0;
    s[i] = 0;
    to[i] = at.value;
    n[i] = at.row < rows_all ? cols - at.t * 128 : 0;
    if (8 * l < n[i]) {
      code[i] = __ldg(reinterpret_cast<const uint32_t*>(qi + i * 128));
      int64_t so = at.scale;
      if (rows != rows_all) {  // a group's scales start at a tile of their own
        const uint32_t g = at.row / static_cast<uint32_t>(rows);
        so = g * per + mx_scale_at(at.row - g * rows, 4 * at.t, kt);
      }
      s[i] = __ldg(scales + so + (l >> 2));
    }
    at.step(kt, out, cols);
  }
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i) {
    const Raw8<T> t = dequantize8<DT>(code[i], s[i]);
    T* o = to[i] + 8 * l;
    if (8 * l + 8 <= n[i]) {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(t) / 16); ++j)
        // written once and larger than the codes: not kept in L2 in their place
        __stcs(reinterpret_cast<uint4*>(o) + j, reinterpret_cast<const uint4*>(&t)[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * l + j < n[i]) o[j] = t.v[j];
    }
  }
}

// ---- other rows.  A warp takes U x 256 values of one row; its lanes read or store neighbouring
// values, 32 at a time, and pass them on through shared memory (5000 rows of 3001 bf16 values:
// 11 and 8 us; with eight strided accesses per lane 12 and 43; as whole vectors between their
// 16-byte boundaries 16 and 12).
template <int DT, int U>
__global__ void __launch_bounds__(32 * kQuantWarps)
    quantize_rows_any_kernel(const typename In<DT>::T* __restrict__ x, int64_t rows, int cols,
                             int64_t stride, uint32_t segs, uint8_t* __restrict__ q,
                             uint8_t* __restrict__ scales) {
  __shared__ float4 shared[kQuantWarps * 64];
  griddep_wait();
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row = w / segs;
  if (row >= rows) return;
  const int c0 = static_cast<int>(w % segs) * (U * 256);
  const int kp = static_cast<int>(mx_cols(cols));
  const typename In<DT>::T* xr = x + row * stride;
  float* buf = reinterpret_cast<float*>(shared + (threadIdx.x >> 5) * 64);
  float v[U][8];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = c0 + i * 256 + 32 * j + lane;
      v[i][j] = k < cols ? In<DT>::f32(__ldg(xr + k)) : 0.0f;
    }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) buf[32 * j + lane] = v[i][j];
    __syncwarp();
    const float4 a = *reinterpret_cast<const float4*>(buf + 8 * lane);
    const float4 b = *reinterpret_cast<const float4*>(buf + 8 * lane + 4);
    float t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t sw;
    const uint32_t code = codes8(t, block_scale(largest(t), lane, &sw));
    const int c = c0 + i * 256 + lane * 8;
    if (c < kp) {
      *reinterpret_cast<uint32_t*>(q + row * static_cast<int64_t>(kp / 2) + c / 2) = code;
      const int64_t so = mx_scale_at(row, c / 128 * 4, kp / 128);
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + so) = sw;
      if (row == rows - 1) pad_tile(scales, so, row, lane & 15);
    }
  }
}

template <int DT, int U>
__global__ void __launch_bounds__(32 * kQuantWarps)
    dequantize_rows_any_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                               int64_t rows, int64_t rows_all, int cols, uint32_t segs,
                               typename In<DT>::T* __restrict__ out) {
  using T = typename In<DT>::T;
  __shared__ Raw8<T> shared[kQuantWarps * 32];
  griddep_wait();
  const uint32_t w = blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t row_all = w / segs;
  if (row_all >= rows_all) return;
  const int64_t g = row_all / rows, row = row_all % rows;
  const int c0 = static_cast<int>(w % segs) * (U * 256);
  const int kp = static_cast<int>(mx_cols(cols));
  const uint8_t* qi = q + row_all * static_cast<int64_t>(kp / 2) + (c0 + lane * 8) / 2;
  const uint8_t* si = scales + g * mx_scale_bytes(rows, cols) +
                      mx_scale_at(row, (c0 + lane * 8) / 32, kp / 128);
  T* o = out + row_all * static_cast<int64_t>(cols);
  Raw8<T>* mine = shared + (threadIdx.x >> 5) * 32;
  uint32_t code[U], s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    code[i] = 0;
    s[i] = 0;
    if (c0 + i * 256 + lane * 8 < cols) {
      code[i] = __ldg(reinterpret_cast<const uint32_t*>(qi + i * 128));
      s[i] = __ldg(si + i * 2 * kMxTileBytes);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    __syncwarp();
    mine[lane] = dequantize8<DT>(code[i], s[i]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = c0 + i * 256 + 32 * j + lane;
      if (k < cols) o[k] = reinterpret_cast<const T*>(mine)[32 * j + lane];
    }
  }
}

// Weights [E, K, N] bf16 -> [E, N, Kp / 2], blocks along K: a CTA transposes 256 K x 64 N
// through shared memory.  Thread (n pair, block) quantises one block of two neighbouring
// columns; codes and scale words leave through shared memory in 16-byte and 4-byte pieces of
// whole rows.
constexpr int kWtK = 256, kWtN = 64;
__global__ void __launch_bounds__(256, 5)
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
  // both columns at a time: magnitudes order like their bits, and a bf16 times a power of two is
  // exact in bf16 (or far below the smallest code)
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = __vmaxu2(top, tile[32 * b + i][np] & 0x7FFF7FFFu);
  const uint32_t s0 = mx_scale_byte(top << 16), s1 = mx_scale_byte(top & 0xFFFF0000u);
  const uint32_t inv = (__float_as_uint(mx_inverse_scale(s0)) >> 16) |
                       (__float_as_uint(mx_inverse_scale(s1)) & 0xFFFF0000u);
  uint32_t w0[4], w1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v0[8], v1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 t =
          __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&tile[32 * b + 8 * i + j][np]),
                  *reinterpret_cast<const __nv_bfloat162*>(&inv));
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&t);
      v0[j] = bf16lo(u);
      v1[j] = bf16hi(u);
    }
    w0[i] = s0 == 255u ? 0u : e2m1x8(v0);
    w1[i] = s1 == 255u ? 0u : e2m1x8(v1);
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

// Blocks of a launch over `rows` rows that start on 16 bytes (u = 0), or warps of u x 256 values
// of a row, `segs` per row, for other rows: the most of 4, 2 and 1 that leaves at most an eighth
// of the lanes without work.  False when a 32-bit index does not hold them.
struct Cut {
  int u;
  uint32_t segs, blocks;
};
bool cut_rows(int64_t rows, int cols, bool vec, Cut* c) {
  const int64_t kp = mx_cols(cols);
  if (rows > (INT32_MAX - 64) / (kp / 128)) return false;
  *c = Cut{0, 0, 0};
  int64_t warps = (rows * (kp / 128) + 2 * kHalfTiles - 1) / (2 * kHalfTiles);
  if (!vec) {
    c->u = 4;
    while (c->u > 1 && (kp + 256 * c->u - 1) / (256 * c->u) * (256 * c->u) * 7 > kp * 8) c->u /= 2;
    c->segs = static_cast<uint32_t>((kp + 256 * c->u - 1) / (256 * c->u));
    warps = rows * c->segs;
  }
  c->blocks = static_cast<uint32_t>((warps + kQuantWarps - 1) / kQuantWarps);
  return true;
}

template <int DT>
cudaError_t launch_quantize(const void* x, int64_t rows, int cols, int64_t stride, const Cut& c,
                            uint8_t* q, uint8_t* scales, cudaStream_t s) {
  const auto* xt = static_cast<const typename In<DT>::T*>(x);
  const dim3 grid(c.blocks), block(32 * kQuantWarps);
  if (c.u == 0)
    return launch_pdl(quantize_rows_kernel<DT>, grid, block, 0, s, xt, rows, cols, stride, q, scales);
  const auto kern = c.u == 4   ? quantize_rows_any_kernel<DT, 4>
                    : c.u == 2 ? quantize_rows_any_kernel<DT, 2>
                               : quantize_rows_any_kernel<DT, 1>;
  return launch_pdl(kern, grid, block, 0, s, xt, rows, cols, stride, c.segs, q, scales);
}
template <int DT>
cudaError_t launch_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows,
                              int64_t rows_all, int cols, const Cut& c, void* out, cudaStream_t s) {
  auto* ot = static_cast<typename In<DT>::T*>(out);
  const dim3 grid(c.blocks), block(32 * kQuantWarps);
  if (c.u == 0)
    return launch_pdl(dequantize_rows_kernel<DT>, grid, block, 0, s, q, scales, rows, rows_all, cols, ot);
  const auto kern = c.u == 4   ? dequantize_rows_any_kernel<DT, 4>
                    : c.u == 2 ? dequantize_rows_any_kernel<DT, 2>
                               : dequantize_rows_any_kernel<DT, 1>;
  return launch_pdl(kern, grid, block, 0, s, q, scales, rows, rows_all, cols, c.segs, ot);
}

int64_t dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }

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
  if (reinterpret_cast<uintptr_t>(x) % dtype_bytes(dtype) != 0) return MOE_ERR_INVALID_ARG;
  Cut cut;
  const bool vec = aligned16(x) && row_stride * dtype_bytes(dtype) % 16 == 0;
  if (cols > kMaxFp4Cols || !cut_rows(rows, cols, vec, &cut)) return MOE_ERR_UNSUPPORTED;
  const auto run = dtype == MOE_DTYPE_BF16  ? launch_quantize<MOE_DTYPE_BF16>
                   : dtype == MOE_DTYPE_F16 ? launch_quantize<MOE_DTYPE_F16>
                                            : launch_quantize<MOE_DTYPE_F32>;
  return cuda_status(run(x, rows, cols, row_stride, cut, q, scales, stream));
}

moe_status_t moe_dequantize_rows_fp4(const uint8_t* q, const uint8_t* scales, int groups,
                                     int64_t rows, int cols, int dtype, void* out,
                                     cudaStream_t stream) {
  if (!known_dtype(dtype) || groups < 0 || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (groups == 0 || rows == 0) return MOE_OK;
  if (!q || !scales || !out || !aligned16(q) || !aligned16(scales) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  if (rows % 128 == 0) {  // groups of whole scale tiles are one matrix
    if (rows > INT32_MAX / groups) return MOE_ERR_UNSUPPORTED;
    rows *= groups;
    groups = 1;
  }
  Cut cut;
  const bool vec = cols * dtype_bytes(dtype) % 16 == 0;  // `out` itself is aligned
  if (cols > kMaxFp4Cols || rows > INT32_MAX / groups || !cut_rows(rows * groups, cols, vec, &cut))
    return MOE_ERR_UNSUPPORTED;
  const auto run = dtype == MOE_DTYPE_BF16  ? launch_dequantize<MOE_DTYPE_BF16>
                   : dtype == MOE_DTYPE_F16 ? launch_dequantize<MOE_DTYPE_F16>
                                            : launch_dequantize<MOE_DTYPE_F32>;
  return cuda_status(run(q, scales, rows, rows * groups, cols, cut, out, stream));
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
