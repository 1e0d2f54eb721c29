// Root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its
// gradient.
//   s = x + r (rounded to the type once: the sum that the next layer adds to)
//   y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps),  in fp32, rounded once per output
//   dx = rstd (g - n mean(g n)) + dsum,  g = dy w, n = s rstd;  dw = sum over rows of dy n
// Bound by HBM: each value is read once (a row stays in registers between the sum and the outputs)
// and each output written once.  A row is cut into segments of 256 values, one or more per warp
// (`V`); a segment's sum is a warp's, and the segments' sums are added in one order, so a row's
// results do not depend on the other rows or on how many warps share it.
#include "fp8.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxSegs = 64;  // cols <= 16384

struct NormArgs {
  const void *x, *residual, *w;
  void *sum, *out;
  uint8_t* q;
  float *scales, *rstd;
  int64_t rows, x_stride;
  int cols, W, w_f32;  // W: warps per row
  float eps;
};

// Eight weights as fp32, laid over a segment as the values are.
template <int DT, bool VEC>
__device__ __forceinline__ void load_weights(const void* w, int w_f32, int c0, int cols, int lane,
                                             float (&f)[8]) {
  if (w_f32) {
    const Raw8<float> r = load_seg<VEC>(static_cast<const float*>(w) + c0, cols - c0, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = r.v[j];
  } else {
    using T = typename In<DT>::T;
    const Raw8<T> r = load_seg<VEC>(static_cast<const T*>(w) + c0, cols - c0, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = In<DT>::f32(r.v[j]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// The sum of a row's segment sums, by every warp for itself in the same order.
__device__ __forceinline__ float sum_parts(const float* part, int segs, int lane) {
  float v = 0.0f;
  for (int i = lane; i < segs; i += 32) v += part[i];
  return warp_sum(v);
}

// One row per CTA of W warps, or (W = 1) a row per warp.
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512)
    rmsnorm_kernel(const NormArgs a) {
  using T = typename In<DT>::T;
  __shared__ float part[kMaxSegs];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = a.W == 1;
  const int64_t row = alone ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  const int w0 = alone ? 0 : warp;
  if (row >= a.rows) return;  // whole warps, and only of CTAs that do not synchronise
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const int64_t at = row * a.cols;
  Raw8<T> s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c0 = (w0 + i * a.W) * kSeg;
    s[i] = load_seg<VEC>(x + c0, a.cols - c0, lane);
  }
  if (a.residual) {
    const T* r = static_cast<const T*>(a.residual) + at;
    Raw8<T> v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      v[i] = load_seg<VEC>(r + c0, a.cols - c0, lane);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i].v[j] = In<DT>::of(In<DT>::f32(s[i].v[j]) + In<DT>::f32(v[i].v[j]));
      store_seg<VEC>(static_cast<T*>(a.sum) + at + c0, a.cols - c0, lane, s[i]);
    }
  }
  float total = 0.0f, sq[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sq[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = In<DT>::f32(s[i].v[j]);
      sq[i] = fmaf(f, f, sq[i]);
    }
    sq[i] = warp_sum(sq[i]);
  }
  if (alone) {  // the order of sum_parts: at most 32 segments, one to a lane
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) v = lane == i ? sq[i] : v;
    total = warp_sum(v);
  } else {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (w0 + i * a.W < segs) part[w0 + i * a.W] = sq[i];
    }
    __syncthreads();
    total = sum_parts(part, segs, lane);
  }
  const float rstd = __frsqrt_rn(total / static_cast<float>(a.cols) + a.eps);
  if (a.rstd && w0 == 0 && lane == 0) a.rstd[row] = rstd;
  const int64_t kp = fp8_cols(a.cols);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c0 = (w0 + i * a.W) * kSeg;
    if (c0 >= a.cols) break;
    float y[8], w[8];
    load_weights<DT, VEC>(a.w, a.w_f32, c0, a.cols, lane, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = In<DT>::f32(s[i].v[j]) * rstd * w[j];
    if (a.out) {
      Raw8<T> o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = In<DT>::of(y[j]);
      store_seg<VEC>(static_cast<T*>(a.out) + at + c0, a.cols - c0, lane, o);
    }
    if (a.q)
      quantize_seg<VEC>(y, a.q + row * kp + c0, a.scales + row * (kp / 128) + c0 / 128,
                        static_cast<int>(kp - c0 < kSeg ? kp - c0 : kSeg), lane);
  }
}

struct NormGradArgs {
  const void *dy, *s, *w, *dsum;
  const float* rstd;
  void* dx;
  float* part;  // [CTAs][cols] sums of dy n, null without dw
  int64_t rows;
  int cols, W, w_f32;
};

// Each CTA (W = 1: each warp) walks over rows and keeps its columns' sums of dy n in registers; a
// second kernel adds the CTAs' sums in their order.  The gradient of the weights is bitwise
// reproducible on one device; it depends on the number of CTAs.
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512)
    rmsnorm_backward_kernel(const NormGradArgs a) {
  using T = typename In<DT>::T;
  __shared__ float part[2][kMaxSegs];
  extern __shared__ float sums[];  // W = 1: [warps][cols]
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = a.W == 1;
  const int w0 = alone ? 0 : warp;
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const int64_t first = alone ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  const int64_t step = alone ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  int turn = 0;
  for (int64_t row = first; row < a.rows; row += step, turn ^= 1) {
    const int64_t at = row * a.cols;
    const float rstd = a.rstd[row];
    Raw8<T> s[V], dy[V], ds[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      s[i] = load_seg<VEC>(static_cast<const T*>(a.s) + at + c0, a.cols - c0, lane);
      dy[i] = load_seg<VEC>(static_cast<const T*>(a.dy) + at + c0, a.cols - c0, lane);
    }
    if (a.dsum) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c0 = (w0 + i * a.W) * kSeg;
        ds[i] = load_seg<VEC>(static_cast<const T*>(a.dsum) + at + c0, a.cols - c0, lane);
      }
    }
    float dot[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      float w[8];
      load_weights<DT, VEC>(a.w, a.w_f32, c0, a.cols, lane, w);
      dot[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = In<DT>::f32(s[i].v[j]) * rstd, d = In<DT>::f32(dy[i].v[j]);
        dw[i][j] = fmaf(d, n, dw[i][j]);
        dot[i] = fmaf(d * w[j], n, dot[i]);
      }
      dot[i] = warp_sum(dot[i]);
    }
    float total;
    if (alone) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) v = lane == i ? dot[i] : v;
      total = warp_sum(v);
    } else {
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (w0 + i * a.W < segs) part[turn][w0 + i * a.W] = dot[i];
      }
      // one barrier a row: the other half of `part` is written before the next one
      __syncthreads();
      total = sum_parts(part[turn], segs, lane);
    }
    const float mean = total / static_cast<float>(a.cols);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      float w[8];
      load_weights<DT, VEC>(a.w, a.w_f32, c0, a.cols, lane, w);
      Raw8<T> o;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = In<DT>::f32(s[i].v[j]) * rstd;
        float v = rstd * fmaf(-n, mean, In<DT>::f32(dy[i].v[j]) * w[j]);
        if (a.dsum) v += In<DT>::f32(ds[i].v[j]);
        o.v[j] = In<DT>::of(v);
      }
      store_seg<VEC>(static_cast<T*>(a.dx) + at + c0, a.cols - c0, lane, o);
    }
  }
  if (!a.part) return;
  float* mine = alone ? sums + warp * a.cols : a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c0 = (w0 + i * a.W) * kSeg;
    Raw8<float> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.v[j] = dw[i][j];
    if (alone || !VEC) {  // (rows of `sums` need not start on 16 bytes)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = c0 + (VEC ? 8 * lane + j : 32 * j + lane);
        if (c < a.cols) mine[c] = v.v[j];
      }
    } else {
      store_seg<true>(mine + c0, a.cols - c0, lane, v);
    }
  }
  if (alone) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float v = 0.0f;
      for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v += sums[i * a.cols + c];
      a.part[static_cast<int64_t>(blockIdx.x) * a.cols + c] = v;
    }
  }
}

// dw[c] = sum over n partial rows: 32 columns a CTA, each of 32 warps every 32nd row, then the
// warps' sums in order.
__global__ void __launch_bounds__(1024) rmsnorm_dweight_kernel(const float* __restrict__ part, int n,
                                                               int cols, float* __restrict__ dw) {
  __shared__ float sums[32][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int r = warp; r < n; r += 32) v += part[static_cast<int64_t>(r) * cols + c];
  }
  sums[warp][lane] = v;
  __syncthreads();
  v = warp_sum(sums[lane][warp]);
  const int o = blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) dw[o] = v;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known_dtype(int dt) {
  return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16 || dt == MOE_DTYPE_F32;
}
int64_t dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Segments per warp and warps per row.  Four segments keep loads of 4 x 16 bytes per lane in flight;
// with no more rows than SMs a row is spread over as many warps as it has segments.
struct Shape {
  int v, W, threads;
};
constexpr int kAloneWarps = 8;  // warps of a CTA whose warps have a row each
Shape shape_of(int64_t rows, int cols, int sms) {
  const int segs = (cols + kSeg - 1) / kSeg;
  Shape s;
  s.v = 1;
  while (s.v < segs && s.v < 4) s.v *= 2;
  if (rows <= sms && segs <= 32) s.v = 1;
  s.W = (segs + s.v - 1) / s.v;
  s.threads = 32 * (s.W == 1 ? kAloneWarps : s.W);
  return s;
}
int64_t grad_ctas(int64_t rows, int cols, int sms) {
  const Shape s = shape_of(rows, cols, sms);
  const int64_t most = s.W == 1 ? (rows + kAloneWarps - 1) / kAloneWarps : rows;
  const int64_t per_sm = s.threads <= 256 ? 4 : s.threads <= 512 ? 2 : 1;
  return most < per_sm * sms ? most : per_sm * sms;
}

template <int DT, int V>
cudaError_t launch_norm(const NormArgs& a, const Shape& s, bool vec, cudaStream_t st) {
  const int64_t per = s.W == 1 ? kAloneWarps : 1;
  const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per)), block(s.threads);
  return vec ? launch_pdl(rmsnorm_kernel<DT, V, true>, grid, block, 0, st, a)
             : launch_pdl(rmsnorm_kernel<DT, V, false>, grid, block, 0, st, a);
}
template <int DT>
cudaError_t launch_norm(const NormArgs& a, const Shape& s, bool vec, cudaStream_t st) {
  return s.v == 1   ? launch_norm<DT, 1>(a, s, vec, st)
         : s.v == 2 ? launch_norm<DT, 2>(a, s, vec, st)
                    : launch_norm<DT, 4>(a, s, vec, st);
}
template <int DT, int V>
cudaError_t launch_grad(const NormGradArgs& a, const Shape& s, int ctas, bool vec, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ctas)), block(s.threads);
  const size_t smem = s.W == 1 ? static_cast<size_t>(kAloneWarps) * a.cols * 4 : 0;  // <= 32 KB
  return vec ? launch_pdl(rmsnorm_backward_kernel<DT, V, true>, grid, block, smem, st, a)
             : launch_pdl(rmsnorm_backward_kernel<DT, V, false>, grid, block, smem, st, a);
}
template <int DT>
cudaError_t launch_grad(const NormGradArgs& a, const Shape& s, int ctas, bool vec, cudaStream_t st) {
  return s.v == 1   ? launch_grad<DT, 1>(a, s, ctas, vec, st)
         : s.v == 2 ? launch_grad<DT, 2>(a, s, ctas, vec, st)
                    : launch_grad<DT, 4>(a, s, ctas, vec, st);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_rmsnorm(const void* x, int64_t x_stride, const void* residual, const void* weight,
                         int dtype, int weight_dtype, int64_t rows, int cols, float eps,
                         void* sum_out, void* out, uint8_t* q, float* scales, float* rstd,
                         cudaStream_t stream) {
  if (!known_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MOE_DTYPE_F32) || rows < 0 ||
      cols < 1 || x_stride < 0 || !(eps >= 0.0f))
    return MOE_ERR_INVALID_ARG;
  if ((residual != nullptr) != (sum_out != nullptr) || (q != nullptr) != (scales != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int size = static_cast<int>(dtype_bytes(dtype));
  if (!x || !weight || (!out && !q)) return MOE_ERR_INVALID_ARG;
  if (rows > 1 && x_stride < cols) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(x, size) || !aligned_to(residual, size) || !aligned_to(sum_out, size) ||
      !aligned_to(out, size) || !aligned_to(weight, static_cast<int>(dtype_bytes(weight_dtype))) ||
      !aligned16(q) || !aligned_to(scales, 4) || !aligned_to(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxSegs * kSeg || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const bool vec = aligned16(x) && x_stride * size % 16 == 0 && cols % 8 == 0 &&
                   cols * size % 16 == 0 && aligned16(residual) && aligned16(sum_out) &&
                   aligned16(out) && aligned16(weight);
  const NormArgs a{x,     residual, weight, sum_out,  out,  q, scales, rstd,
                   rows,  x_stride, cols,   0,        weight_dtype == MOE_DTYPE_F32, eps};
  const Shape s = shape_of(rows, cols, num_sms_of_current_device());
  NormArgs b = a;
  b.W = s.W;
  return cuda_status(dtype == MOE_DTYPE_BF16  ? launch_norm<MOE_DTYPE_BF16>(b, s, vec, stream)
                     : dtype == MOE_DTYPE_F16 ? launch_norm<MOE_DTYPE_F16>(b, s, vec, stream)
                                              : launch_norm<MOE_DTYPE_F32>(b, s, vec, stream));
}

size_t moe_rmsnorm_workspace_bytes(int64_t rows, int cols) {
  if (rows < 0 || cols < 1 || cols > kMaxSegs * kSeg || rows > INT32_MAX) return 0;
  const int64_t n = grad_ctas(rows, cols, num_sms_of_current_device());
  const int64_t bytes = (n * cols * 4 + 255) / 256 * 256;
  return static_cast<size_t>(bytes < 256 ? 256 : bytes);
}

moe_status_t moe_rmsnorm_backward(const void* dy, const void* s, const void* weight,
                                  const float* rstd, const void* dsum, int dtype, int weight_dtype,
                                  int64_t rows, int cols, void* dx, float* dweight, void* ws,
                                  size_t ws_bytes, cudaStream_t stream) {
  if (!known_dtype(dtype) || (weight_dtype != dtype && weight_dtype != MOE_DTYPE_F32) || rows < 0 ||
      cols < 1)
    return MOE_ERR_INVALID_ARG;
  const int size = static_cast<int>(dtype_bytes(dtype));
  if (rows > 0 && (!dy || !s || !weight || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(dy, size) || !aligned_to(s, size) || !aligned_to(dsum, size) ||
      !aligned_to(dx, size) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) ||
      !aligned_to(weight, static_cast<int>(dtype_bytes(weight_dtype))))
    return MOE_ERR_INVALID_ARG;
  if (cols > kMaxSegs * kSeg || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (dweight) {
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_rmsnorm_workspace_bytes(rows, cols)) return MOE_ERR_WORKSPACE;
  }
  if (rows == 0)
    return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, 4ull * cols, stream)) : MOE_OK;
  const int sms = num_sms_of_current_device();
  const Shape sh = shape_of(rows, cols, sms);
  const int ctas = static_cast<int>(grad_ctas(rows, cols, sms));
  const bool vec = cols % 8 == 0 && aligned16(dy) && aligned16(s) && aligned16(dsum) &&
                   aligned16(dx) && aligned16(weight);
  const NormGradArgs a{dy,   s,    weight, dsum, rstd, dx, dweight ? static_cast<float*>(ws) : nullptr,
                       rows, cols, sh.W,   weight_dtype == MOE_DTYPE_F32};
  cudaError_t st = dtype == MOE_DTYPE_BF16  ? launch_grad<MOE_DTYPE_BF16>(a, sh, ctas, vec, stream)
                   : dtype == MOE_DTYPE_F16 ? launch_grad<MOE_DTYPE_F16>(a, sh, ctas, vec, stream)
                                            : launch_grad<MOE_DTYPE_F32>(a, sh, ctas, vec, stream);
  if (st == cudaSuccess && dweight)
    st = launch_pdl(rmsnorm_dweight_kernel, dim3((cols + 31) / 32), dim3(1024), 0, stream,
                    static_cast<const float*>(ws), ctas, cols, dweight);
  return cuda_status(st);
}

}  // extern "C"
