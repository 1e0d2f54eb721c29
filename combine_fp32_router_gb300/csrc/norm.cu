// Root-mean-square norm of rows, with the residual's addition and an output in 8 bits, and its
// gradient.
//   s = x + r (rounded to the type once: the sum that the next layer adds to)
//   y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps),  in fp32, rounded once per output
//   dx = rstd (g - n mean(g n)) + dsum,  g = dy w, n = s rstd;  dw = sum over rows of dy n
// Bound by HBM: each value is read once (a row stays in registers between the sum and the outputs)
// and each output written once.  A row is cut into segments of 256 values, one or more per warp
// (`V`); a segment's sum is a warp's, and the segments' sums are added in one order, so a row's
// results do not depend on the other rows or on how many warps share it.
#include <atomic>

#include "fp8.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxSegs = 64;  // cols <= 16384
constexpr int kStreamThreads = 512;

struct NormArgs {
  const void *x, *residual, *w;
  void *sum, *out;
  uint8_t* q;
  float *scales, *rstd;
  int64_t rows, x_stride;
  int cols, W, w_f32;  // W: warps per row
  float eps;
};

template <int DT>
__device__ __forceinline__ void to_f32(const Raw8<typename In<DT>::T>& r, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 x = get2<DT>(r, j);
    f[j] = x.x;
    f[j + 1] = x.y;
  }
}
// x + r, rounded to the type (written in pairs of values the norm took 178 us where it takes 168)
template <int DT>
__device__ __forceinline__ void add_to(Raw8<typename In<DT>::T>& x, const Raw8<typename In<DT>::T>& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x.v[j] = In<DT>::of(In<DT>::f32(x.v[j]) + In<DT>::f32(r.v[j]));
}

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
    to_f32<DT>(load_seg<VEC>(static_cast<const T*>(w) + c0, cols - c0, lane), f);
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

// The sum over a row of its segments' per-lane sums v: a warp's for each segment, then the segments'
// in one order, whatever V and W are.  With several warps per row all threads synchronise once; the
// caller alternates between two arrays `part`.
template <int V>
__device__ __forceinline__ float row_total(float (&v)[V], float* part, int w0, int W, int segs, int lane) {
  // The sums of several segments at once: a step of 16 lanes leaves segment 2 i to the lanes below 16
  // and 2 i + 1 to the others, a step of 8 then halves these; every sum is formed in warp_sum's order.
  const bool hi = lane & 16, second = lane & 8;
  float u = v[0];
  if constexpr (V == 1) {
    u += __shfl_xor_sync(0xFFFFFFFFu, u, 16);
    u += __shfl_xor_sync(0xFFFFFFFFu, u, 8);
  } else {
    u = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? v[0] : v[1], 16);
    if constexpr (V == 4) {
      const float t = (hi ? v[3] : v[2]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? v[2] : v[3], 16);
      u = (second ? t : u) + __shfl_xor_sync(0xFFFFFFFFu, second ? u : t, 8);
    } else {
      u += __shfl_xor_sync(0xFFFFFFFFu, u, 8);
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
  const int i = V == 1 ? 0 : V == 2 ? hi : 2 * second + hi;  // the segment whose sum this lane has
  if (W == 1) {  // the order of sum_parts: one segment to a lane
    u = __shfl_sync(0xFFFFFFFFu, u, V == 1 ? 0 : V == 2 ? (lane & 1) * 16 : (lane & 1) * 16 + (lane & 2) * 4);
    return warp_sum(lane < V ? u : 0.0f);
  }
  if ((lane & (V == 1 ? 31 : V == 2 ? 15 : 7)) == 0 && w0 + i * W < segs) part[w0 + i * W] = u;
  __syncthreads();
  return sum_parts(part, segs, lane);
}

// The sum of eight squares, every kernel's in this order.
__device__ __forceinline__ float squares(const float (&s)[8]) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) fma2(a, b, s[j], s[j + 1], s[j], s[j + 1]);
  return a + b;
}

// The outputs of a warp's segments (the i-th from column c0 + i step on): y = s rstd w in the type and in
// 8 bits.
template <int DT, int V, bool VEC>
__device__ __forceinline__ void emit(const NormArgs& a, int64_t row, int c0, int step, int lane,
                                     float (&y)[V][8], float rstd, const float (&w)[V][8]) {
  using T = typename In<DT>::T;
  const int64_t kp = fp8_cols(a.cols);
  uint8_t* q = a.q + row * kp;
  float* scales = a.scales + row * (kp / 128);
  uint32_t m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = c0 + i * step;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      mul2(y[i][j], y[i][j + 1], rstd, rstd);
      mul2(y[i][j], y[i][j + 1], w[i][j], w[i][j + 1]);
    }
    if (a.out && c < a.cols) {
      Raw8<T> o;
#pragma unroll
      for (int j = 0; j < 8; j += 2) set2<DT>(o, j, y[i][j], y[i][j + 1]);
      store_seg<VEC>(static_cast<T*>(a.out) + row * a.cols + c, a.cols - c, lane, o);
    }
    if constexpr (VEC) m[i] = amax8(y[i]);
    else if (a.q && c < a.cols)
      quantize_seg(y[i], q + c, scales + c / 128, static_cast<int>(kp - c < kSeg ? kp - c : kSeg), lane);
  }
  if constexpr (VEC) {
    if (!a.q) return;
    const Scales<V> s(m, lane);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * step + 8 * lane;
      if (c < kp) *reinterpret_cast<uint2*>(q + c) = codes8(y[i], s.inv[i]);
    }
    const int b = (c0 + s.which(lane) * step) / 128 + (lane >> 4);
    if (s.stores(lane) && b < kp / 128) scales[b] = s.scale;
  }
}

// One row per CTA of W warps, or (W = 1) a row per warp.
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(1024, V == 1 ? 2 : 1)
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
      add_to<DT>(s[i], v[i]);
      store_seg<VEC>(static_cast<T*>(a.sum) + at + c0, a.cols - c0, lane, s[i]);
    }
  }
  float sq[V], y[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    to_f32<DT>(s[i], y[i]);
    sq[i] = squares(y[i]);
  }
  const float total = row_total<V>(sq, part, w0, a.W, segs, lane);
  const float rstd = __frsqrt_rn(total / static_cast<float>(a.cols) + a.eps);
  if (a.rstd && w0 == 0 && lane == 0) a.rstd[row] = rstd;
  float w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) load_weights<DT, VEC>(a.w, a.w_f32, (w0 + i * a.W) * kSeg, a.cols, lane, w[i]);
  emit<DT, V, VEC>(a, row, w0 * kSeg, a.W * kSeg, lane, y, rstd, w);
}

// ---- many rows that start on 16 bytes.  Persistent CTAs; the next kAhead rows are on their way to
// shared memory (cp.async, every thread its own values, so nothing is waited for but the thread's own
// copies) while a row is normalised.  The weights stay in registers.  16384 x 7168 bf16 with
// residual and both outputs: 168 us, 6.3 TB/s; without the residual 129 us, 4.6 TB/s, bound by issuing.
constexpr int kAhead = 2;
// A thread's places: kAhead rows of `tensors` tensors of V segments, 16-byte pieces a CTA apart.
template <int DT, int V>
struct Ring {
  static constexpr int kPieces = 8 * sizeof(typename In<DT>::T) / 16;
  uint4* base;
  int tensors;
  __device__ __forceinline__ uint4* at(int slot, int t, int i) const {
    return base + ((slot * tensors + t) * V + i) * kPieces * blockDim.x;
  }
  __device__ __forceinline__ void copy(int slot, int t, int i, const typename In<DT>::T* src) const {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      cp_async_16(smem_u32(at(slot, t, i) + k * blockDim.x), reinterpret_cast<const char*>(src) + 16 * k);
  }
  __device__ __forceinline__ Raw8<typename In<DT>::T> get(int slot, int t, int i) const {
    Raw8<typename In<DT>::T> r;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) reinterpret_cast<uint4*>(&r)[k] = at(slot, t, i)[k * blockDim.x];
    return r;
  }
};
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int DT, int V>
__global__ void __launch_bounds__(kStreamThreads, V == 4 ? 1 : 2) rmsnorm_stream_kernel(const NormArgs a) {
  using T = typename In<DT>::T;
  constexpr int D = kAhead;
  __shared__ float part[2][kMaxSegs];
  extern __shared__ uint4 ring_mem[];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = a.W == 1;
  const int w0 = alone ? 0 : warp;
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const int64_t first = alone ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  const int64_t step = alone ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
  const Ring<DT, V> ring{ring_mem + threadIdx.x, a.residual ? 2 : 1};
  const auto fetch = [&](int64_t row, int slot) {
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (w0 + i * a.W) * kSeg + 8 * lane;
        if (c < a.cols) {
          ring.copy(slot, 0, i, static_cast<const T*>(a.x) + row * a.x_stride + c);
          if (a.residual) ring.copy(slot, 1, i, static_cast<const T*>(a.residual) + row * a.cols + c);
        }
      }
    }
    cp_async_close();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(first + d * step, d);
  float w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) load_weights<DT, true>(a.w, a.w_f32, (w0 + i * a.W) * kSeg, a.cols, lane, w[i]);
  int turn = 0, slot = 0;
  for (int64_t row = first; row < a.rows; row += step, turn ^= 1) {
    cp_async_wait<D - 1>();
    float s[V][8], sq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = 0.0f;
      if (c0 + 8 * lane < a.cols) {
        Raw8<T> x = ring.get(slot, 0, i);
        if (a.residual) {
          add_to<DT>(x, ring.get(slot, 1, i));
          store_seg<true>(static_cast<T*>(a.sum) + row * a.cols + c0, a.cols - c0, lane, x);
        }
        to_f32<DT>(x, s[i]);
      }
      sq[i] = squares(s[i]);
    }
    fetch(row + D * step, slot);
    if (++slot == D) slot = 0;
    const float total = row_total<V>(sq, part[turn], w0, a.W, segs, lane);
    const float rstd = __frsqrt_rn(total / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && w0 == 0 && lane == 0) a.rstd[row] = rstd;
    emit<DT, V, true>(a, row, w0 * kSeg, a.W * kSeg, lane, s, rstd, w);
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

// The gradient's sums over eight values: n = s rstd first, which is of the order of one whatever the row's
// size is, so that no sum leaves fp32's range where the gradients do not (sums of dy s,
// an instruction a pair less and 1 % faster, did for rows of 1e17 with dy of 1e20, or of 1e-16 with 1e-25).
// <dy n, w> is returned, and dy n goes into the columns' sums.
template <int DT>
__device__ __forceinline__ float grad_sums(const Raw8<typename In<DT>::T>& s, const Raw8<typename In<DT>::T>& dy,
                                           const float (&w)[8], float rstd, float (&dw)[8]) {
  float p = 0.0f, q = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 a = get2<DT>(s, j), d = get2<DT>(dy, j);
    float n = a.x, m = a.y;
    mul2(n, m, rstd, rstd);
    fma2(dw[j], dw[j + 1], d.x, d.y, n, m);
    mul2(n, m, d.x, d.y);
    fma2(p, q, n, m, w[j], w[j + 1]);
  }
  return p + q;
}
// What a row's n are subtracted with, from its total <dy n, w>.
__device__ __forceinline__ float grad_factor(float total, float rstd, int cols) {
  return rstd * (total / static_cast<float>(cols));
}
// dx = dsum + dy (rstd w) - n c, n = s rstd
template <int DT>
__device__ __forceinline__ Raw8<typename In<DT>::T> grad_out(const Raw8<typename In<DT>::T>& s,
                                                             const Raw8<typename In<DT>::T>& dy, const float (&w)[8],
                                                             float rstd, float c, const float (&dsum)[8]) {
  Raw8<typename In<DT>::T> o;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 a = get2<DT>(s, j), d = get2<DT>(dy, j);
    float n0 = a.x, n1 = a.y;
    mul2(n0, n1, rstd, rstd);
    set2<DT>(o, j, fmaf(-c, n0, fmaf(d.x, rstd * w[j], dsum[j])),
             fmaf(-c, n1, fmaf(d.y, rstd * w[j + 1], dsum[j + 1])));
  }
  return o;
}

// A CTA's sums of dy n to its row of `part`; with a row per warp through `sums` [warps][cols].
template <int V, bool VEC>
__device__ __forceinline__ void flush_dw(const NormGradArgs& a, const float (&dw)[V][8], float* sums, int w0,
                                         int lane) {
  if (!a.part) return;
  const bool alone = a.W == 1;
  const int warp = threadIdx.x >> 5;
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

// Each CTA (W = 1: each warp) walks over rows and keeps its columns' sums of dy n in registers; a
// second kernel adds the CTAs' sums in their order.  The gradient of the weights is bitwise
// reproducible on one device; it depends on the number of CTAs.
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(1024)
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
      dot[i] = grad_sums<DT>(s[i], dy[i], w, rstd, dw[i]);
    }
    const float c = grad_factor(row_total<V>(dot, part[turn], w0, a.W, segs, lane), rstd, a.cols);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      float w[8], v[8] = {};
      load_weights<DT, VEC>(a.w, a.w_f32, c0, a.cols, lane, w);
      if (a.dsum) to_f32<DT>(ds[i], v);
      store_seg<VEC>(static_cast<T*>(a.dx) + at + c0, a.cols - c0, lane, grad_out<DT>(s[i], dy[i], w, rstd, c, v));
    }
  }
  flush_dw<V, VEC>(a, dw, sums, w0, lane);
}

// The same with the next rows on their way (as in rmsnorm_stream_kernel): dy, s and dsum are read from
// shared memory where they are used.  8192 x 4096 bf16 with dsum: 52 us, 5.2 TB/s, the second kernel's
// 4 among them; three rows ahead leave an SM two CTAs instead of four and took 73 us where two took 56.
// Bound by issuing (68 % of all slots) and by each row's one synchronisation.
template <int DT, int V>
__global__ void __launch_bounds__(kStreamThreads, V == 4 ? 1 : 2)
    rmsnorm_backward_stream_kernel(const NormGradArgs a) {
  using T = typename In<DT>::T;
  constexpr int D = kAhead;
  __shared__ float part[2][kMaxSegs];
  extern __shared__ uint4 ring_mem[];  // and, with a row per warp, their sums at the end
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = a.W == 1;
  const int w0 = alone ? 0 : warp;
  const int segs = (a.cols + kSeg - 1) / kSeg;
  const int64_t first = alone ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  const int64_t step = alone ? static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) : gridDim.x;
  const Ring<DT, V> ring{ring_mem + threadIdx.x, a.dsum ? 3 : 2};
  const auto fetch = [&](int64_t row, int slot) {
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (w0 + i * a.W) * kSeg + 8 * lane;
        const int64_t at = row * a.cols + c;
        if (c < a.cols) {
          ring.copy(slot, 0, i, static_cast<const T*>(a.s) + at);
          ring.copy(slot, 1, i, static_cast<const T*>(a.dy) + at);
          if (a.dsum) ring.copy(slot, 2, i, static_cast<const T*>(a.dsum) + at);
        }
      }
    }
    cp_async_close();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(first + d * step, d);
  float w[V][8], dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    load_weights<DT, true>(a.w, a.w_f32, (w0 + i * a.W) * kSeg, a.cols, lane, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0, slot = 0;
  for (int64_t row = first; row < a.rows; row += step, turn ^= 1) {
    const float rstd = a.rstd[row];
    cp_async_wait<D - 1>();
    float dot[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dot[i] = 0.0f;
      if ((w0 + i * a.W) * kSeg + 8 * lane < a.cols) {
        const Raw8<T> s = ring.get(slot, 0, i), dy = ring.get(slot, 1, i);
        dot[i] = grad_sums<DT>(s, dy, w[i], rstd, dw[i]);
      }
    }
    const float c = grad_factor(row_total<V>(dot, part[turn], w0, a.W, segs, lane), rstd, a.cols);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c0 = (w0 + i * a.W) * kSeg;
      if (c0 + 8 * lane < a.cols) {
        const Raw8<T> s = ring.get(slot, 0, i), dy = ring.get(slot, 1, i);
        float v[8] = {};
        if (a.dsum) to_f32<DT>(ring.get(slot, 2, i), v);
        store_seg<true>(static_cast<T*>(a.dx) + row * a.cols + c0, a.cols - c0, lane,
                        grad_out<DT>(s, dy, w[i], rstd, c, v));
      }
    }
    fetch(row + D * step, slot);
    if (++slot == D) slot = 0;
  }
  cp_async_wait<0>();
  flush_dw<V, true>(a, dw, reinterpret_cast<float*>(ring_mem + static_cast<size_t>(D) * ring.tensors * V *
                                                                  Ring<DT, V>::kPieces * blockDim.x), w0, lane);
}

// dw[c] = sum over n partial rows: 32 columns a cluster of C CTAs, whose warps take every C * kSumWarps-th
// row; the sums of a CTA's warps and then of the CTAs are added in order.  Eight CTAs where all clusters
// fit the SMs at once, four beyond: the gradient of 2048 x 2048 bf16 takes 13.4 and 14.6 us, of
// 8192 x 7168 91.6 and 88.3 (one CTA of 32 warps: 2 us more than eight of them at 2048 x 2048).
constexpr int kSumWarps = 8;
template <int C>
__global__ void __cluster_dims__(1, C, 1) __launch_bounds__(32 * kSumWarps)
    rmsnorm_dweight_kernel(const float* __restrict__ part, int n, int cols, float* __restrict__ dw) {
  __shared__ float sums[kSumWarps][32];
  __shared__ uint32_t all[C][32];  // rank 0's: every CTA's
  cluster_sync_all();  // rank 0 runs: its shared memory can be written
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int r = rank * kSumWarps + warp; r < n; r += C * kSumWarps)
      v += part[static_cast<int64_t>(r) * cols + c];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) v += sums[i][lane];
    st_shared_cluster_u32(mapa_shared(smem_u32(&all[rank][lane]), 0), __float_as_uint(v));
  }
  cluster_sync_all();
  if (rank == 0 && warp == 0 && c < cols) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) v += __uint_as_float(all[i][lane]);
    dw[c] = v;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known_dtype(int dt) {
  return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16 || dt == MOE_DTYPE_F32;
}
int64_t dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// How rows are cut: segments per warp, warps per row, threads of a CTA (a row, or kAloneWarps rows of
// one warp each).
//   kStream  16-bit rows that start on 16 bytes, more of them than SMs: two segments a warp, four beyond
//            32 segments.  (16384 x 7168 bf16 with residual and both outputs 168 us, 211 as kFew; the
//            gradient of 8192 x 4096 52 us, 69 as kFew.  fp32, 8192 x 4096: 120 us, 88 as kFew, the
//            gradient 148 and 116, since an SM then holds few rows.)
//   kFew     others that start on 16 bytes: a row over as many warps as it has segments, up to 32
//   kAny     rows that do not: the same cut (16384 x 1925 fp32 58 us, 4.9 TB/s; bf16 60 us, 2.6 TB/s, bound
//            by one value an instruction)
enum Path { kStream, kFew, kAny };
struct Shape {
  int v, W, threads;
};
constexpr int kAloneWarps = 8;
constexpr Shape shape_of(Path path, int cols) {
  const int segs = (cols + kSeg - 1) / kSeg;
  const int most = path != kStream ? (segs > 32 ? 2 : 1) : segs > 32 ? 4 : 2;
  Shape s{1, 0, 0};
  while (s.v < segs && s.v < most) s.v *= 2;
  s.W = (segs + s.v - 1) / s.v;
  s.threads = 32 * (s.W == 1 ? kAloneWarps : s.W);
  return s;
}
// Shared memory of the gradient's rows of one warp each: a CTA's sums by column, at most 16 KB beside a
// stream's ring.  The other kernels' is not asked for beforehand, so it has to stay below 48 KB.
constexpr size_t sums_bytes(const Shape& s, int cols) {
  return s.W == 1 ? static_cast<size_t>(kAloneWarps) * cols * 4 : 0;
}
constexpr size_t most_sums(Path path) {
  size_t most = 0;
  for (int cols = kSeg; cols <= kMaxSegs * kSeg; cols += kSeg) {  // a cut's widest rows
    const size_t n = sums_bytes(shape_of(path, cols), cols);
    if (n > most) most = n;
  }
  return most;
}
constexpr size_t kMostSums = 16384;
static_assert(most_sums(kStream) <= kMostSums, "");
static_assert(most_sums(kFew) <= 40960 && most_sums(kAny) <= 40960, "launched without being allowed more");
constexpr size_t kMostRing = 110000;  // two CTAs share an SM's memory
size_t ring_bytes(const Shape& s, int tensors) {
  return static_cast<size_t>(kAhead) * tensors * s.v * 16 * s.threads;
}
Path path_of(int64_t rows, int cols, int size, int tensors, bool vec, int sms) {
  if (!vec) return kAny;
  return size == 2 && rows > sms && ring_bytes(shape_of(kStream, cols), tensors) <= kMostRing ? kStream : kFew;
}
int64_t units(int64_t rows, const Shape& s) { return s.W == 1 ? (rows + kAloneWarps - 1) / kAloneWarps : rows; }
// CTAs that walk over rows: as many as make 32 warps an SM, fewer where shared memory holds fewer.
int64_t walkers(int64_t rows, const Shape& s, size_t smem, int sms) {
  int64_t per_sm = 1024 / s.threads;
  if (per_sm > 16) per_sm = 16;
  if (smem > 0 && per_sm > static_cast<int64_t>(2 * kMostRing / smem))
    per_sm = static_cast<int64_t>(2 * kMostRing / smem);
  if (per_sm < 1) per_sm = 1;
  const int64_t n = units(rows, s);
  return n < per_sm * sms ? n : per_sm * sms;
}
int64_t most_walkers(int64_t rows, int cols, int sms) {
  int64_t most = 0;
  for (Path path : {kStream, kFew, kAny}) {
    const int64_t n = walkers(rows, shape_of(path, cols), 0, sms);
    if (n > most) most = n;
  }
  return most;
}
// Allows a kernel its dynamic shared memory (once per device).
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(done.load(std::memory_order_acquire) & bit)) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kMostRing + kMostSums));
    if (st != cudaSuccess) return st;
    done.fetch_or(bit, std::memory_order_release);
  }
  return cudaSuccess;
}

template <int DT, int V>
cudaError_t launch_norm(const NormArgs& a, Path path, const Shape& s, int sms, cudaStream_t st) {
  if constexpr (DT != MOE_DTYPE_F32)
    if (path == kStream) {
      static std::atomic<unsigned long long> done{0ull};
      const cudaError_t e = allow_smem(rmsnorm_stream_kernel<DT, V>, done);
      if (e != cudaSuccess) return e;
      const size_t smem = ring_bytes(s, a.residual ? 2 : 1);
      return launch_pdl(rmsnorm_stream_kernel<DT, V>, dim3(static_cast<unsigned>(walkers(a.rows, s, smem, sms))),
                        dim3(s.threads), smem, st, a);
    }
  if constexpr (V <= 2) {
    const dim3 grid(static_cast<unsigned>(units(a.rows, s))), block(s.threads);
    return path == kFew ? launch_pdl(rmsnorm_kernel<DT, V, true>, grid, block, 0, st, a)
                        : launch_pdl(rmsnorm_kernel<DT, V, false>, grid, block, 0, st, a);
  }
  return cudaErrorInvalidValue;
}
template <int DT>
cudaError_t launch_norm(const NormArgs& a, Path path, const Shape& s, int sms, cudaStream_t st) {
  return s.v == 1   ? launch_norm<DT, 1>(a, path, s, sms, st)
         : s.v == 2 ? launch_norm<DT, 2>(a, path, s, sms, st)
                    : launch_norm<DT, 4>(a, path, s, sms, st);
}
// *ctas: rows of partial sums that the launch leaves in a.part
template <int DT, int V>
cudaError_t launch_grad(const NormGradArgs& a, Path path, const Shape& s, int sms, int* ctas, cudaStream_t st) {
  const size_t sums = sums_bytes(s, a.cols);
  const size_t smem = sums + (path == kStream ? ring_bytes(s, a.dsum ? 3 : 2) : 0);
  *ctas = static_cast<int>(walkers(a.rows, s, smem, sms));
  const dim3 grid(static_cast<unsigned>(*ctas)), block(s.threads);
  if constexpr (DT != MOE_DTYPE_F32)
    if (path == kStream) {
      static std::atomic<unsigned long long> done{0ull};
      const cudaError_t e = allow_smem(rmsnorm_backward_stream_kernel<DT, V>, done);
      return e != cudaSuccess ? e : launch_pdl(rmsnorm_backward_stream_kernel<DT, V>, grid, block, smem, st, a);
    }
  if constexpr (V <= 2)
    return path == kFew ? launch_pdl(rmsnorm_backward_kernel<DT, V, true>, grid, block, smem, st, a)
                        : launch_pdl(rmsnorm_backward_kernel<DT, V, false>, grid, block, smem, st, a);
  return cudaErrorInvalidValue;
}
template <int DT>
cudaError_t launch_grad(const NormGradArgs& a, Path path, const Shape& s, int sms, int* ctas, cudaStream_t st) {
  return s.v == 1   ? launch_grad<DT, 1>(a, path, s, sms, ctas, st)
         : s.v == 2 ? launch_grad<DT, 2>(a, path, s, sms, ctas, st)
                    : launch_grad<DT, 4>(a, path, s, sms, ctas, st);
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
  const int sms = num_sms_of_current_device();
  const Path path = path_of(rows, cols, size, residual ? 2 : 1, vec, sms);
  const Shape s = shape_of(path, cols);
  NormArgs b = a;
  b.W = s.W;
  return cuda_status(dtype == MOE_DTYPE_BF16  ? launch_norm<MOE_DTYPE_BF16>(b, path, s, sms, stream)
                     : dtype == MOE_DTYPE_F16 ? launch_norm<MOE_DTYPE_F16>(b, path, s, sms, stream)
                                              : launch_norm<MOE_DTYPE_F32>(b, path, s, sms, stream));
}

size_t moe_rmsnorm_workspace_bytes(int64_t rows, int cols) {
  if (rows < 0 || cols < 1 || cols > kMaxSegs * kSeg || rows > INT32_MAX) return 0;
  const int64_t n = most_walkers(rows, cols, num_sms_of_current_device());
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
  const bool vec = cols % 8 == 0 && aligned16(dy) && aligned16(s) && aligned16(dsum) &&
                   aligned16(dx) && aligned16(weight);
  const Path path = path_of(rows, cols, size, dsum ? 3 : 2, vec, sms);
  const Shape sh = shape_of(path, cols);
  int ctas = 0;
  const NormGradArgs a{dy,   s,    weight, dsum, rstd, dx, dweight ? static_cast<float*>(ws) : nullptr,
                       rows, cols, sh.W,   weight_dtype == MOE_DTYPE_F32};
  cudaError_t st = dtype == MOE_DTYPE_BF16  ? launch_grad<MOE_DTYPE_BF16>(a, path, sh, sms, &ctas, stream)
                   : dtype == MOE_DTYPE_F16 ? launch_grad<MOE_DTYPE_F16>(a, path, sh, sms, &ctas, stream)
                                            : launch_grad<MOE_DTYPE_F32>(a, path, sh, sms, &ctas, stream);
  if (st == cudaSuccess && dweight) {
    const int groups = (cols + 31) / 32, ctas_per_sm = 2048 / (32 * kSumWarps);
    const bool eight = groups * 8 <= sms * ctas_per_sm;
    st = launch_pdl(eight ? rmsnorm_dweight_kernel<8> : rmsnorm_dweight_kernel<4>, dim3(groups, eight ? 8 : 4),
                    dim3(32 * kSumWarps), 0, stream, static_cast<const float*>(ws), ctas, cols, dweight);
  }
  return cuda_status(st);
}

}  // extern "C"
