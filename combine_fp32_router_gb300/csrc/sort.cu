// Tokens sorted by expert and back, with weights applied, and the gradients of both.
//   sort     pair p = (t, j) of expert e goes to row seg(e) + #{p' < p : e(p') = e}; seg(e) is a
//            multiple of 128 (the layout of the grouped products); rows[row] = x[t]
//   sort'    dx[t] = sum_j drows[pos[t, j]]
//   unsort   out[t] = sum_j gate[t, j] rows[pos[t, j]]
//   unsort'  drows[pos[t, j]] = gate[t, j] dout[t],  dgate[t, j] = <rows[pos[t, j]], dout[t]>
// in fp32, slots in order, rounded once.  Bound by HBM: a token's row is read once and written for
// each of its pairs, or the other way round.  Ranks come from ballots and prefix sums, never from
// the order of atomics, so every result is bitwise reproducible.  8192 tokens, 8 of 128 experts, 4096
// values bf16: sort 106 us, 5.7 TB/s, unsort and sort' 100, 6.1 TB/s, unsort' 187, 6.1 TB/s.
#include "fp8.cuh"
#include "internal.h"

namespace moe {

namespace {

// Pairs that every CTA of the one-launch form ranks by itself.  300 tokens of 8 pairs, 7168 bf16 each:
// 10.3 us, 23 in three launches; 1000 of 2048: 18 us, 12.7 in three.
constexpr int kSmallPairs = 4096;
constexpr int kChunk = 2048;       // pairs of a ranking CTA
constexpr int kThreads = 256;

// What is copied per pair: nv vectors of a row, and ns fp32 scales of it (0: none).
struct Payload {
  const void* x;
  void* rows;
  const float* xs;
  float* rs;
  int64_t nv;
  int ns;
};

// off[e]: first row of expert e, off[E]: rows in all, from the counts in cnt (both shared); by
// kThreads threads.
__device__ __forceinline__ void segment_starts(const int32_t* cnt, int32_t* off, int E) {
  __shared__ int32_t warp_sum_s[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = kMaxE / kThreads;
  int32_t v[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    v[i] = e < E ? (cnt[e] + 127) / 128 * 128 : 0;
    sum += v[i];
  }
  int32_t scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) warp_sum_s[warp] = scan;
  __syncthreads();
  int32_t at = scan - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum_s[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < E) off[e] = at;
    at += v[i];
    if (e == E - 1) off[E] = at;
  }
  __syncthreads();
}

// perm = -1 where no pair goes, by all warps of the grid.
__device__ __forceinline__ void clear_padding(const int32_t* cnt, const int32_t* off, int E,
                                              int32_t* perm, int64_t n_rows) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  for (int64_t e = w; e < E; e += warps)
    for (int r = off[e] + cnt[e] + lane; r < off[e + 1]; r += 32) perm[r] = -1;
  for (int64_t r = off[E] + w * 32 + lane; r < n_rows; r += warps * 32) perm[r] = -1;
}

// Copies vectors c .. end - 1 of a token's row (by `n` threads, c is this one's first) to the rows of
// its k pairs (those >= 0), and its scales.
template <typename V>
__device__ __forceinline__ void copy_row(const Payload& p, int64_t t, int k, const int32_t* rows, int64_t c,
                                         int64_t end, int i, int n, bool scales) {
  const V* src = static_cast<const V*>(p.x) + t * p.nv;
  V* dst = static_cast<V*>(p.rows);
  for (; c + 3 * n < end; c += 4 * n) {
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = src[c + u * n];
    for (int j = 0; j < k; ++j) {
      const int32_t r = rows[j];
      if (r < 0) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) dst[r * p.nv + c + u * n] = v[u];
    }
  }
  for (; c < end; c += n) {
    const V v = src[c];
    for (int j = 0; j < k; ++j)
      if (rows[j] >= 0) dst[rows[j] * p.nv + c] = v;
  }
  if (!scales) return;
  for (int s = i; s < p.ns; s += n) {
    const float v = p.xs[t * p.ns + s];
    for (int j = 0; j < k; ++j)
      if (rows[j] >= 0) p.rs[static_cast<int64_t>(rows[j]) * p.ns + s] = v;
  }
}

// One launch for up to kSmallPairs pairs: every CTA counts all of them, ranks its own tokens' pairs
// against the earlier ones and copies those tokens' rows.
template <typename V>
__global__ void __launch_bounds__(kThreads)
    sort_small_kernel(const int32_t* __restrict__ idx, int T, int k, int E, Payload p,
                      int32_t* __restrict__ counts, int32_t* __restrict__ perm,
                      int32_t* __restrict__ pos, int64_t n_rows, DevErr* err) {
  __shared__ int32_t cnt[kMaxE], off[kMaxE + 1], mine[kMaxK];
  __shared__ int16_t ex[kSmallPairs];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = T * k;
  // CTA 0, which alone records errors here, clears the record first
  if (blockIdx.x == 0 && tid == 0) *err = DevErr{};
  for (int e = tid; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads) {
    const int e = idx[i];
    const bool real = e >= 0 && e < E;
    if (!real && e != -1 && blockIdx.x == 0) set_error(err, MOE_ERR_DEVICE_BOUNDS, 300);
    ex[i] = static_cast<int16_t>(real ? e : -1);
    if (real) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  segment_starts(cnt, off, E);
  if (blockIdx.x == 0)
    for (int e = tid; e < E; e += kThreads) counts[e] = cnt[e];
  clear_padding(cnt, off, E, perm, n_rows);
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    __syncthreads();  // the previous token's `mine` has been read
    for (int j = warp; j < k; j += kThreads / 32) {
      const int q = t * k + j, e = ex[q];
      int rank = 0;
      for (int i = lane; i < q; i += 32) rank += ex[i] == e;
      rank = __reduce_add_sync(0xFFFFFFFFu, rank);
      if (lane == 0) {
        const int32_t row = e < 0 ? -1 : off[e] + rank;
        mine[j] = row;
        pos[q] = row;
        if (row >= 0) perm[row] = q;
      }
    }
    __syncthreads();
    copy_row<V>(p, t, k, mine, tid, p.nv, tid, kThreads, true);
  }
}

// Larger batches, first launch: each CTA ranks kChunk pairs among themselves (rank_of) and counts
// them by expert (hist [E][chunks]).
__global__ void __launch_bounds__(kThreads)
    sort_rank_kernel(const int32_t* __restrict__ idx, int64_t pairs, int E, int64_t chunks,
                     int32_t* __restrict__ hist, int32_t* __restrict__ rank_of, DevErr* err) {
  extern __shared__ int32_t wcnt[];  // [warps][E]
  constexpr int kWarps = kThreads / 32, kPer = kChunk / kThreads;
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && tid == 0) *err = DevErr{};  // (recorded into by the third launch)
  for (int i = tid; i < kWarps * E; i += kThreads) wcnt[i] = 0;
  __syncthreads();
  int32_t* cnt = wcnt + warp * E;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kChunk + warp * (32 * kPer) + lane;
  int e[kPer], rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = p0 + 32 * i;
    e[i] = p < pairs ? idx[p] : -1;
    if (e[i] < 0 || e[i] >= E) e[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e[i]);
    rank[i] = 0;
    if (e[i] >= 0) rank[i] = cnt[e[i]] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (e[i] >= 0 && lane == __ffs(peers) - 1) cnt[e[i]] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int x = tid; x < E; x += kThreads) {  // counts before each warp, and of the chunk
    int32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int32_t v = wcnt[w * E + x];
      wcnt[w * E + x] = sum;
      sum += v;
    }
    hist[x * chunks + blockIdx.x] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = p0 + 32 * i;
    if (p < pairs) rank_of[p] = e[i] < 0 ? -1 : cnt[e[i]] + rank[i];
  }
}

// Second: a warp per expert turns its chunks' counts into the counts before each chunk.
__global__ void __launch_bounds__(kThreads)
    sort_scan_kernel(int32_t* __restrict__ hist, int E, int64_t chunks, int32_t* __restrict__ counts) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (e >= E) return;
  int32_t* h = hist + e * chunks;
  int32_t sum = 0;
  for (int64_t c0 = 0; c0 < chunks; c0 += 32) {
    const int32_t own = c0 + lane < chunks ? h[c0 + lane] : 0;
    int32_t v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    if (c0 + lane < chunks) h[c0 + lane] = sum + v - own;
    sum += __shfl_sync(0xFFFFFFFFu, v, 31);
  }
  if (lane == 0) counts[e] = sum;
}

// Third: rows of the pairs, and the copies: a warp per token and part of its row (`parts` of `per`
// vectors; the first part's warp writes the indices and copies the scales).
template <typename V>
__global__ void __launch_bounds__(kThreads)
    sort_copy_kernel(const int32_t* __restrict__ idx, int64_t T, int k, int E, int64_t chunks,
                     const int32_t* __restrict__ hist, const int32_t* __restrict__ rank_of,
                     const int32_t* __restrict__ counts, Payload p, int parts, int per,
                     int32_t* __restrict__ perm, int32_t* __restrict__ pos, int64_t n_rows, DevErr* err) {
  __shared__ int32_t cnt[kMaxE], off[kMaxE + 1], rows_s[kThreads / 32][kMaxK];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < E; e += kThreads) cnt[e] = counts[e];
  __syncthreads();
  segment_starts(cnt, off, E);
  clear_padding(cnt, off, E, perm, n_rows);
  int32_t* rows = rows_s[warp];
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp; u < T * parts; u += warps) {
    const int64_t t = u / parts;
    const int part = static_cast<int>(u - t * parts);
    if (lane < k) {
      const int64_t q = t * k + lane;
      const int e = idx[q];
      int32_t row = -1;
      if (e >= 0 && e < E) row = off[e] + hist[e * chunks + q / kChunk] + rank_of[q];
      else if (e != -1) set_error(err, MOE_ERR_DEVICE_BOUNDS, 301);
      rows[lane] = row;
      if (part == 0) {
        pos[q] = row;
        if (row >= 0) perm[row] = static_cast<int32_t>(q);
      }
    }
    __syncwarp();
    const int64_t c0 = static_cast<int64_t>(part) * per;
    copy_row<V>(p, t, k, rows, c0 + lane, c0 + per < p.nv ? c0 + per : p.nv, lane, 32, part == 0);
    __syncwarp();
  }
}

struct BackArgs {
  const void *rows, *dout;  // dout: unsort' alone
  const float* gate;        // null: ones
  const int32_t* pos;
  void *out, *drows;
  float* dgate;
  int64_t T, n_rows;
  int k, d, per;  // per: segments of a warp's unit (unsort)
  DevErr* err;
};

// A lane's pair (lane < k): its row, -1 without one, and its weight.
__device__ __forceinline__ int32_t pair_row(const BackArgs& a, int64_t t, int lane, float* g, bool report) {
  int32_t row = -1;
  *g = 1.0f;
  if (lane < a.k) {
    row = a.pos[t * a.k + lane];
    if (a.gate) *g = a.gate[t * a.k + lane];
    if (row < -1 || row >= a.n_rows) {
      if (report) set_error(a.err, MOE_ERR_DEVICE_BOUNDS, 302);
      row = -1;
    }
  }
  return row;
}

// out[t] = sum_j g_j rows[pos_j]: a warp per token and `per` segments, KB rows' loads in flight.
template <int DT, int KB, bool VEC>
__global__ void __launch_bounds__(kThreads) unsort_kernel(const BackArgs a) {
  using T = typename In<DT>::T;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int segs = (a.d + kSeg - 1) / kSeg;
  const int upt = (segs + a.per - 1) / a.per;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       u < a.T * upt; u += warps) {
    const int64_t t = u / upt;
    const int s0 = static_cast<int>(u - t * upt) * a.per;
    float g;
    const int32_t row = pair_row(a, t, lane, &g, s0 == 0);
    for (int s = s0; s < s0 + a.per && s < segs; ++s) {
      const int c0 = s * kSeg, n = a.d - c0;
      float acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
      for (int j0 = 0; j0 < a.k; j0 += KB) {
        Raw8<T> v[KB];
        float gs[KB];
        int32_t rs[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          rs[j] = __shfl_sync(0xFFFFFFFFu, row, (j0 + j) & 31);
          gs[j] = __shfl_sync(0xFFFFFFFFu, g, (j0 + j) & 31);
          if (rs[j] >= 0)
            v[j] = load_seg<VEC>(static_cast<const T*>(a.rows) + static_cast<int64_t>(rs[j]) * a.d + c0, n, lane);
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (rs[j] >= 0) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float2 x = get2<DT>(v[j], i);
              fma2(acc[i], acc[i + 1], x.x, x.y, gs[j], gs[j]);
            }
          }
      }
      Raw8<T> o;
#pragma unroll
      for (int i = 0; i < 8; i += 2) set2<DT>(o, i, acc[i], acc[i + 1]);
      store_seg<VEC>(static_cast<T*>(a.out) + t * a.d + c0, n, lane, o);
    }
  }
}

// drows and dgate: a CTA per token; a warp's sums over its segments, then the warps' in order.
template <int DT, int KC, bool VEC>
__global__ void __launch_bounds__(kThreads) unsort_backward_kernel(const BackArgs a) {
  using T = typename In<DT>::T;
  constexpr int KB = KC < 8 ? KC : 8;
  __shared__ float part[kThreads / 32][KC];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int segs = (a.d + kSeg - 1) / kSeg;
  const int64_t t = blockIdx.x;
  float g;
  const int32_t row = pair_row(a, t, lane, &g, warp == 0);
  float acc[KC];
#pragma unroll
  for (int j = 0; j < KC; ++j) acc[j] = 0.0f;
  for (int s = warp; s < segs; s += W) {
    const int c0 = s * kSeg, n = a.d - c0;
    const Raw8<T> dy = load_seg<VEC>(static_cast<const T*>(a.dout) + t * a.d + c0, n, lane);
#pragma unroll
    for (int j0 = 0; j0 < KC; j0 += KB) {
      if (j0 >= a.k) break;
      Raw8<T> y[KB];
      int32_t rs[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        rs[j] = __shfl_sync(0xFFFFFFFFu, row, j0 + j);
        if (a.dgate && rs[j] >= 0)
          y[j] = load_seg<VEC>(static_cast<const T*>(a.rows) + static_cast<int64_t>(rs[j]) * a.d + c0, n, lane);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const float gj = __shfl_sync(0xFFFFFFFFu, g, j0 + j);
        if (rs[j] < 0) continue;
        Raw8<T> o;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 f = get2<DT>(dy, i);
          if (a.dgate) {
            const float2 v = get2<DT>(y[j], i);
            acc[j0 + j] = fmaf(v.y, f.y, fmaf(v.x, f.x, acc[j0 + j]));
          }
          set2<DT>(o, i, gj * f.x, gj * f.y);
        }
        store_seg<VEC, true>(static_cast<T*>(a.drows) + static_cast<int64_t>(rs[j]) * a.d + c0, n, lane, o);
      }
    }
  }
  if (!a.dgate) return;
#pragma unroll
  for (int j = 0; j < KC; ++j) {
    float v = acc[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) part[warp][j] = v;
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < a.k) {
    float v = 0.0f;
    for (int w = 0; w < W; ++w) v += part[w][threadIdx.x];
    a.dgate[t * a.k + threadIdx.x] = v;
  }
}

bool aligned_to(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known_dtype(int dt) {
  return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16 || dt == MOE_DTYPE_F32;
}
int64_t dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }
moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool sizes_ok(int64_t T, int k, int E) {
  return k <= kMaxK && E <= kMaxE && T <= (INT32_MAX - 128 * (static_cast<int64_t>(E) + 1)) / k;
}
int64_t bound_rows(int64_t T, int k, int E) {
  const int64_t pairs = T * k;
  return (pairs + 127 * (E < pairs ? E : pairs) + 127) / 128 * 128;
}
int64_t chunks_of(int64_t pairs) { return (pairs + kChunk - 1) / kChunk; }
size_t ws_bytes_of(int64_t T, int k, int E) {
  const int64_t words = T * k <= kSmallPairs ? 0 : chunks_of(T * k) * E + T * k;  // hist, rank_of
  return static_cast<size_t>(256 + (4 * words + 255) / 256 * 256);
}

template <typename V>
cudaError_t launch_sort(const int32_t* idx, int64_t T, int k, int E, const Payload& p, int32_t* counts,
                        int32_t* perm, int32_t* pos, int64_t n_rows, char* ws, int sms, cudaStream_t s) {
  auto* err = reinterpret_cast<DevErr*>(ws);
  const int64_t pairs = T * k;
  if (pairs <= kSmallPairs) {
    const int64_t g = T < 1 ? 1 : T < 4 * sms ? T : 4 * sms;
    return launch_pdl(sort_small_kernel<V>, dim3(static_cast<unsigned>(g)), dim3(kThreads), 0, s, idx,
                      static_cast<int>(T), k, E, p, counts, perm, pos, n_rows, err);
  }
  auto* hist = reinterpret_cast<int32_t*>(ws + 256);
  const int64_t chunks = chunks_of(pairs);
  int32_t* rank_of = hist + chunks * E;
  cudaError_t st = launch_pdl(sort_rank_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kThreads),
                              sizeof(int32_t) * (kThreads / 32) * E, s, idx, pairs, E, chunks, hist, rank_of, err);
  if (st == cudaSuccess)
    st = launch_pdl(sort_scan_kernel, dim3((E + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0,
                    s, hist, E, chunks, counts);
  // few tokens are cut into parts of 128 vectors or more, for 32 warps an SM
  int64_t parts = (32ll * sms + T - 1) / T;
  if (parts > p.nv / 128) parts = p.nv / 128;
  if (parts < 1) parts = 1;
  const int64_t per = (p.nv + parts - 1) / parts;
  const int64_t want = (T * parts + kThreads / 32 - 1) / (kThreads / 32), most = 8 * sms;
  if (st == cudaSuccess)
    st = launch_pdl(sort_copy_kernel<V>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kThreads), 0,
                    s, idx, T, k, E, chunks, hist, rank_of, counts, p, static_cast<int>(parts),
                    static_cast<int>(per), perm, pos, n_rows, err);
  return st;
}

template <int DT, bool VEC>
cudaError_t launch_unsort(BackArgs a, int sms, cudaStream_t s) {
  const int segs = (a.d + kSeg - 1) / kSeg;
  a.per = a.T * segs <= 64ll * sms ? 1 : 4;
  const int64_t units = a.T * ((segs + a.per - 1) / a.per), want = (units + kThreads / 32 - 1) / (kThreads / 32);
  const dim3 grid(static_cast<unsigned>(want < 65536 ? want : 65536)), block(kThreads);
  return a.k <= 2   ? launch_pdl(unsort_kernel<DT, 2, VEC>, grid, block, 0, s, a)
         : a.k <= 4 ? launch_pdl(unsort_kernel<DT, 4, VEC>, grid, block, 0, s, a)
                    : launch_pdl(unsort_kernel<DT, 8, VEC>, grid, block, 0, s, a);
}
template <int DT, bool VEC>
cudaError_t launch_unsort_backward(const BackArgs& a, cudaStream_t s) {
  const int segs = (a.d + kSeg - 1) / kSeg, W = segs < kThreads / 32 ? segs : kThreads / 32;
  const dim3 grid(static_cast<unsigned>(a.T)), block(32 * W);
  return a.k <= 4   ? launch_pdl(unsort_backward_kernel<DT, 4, VEC>, grid, block, 0, s, a)
         : a.k <= 8 ? launch_pdl(unsort_backward_kernel<DT, 8, VEC>, grid, block, 0, s, a)
                    : launch_pdl(unsort_backward_kernel<DT, 16, VEC>, grid, block, 0, s, a);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_sort_rows_bound(int64_t T, int k, int E) {
  return T < 0 || k < 1 || E < 1 || !sizes_ok(T, k, E) ? 0 : bound_rows(T, k, E);
}

size_t moe_sort_workspace_bytes(int64_t T, int E, int k) {
  return T < 0 || k < 1 || E < 1 || !sizes_ok(T, k, E) ? 0 : ws_bytes_of(T, k, E);
}

moe_status_t moe_sort_tokens(const void* x, int64_t row_bytes, const float* x_scales, int n_scales,
                             const int32_t* topk_idx, int64_t T, int k, int E, void* rows,
                             int64_t n_rows, float* rows_scales, int32_t* counts, int32_t* perm,
                             int32_t* pos, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (T < 0 || k < 1 || E < 1 || row_bytes < 1 || n_scales < 0) return MOE_ERR_INVALID_ARG;
  if (!sizes_ok(T, k, E) || row_bytes > (1 << 20) || n_scales > kMaxFp8Cols) return MOE_ERR_UNSUPPORTED;
  if (!counts || !ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || !aligned_to(counts, 4) ||
      !aligned_to(perm, 4) || !aligned_to(pos, 4) || !aligned_to(topk_idx, 4) ||
      !aligned_to(x_scales, 4) || !aligned_to(rows_scales, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !topk_idx || !rows || !perm || !pos)) return MOE_ERR_INVALID_ARG;
  if ((n_scales > 0) != (x_scales != nullptr) || (n_scales > 0) != (rows_scales != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (n_rows < bound_rows(T, k, E) || n_rows > INT32_MAX || (n_rows > 0 && !perm)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < ws_bytes_of(T, k, E)) return MOE_ERR_WORKSPACE;
  int64_t v = 16;  // bytes of the widest vector that every row of both sides starts on
  while (row_bytes % v != 0 || !aligned_to(x, v) || !aligned_to(rows, v)) v /= 2;
  const Payload p{x, rows, x_scales, rows_scales, row_bytes / v, n_scales};
  const auto run = v == 16  ? launch_sort<uint4>
                   : v == 8 ? launch_sort<uint2>
                   : v == 4 ? launch_sort<uint32_t>
                   : v == 2 ? launch_sort<uint16_t>
                            : launch_sort<uint8_t>;
  return cuda_status(run(topk_idx, T, k, E, p, counts, perm, pos, n_rows, static_cast<char*>(ws),
                         num_sms_of_current_device(), stream));
}

moe_status_t moe_unsort_tokens(const void* rows, int dtype, int64_t n_rows, const float* gate,
                               const int32_t* pos, int64_t T, int k, int d, void* out, void* err_word,
                               cudaStream_t stream) {
  if (!known_dtype(dtype) || T < 0 || k < 1 || d < 1 || n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (k > kMaxK || d > 65536 || T > INT32_MAX / k || n_rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int64_t size = dtype_bytes(dtype);
  if ((!rows && n_rows > 0) || !pos || !out || !err_word || !aligned_to(rows, size) ||
      !aligned_to(out, size) || !aligned_to(gate, 4) || !aligned_to(pos, 4) || !aligned_to(err_word, 16))
    return MOE_ERR_INVALID_ARG;
  BackArgs a{};
  a.rows = rows;
  a.gate = gate;
  a.pos = pos;
  a.out = out;
  a.T = T;
  a.n_rows = n_rows;
  a.k = k;
  a.d = d;
  a.err = static_cast<DevErr*>(err_word);
  const bool vec = d % 8 == 0 && aligned_to(rows, 16) && aligned_to(out, 16);
  const int sms = num_sms_of_current_device();
  const auto run = dtype == MOE_DTYPE_BF16
                       ? (vec ? launch_unsort<MOE_DTYPE_BF16, true> : launch_unsort<MOE_DTYPE_BF16, false>)
                   : dtype == MOE_DTYPE_F16
                       ? (vec ? launch_unsort<MOE_DTYPE_F16, true> : launch_unsort<MOE_DTYPE_F16, false>)
                       : (vec ? launch_unsort<MOE_DTYPE_F32, true> : launch_unsort<MOE_DTYPE_F32, false>);
  return cuda_status(run(a, sms, stream));
}

moe_status_t moe_sort_tokens_backward(const void* drows, int dtype, int64_t n_rows, const int32_t* pos,
                                      int64_t T, int k, int d, void* dx, void* err_word,
                                      cudaStream_t stream) {
  return moe_unsort_tokens(drows, dtype, n_rows, nullptr, pos, T, k, d, dx, err_word, stream);
}

moe_status_t moe_unsort_tokens_backward(const void* dout, const void* rows, int dtype, int64_t n_rows,
                                        const float* gate, const int32_t* pos, int64_t T, int k, int d,
                                        void* drows, float* dgate, void* err_word, cudaStream_t stream) {
  if (!known_dtype(dtype) || T < 0 || k < 1 || d < 1 || n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (k > kMaxK || d > 65536 || T > INT32_MAX / k || n_rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int64_t size = dtype_bytes(dtype);
  if (!dout || !pos || !err_word || (n_rows > 0 && !drows) || (dgate && (!gate || (n_rows > 0 && !rows))) ||
      !aligned_to(dout, size) || !aligned_to(rows, size) || !aligned_to(drows, size) ||
      !aligned_to(gate, 4) || !aligned_to(pos, 4) || !aligned_to(dgate, 4) || !aligned_to(err_word, 16))
    return MOE_ERR_INVALID_ARG;
  BackArgs a{};
  a.rows = rows;
  a.dout = dout;
  a.gate = gate;
  a.pos = pos;
  a.drows = drows;
  a.dgate = dgate;
  a.T = T;
  a.n_rows = n_rows;
  a.k = k;
  a.d = d;
  a.err = static_cast<DevErr*>(err_word);
  const bool vec = d % 8 == 0 && aligned_to(dout, 16) && aligned_to(drows, 16) &&
                   (!dgate || aligned_to(rows, 16));
  const auto run = dtype == MOE_DTYPE_BF16  ? (vec ? launch_unsort_backward<MOE_DTYPE_BF16, true>
                                                   : launch_unsort_backward<MOE_DTYPE_BF16, false>)
                   : dtype == MOE_DTYPE_F16 ? (vec ? launch_unsort_backward<MOE_DTYPE_F16, true>
                                                   : launch_unsort_backward<MOE_DTYPE_F16, false>)
                                            : (vec ? launch_unsort_backward<MOE_DTYPE_F32, true>
                                                   : launch_unsort_backward<MOE_DTYPE_F32, false>);
  return cuda_status(run(a, stream));
}

}  // extern "C"
