// Product of MXFP4 rows and MXFP4 expert weights on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4, one E8M0 scale per 32 values, fp32 accumulation):
//   out[r, n] = sum_k A[r, k] B[e(r)][n, k],  rows grouped by expert in 128-row segments.
//
// One persistent launch.  A tile is 128 weight rows (the M operand) x a block of up to 192
// activation rows of one expert (the N operand, so a block costs MMAs for the rows it has):
//   warp 0      producer: codes by 2-D TMA (128-byte swizzle), scale tiles by bulk copies
//   warp 1      one lane: scale tiles shared memory -> TMEM (tcgen05.cp), then the MMAs, which
//               the hardware runs in that order
//   warp 2      TMEM allocator
//   warps 4..7  epilogue: accumulator column = output row, lane = output column, so a warp
//               stores 32 neighbouring outputs of a row at a time
// The K order of every output is that of its stages, whatever the other rows are.
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

CUtensorMap make_map_u8(const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                        cudaError_t* st);

namespace {

// Device-side problems of the 4-bit product (a bounded wait that ran out, counts that do not
// fit the rows): first error since moe_gemm_fp4_get_error last read it.
__device__ DevErr g_gemm_err;

constexpr int kRows = 192;  // N of a tile: two 192-column accumulators + scales fill TMEM
constexpr int kStages = 5;
constexpr int kKStage = 256;                   // values of K per stage (128 bytes of codes)
constexpr uint32_t kABytes = 128 * 128;        // weight codes
constexpr uint32_t kBBytes = kRows * 128;      // activation codes
constexpr uint32_t kSfaBytes = 2 * kMxTileBytes;
constexpr uint32_t kSfbBytes = 4 * kMxTileBytes;  // up to two 128-row tiles
constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
constexpr uint32_t kSfCols = 24;               // TMEM columns of a stage's scales: 8 + 16
constexpr uint32_t kSfCol0 = 2 * kRows;
static_assert(kSfCol0 + kStages * kSfCols <= 512, "TMEM columns");
static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024 bytes");
constexpr int kBars = 2 * kStages + 5;
constexpr int kThreads = 256;

struct Params {
  const uint8_t* sa;  // scales of the activation rows
  const uint8_t* sb;  // scales of the weights, [E] arrays of sb_bytes
  const int32_t* counts;
  int64_t rows, sb_bytes;
  int N, kt, E, nt;   // outputs, 128-value K tiles, experts, 128-row weight tiles per expert
  int64_t ldo;
  void* out;
  uint64_t wait_ns;
  CUtensorMap mapA;      // weight codes, boxes of 128 rows
  CUtensorMap mapB[4];   // activation codes, boxes of 16, 64, 128 and 192 rows
};

constexpr size_t kTable = 2 * (kMaxE + 1) * sizeof(int32_t);
constexpr size_t kSmemBytes = kStages * kStageBytes + 1024 + 8 * kBars + 64 + kTable;
static_assert(kSmemBytes <= 232448, "fits the opt-in shared memory of a CTA (227 KB)");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
struct Tile {
  int e, row0, nvalid, n0;
};

// first_block[e], first_row[e]: blocks and rows before expert e (E + 1 entries each)
__device__ __forceinline__ Tile decode(const Params& p, const int32_t* first_block,
                                       const int32_t* first_row, int64_t tile) {
  const int b = static_cast<int>(tile / p.nt);
  int lo = 0, hi = p.E;  // the last expert with first_block[e] <= b
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first_block[mid] <= b) lo = mid;
    else hi = mid;
  }
  Tile t;
  t.e = lo;
  const int i = b - first_block[lo];
  t.row0 = first_row[lo] + i * kRows;
  const int cnt = p.counts ? p.counts[lo] : static_cast<int>(p.rows);
  t.nvalid = min(cnt - i * kRows, kRows);
  t.n0 = static_cast<int>(tile % p.nt) * 128;
  return t;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp4_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const uint32_t bars = base + kStages * kStageBytes;
  const auto full = [&](int s) { return bars + 8u * s; };
  const auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  const auto tfull = [&](int s) { return bars + 8u * (2 * kStages + s); };
  const auto tempty = [&](int s) { return bars + 8u * (2 * kStages + 2 + s); };
  const uint32_t drain = bars + 8u * (2 * kStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kStages * kStageBytes + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* first_block = reinterpret_cast<int32_t*>(tmem_slot + 4);
  int32_t* first_row = first_block + kMaxE + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  DevErr* err = &g_gemm_err;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull(s), 1);
      mbar_init(tempty(s), 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
    tma_prefetch_desc(&p.mapA);
  }
  if (warp == 2) tmem_alloc(smem_u32(tmem_slot), 512);
  griddep_wait();
  if (warp == 3) {  // the experts' first blocks and rows
    int nb = 0, nr = 0;
    bool bad = false;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < p.E) c = p.counts ? p.counts[e] : static_cast<int>(p.rows);
      bad |= c < 0 || c > p.rows;
      if (bad) c = 0;
      int b = (c + kRows - 1) / kRows, r = p.counts ? (c + 127) / 128 : 0;
      const int b_own = b, r_own = r;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int ub = __shfl_up_sync(0xFFFFFFFFu, b, o), ur = __shfl_up_sync(0xFFFFFFFFu, r, o);
        if (lane >= o) {
          b += ub;
          r += ur;
        }
      }
      if (e < p.E) {
        first_block[e] = nb + b - b_own;
        first_row[e] = (nr + r - r_own) * 128;
        // the last row that is read has to exist (the padding after it need not)
        bad |= static_cast<int64_t>(nr + r - r_own) * 128 + c > p.rows;
      }
      nb += __shfl_sync(0xFFFFFFFFu, b, 31);
      nr += __shfl_sync(0xFFFFFFFFu, r, 31);
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      first_block[p.E] = bad ? 0 : nb;  // no block at all when the counts do not fit
      if (bad) set_error(err, MOE_ERR_DEVICE_BOUNDS, 60);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t tiles = static_cast<int64_t>(first_block[p.E]) * p.nt;
  const int nks = (p.kt + 1) / 2;

  if (warp == 0) {
    uint32_t it = 0, s = 0, phase = 1;
    bool ok = true;
    for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      const Tile t = decode(p, first_block, first_row, tile);
      const int bi = t.nvalid <= 16 ? 0 : (t.nvalid <= 64 ? 1 : (t.nvalid <= 128 ? 2 : 3));
      const uint32_t bbytes = (bi == 0 ? 16 : (bi == 1 ? 64 : (bi == 2 ? 128 : kRows))) * 128;
      const CUtensorMap* mb = &p.mapB[bi];
      const int rt0 = t.row0 / 128, nsb = (t.row0 + t.nvalid - 1) / 128 - rt0 + 1;
      const uint8_t* sfa = p.sb + t.e * p.sb_bytes + static_cast<int64_t>(t.n0 / 128) * p.kt * kMxTileBytes;
      const uint8_t* sfb = p.sa + static_cast<int64_t>(rt0) * p.kt * kMxTileBytes;
      const uint8_t* sfb1 = sfb + static_cast<int64_t>(p.kt) * kMxTileBytes;
      const int wrow = t.e * p.N + t.n0;
      for (int ks = 0; ks < nks; ++ks, ++it) {
        if (it >= kStages) ok = warp_wait(empty(s), phase, abort_flag, err, 61, p.wait_ns);
        if (!ok) break;
        const uint32_t st = base + s * kStageBytes, ssf = st + kABytes + kBBytes;
        const uint32_t sfbytes = min(2, p.kt - 2 * ks) * kMxTileBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(full(s), kABytes + bbytes + sfbytes * (1 + nsb));
          tma_load_2d(st, &p.mapA, full(s), ks * 128, wrow);
          tma_load_2d(st + kABytes, mb, full(s), ks * 128, t.row0);
          bulk_load(ssf, sfa + 2 * ks * kMxTileBytes, sfbytes, full(s));
          bulk_load(ssf + kSfaBytes, sfb + 2 * ks * kMxTileBytes, sfbytes, full(s));
          if (nsb > 1)
            bulk_load(ssf + kSfaBytes + 2 * kMxTileBytes, sfb1 + 2 * ks * kMxTileBytes, sfbytes, full(s));
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // copies still in flight land before the CTA ends (only after an abort are there any that
    // the MMA warp has not waited for)
    if (*abort_flag)
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
        mbar_wait(full(i % kStages), (i / kStages) & 1, nullptr, err, 62, p.wait_ns);
  } else if (warp == 1) {
    uint32_t s = 0, phase = 0, n = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++n) {
      const Tile t = decode(p, first_block, first_row, tile);
      const uint32_t acc = n & 1, tacc = tmem + acc * kRows;
      if (n >= 2 && !warp_wait(tempty(acc), (n / 2 - 1) & 1, abort_flag, err, 63, p.wait_ns)) break;
      tc_fence_after();
      // the block may start in the middle of a scale tile (row 64 of it: column 2)
      const uint32_t sf_shift = (t.row0 % 128) / 32;
      const int nsb = (t.row0 + t.nvalid - 1) / 128 - t.row0 / 128 + 1;
      const uint32_t idesc = idesc_mxf4(128, (t.nvalid + 15) / 16 * 16);
      for (int ks = 0; ks < nks; ++ks) {
        ok = warp_wait(full(s), phase, abort_flag, err, 64, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = base + s * kStageBytes;
        const uint32_t ssf = st + kABytes + kBBytes;
        const uint32_t tsf = tmem + kSfCol0 + s * kSfCols;
        const int nkt = min(2, p.kt - 2 * ks);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i < nkt) {
              tmem_cp_scales(tsf + 4 * i, ssf + i * kMxTileBytes);
              tmem_cp_scales(tsf + 8 + 8 * i, ssf + kSfaBytes + i * kMxTileBytes);
              if (nsb > 1) tmem_cp_scales(tsf + 12 + 8 * i, ssf + kSfaBytes + (2 + i) * kMxTileBytes);
            }
          }
          const uint64_t da = smem_desc_sw128(st, 16, 1024);
          const uint64_t db = smem_desc_sw128(st + kABytes, 16, 1024);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t id = (j & 1) * 2;
            if (j < 2 * nkt)
              umma_mxf4(tacc, da + 2 * j, db + 2 * j, idesc | (id << 4) | (id << 29),
                        tsf + 4 * (j >> 1), tsf + 8 + 8 * (j >> 1) + sf_shift, ks > 0 || j > 0);
          }
          umma_commit(empty(s));
          if (ks == nks - 1) umma_commit(tfull(acc));
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (elect_one()) umma_commit(drain);  // every MMA issued is complete before TMEM is freed
    mbar_wait(drain, 0, nullptr, err, 65, p.wait_ns);
  } else if (warp >= 4) {
    const int q = warp - 4;
    uint32_t n = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++n) {
      const Tile t = decode(p, first_block, first_row, tile);
      const uint32_t acc = n & 1;
      if (!mbar_wait(tfull(acc), (n / 2) & 1, abort_flag, err, 66, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t tacc = tmem + acc * kRows + (static_cast<uint32_t>(32 * q) << 16);
      const int col = t.n0 + 32 * q + lane;
      for (int r0 = 0; r0 < t.nvalid; r0 += 32) {
        float a[16], b[16];
        tmem_ld16x2(tacc + r0, tacc + r0 + 16, a, b);
        if (r0 + 32 >= t.nvalid) {  // the last read of this accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty(acc));
        }
        if (col < p.N) {
          const int64_t at = static_cast<int64_t>(t.row0 + r0) * p.ldo + col;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = j < 16 ? a[j & 15] : b[j & 15];
            if (r0 + j < t.nvalid) {
              if constexpr (F32) static_cast<float*>(p.out)[at + j * p.ldo] = v;
              else static_cast<uint16_t*>(p.out)[at + j * p.ldo] = bf16_bits(v);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool F32>
cudaError_t launch(const Params& p, int grid, cudaStream_t s) {
  auto kern = gemm_fp4_kernel<F32>;
  static std::atomic<unsigned long long> attr_set_mask{0ull};
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(attr_set_mask.load(std::memory_order_acquire) & bit)) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmemBytes));
    if (st != cudaSuccess) return st;
    attr_set_mask.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, s, p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

// 2-D map of `rows` rows of `inner` bytes, 128-byte swizzle, boxes of 128 bytes x box_rows
// (bytes past the row's end and rows past the last are read as zeros).
CUtensorMap make_map_u8(const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                        cudaError_t* st) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  CUtensorMap m = {};
  auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {inner};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t ones[2] = {1, 1};
  if (!enc || enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    *st = cudaErrorInvalidValue;
  return m;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_gemm_fp4(const uint8_t* a, const uint8_t* a_scales, int64_t rows,
                          const int32_t* counts, const uint8_t* b, const uint8_t* b_scales, int E,
                          int N, int K, void* out, int out_dtype, cudaStream_t stream) {
  if (rows < 0 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (!counts && E != 1) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!a || !a_scales || !b || !b_scales || !out || !aligned16(a) || !aligned16(a_scales) ||
      !aligned16(b) || !aligned16(b_scales) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(counts) & 3) != 0)
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || N > kMaxFp4Cols || K > kMaxFp4Cols || rows > INT32_MAX - 256 ||
      static_cast<int64_t>(E) * N > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  const uint64_t inner = static_cast<uint64_t>(mx_cols(K) / 2);
  cudaError_t st = cudaSuccess;
  Params p = {};
  p.sa = a_scales;
  p.sb = b_scales;
  p.counts = counts;
  p.rows = rows;
  p.sb_bytes = mx_scale_bytes(N, K);
  p.N = N;
  p.kt = static_cast<int>(mx_cols(K) / 128);
  p.E = E;
  p.nt = (N + 127) / 128;
  p.ldo = N;
  p.out = out;
  p.wait_ns = wait_limit_ns();
  p.mapA = make_map_u8(b, inner, static_cast<uint64_t>(E) * N, 128, &st);
  const uint32_t boxes[4] = {16, 64, 128, kRows};
  for (int i = 0; i < 4; ++i)
    p.mapB[i] = make_map_u8(a, inner, static_cast<uint64_t>(rows), boxes[i], &st);
  const int sms = num_sms_of_current_device();
  if (st != cudaSuccess) return MOE_ERR_CUDA;
  const int64_t blocks = (rows + kRows - 1) / kRows + (counts ? E : 0);
  const int64_t tiles = blocks * p.nt;
  const int grid = static_cast<int>(tiles < sms ? tiles : sms);
  st = out_dtype == MOE_DTYPE_F32 ? launch<true>(p, grid, stream) : launch<false>(p, grid, stream);
  return st == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_gemm_fp4_get_error(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
  DevErr e = {}, none = {};
  if (cudaMemcpyFromSymbol(&e, g_gemm_err, sizeof(e)) != cudaSuccess) return MOE_ERR_CUDA;
  if (e.status != 0 && cudaMemcpyToSymbol(g_gemm_err, &none, sizeof(none)) != cudaSuccess)
    return MOE_ERR_CUDA;
  return static_cast<moe_status_t>(e.status);
}

}  // extern "C"
