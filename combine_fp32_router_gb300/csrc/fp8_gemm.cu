// Product of 8-bit rows and 8-bit expert weights with a scale per 128 values (format: fp8.cuh):
//   out[r, n] = sum_kb sa[r, kb] sb[e(r)][n / 128, kb] sum_{k in kb} A[r, k] B[e(r)][n, k],
// rows grouped by expert in 128-row segments, or one matrix.
//
// One persistent launch.  A tile is 256 x 256 on a CTA pair (cta_group::2: each CTA holds 128 rows
// and half of the weights) or 128 rows x 128 or 64, or 64 rows x 32 weight rows on one CTA.  The
// tensor cores (tcgen05.mma kind::f8f6f4) sum the 128 values of a block of K into TMEM; scales differ
// from block to block, so the sum of each block is taken out of TMEM, scaled and added to the tile's
// sums, which stay in registers:  acc = fma(sum, sa sb, acc), two values an instruction.  Every shape
// adds the same products in the same order, so a row's results do not depend on the other rows.
//
// 8192 x 7168 x 7168 takes 308 to 314 us in bf16, 2.7 PFLOP/s (335 call after call, at the power limit):
// twelve rounds of tiles, 32 KB a block of K into each SM, 71 GB/s.  With all sums and scales and three
// quarters of the MMAs left out it takes 266, 83 GB/s: most of it is bringing codes into the SMs, and 42
// us are sums and the MMAs' hand-over that no load covers.  One row of 7168 x 4096 takes 11 us, 7.6 and
// 4.1 with a half and none of K: 4 KB a block from HBM on 128 SMs, 4.3 TB/s.  Warps:
//   0..7    sums: lanes 32 (w % 4) .. of TMEM, half w / 4 of the columns; then the output
//   8       producer: codes by TMA (128-byte swizzle)
//   9, 10   MMAs, groups of blocks of K in turn: what one spends on waiting, committing and looping
//           (400 cycles a group) passes while the other's MMAs run; TMEM allocation
//   11      scales: sa sb of every row and 8 blocks of K at a time, to shared memory
// The summing warps take registers from the others: 128 sums and 64 values in flight.
#include <cuda.h>

#include <atomic>
#include <cstddef>
#include <cstdlib>
#include <mutex>

#include "fp8.cuh"
#include "internal.h"

namespace moe {

namespace {

// Device-side problems of the 8-bit product (a bounded wait that ran out, counts that do not fit
// the rows): first error since moe_gemm_fp8_get_error last read it.
__device__ DevErr g_gemm8_err;

// Reads and clears it in one step: an error that comes between the two would be lost.
__device__ int g_taken8_status;
__global__ void take_error_kernel() { g_taken8_status = atomicExch(&g_gemm8_err.status, 0); }

constexpr int kMaxStages = 32;
constexpr int kBufs = 2;
constexpr int kSumWarps = 8, kLoader = 8, kIssuer = 9, kScaler = 11;
constexpr int kThreads = 384;
// Registers of a thread: launched with 168 (65536 / 384, which ptxas gives to the launch bounds), of
// which the last four warps keep 88 and the others get 208.
constexpr int kLaunchRegs = 168, kSumRegs = 208, kOtherRegs = 88;
static_assert(2 * kSumRegs + kOtherRegs <= 3 * kLaunchRegs, "registers at launch");
constexpr int kBoxes = 5;  // box heights of the rows: 8, 16, 32, 64, 128
// The stages, and behind them each summing warp's place for outputs: 32 rows of 128 bytes, once or twice.
constexpr uint32_t kBufferBytes = 192 * 1024;
// Factors of 8 blocks of K at a time; rows of one block 132 words apart, so that four rows of eight
// blocks meet no bank twice.  Read from global memory by each summing lane for itself, the scales
// took a warp 210 cycles of the 512 of a block of K.
constexpr int kScaleBlocks = 8, kScaleRow = 132;

template <int NT, bool PAIR>
struct Cfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  // Rows of a CTA's MMAs.  Few columns go with few rows: 64 rows take 96 cycles a block of K with 32
  // columns, 128 take 160.  64 rows lie in lanes 0 .. 15 of each of the four quarters of TMEM.
  static constexpr int kM = NT == 32 ? 64 : 128;
  static constexpr int kRows = kM * kCtas;      // rows of a tile
  static constexpr int kLocalN = NT / kCtas;    // weight rows that a CTA loads
  static constexpr int kCols = NT / 2;          // columns of a warp's sums
  // Blocks of K between two arrivals of the summing warps, and at most per stage: an MMA warp's turn
  // (wait, issue, commit) takes 350 cycles, the MMAs of a block 160 with 32 columns, 256 with 128
  static constexpr int kG = NT == 32 ? 4 : NT == 256 ? 1 : 2;
  static constexpr uint32_t kTmemCols = kBufs * kG * NT;
  static constexpr uint32_t kOutBytes = PAIR ? 8192 : 4096;
  static constexpr uint32_t kRingBytes = kBufferBytes - kSumWarps * kOutBytes;
  static_assert(kTmemCols <= 512, "");
  static_assert(kRingBytes >= kBufs * kG * (kM + kLocalN) * 128, "the ring holds kBufs groups");
};

struct Params {
  const int32_t* counts;
  const float *sa, *sb;
  int64_t rows;
  int N, kt, E, nt, nb;  // outputs, blocks of K, experts, weight tiles and scale blocks per expert
  int stages, ks;        // stages, and blocks of K in one
  uint32_t abytes;       // place for the rows of a block of K
  int vec;               // output rows start on 32 (2), 16 (1) bytes or neither (0)
  int f32, tma_out;      // tma_out: rows of the output can be stored by TMA
  void* out;
  uint64_t wait_ns;
  uint32_t withhold;     // test hook: bit 0, 1: CTA 0, 1 loads nothing
  CUtensorMap mapB, mapA[kBoxes], mapOut;
};

// behind the stages (an MMA whose box has fewer than 128 rows reads up to 16 KB past its stage: what
// it finds there meets rows that are not stored)
struct Shared {
  alignas(16) float factors[2][2][kScaleBlocks][kScaleRow];  // slot, half of the columns
  int4 info[2];  // per slot: its tile's first row, valid rows and first column
  uint64_t bars[2 * kMaxStages + 2 * kBufs + 5];
  uint32_t tmem;
  int32_t abort_flag;
  uint32_t peer_issued;                          // fills issued by the peer
  uint32_t tx[kMaxStages], peer_tx[kMaxStages];  // bytes of the fill in a stage
  int32_t first_block[kMaxE + 1], first_row[kMaxE + 1], count[kMaxE];
};
constexpr size_t kSmemBytes = kBufferBytes + 1024 + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "fits the opt-in shared memory of a CTA (227 KB)");
static_assert(sizeof(Shared) >= 16384, "what a box of fewer than 128 rows leaves out can be read");

struct Tile {
  int e, row0, nvalid, n0;
  int box;  // index of the box height, the same on both CTAs of a pair
};

template <int NT, bool PAIR>
__device__ __forceinline__ Tile decode(const Params& p, const Shared& sh, uint32_t tile) {
  constexpr int R = Cfg<NT, PAIR>::kRows;
  const uint32_t nt = static_cast<uint32_t>(p.nt);
  const int b = static_cast<int>(tile / nt);
  int lo = 0, hi = p.E;  // the last expert with first_block[e] <= b
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sh.first_block[mid] <= b) lo = mid;
    else hi = mid;
  }
  Tile t;
  t.e = lo;
  const int i = b - sh.first_block[lo];
  t.row0 = sh.first_row[lo] + i * R;
  t.nvalid = min(sh.count[lo] - i * R, R);
  t.n0 = static_cast<int>(tile - b * nt) * NT;
  t.box = t.nvalid <= 8 ? 0 : t.nvalid <= 16 ? 1 : t.nvalid <= 32 ? 2 : t.nvalid <= 64 ? 3 : 4;
  return t;
}

__device__ __forceinline__ bool mbar_try_wait_relaxed(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 16 columns of this thread's lane, and the wait for them.
__device__ __forceinline__ void tmem_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_done(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Eight words to a place of its alignment (vec as in Params)
__device__ __forceinline__ void store8(uint32_t* o, int vec, const uint32_t (&w)[8]) {
  if (vec == 2) {
    st_v8(o, w);
  } else {
    st_v4(o, make_uint4(w[0], w[1], w[2], w[3]));
    st_v4(o + 4, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

// A warp's 16 sums of `n` rows (lane = row, from `row` on) to their columns col .. col + 15 (those
// below N).  Where rows do not start on 16 bytes they go through shared memory, so that lanes store
// neighbouring values.
__device__ __forceinline__ void store16(const Params& p, int64_t row, int n, int col, const float* acc,
                                        uint32_t* buf, int lane) {
  if (p.vec && col + 16 <= p.N) {
    if (lane >= n) return;
    const int64_t at = (row + lane) * p.N + col;
    uint32_t w[8];
    if (p.f32) {
      uint32_t* o = static_cast<uint32_t*>(p.out) + at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(acc[8 * h + i]);
        store8(o + 8 * h, p.vec, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
      store8(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at), p.vec, w);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i) buf[lane * 17 + i] = __float_as_uint(acc[i]);
  __syncwarp();
  const int c = lane & 15;
  if (col + c < p.N) {
#pragma unroll 8
    for (int r = lane >> 4; r < n; r += 2) {
      const int64_t at = (row + r) * p.N + col + c;
      if (p.f32) static_cast<uint32_t*>(p.out)[at] = buf[r * 17 + c];
      else static_cast<uint16_t*>(p.out)[at] = bf16_bits(__uint_as_float(buf[r * 17 + c]));
    }
  }
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint4 u) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w)
               : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// 16 bytes of output: W = 32: four sums in fp32, 64: eight in bf16
template <int W>
__device__ __forceinline__ uint4 pack16(const float* v) {
  if constexpr (W == 32)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}
// 128 bytes of each of a warp's 32 rows (W sums, from column col on) through shared memory as one
// TMA store, which leaves out columns past N: lanes storing their own rows take 32 memory lines an
// instruction.  16-byte pieces are swizzled as the tensor map has it.
template <int W>
__device__ __forceinline__ void store_tile(const Params& p, int row, int col, const float* acc, uint32_t buf,
                                           int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    st_shared_v4(buf + 128 * lane + 16 * (i ^ (lane & 7)), pack16<W>(acc + i * (W / 8)));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&p.mapOut, buf, col, row);
    bulk_commit();
  }
}

// The same for rows that start anywhere.  fp32: a row at a time.  bf16: eight lanes take a row, its
// 16-byte pieces where its place in memory has them, and value by value the 16 bytes before the first
// and behind the last of them.  8192 x 7161 x 2048: bf16 134 us, fp32 144, both 164 with 16 columns at a
// time as in store16; bf16 a row at a time in words of two: 182 (7168 columns, by TMA: 102 and 121).
template <int W>
__device__ __forceinline__ void store_rows(const Params& p, int64_t row, int n, int col, const float* acc,
                                           uint32_t buf, int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) st_shared_v4(buf + 128 * lane + 16 * (i ^ (lane & 7)), pack16<W>(acc + i * (W / 8)));
  __syncwarp();
  const auto word = [&](int r, uint32_t b) {  // the one at byte b of row r
    return ld_shared_u32(buf + 128 * r + ((b & ~15u) ^ 16 * (r & 7)) + (b & 12));
  };
  if constexpr (W == 32) {
    uint32_t* o = static_cast<uint32_t*>(p.out) + row * p.N + col + lane;
#pragma unroll 8
    for (int r = 0; r < n; ++r, o += p.N) *o = word(r, 4 * lane);
  } else {
    const int j = lane & 7;
    uint16_t* o = static_cast<uint16_t*>(p.out) + (row + (lane >> 3)) * p.N + col;
#pragma unroll 2
    for (int r = lane >> 3; r < n; r += 4, o += 4 * static_cast<int64_t>(p.N)) {
      const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(o)) & 15;
      if (j > 0) {
        uint32_t x[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) x[i] = word(r, min(((16 * j - off) & ~3u) + 4 * i, 124u));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 8 * (off & 2));
        st_v4(reinterpret_cast<char*>(o) + 16 * j - off, make_uint4(x[0], x[1], x[2], x[3]));
      }
      const int e = j < static_cast<int>(16 - off) / 2 ? j : 56 + j;
      o[e] = static_cast<uint16_t>(word(r, 2 * e) >> (16 * (e & 1)));
    }
  }
}

template <int NT, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp8_kernel(const __grid_constant__ Params p) {
  using C = Cfg<NT, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw + (base - raw) + kBufferBytes);
  const uint32_t S = static_cast<uint32_t>(p.stages);
  const uint32_t kb_bytes = p.abytes + C::kLocalN * 128, stage_bytes = p.ks * kb_bytes;
  const auto full = [&](uint32_t s) { return smem_u32(&sh.bars[s]); };
  const auto empty = [&](uint32_t s) { return smem_u32(&sh.bars[kMaxStages + s]); };
  const auto tfull = [&](uint32_t a) { return smem_u32(&sh.bars[2 * kMaxStages + a]); };
  const auto tempty = [&](uint32_t a) { return smem_u32(&sh.bars[2 * kMaxStages + kBufs + a]); };
  const auto sfull = [&](uint32_t i) { return smem_u32(&sh.bars[2 * kMaxStages + 2 * kBufs + i]); };
  const auto sempty = [&](uint32_t i) { return smem_u32(&sh.bars[2 * kMaxStages + 2 * kBufs + 2 + i]); };
  const uint32_t drain = smem_u32(&sh.bars[2 * kMaxStages + 2 * kBufs + 4]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&sh.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C::kCtas, units = gridDim.x / C::kCtas;
  DevErr* err = &g_gemm8_err;
  // the peer arrives on a pair's barriers too: those waits acquire at cluster scope
  const auto wait = [&](uint32_t bar, uint32_t parity, volatile int* ab, int site) {
    if constexpr (PAIR) return mbar_wait_cluster(bar, parity, ab, err, site, p.wait_ns);
    else return mbar_wait(bar, parity, ab, err, site, p.wait_ns);
  };
  const auto warp_wait = [&](uint32_t bar, uint32_t parity, int site) {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity, abort_flag, site)) != 0;
  };
  // factors pass between warps of one CTA
  const auto own_wait = [&](uint32_t bar, uint32_t parity, int site) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, err, site, p.wait_ns)) != 0;
  };
  // TMEM alone passes over tfull and tempty, ordered by the tcgen05 fences on both sides, so the first
  // look need not acquire: at cluster scope that took 5 % of the whole product.
  const auto tmem_wait = [&](uint32_t bar, uint32_t parity, int site) {
    if constexpr (PAIR)
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait_relaxed(bar, parity))) return true;
    return warp_wait(bar, parity, site);
  };

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(full(s), 1);  // rank 0's: its arming arrival and both CTAs' bytes
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), kSumWarps * C::kCtas);  // rank 0's: an arrival of every summing warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull(i), 1);
      mbar_init(sempty(i), kSumWarps);
    }
    mbar_init(drain, 2);
    fence_mbar_init();
    sh.abort_flag = 0;
    sh.peer_issued = 0u;
    tma_prefetch_desc(&p.mapB);
    if (p.tma_out) tma_prefetch_desc(&p.mapOut);
  }
  if (warp == kIssuer) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(&sh.tmem), C::kTmemCols);
    else tmem_alloc(smem_u32(&sh.tmem), C::kTmemCols);
  }
  griddep_wait();
  if (warp == kLoader) {  // the experts' first blocks and rows
    int nb = 0, nr = 0;
    bool bad = false;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < p.E) c = p.counts ? p.counts[e] : static_cast<int>(p.rows);
      bad |= c < 0 || c > p.rows;
      if (bad) c = 0;
      int b = (c + C::kRows - 1) / C::kRows, r = p.counts ? (c + 127) / 128 : 0;
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
        sh.first_block[e] = nb + b - b_own;
        sh.first_row[e] = (nr + r - r_own) * 128;
        sh.count[e] = c;
        // the last row that is read has to exist (the padding after it need not, nor the place
        // where an expert without rows would start)
        bad |= c > 0 && static_cast<int64_t>(nr + r - r_own) * 128 + c > p.rows;
      }
      nb += __shfl_sync(0xFFFFFFFFu, b, 31);
      nr += __shfl_sync(0xFFFFFFFFu, r, 31);
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      sh.first_block[p.E] = bad ? 0 : nb;  // no block at all when the counts do not fit
      if (bad && rank == 0) set_error(err, MOE_ERR_DEVICE_BOUNDS, 80);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t tiles = static_cast<uint32_t>(sh.first_block[p.E]) * p.nt;
  uint32_t issued = 0;  // fills that this CTA's producer issued
  if (warp >= kSumWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoader) {
      uint32_t s = 0, phase = 1;
      bool ok = blockIdx.x > 1 || ((p.withhold >> blockIdx.x) & 1u) == 0u;
      const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
        if constexpr (PAIR) tma_load_2d_pair(dst, m, bar, x, y);
        else tma_load_2d(dst, m, bar, x, y);
      };
      for (uint32_t tile = unit; ok && tile < tiles; tile += units) {
        const Tile t = decode<NT, PAIR>(p, sh, tile);
        const CUtensorMap* ma = &p.mapA[t.box];
        const uint32_t kb_tx = (8u << t.box) * 128u + C::kLocalN * 128u;
        const int wrow = t.e * p.N + t.n0 + C::kLocalN * rank, arow = t.row0 + 128 * rank;
        for (int k0 = 0; k0 < p.kt; k0 += p.ks) {
          if (issued >= S) ok = warp_wait(empty(s), phase, 81);
          if (!ok) break;
          const int nk = min(p.ks, p.kt - k0);
          const uint32_t bytes = nk * kb_tx;
          const uint32_t bar = PAIR ? mapa_shared(full(s), 0) : full(s);
          if (elect_one()) {
            sh.tx[s] = bytes;
            if (rank == 0) mbar_arrive_expect_tx(full(s), bytes * C::kCtas);
            for (int j = 0; j < nk; ++j) {
              const uint32_t st = base + s * stage_bytes + j * kb_bytes;
              load(st, ma, bar, (k0 + j) * 128, arow);
              load(st + p.abytes, &p.mapB, bar, (k0 + j) * 128, wrow);
            }
          }
          __syncwarp();
          ++issued;
          if (++s == S) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    } else if (warp < kScaler && rank == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(C::kRows, NT);
      uint32_t s = 0, phase = 0, a = 0, aphase = 1, group = 0;
      bool ok = true;
      for (uint32_t tile = unit; ok && tile < tiles; tile += units) {
        for (int left = p.kt; ok && left > 0; left -= C::kG, ++group) {
          const int nk = min(C::kG, left);
          const bool mine = (group & 1) == static_cast<uint32_t>(warp - kIssuer);
          // A wait by parity for a fill needs the stage's fill before it to have landed; while that is on
          // its way it takes the one before for its own.  That fill is this warp's own where groups are
          // a stage and the stages even; elsewhere the buffer is waited for first: its last sums taken,
          // every fill up to its last group's has landed, and the ring holds kBufs groups.
          const bool wait_buffer = mine && group >= kBufs;
          if (C::kG > 1 && wait_buffer && !(ok = tmem_wait(tempty(a), aphase, 83))) break;
          for (int j0 = 0; j0 < nk; j0 += p.ks) {  // ks divides kG: a stage
            if (mine) {
              ok = warp_wait(full(s), phase, 84);
              // (of the pairs, what an MMA warp waits for last: with the stage after it 5 % slower)
              if (ok && C::kG == 1 && wait_buffer) ok = tmem_wait(tempty(a), aphase, 83);
              if (!ok) break;
              tc_fence_after();
              const int n = min(p.ks, nk - j0);
              if (elect_one()) {
                for (int j = 0; j < n; ++j) {
                  const uint32_t st = base + s * stage_bytes + j * kb_bytes;
                  const uint32_t d = tmem + (a * C::kG + j0 + j) * NT;
                  const uint64_t da = smem_desc_sw128(st, 16, 1024);
                  const uint64_t db = smem_desc_sw128(st + p.abytes, 16, 1024);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {  // 32 values of K each
                    if constexpr (PAIR) umma_f8_pair(d, da + 2 * i, db + 2 * i, idesc, i > 0);
                    else umma_f8(d, da + 2 * i, db + 2 * i, idesc, i > 0);
                  }
                }
                if constexpr (PAIR) {
                  if (j0 + n == nk) umma_commit_pair(tfull(a), 3);
                  umma_commit_pair(empty(s), 3);
                } else {
                  if (j0 + n == nk) umma_commit(tfull(a));
                  umma_commit(empty(s));
                }
              }
              __syncwarp();
            }
            if (++s == S) {
              s = 0;
              phase ^= 1;
            }
          }
          if (++a == kBufs) {
            a = 0;
            aphase ^= 1;
          }
        }
      }
      __syncwarp();
      if (elect_one()) {  // every MMA issued is complete before TMEM is freed
        if constexpr (PAIR) umma_commit_pair(drain, 1);
        else umma_commit(drain);
      }
      mbar_wait(drain, 0, nullptr, err, 85, p.wait_ns);
    } else if (warp == kScaler) {
      uint32_t slot = 0, phase = 1, fills = 0;
      bool ok = true;
      for (uint32_t tile = unit; ok && tile < tiles; tile += units) {
        const Tile t = decode<NT, PAIR>(p, sh, tile);
        const int nrows = min(t.nvalid - 128 * rank, 128);  // none: the factors are not used
        const float* sa = p.sa + static_cast<int64_t>(t.row0 + 128 * rank) * p.kt;
        // columns past N take the last block's
        const float* sb0 = p.sb + (static_cast<int64_t>(t.e) * p.nb + t.n0 / 128) * p.kt;
        const float* sb1 = p.sb + (static_cast<int64_t>(t.e) * p.nb + min(t.n0 / 128 + 1, p.nb - 1)) * p.kt;
        for (int k0 = 0; k0 < p.kt; k0 += kScaleBlocks) {
          const int kb = min(k0 + (lane & 7), p.kt - 1);
          const float b0 = __ldg(sb0 + kb), b1 = NT == 256 ? __ldg(sb1 + kb) : 0.0f;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int r0 = 64 * part + (lane >> 3);
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = r0 + 4 * i < nrows ? __ldg(sa + static_cast<int64_t>(r0 + 4 * i) * p.kt + kb) : 0.0f;
            if (part == 0 && fills >= 2) ok = own_wait(sempty(slot), phase, 87);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              sh.factors[slot][0][lane & 7][r0 + 4 * i] = v[i] * b0;
              if (NT == 256) sh.factors[slot][1][lane & 7][r0 + 4 * i] = v[i] * b1;
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) {
            sh.info[slot] = make_int4(t.row0, t.nvalid, t.n0, 0);
            mbar_arrive(sfull(slot));
          }
          ++fills;
          if (++slot == 2) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    constexpr int kCols = C::kCols, G = C::kG, B = 16;  // B: columns taken at a time
    const int q = warp & 3, part = warp >> 2, half = part * kCols / 128;
    // addresses of this warp's TMEM lanes and columns, its factors, and the buffers' barriers
    const uint32_t shared = base + kBufferBytes;
    const uint32_t tcols = tmem + part * kCols + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t factors = shared + static_cast<uint32_t>(offsetof(Shared, factors)) +
                             4 * ((NT == 256 ? half : 0) * (kScaleBlocks * kScaleRow) + C::kM / 4 * q + lane);
    constexpr uint32_t kOutBytes = C::kOutBytes;
    const uint32_t out_buf = base + C::kRingBytes + warp * kOutBytes;
    const uint32_t tfull0 = tfull(0);
    const uint32_t tempty0 = PAIR ? mapa_shared(tempty(0), 0) : tempty(0);
    uint32_t a = 0, aphase = 0, slot = 0, sphase = 0;
    bool ok = true;
    for (uint32_t tile = unit; ok && tile < tiles; tile += units) {
      if (!(ok = own_wait(sfull(slot), sphase, 88))) break;
      const int4 t = sh.info[slot];
      const int r0 = 128 * rank + C::kM / 4 * q, col0 = t.z + part * kCols;
      const bool live = r0 < t.y && col0 < p.N;  // else nothing of it is stored
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
      for (int left = p.kt; left > 0; left -= kScaleBlocks) {
        if (left < p.kt) ok = ok && own_wait(sfull(slot), sphase, 88);
        if (!ok) break;
        uint32_t f = factors + slot * (2 * kScaleBlocks * kScaleRow * 4);
#pragma unroll 1
        for (int n = min(left, kScaleBlocks); n > 0; n -= G) {
          // one answer for the warp: the tcgen05.ld below is .sync.aligned
          ok = tmem_wait(tfull0 + 8 * a, aphase, 86);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = tcols + a * (G * NT);
#pragma unroll
          for (int j = 0; j < G; ++j) {
            if (live && j < n) {
              float scale;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(scale) : "r"(f + j * (kScaleRow * 4)));
              uint32_t v[2][B];
              tmem_start(ta + j * NT, v[0]);
#pragma unroll
              for (int c = 0; c < kCols; c += B) {
                const int b = c / B & 1;
                tmem_done(v[b]);
                if (c + B < kCols) tmem_start(ta + j * NT + c + B, v[b ^ 1]);
                if (c + B == kCols && (j == G - 1 || j + 1 == n)) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster_relaxed(tempty0 + 8 * a);
                    else mbar_arrive(tempty0 + 8 * a);
                  }
                }
#pragma unroll
                for (int i = 0; i < B; i += 2)
                  asm("{\n\t.reg .b64 v, s, a;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
                      "mov.b64 a, {%0, %1};\n\tfma.rn.f32x2 a, v, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
                      : "+f"(acc[c + i]), "+f"(acc[c + i + 1])
                      : "r"(v[b][i]), "r"(v[b][i + 1]), "f"(scale));
              }
            }
          }
          if (!live) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) mbar_arrive_cluster_relaxed(tempty0 + 8 * a);
              else mbar_arrive(tempty0 + 8 * a);
            }
          }
          f += G * kScaleRow * 4;
          if (++a == kBufs) {
            a = 0;
            aphase ^= 1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty(slot));
        if (++slot == 2) {
          slot = 0;
          sphase ^= 1;
        }
      }
      if (ok && live) {
        const int n = min(t.y - r0, C::kM / 4), row = t.x + r0;
        if (lane == 0) bulk_wait_read_all();  // the last tile's stores have left the buffer
        __syncwarp();
        if (kCols % 64 == 0 && p.tma_out && !p.f32 && n == 32) {
#pragma unroll
          for (int c = 0; c < kCols / 64 * 64; c += 64) {
            if (c * 64 >= static_cast<int>(kOutBytes)) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
            if (col0 + c < p.N) store_tile<64>(p, row, col0 + c, acc + c, out_buf + c * 64 % kOutBytes, lane);
          }
        } else if (kCols % 32 == 0 && p.tma_out && p.f32 && n == 32) {
#pragma unroll
          for (int c = 0; c < kCols / 32 * 32; c += 32) {
            if (c * 128 >= static_cast<int>(kOutBytes)) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
            if (col0 + c < p.N) store_tile<32>(p, row, col0 + c, acc + c, out_buf + c * 128 % kOutBytes, lane);
          }
        } else {
          uint32_t* buf = reinterpret_cast<uint32_t*>(smem_raw + (out_buf - raw));
          const int w = p.vec ? 0 : p.f32 ? 32 : 64;  // columns that store_rows takes
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            const int b = col0 + c / 64 * 64;
            if (kCols % 64 == 0 && w == 64 && b + 64 <= p.N) {
              if (c % 64 == 0) store_rows<64>(p, row, n, b, acc + c, out_buf, lane);
            } else if (kCols % 32 == 0 && w == 32 && col0 + c / 32 * 32 + 32 <= p.N) {
              if (c % 32 == 0) store_rows<32>(p, row, n, col0 + c, acc + c, out_buf, lane);
            } else {
              store16(p, row, n, col0 + c, acc + c, buf, lane);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  // After an abort, loads may still be in flight: they land before TMEM is released and the
  // CTAs exit.  With pairs all complete on rank 0's barriers: rank 1 reports its fills, rank 0
  // balances the bytes of fills that only one CTA issued and waits, then both leave together.
  if constexpr (PAIR) {
    if (rank == 1 && warp == kLoader && lane == 0) {
      st_shared_cluster_u32(mapa_shared(smem_u32(&sh.peer_issued), 0), issued);
      for (uint32_t s = 0; s < S; ++s)
        st_shared_cluster_u32(mapa_shared(smem_u32(&sh.peer_tx[s]), 0), sh.tx[s]);
    }
    cluster_sync_all();
  }
  if (rank == 0 && warp == kLoader && lane == 0) {
    const uint32_t peer = PAIR ? *const_cast<volatile uint32_t*>(&sh.peer_issued) : issued;
    const uint32_t end = issued > peer ? issued : peer;
    // (the last S fills: earlier ones have landed, or their stages would not have been filled again)
    for (uint32_t f = end > S ? end - S : 0; f < end; ++f) {
      const uint32_t s = f % S;
      if (f >= issued) mbar_arrive_expect_tx(full(s), sh.peer_tx[s]);
      else if (f >= peer) mbar_complete_tx(full(s), sh.tx[s]);
      wait(full(s), (f / S) & 1, nullptr, 82);
    }
  }
  if constexpr (PAIR) {
    __syncthreads();
    cluster_sync_all();  // no load, remote arrival or MMA into the peer after this point
  }
  if (warp == kIssuer) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int NT, bool PAIR>
cudaError_t launch(const Params& p, int units, cudaStream_t s) {
  auto kern = gemm_fp8_kernel<NT, PAIR>;
  static std::atomic<unsigned long long> attr_set_mask{0ull};
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(attr_set_mask.load(std::memory_order_acquire) & bit)) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmemBytes));
    if (st != cudaSuccess) return st;
    cudaFuncAttributes fa;  // the split of the registers has to fit the launch's
    if ((st = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return st;
    if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    attr_set_mask.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(Cfg<NT, PAIR>::kCtas * units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                            const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Codes: `rows` rows of K values, fp8_cols(K) bytes apart, 128-byte swizzle, boxes of 128 values x
// box_rows.  Values past K and rows past the last are read as zeros, whatever is there.
CUtensorMap code_map(const void* base, int K, uint64_t rows, uint32_t box_rows, cudaError_t* st) {
  CUtensorMap m = {};
  auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(fp8_cols(K))};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t ones[2] = {1, 1};
  if (!enc || enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    *st = cudaErrorInvalidValue;
  return m;
}

// Tile shapes: 256 x 256 on pairs, or 128 x 128, 128 x 64 or 64 x 32 on single CTAs; by the rounds of
// tiles that each takes over the SMs, times what a block of K of a tile costs there and a tile besides
// (ns, of 8192 x 7168 x 7168 and 4000 x 7168 x 512 in each shape: 306, 465, 567, 1205 us and 26, 30,
// 46, 90; one row of 7168 x 4096 takes 28, 18, 16 and 11 us).  With `counts`, which are on the device,
// `rows` is taken for moe_sort_rows_bound of the pairs, and the pairs for equal shares of the experts
// (37 pairs over 49 experts, 84 x 6373: 10.7 us, 15.6 when the padding counted as rows by half).
// MOE_FP8_SHAPE = 0 .. 3 sets the shape; every shape gives the same bits.
struct Shape {
  int rows, n, ctas, block, tile;
};
constexpr int kNumShapes = 4;
constexpr Shape kShapes[kNumShapes] = {
    {256, 256, 2, 450, 1800}, {128, 128, 1, 345, 870}, {128, 64, 1, 210, 900}, {64, 32, 1, 115, 470}};
int choose_shape(int64_t rows, int N, int kt, int E, bool grouped, int sms) {
  static const int forced = [] {
    const char* v = std::getenv("MOE_FP8_SHAPE");
    return v && *v >= '0' && *v <= '3' ? *v - '0' : -1;
  }();
  if (forced >= 0) return forced;
  if (grouped) rows = rows > 128 * static_cast<int64_t>(E) ? rows - 127 * static_cast<int64_t>(E) : E;
  const int64_t share = (rows + E - 1) / E;
  int best = 0;
  int64_t least = INT64_MAX;
  for (int i = 0; i < kNumShapes; ++i) {
    const Shape& s = kShapes[i];
    const int64_t tiles = E * ((share + s.rows - 1) / s.rows) * ((N + s.n - 1) / s.n);
    const int64_t units = sms / s.ctas, cost = (tiles + units - 1) / units * (kt * s.block + s.tile);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

template <int NT, bool PAIR>
cudaError_t run(Params& p, const uint8_t* a, const uint8_t* b, int K, int sms, cudaStream_t stream) {
  using C = Cfg<NT, PAIR>;
  cudaError_t st = cudaSuccess;
  const int64_t blocks = (p.rows + C::kRows - 1) / C::kRows + (p.counts ? p.E : 0);
  p.nt = (p.N + NT - 1) / NT;
  p.mapB = code_map(b, K, static_cast<uint64_t>(p.E) * p.N, C::kLocalN, &st);
  for (int i = 0; i < kBoxes && (8 << i) <= C::kM; ++i)  // no block has more than `rows`
    if (i == 0 || p.rows > (4 << i)) {
      p.mapA[i] = code_map(a, K, static_cast<uint64_t>(p.rows), 8u << i, &st);
      p.abytes = (8u << i) * 128u;
    }
  if (p.vec) {  // rows start on 16 bytes
    auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
    const cuuint64_t size = p.f32 ? 4 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.rows)};
    const cuuint64_t strides[1] = {p.N * size};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), 32}, ones[2] = {1, 1};
    if (!enc || enc(&p.mapOut, p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out,
                    dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    p.tma_out = 1;
  }
  if (st != cudaSuccess) return st;
  // as many blocks of K in a stage as leave three of them
  const uint32_t kb_bytes = p.abytes + C::kLocalN * 128u;
  for (p.ks = C::kG; p.ks > 1 && 3 * p.ks * kb_bytes > C::kRingBytes;) p.ks /= 2;
  const int stages = static_cast<int>(C::kRingBytes / (p.ks * kb_bytes));
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  if (C::kG == 1) p.stages &= ~1;
  const int64_t tiles = blocks * p.nt;  // checked by the caller to fit 31 bits
  const int units = static_cast<int>(tiles < sms / C::kCtas ? tiles : sms / C::kCtas);
  return launch<NT, PAIR>(p, units, stream);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_gemm_fp8(const uint8_t* a, const float* a_scales, int64_t rows,
                          const int32_t* counts, const uint8_t* b, const float* b_scales, int E, int N,
                          int K, void* out, int out_dtype, cudaStream_t stream) {
  if (rows < 0 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (!counts && E != 1) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int size = out_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!a || !a_scales || !b || !b_scales || !out || !aligned_to(a, 16) || !aligned_to(b, 16) ||
      !aligned_to(a_scales, 4) || !aligned_to(b_scales, 4) || !aligned_to(counts, 4) || !aligned_to(out, size))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || N > kMaxFp8Cols || K > kMaxFp8Cols || rows > INT32_MAX - 256 ||
      static_cast<int64_t>(E) * N > INT32_MAX - 256)  // rows of a tile past the last expert count too
    return MOE_ERR_UNSUPPORTED;
  // tiles of 64 x 32 at the least
  if (((rows + 63) / 64 + E) * ((N + 31) / 32) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  Params p = {};
  p.counts = counts;
  p.sa = a_scales;
  p.sb = b_scales;
  p.rows = rows;
  p.N = N;
  p.kt = static_cast<int>(fp8_cols(K) / 128);
  p.E = E;
  p.nb = (N + 127) / 128;
  const int64_t row = static_cast<int64_t>(N) * size;
  p.vec = aligned_to(out, 32) && row % 32 == 0 ? 2 : aligned_to(out, 16) && row % 16 == 0 ? 1 : 0;
  p.f32 = out_dtype == MOE_DTYPE_F32;
  p.out = out;
  p.wait_ns = wait_limit_ns();
  p.withhold = withheld_loaders();
  const int sms = num_sms_of_current_device();
  const int shape = choose_shape(rows, N, p.kt, E, counts != nullptr, sms);
  const cudaError_t st = shape == 0   ? run<256, true>(p, a, b, K, sms, stream)
                         : shape == 1 ? run<128, false>(p, a, b, K, sms, stream)
                         : shape == 2 ? run<64, false>(p, a, b, K, sms, stream)
                                      : run<32, false>(p, a, b, K, sms, stream);
  return st == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_gemm_fp8_get_error(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
  static std::mutex m;  // g_taken8_status is one caller's at a time
  const std::lock_guard<std::mutex> lock(m);
  int status = 0;
  if (cudaLaunchKernel(reinterpret_cast<const void*>(take_error_kernel), dim3(1), dim3(1), nullptr, 0,
                       stream) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&status, g_taken8_status, sizeof(status), 0, cudaMemcpyDeviceToHost,
                                stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  return static_cast<moe_status_t>(status);
}

}  // extern "C"
