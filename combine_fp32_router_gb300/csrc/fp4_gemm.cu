// Product of MXFP4 rows and MXFP4 expert weights on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4, one E8M0 scale per 32 values, fp32 accumulation):
//   out[r, n] = sum_k A[r, k] B[e(r)][n, k],  rows grouped by expert in 128-row segments.
//
// One persistent launch.  A tile is weight rows (the M operand) x a block of activation rows of
// one expert (the N operand, so a block costs MMAs for the rows it has), in one of two shapes:
//   pairs    256 weight rows x up to 192 rows on a CTA pair (cta_group::2): each CTA loads its
//            half of both, 31 KB per 256 values of K for 128 x 192 outputs
//   singles  128 weight rows (or 64 or 32 of them) x up to 128 rows on one CTA, where pairs would
//            leave SMs idle
// Both add the same products in the same order: K runs through the tensor cores 64 values at a
// time, whatever the other rows are.  Warps:
//   0      producer: codes by TMA (128-byte swizzle), scale tiles by TMA (plain)
//   1      scale tiles shared memory -> TMEM (tcgen05.cp), then the MMAs, which the hardware
//          runs in that order
//   2      TMEM allocator, 3 the experts' first rows and blocks
//   4..7   epilogue: accumulator column = output row, lane = output column
// Bound, with full blocks of pairs, by the tensor pipe and the thread that feeds it: a stage of
// 256 values of K takes some 540 cycles, 408 of them MMAs (8192 x 7168 x 7168: 131 to 141 us by box
// and clocks, 6.0 to 6.4 PFLOP/s; 128 x 192 tiles on single CTAs, which take in 43 KB for the same
// work, 175 us); with few rows by the issuing thread: 3 rows of 4096 x 7168, 10.1 us, spend 16.8
// thousand cycles in its loop, 3.6 of them waiting for loads, the others some 470 for each of 28
// stages, of which 280 are MMAs (70 per 64 values of K, since an MMA reads 128 weight rows whatever
// part of them is real).
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

namespace {

// Device-side problems of the 4-bit product (a bounded wait that ran out, counts that do not
// fit the rows): first error since moe_gemm_fp4_get_error last read it.
__device__ DevErr g_gemm_err;

// Reads and clears it in one step: an error that comes between the two would be lost.
__device__ int g_taken_status;
__global__ void take_error_kernel() { g_taken_status = atomicExch(&g_gemm_err.status, 0); }

template <bool PAIR>
struct Cfg {
  static constexpr int kRows = PAIR ? 192 : 128;  // N of a tile
  static constexpr int kLocal = PAIR ? kRows / 2 : kRows;  // rows a CTA loads
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kStages = 5;
  static constexpr int kSfTiles = PAIR ? 2 : 1;  // 128-row scale tiles a block can touch
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = kLocal * 128;
  static constexpr uint32_t kSfaBytes = 2 * kMxTileBytes;
  static constexpr uint32_t kSfbBytes = 2 * kSfTiles * kMxTileBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr uint32_t kSfCols = 8 + 8 * kSfTiles;  // TMEM columns of a stage's scales
  static constexpr uint32_t kSfCol0 = 2 * kRows;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSfCol0 + kStages * kSfCols <= kTmemCols, "TMEM columns");
  static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024 bytes");
};
constexpr int kBoxes = 4;  // box heights of the activation rows: 16, 32, 64, and 96 (pairs) or 128
constexpr int kThreads = 256;
constexpr int kMaxStages = 5;
constexpr int kTrRow = 36;  // words of a transpose row: 32 columns, padded against bank conflicts

struct Params {
  const int32_t* counts;
  int64_t rows;
  int N, kt, E, nt;   // outputs, 128-value K tiles, experts, weight tiles per expert
  int mt;             // weight rows of a CTA's tile: 128; 64 or 32 of the 128 (singles)
  int sf_tiles;       // 128-row scale tiles per expert
  int64_t ldo;
  int vec;  // output rows start on 16 bytes
  void* out;
  uint64_t wait_ns;
  uint32_t withhold;  // test hook: bit 0, 1: CTA 0, 1 loads nothing
  CUtensorMap mapA, mapSa;          // weight codes (boxes of 128 rows) and scale tiles
  CUtensorMap mapB[kBoxes], mapSb;  // activation codes and scale tiles
};

// behind the stages
struct Shared {
  uint64_t bars[2 * kMaxStages + 5];
  uint32_t tmem;
  int32_t abort_flag;
  uint32_t consumed, peer_issued;          // fills used by MMAs, fills issued by the peer
  uint32_t tx[kMaxStages], peer_tx[kMaxStages];  // bytes of the fill in a stage
  int32_t first_block[kMaxE + 1], first_row[kMaxE + 1], count[kMaxE];
  alignas(16) uint32_t transpose[4 * 16 * kTrRow];
};
template <bool PAIR>
constexpr size_t smem_bytes() {
  return Cfg<PAIR>::kStages * Cfg<PAIR>::kStageBytes + 1024 + sizeof(Shared);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448,
              "fits the opt-in shared memory of a CTA (227 KB)");

__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void umma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
      "\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

struct Tile {
  int e, row0, nvalid, n0;
  int box;    // index of the box height
  int local;  // rows each CTA loads
};

// first_block[e], first_row[e]: blocks and rows before expert e (E + 1 entries each)
template <bool PAIR>
__device__ __forceinline__ Tile decode(const Params& p, const Shared& sh, uint32_t tile) {
  constexpr int R = Cfg<PAIR>::kRows;
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
  t.n0 = static_cast<int>(tile - b * nt) * (PAIR ? 256 : p.mt);
  const int half = PAIR ? (t.nvalid + 1) / 2 : t.nvalid;
  t.box = half <= 16 ? 0 : (half <= 32 ? 1 : (half <= 64 ? 2 : 3));
  t.local = PAIR && t.box == 3 ? 96 : 16 << t.box;
  return t;
}

template <bool F32, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp4_kernel(const __grid_constant__ Params p) {
  using C = Cfg<PAIR>;
  constexpr uint32_t S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw + (base - raw) + S * C::kStageBytes);
  const auto full = [&](uint32_t s) { return smem_u32(&sh.bars[s]); };
  const auto empty = [&](uint32_t s) { return smem_u32(&sh.bars[kMaxStages + s]); };
  const auto tfull = [&](uint32_t a) { return smem_u32(&sh.bars[2 * kMaxStages + a]); };
  const auto tempty = [&](uint32_t a) { return smem_u32(&sh.bars[2 * kMaxStages + 2 + a]); };
  const uint32_t drain = smem_u32(&sh.bars[2 * kMaxStages + 4]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&sh.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / C::kCtas, units = gridDim.x / C::kCtas;
  DevErr* err = &g_gemm_err;
  // the peer arrives on a pair's barriers too: those waits acquire at cluster scope
  const auto wait = [&](uint32_t bar, uint32_t parity, volatile int* ab, int site) {
    if constexpr (PAIR) return mbar_wait_cluster(bar, parity, ab, err, site, p.wait_ns);
    else return mbar_wait(bar, parity, ab, err, site, p.wait_ns);
  };
  const auto warp_wait = [&](uint32_t bar, uint32_t parity, int site) {
    return __all_sync(0xFFFFFFFFu, wait(bar, parity, abort_flag, site)) != 0;
  };

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(full(s), 1);  // rank 0's: its arming arrival and both CTAs' bytes
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 4 * C::kCtas);  // rank 0's: an arrival of every epilogue warp
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    sh.abort_flag = 0;
    sh.consumed = sh.peer_issued = 0u;
    tma_prefetch_desc(&p.mapA);
    tma_prefetch_desc(&p.mapSa);
    tma_prefetch_desc(&p.mapSb);
  }
  if (warp == 2) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(&sh.tmem), C::kTmemCols);
    else tmem_alloc(smem_u32(&sh.tmem), C::kTmemCols);
  }
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
      if (bad && rank == 0) set_error(err, MOE_ERR_DEVICE_BOUNDS, 60);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t tiles = static_cast<uint32_t>(sh.first_block[p.E]) * p.nt;
  const int nks = (p.kt + 1) / 2;
  uint32_t issued = 0;  // fills that this CTA's producer issued

  if (warp == 0) {
    uint32_t s = 0, phase = 1;
    bool ok = blockIdx.x > 1 || ((p.withhold >> blockIdx.x) & 1u) == 0u;
    const auto load = [&](uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
      if constexpr (PAIR) tma_load_2d_pair(dst, m, bar, x, y);
      else tma_load_2d(dst, m, bar, x, y);
    };
    for (uint32_t tile = unit; ok && tile < tiles; tile += units) {
      const Tile t = decode<PAIR>(p, sh, tile);
      const CUtensorMap* mb = &p.mapB[t.box];
      const uint32_t bytes = (PAIR ? 128 : p.mt) * 128u + t.local * 128u + C::kSfaBytes + C::kSfbBytes;
      const int wrow = t.e * p.N + t.n0 + 128 * rank, brow = t.row0 + t.local * rank;
      const int wtile = t.e * p.sf_tiles + t.n0 / 128 + rank, btile = t.row0 / 128;
      // fewer than 128 weight rows lie at their own place among their scale tile's 128 (what is
      // around them meets outputs that are not stored)
      const uint32_t aplace = (t.n0 % 128) * 128u;
      for (int ks = 0; ks < nks; ++ks) {
        if (issued >= S) ok = warp_wait(empty(s), phase, 61);
        if (!ok) break;
        const uint32_t st = base + s * C::kStageBytes, ssf = st + C::kABytes + C::kBBytes;
        const uint32_t bar = PAIR ? mapa_shared(full(s), 0) : full(s);
        if (elect_one()) {
          sh.tx[s] = bytes;
          if (rank == 0) mbar_arrive_expect_tx(full(s), bytes * C::kCtas);
          load(st + aplace, &p.mapA, bar, ks * 128, wrow);
          load(st + C::kABytes, mb, bar, ks * 128, brow);
          load(ssf, &p.mapSa, bar, ks * 256, wtile);  // in words; zeros past the last K tile
          load(ssf + C::kSfaBytes, &p.mapSb, bar, ks * 256, btile);
        }
        __syncwarp();
        ++issued;
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    uint32_t s = 0, phase = 0, n = 0, used = 0;
    bool ok = true;
    for (uint32_t tile = unit; ok && tile < tiles; tile += units, ++n) {
      const Tile t = decode<PAIR>(p, sh, tile);
      const uint32_t acc = n & 1, tacc = tmem + acc * C::kRows;
      if (n >= 2 && !warp_wait(tempty(acc), (n / 2 - 1) & 1, 63)) break;
      tc_fence_after();
      // the block may start inside a scale tile (row 64 of it: column 2)
      const uint32_t sf_shift = (t.row0 % 128) / 32;
      const uint32_t idesc = idesc_mxf4(128 * C::kCtas, t.local * C::kCtas);
      for (int ks = 0; ks < nks; ++ks) {
        ok = warp_wait(full(s), phase, 64);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = base + s * C::kStageBytes;
        const uint32_t ssf = st + C::kABytes + C::kBBytes;
        const uint32_t tsf = tmem + C::kSfCol0 + s * C::kSfCols;
        const int nkt = min(2, p.kt - 2 * ks);
        if (elect_one()) {
          const auto copy = [&](uint32_t dst, uint32_t src) {
            if constexpr (PAIR) tmem_cp_scales_pair(dst, src);
            else tmem_cp_scales(dst, src);
          };
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i < nkt) {
              copy(tsf + 4 * i, ssf + i * kMxTileBytes);
#pragma unroll
              for (int j = 0; j < C::kSfTiles; ++j)
                copy(tsf + 8 + 4 * (C::kSfTiles * i + j), ssf + C::kSfaBytes + (2 * j + i) * kMxTileBytes);
            }
          }
          const uint64_t da = smem_desc_sw128(st, 16, 1024);
          const uint64_t db = smem_desc_sw128(st + C::kABytes, 16, 1024);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t id = (j & 1) * 2, d = idesc | (id << 4) | (id << 29);
            const uint32_t sfa = tsf + 4 * (j >> 1);
            const uint32_t sfb = tsf + 8 + 4 * C::kSfTiles * (j >> 1) + sf_shift;
            if (j < 2 * nkt) {
              if constexpr (PAIR) umma_mxf4_pair(tacc, da + 2 * j, db + 2 * j, d, sfa, sfb, ks > 0 || j > 0);
              else umma_mxf4(tacc, da + 2 * j, db + 2 * j, d, sfa, sfb, ks > 0 || j > 0);
            }
          }
          if constexpr (PAIR) {
            umma_commit_pair(empty(s), 3);
            if (ks == nks - 1) umma_commit_pair(tfull(acc), 3);
          } else {
            umma_commit(empty(s));
            if (ks == nks - 1) umma_commit(tfull(acc));
          }
        }
        __syncwarp();
        ++used;
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (elect_one()) {  // every MMA issued is complete before TMEM is freed
      sh.consumed = used;
      if constexpr (PAIR) umma_commit_pair(drain, 1);
      else umma_commit(drain);
    }
    mbar_wait(drain, 0, nullptr, err, 65, p.wait_ns);
  } else if (warp >= 4) {
    const int q = warp - 4;
    uint32_t* tr = sh.transpose + q * 16 * kTrRow;
    uint32_t n = 0;
    for (uint32_t tile = unit; tile < tiles; tile += units, ++n) {
      const Tile t = decode<PAIR>(p, sh, tile);
      const uint32_t acc = n & 1;
      // one answer for the warp: the tcgen05.ld below is .sync.aligned
      if (!warp_wait(tfull(acc), (n / 2) & 1, 66)) break;
      tc_fence_after();
      const uint32_t tacc = tmem + acc * C::kRows + (static_cast<uint32_t>(32 * q) << 16);
      const int col0 = t.n0 / 128 * 128 + 128 * rank + 32 * q;  // this warp's 32 output columns
      for (int r0 = 0; r0 < t.nvalid; r0 += 32) {
        float a[16], b[16];
        tmem_ld16x2(tacc + r0, tacc + r0 + 16, a, b);
        if (r0 + 32 >= t.nvalid) {  // the last read of this accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) mbar_arrive_cluster_relaxed(mapa_shared(tempty(acc), 0));
            else mbar_arrive(tempty(acc));
          }
        }
        if (!PAIR && (32 * q < t.n0 % 128 || 32 * q >= t.n0 % 128 + p.mt)) continue;  // not of this tile
        const int left = t.nvalid - r0;         // rows of this chunk (may exceed 32)
        if (F32 || !p.vec) {
          const int col = col0 + lane;
          if (col < p.N) {
            const int64_t at = static_cast<int64_t>(t.row0 + r0) * p.ldo + col;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float v = j < 16 ? a[j & 15] : b[j & 15];
              if (j < left) {
                if constexpr (F32) static_cast<float*>(p.out)[at + j * p.ldo] = v;
                else static_cast<uint16_t*>(p.out)[at + j * p.ldo] = bf16_bits(v);
              }
            }
          }
        } else {
          // rows 2 i and 2 i + 1 of a column as one word, through shared memory: a lane then
          // holds eight columns of two rows and stores 16 bytes of each (storing 2 bytes per
          // lane instead took longer than the MMAs of a tile with K = 2048)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tr[i * kTrRow + lane] = i < 8 ? pack_bf16x2(a[2 * i & 15], a[(2 * i + 1) & 15])
                                          : pack_bf16x2(b[2 * i & 15], b[(2 * i + 1) & 15]);
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = (lane >> 2) + 8 * h, c = 8 * (lane & 3);
            const uint4 u = *reinterpret_cast<const uint4*>(&tr[i * kTrRow + c]);
            const uint4 w = *reinterpret_cast<const uint4*>(&tr[i * kTrRow + c + 4]);
            if (col0 + c < p.N) {
              uint16_t* o = static_cast<uint16_t*>(p.out) +
                            static_cast<int64_t>(t.row0 + r0 + 2 * i) * p.ldo + col0 + c;
              if (2 * i < left)
                st_v4(o, make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410),
                                    __byte_perm(w.x, w.y, 0x5410), __byte_perm(w.z, w.w, 0x5410)));
              if (2 * i + 1 < left)
                st_v4(o + p.ldo,
                      make_uint4(__byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x7632),
                                 __byte_perm(w.x, w.y, 0x7632), __byte_perm(w.z, w.w, 0x7632)));
            }
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // After an abort, loads may still be in flight: they land before TMEM is released and the
  // CTAs exit.  With pairs all complete on rank 0's barriers: rank 1 reports its fills, rank 0
  // balances the bytes of fills that only one CTA issued and waits, then both leave together.
  if constexpr (PAIR) {
    if (rank == 1 && warp == 0 && lane == 0) {
      st_shared_cluster_u32(mapa_shared(smem_u32(&sh.peer_issued), 0), issued);
      for (uint32_t s = 0; s < S; ++s)
        st_shared_cluster_u32(mapa_shared(smem_u32(&sh.peer_tx[s]), 0), sh.tx[s]);
    }
    cluster_sync_all();
  }
  if (rank == 0 && warp == 0 && lane == 0) {
    const uint32_t peer = PAIR ? *const_cast<volatile uint32_t*>(&sh.peer_issued) : issued;
    const uint32_t end = issued > peer ? issued : peer;
    for (uint32_t f = *const_cast<volatile uint32_t*>(&sh.consumed); f < end; ++f) {
      const uint32_t s = f % S;
      if (f >= issued) mbar_arrive_expect_tx(full(s), sh.peer_tx[s]);
      else if (f >= peer) mbar_complete_tx(full(s), sh.tx[s]);
      wait(full(s), (f / S) & 1, nullptr, 62);
    }
  }
  if constexpr (PAIR) {
    __syncthreads();
    cluster_sync_all();  // no load, remote arrival or MMA into the peer after this point
  }
  if (warp == 2) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <bool F32, bool PAIR>
cudaError_t launch(const Params& p, int units, cudaStream_t s) {
  auto kern = gemm_fp4_kernel<F32, PAIR>;
  static std::atomic<unsigned long long> attr_set_mask{0ull};
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(attr_set_mask.load(std::memory_order_acquire) & bit)) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_bytes<PAIR>()));
    if (st != cudaSuccess) return st;
    attr_set_mask.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(Cfg<PAIR>::kCtas * units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<PAIR>();
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                            const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Codes: `rows` rows of `inner` bytes, 128-byte swizzle, boxes of 128 bytes x box_rows (bytes
// past the row's end and rows past the last are read as zeros).
CUtensorMap code_map(const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                     cudaError_t* st) {
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

// Scale tiles: `tiles` rows of kt tiles (128 words each), boxes of two tiles x box_tiles rows.
CUtensorMap scale_map(const void* base, int kt, uint64_t tiles, uint32_t box_tiles, cudaError_t* st) {
  CUtensorMap m = {};
  auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
  const cuuint64_t dims[2] = {128ull * kt, tiles};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kt) * kMxTileBytes};
  const cuuint32_t box[2] = {256, box_tiles};
  const cuuint32_t ones[2] = {1, 1};
  if (!enc || enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    *st = cudaErrorInvalidValue;
  return m;
}

// Pairs or singles, by the rounds of tiles that each takes over the SMs: a full round of pairs
// costs 9/8 of one of singles (both then take in what an SM can, 955 and 843 cycles a stage over
// 64 experts).  Measured on GB300, single and pair: 3 rows of N 4096, K 7168 10.0 and 10.6 us; 777
// of 1545 x 2976 9.6 and 11.8; 1024 of 2048 x 2048 6.0 and 7.1; 4096 of 1024 x 2048 8.8 and 9.7;
// over 64 experts of 1024 x 2048 300 rows 11.2 and 12.2, 24576 rows 42.6 and 36.2; 8192 of 7168 x
// 7168 175 (128 x 192 singles) and 131.  With `counts`, which are on the device, the experts are
// taken to have equal shares of the rows less half a tile of padding each; both shapes give the
// same bits.
bool use_pairs(int64_t rows, int N, int E, bool grouped, int sms) {
  if (grouped) rows = rows > 65 * static_cast<int64_t>(E) ? rows - 64 * static_cast<int64_t>(E) : E;
  const int64_t share = (rows + E - 1) / E;
  const auto rounds = [&](int height, int width, int units) {
    const int64_t tiles = E * ((share + height - 1) / height) * ((N + width - 1) / width);
    return (tiles + units - 1) / units;
  };
  return 9 * rounds(Cfg<true>::kRows, 256, sms / 2) < 8 * rounds(Cfg<false>::kRows, 128, sms);
}

template <bool PAIR>
cudaError_t run(Params& p, const uint8_t* a, const uint8_t* a_scales, const uint8_t* b,
                const uint8_t* b_scales, int K, int out_dtype, int sms, cudaStream_t stream) {
  using C = Cfg<PAIR>;
  cudaError_t st = cudaSuccess;
  const uint64_t inner = static_cast<uint64_t>(mx_cols(K) / 2);
  const int64_t blocks = (p.rows + C::kRows - 1) / C::kRows + (p.counts ? p.E : 0);
  p.mt = 128;
  if (!PAIR && !p.counts)
    while (p.mt > 32 && 2 * blocks * ((p.N + p.mt - 1) / p.mt) <= sms) p.mt /= 2;
  p.nt = (p.N + p.mt * C::kCtas - 1) / (p.mt * C::kCtas);
  p.mapA = code_map(b, inner, static_cast<uint64_t>(p.E) * p.N, p.mt, &st);
  p.mapSa = scale_map(b_scales, p.kt, static_cast<uint64_t>(p.E) * p.sf_tiles, 1, &st);
  p.mapSb = scale_map(a_scales, p.kt, static_cast<uint64_t>((p.rows + 127) / 128), C::kSfTiles, &st);
  const int boxes[kBoxes] = {16, 32, 64, PAIR ? 96 : 128};
  for (int i = 0; i < kBoxes; ++i)  // no block has more than `rows`
    if (i == 0 || p.rows > boxes[i - 1])
      p.mapB[i] = code_map(a, inner, static_cast<uint64_t>(p.rows), boxes[i], &st);
  if (st != cudaSuccess) return st;
  const int64_t tiles = blocks * p.nt;  // checked by the caller to fit 31 bits
  const int units = static_cast<int>(tiles < sms / C::kCtas ? tiles : sms / C::kCtas);
  return out_dtype == MOE_DTYPE_F32 ? launch<true, PAIR>(p, units, stream)
                                    : launch<false, PAIR>(p, units, stream);
}

}  // namespace

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
      static_cast<int64_t>(E) * N > INT32_MAX - 256)  // rows of a tile past the last expert count too
    return MOE_ERR_UNSUPPORTED;
  // tiles of 64 x 32 at the least
  if (((rows + 63) / 64 + E) * ((N + 31) / 32) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  Params p = {};
  p.counts = counts;
  p.rows = rows;
  p.N = N;
  p.kt = static_cast<int>(mx_cols(K) / 128);
  p.E = E;
  p.sf_tiles = (N + 127) / 128;
  p.ldo = N;
  p.vec = N % 8 == 0;
  p.out = out;
  p.wait_ns = wait_limit_ns();
  p.withhold = withheld_loaders();
  const int sms = num_sms_of_current_device();
  const cudaError_t st =
      use_pairs(rows, N, E, counts != nullptr, sms)
          ? run<true>(p, a, a_scales, b, b_scales, K, out_dtype, sms, stream)
          : run<false>(p, a, a_scales, b, b_scales, K, out_dtype, sms, stream);
  return st == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_gemm_fp4_get_error(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
  static std::mutex m;  // g_taken_status is one caller's at a time
  const std::lock_guard<std::mutex> lock(m);
  int status = 0;
  if (cudaLaunchKernel(reinterpret_cast<const void*>(take_error_kernel), dim3(1), dim3(1), nullptr, 0,
                       stream) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&status, g_taken_status, sizeof(status), 0, cudaMemcpyDeviceToHost,
                                stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  return static_cast<moe_status_t>(status);
}

}  // extern "C"
