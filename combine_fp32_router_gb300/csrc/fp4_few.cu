// The whole MoE layer for a few tokens (T <= 32) on MXFP4 experts, in two launches:
//   few_router_kernel  logits = x R^T in fp32 (unless the caller has them), x in MXFP4 terms,
//                      counters cleared
//   few_experts_kernel top-k and gates, both expert products with SwiGLU between, the combine
//
// Bound by reading the chosen experts' weights, 17/32 byte a value, once for up to 8 tokens that
// chose an expert (9 to 16 tokens read it twice, and so on: 32 tokens over 8 experts of d = 7168,
// d_ff = 2048, top-2, met in 11.2 groups, 83.8 us; one reading each would be 27.7).  The block-scaled
// tensor cores (tcgen05 kind::mxf4) take the weights as they lie in memory; the activations
// have to be 4-bit operands too, so each is written as a sum of kTerms = 6 MXFP4 numbers, the
// residual of each being quantised again: a term leaves at most 1/5 of its block's largest
// value, six at most 2^-13.9 of it (2^-19 is usual), which is below what rounding to bf16
// would cost.  A token's terms are six columns of the N operand, the partial products are
// added in fp32.  (Converting the weights to fp16 for mma.sync took 502 us for 16 tokens over 64
// experts of d = 7168, d_ff = 2048; this takes 218 us, 6.9 TB/s.)
//
// Units of work are 128 weight rows x a range of K for up to 8 tokens of an expert, first of
// W1 and W3, then of W2, at last the tokens' combines.  CTAs take them from a counter in that
// order, so whoever waits for an h (or a row of y) waits only for units that running CTAs hold.
// Every sum's order is fixed by the sizes: results do not depend on the batch or on which CTA did
// what.
#include <cuda.h>

#include <atomic>

#include "fp4.cuh"
#include "internal.h"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kMaxT = kFewMaxTokens;
constexpr int kMaxRows = kMaxT * kMaxK;  // (token, slot) pairs
constexpr int kTok = 8;                  // token columns of a unit
constexpr int kTerms = 6;
constexpr int kMaxN = kTok * kTerms;
constexpr int kStageKt = 4;              // 128-value K tiles per stage
constexpr int kPartStages = 4;           // stages of a K range of W1 and W3 (at most)
constexpr uint32_t kABytes = 128 * kStageKt * 64;
constexpr uint32_t kSfBytes = kStageKt * kMxTileBytes;
constexpr int kMaxStages = 4;  // 160 KB in flight per SM; more only lengthens every other round trip
// Four groups of four warps finish units in turn, each with an accumulator of its own: waiting
// for a tile's other sums, SwiGLU and the terms of h take longer than streaming the next unit's
// weights (round trips take 2 to 4 us beside a full ring).  With one group the stream waited for
// it: 320 us instead of 253 us for 16 tokens over 64 experts, the rest being equal.
constexpr int kGroups = 4;
constexpr uint32_t kAccCols = 64;        // TMEM: the accumulators, then the stages' scales
constexpr uint32_t kSfCol0 = kGroups * kAccCols;
constexpr uint32_t kSfCols = 8 * kStageKt;
static_assert(kSfCol0 + kMaxStages * kSfCols <= 512 && kMaxN <= static_cast<int>(kAccCols),
              "TMEM columns");
// warps 0 and 3 load weights and activations, 1 issues MMAs, 2 owns TMEM, 4 on finish units
constexpr int kThreads = 128 + 128 * kGroups;

struct FewLayout {
  size_t err, ticket, done1, xdone, clear_end, xq, xs, gq, gs, hq, hs, part, y, total;
  int cols, parts;
  int64_t groups;
};
// Tokens up to 8 are columns by themselves, the same for every expert; more are gathered into
// groups of up to 8 per expert.
FewLayout few_layout(int64_t T, int d, int E, int k, int dff) {
  FewLayout L;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t r = at;
    at = (at + n + 255) / 256 * 256;
    return r;
  };
  const size_t P = static_cast<size_t>(T) * k, G = T <= kTok && static_cast<size_t>(E) < P ? E : P;
  const int stages = (d / 128 + kStageKt - 1) / kStageKt;
  L.groups = static_cast<int64_t>(G);
  L.cols = static_cast<int>(T < kTok ? T : kTok);
  L.parts = (stages + kPartStages - 1) / kPartStages;
  const size_t rows = static_cast<size_t>(L.cols) * kTerms;
  L.err = take(sizeof(DevErr));
  L.ticket = take(4);
  L.done1 = take(G * 4);
  L.xdone = take(G * 4);
  L.clear_end = at;
  L.xq = take(T * kTerms * (d / 2));
  // scale tiles [d / 128][512] of up to 8 tokens, or words [d / 128][T kTerms] of more
  L.xs = take(static_cast<size_t>(d / 128) * (T <= kTok ? kMxTileBytes : T * kTerms * 4));
  L.gq = take(T <= kTok ? 0 : G * rows * (d / 2));
  L.gs = take(T <= kTok ? 0 : G * (d / 128) * kMxTileBytes);
  L.hq = take(G * rows * (dff / 2));
  L.hs = take(G * (dff / 128) * kMxTileBytes);
  L.part = take(P * (dff / 128) * 2 * L.parts * 128 * 4);
  L.y = take(P * d * 4);
  L.total = at;
  return L;
}

// Scale byte of a term: the smallest power of two that keeps the block's largest magnitude
// within E2M1's 6, so that no term saturates (255 for a block that is not finite).
__device__ __forceinline__ uint32_t term_scale(uint32_t amax) {
  const uint32_t s = mx_scale_byte(amax);
  return s + ((amax & 0x7FFFFFu) > 0x400000u && amax >= 0x01000000u && s < 255u ? 1u : 0u);
}
// Sums that pass between CTAs (of K ranges, and the rows of y) are their own arrival flags: the
// router's launch fills their places with this NaN, which no sum is stored as, and who needs
// them reads until it is gone.  (A counter needs the stores released first, which took 5 us
// per unit under the weight stream.)
constexpr uint32_t kNotYet = 0xFFFFFFFFu;
__device__ __forceinline__ void put_sum(float* p, float v) {
  const uint32_t u = __float_as_uint(v);
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(u == kNotYet ? 0x7FFFFFFFu : u)
               : "memory");
}
__device__ __forceinline__ uint32_t look(const float* p) {
  uint32_t u;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(u) : "l"(p) : "memory");
  return u;
}
// n <= 8 sums (0 past them) for a whole warp, each lane its own, from at(0), at(1), ...  False
// after `limit_ns` or an abort.
template <typename At>
__device__ __forceinline__ bool get_sums(const At& at, int n, float (&v)[8], volatile int* abort_flag,
                                         DevErr* err, int site, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t turn = 0;; ++turn) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = i < n ? look(at(i)) : 0u;
    bool there = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      there = there && u[i] != kNotYet;
      v[i] = __uint_as_float(u[i]);
    }
    if (__all_sync(0xFFFFFFFFu, there)) return true;
    if (turn == 64) t0 = global_ns();
    if (turn > 64 && (turn & 63u) == 0u) {
      const bool late = global_ns() - t0 > limit_ns;
      if (late) {
        *abort_flag = 1;
        set_error(err, MOE_ERR_TIMEOUT, site);
      }
      if (__any_sync(0xFFFFFFFFu, late || *abort_flag != 0)) return false;
    }
  }
}

// Byte of (row n < 48, block b of the 128-value tile) in a scale tile
__device__ __forceinline__ uint32_t sf_at(int n, int b) {
  return (n & 31) * 16 + (n >> 5) * 4 + b;
}

// ------------------------------------------------------------------------------ router
struct RouterParams {
  const uint16_t* x;
  const float* router;  // null: the logits are given
  float* logits;
  int T, d, E;
  int conv;  // the first CTAs, which write x in terms
  DevErr* err;
  int32_t* clear;  // counters, contiguous
  int64_t n_clear;
  uint4* places;   // of sums that pass between CTAs, to be marked kNotYet
  int64_t n_places;  // in 16 bytes
  uint8_t* xq;
  uint8_t* xs;
};

constexpr int kRouterExperts = 2;  // per CTA
constexpr int kRouterThreads = 256;

// Every CTA clears its share of the counters and marks its share of the sums' places; the first
// `conv` write x in MXFP4 terms; each of the next computes the logits of two experts for up to TB
// tokens (blockIdx.y: which): warp w sums the 128-value pieces w, w + 8, ... of d, lanes then warps
// are added in a fixed order, the same for every U.  Any others only mark.
template <int TB, int U>
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(RouterParams p) {
  griddep_wait();
  // the experts' kernel may take its places now; it waits for this one's results itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float red[8][TB][kRouterExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.y == 0) {
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRouterThreads) + threadIdx.x; i < p.n_clear;
         i += static_cast<int64_t>(gridDim.x) * kRouterThreads)
      p.clear[i] = 0;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRouterThreads) + threadIdx.x; i < p.n_places;
         i += static_cast<int64_t>(gridDim.x) * kRouterThreads)
      p.places[i] = make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = DevErr{};
  }
  if (static_cast<int>(blockIdx.x) < p.conv) {
    // 2048 values of a token: d is a multiple of 128, so blocks are whole
    const int per = (p.d + kRouterThreads * 8 - 1) / (kRouterThreads * 8);
    for (int i0 = blockIdx.x; blockIdx.y == 0 && i0 < p.T * per; i0 += p.conv) {
      const int t = i0 / per, row_bytes = p.d / 2;
      const int c = (i0 % per) * kRouterThreads * 8 + threadIdx.x * 8;
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (c < p.d) u = ld_v4(p.x + static_cast<int64_t>(t) * p.d + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
      }
#pragma unroll
      for (int r = 0; r < kTerms; ++r) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const uint32_t s = term_scale(amax);
        const float inv = mx_inverse_scale(s), f = mx_scale(s);
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = s == 255u ? 0.0f : v[i] * inv;
        const uint32_t code = e2m1x8(z);
        uint32_t h[4];
        e2m1x8_to_half(code, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
          v[2 * i] = fmaf(-q.x, f, v[2 * i]);  // exact: at most 24 bits are left
          v[2 * i + 1] = fmaf(-q.y, f, v[2 * i + 1]);
        }
        const int n = t * kTerms + r;
        if (c < p.d) {
          *reinterpret_cast<uint32_t*>(p.xq + n * static_cast<int64_t>(row_bytes) + c / 2) = code;
          if ((lane & 3) == 0) {
            const int b = (c >> 5) & 3;
            uint8_t* o = p.T <= kTok
                             ? p.xs + static_cast<int64_t>(c >> 7) * kMxTileBytes + sf_at(n, b)
                             : p.xs + (static_cast<int64_t>(c >> 7) * p.T * kTerms + n) * 4 + b;
            *o = static_cast<uint8_t>(s);
          }
        }
      }
    }
  }
  const int e0 = (static_cast<int>(blockIdx.x) - p.conv) * kRouterExperts;
  if (!p.router || e0 < 0 || e0 >= p.E) return;
  const int t0 = blockIdx.y * TB, tn = min(TB, p.T - t0);
  const int ne = min(kRouterExperts, p.E - e0);
  const float* r0 = p.router + static_cast<int64_t>(e0) * p.d;
  const float* r1 = r0 + (ne > 1 ? p.d : 0);
  float acc[TB][kRouterExperts];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t][0] = acc[t][1] = 0.0f;
  for (int c0 = warp * 128; c0 < p.d; c0 += U * 1024) {
    float4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 1024 + lane * 4;
      a[u] = b[u] = make_float4(0, 0, 0, 0);
      if (c < p.d) {
        a[u] = __ldg(reinterpret_cast<const float4*>(r0 + c));
        b[u] = __ldg(reinterpret_cast<const float4*>(r1 + c));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // loads without branches, so that they run ahead of the sums: past d the factors are zero
      const int c = min(c0 + u * 1024, p.d - 128) + lane * 4;
      const bool in = c0 + u * 1024 < p.d;
      uint2 xv[TB];
#pragma unroll
      for (int t = 0; t < TB; ++t)
        xv[t] = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<int64_t>(t0 + min(t, tn - 1)) * p.d + c));
      if (in) {
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const float x0 = bf16lo(xv[t].x), x1 = bf16hi(xv[t].x), x2 = bf16lo(xv[t].y), x3 = bf16hi(xv[t].y);
          acc[t][0] = fmaf(x3, a[u].w, fmaf(x2, a[u].z, fmaf(x1, a[u].y, fmaf(x0, a[u].x, acc[t][0]))));
          acc[t][1] = fmaf(x3, b[u].w, fmaf(x2, b[u].z, fmaf(x1, b[u].y, fmaf(x0, b[u].x, acc[t][1]))));
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int j = 0; j < kRouterExperts; ++j) {
      float v = acc[t][j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == 0) red[warp][t][j] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < tn * ne; i += kRouterThreads) {
    const int t = i / ne, j = i % ne;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][t][j];
    p.logits[static_cast<int64_t>(t0 + t) * p.E + e0 + j] = v;
  }
}

// ------------------------------------------------------------------------------ experts
struct ExpertParams {
  const float* logits;
  int T, d, E, k, dff;
  int cols, n, parts;  // token columns, N of the MMAs, K ranges of W1 and W3
  int stages;
  uint32_t stage_bytes;
  const uint8_t *s1, *s3, *s2;
  int64_t s1_bytes, s2_bytes;  // scale bytes per expert
  const uint8_t *xq, *xs;      // the tokens' terms
  uint8_t *gq, *gs, *hq, *hs;  // terms of gathered tokens and of h, per group
  float *part, *y;
  uint16_t* out;
  int32_t *ticket, *done1, *xdone;
  DevErr* err;
  uint64_t wait_ns;
  uint32_t withhold;  // test hook, CTA 0: bit 0 no weights are loaded, bit 1 no activations
  // codes of W1, W3, W2 (boxes of 128 rows) and of x and h terms (boxes of n rows), 128 bytes
  // wide; where rows are whole numbers of 128-byte pieces (wide) a box holds two of them
  CUtensorMap map1, map3, map2, mapx, maph;
  int wide1, wide2;
};

// Up to 8 tokens of an expert: their bits, and the row of the first in `part` and y.
struct Group {
  int32_t e;
  uint32_t tokens;
  int32_t row0;
  int32_t n;
};
struct Unit {
  int32_t kind;  // 0: no more work, 1: W1 or W3 rows, 2: W2 rows, 3: a token's combine
  int32_t group, tile, q;  // q: matrix + 2 * K range; kind 3: group is the token
};
struct StageMeta {
  Unit u;
  int32_t ks, nkt;  // stage along K, K tiles in it
  int32_t flags;  // 1: first stage of its unit, 2: last
};

struct Shared {
  Group group[kMaxRows];
  uint32_t mask[kMaxE];
  int32_t base[kMaxE];  // first row of an expert's tokens
  float gate[kMaxT][kMaxK];
  uint16_t slot_e[kMaxT][kMaxK];
  StageMeta meta[kMaxStages];
  Unit acc_unit[kGroups];
  uint64_t bars[3 * kMaxStages + 2 * kGroups + 1];
  int2 total[kMaxE / 32];  // rows and groups of 32 experts
  int32_t groups, ticket;
  int32_t abort_flag;
  uint32_t tmem;
  // fills of the ring: given out by the weights' loader, joined by the activations', and landed
  // before their MMAs
  uint32_t given, joined, landed;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, uint32_t bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Routing of one token by one warp.  (Lists of logits sorted per lane, or every logit's rank counted
// by a thread, were no faster: each CTA runs this code once per launch.)
template <int EPL>
__device__ __forceinline__ void route_token(const ExpertParams& p, Shared& sh, int t, int lane) {
  float v[EPL];
#pragma unroll
  for (int c = 0; c < EPL; ++c)
    v[c] = lane + 32 * c < p.E ? __ldcg(p.logits + static_cast<int64_t>(t) * p.E + lane + 32 * c) : 0.0f;
  int e;
  float g;
  topk_token<EPL>(v, p.E, p.k, lane, &e, &g);
  if (lane < p.k) {
    sh.slot_e[t][lane] = static_cast<uint16_t>(e);
    sh.gate[t][lane] = g;
    atomicOr(&sh.mask[e], 1u << t);
  }
}

// Row of (token, slot) in h and y: rows by (expert, token)
__device__ __forceinline__ int row_of(const Shared& sh, int t, int j) {
  const int e = sh.slot_e[t][j];
  return sh.base[e] + __popc(sh.mask[e] & ((1u << t) - 1u));
}

// The terms of a group's tokens and their scale words, copied into the layout that h has.  By
// the whole CTA: 16 bytes of codes per thread, then the scale words.
__device__ void gather_group(const ExpertParams& p, const Shared& sh, int gi) {
  const Group gr = sh.group[gi];
  const int row_bytes = p.d / 2, kt = p.d / 128, rows = p.cols * kTerms;
  const int n16 = kTerms * row_bytes / 16, words = kt * kTerms;  // of a token
  for (int i = threadIdx.x; i < gr.n * (n16 + words); i += kThreads) {
    const int c = i / (n16 + words), o = i % (n16 + words);
    uint32_t left = gr.tokens;
    for (int j = 0; j < c; ++j) left &= left - 1u;
    const int t = __ffs(left) - 1;
    if (o < n16) {
      st_v4(p.gq + (static_cast<int64_t>(gi) * rows + c * kTerms) * row_bytes + 16 * o,
            ld_v4(p.xq + static_cast<int64_t>(t) * kTerms * row_bytes + 16 * o));
    } else {
      const int tile = (o - n16) / kTerms, r = (o - n16) % kTerms;
      *reinterpret_cast<uint32_t*>(p.gs + (static_cast<int64_t>(gi) * kt + tile) * kMxTileBytes +
                                   sf_at(c * kTerms + r, 0)) =
          __ldcg(reinterpret_cast<const uint32_t*>(
              p.xs + (static_cast<int64_t>(tile) * p.T * kTerms + t * kTerms + r) * 4));
    }
  }
  fence_proxy_async_global();
}

__global__ void __launch_bounds__(kThreads, 1)
    few_experts_kernel(const __grid_constant__ ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Shared& sh = *reinterpret_cast<Shared*>(
      smem_raw + (base - raw) + static_cast<size_t>(p.stages) * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t S = p.stages;
  const auto full = [&](uint32_t s) { return smem_u32(&sh.bars[s]); };
  const auto empty = [&](uint32_t s) { return smem_u32(&sh.bars[kMaxStages + s]); };
  const auto told = [&](uint32_t s) { return smem_u32(&sh.bars[2 * kMaxStages + s]); };
  const auto tfull = [&](uint32_t a) { return smem_u32(&sh.bars[3 * kMaxStages + a]); };
  const auto tempty = [&](uint32_t a) { return smem_u32(&sh.bars[3 * kMaxStages + kGroups + a]); };
  const uint32_t drain = smem_u32(&sh.bars[3 * kMaxStages + 2 * kGroups]);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&sh.abort_flag);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(full(s), 2);   // the weights' loads and the activations'
      mbar_init(empty(s), 1);
      mbar_init(told(s), 1);   // the stage's meta is written
    }
    for (int a = 0; a < kGroups; ++a) {
      mbar_init(tfull(a), 2);   // the accumulator is complete, its unit is written down
      mbar_init(tempty(a), 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    sh.abort_flag = 0;
    sh.given = sh.joined = sh.landed = 0u;
    tma_prefetch_desc(&p.map1);
    tma_prefetch_desc(&p.map3);
    tma_prefetch_desc(&p.map2);
    tma_prefetch_desc(&p.mapx);
    tma_prefetch_desc(&p.maph);
  }
  if (warp == 2) tmem_alloc(smem_u32(&sh.tmem), 512);
  for (int e = threadIdx.x; e < p.E; e += kThreads) sh.mask[e] = 0u;
  __syncthreads();
  griddep_wait();
  int next = 0;
  if (warp == 0 && lane == 0) next = atomicAdd(p.ticket, 1);
  for (int t = warp; t < p.T; t += kThreads / 32) {
    if (p.E <= 64) route_token<2>(p, sh, t, lane);
    else if (p.E <= 256) route_token<8>(p, sh, t, lane);
    else route_token<kMaxE / 32>(p, sh, t, lane);
  }
  __syncthreads();
  // groups of up to 8 tokens per chosen expert, in expert order; 32 experts per warp at a time
  constexpr int kWarps = kThreads / 32, kRounds = (kMaxE / 32 + kWarps - 1) / kWarps;
  uint32_t mine[kRounds];
  int pn[kRounds], pg[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int e = (warp + i * kWarps) * 32 + lane;
    mine[i] = e < p.E ? sh.mask[e] : 0u;
    pn[i] = __popc(mine[i]);
    pg[i] = (pn[i] + kTok - 1) / kTok;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int un = __shfl_up_sync(0xFFFFFFFFu, pn[i], o), ug = __shfl_up_sync(0xFFFFFFFFu, pg[i], o);
      if (lane >= o) {
        pn[i] += un;
        pg[i] += ug;
      }
    }
    if (lane == 31 && warp + i * kWarps < kMaxE / 32) sh.total[warp + i * kWarps] = make_int2(pn[i], pg[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int w32 = warp + i * kWarps, e = w32 * 32 + lane;
    const int2 before = lane < w32 && lane < kMaxE / 32 ? sh.total[lane] : make_int2(0, 0);
    const int rows = __reduce_add_sync(0xFFFFFFFFu, before.x);
    const int groups = __reduce_add_sync(0xFFFFFFFFu, before.y);
    const int n = __popc(mine[i]);
    int r = rows + pn[i] - n, gi = groups + pg[i] - (n + kTok - 1) / kTok;
    if (e < p.E) sh.base[e] = r;
    uint32_t left = mine[i];
    while (left) {
      uint32_t take = left;
      if (__popc(left) > kTok) {  // the lowest 8 bits that are set
        uint32_t rest = left;
        for (int c = 0; c < kTok; ++c) rest &= rest - 1u;
        take = left & ~rest;
      }
      const int c = __popc(take);
      sh.group[gi++] = Group{e, take, r, c};
      r += c;
      left &= ~take;
    }
    if (w32 == (p.E - 1) / 32 && lane == 31) sh.groups = groups + pg[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const bool direct = p.T <= kTok;  // column = token; else column = place in the group
  const int groups = sh.groups;
  const int ht = p.dff / 128, yt = p.d / 128, Q = 2 * p.parts;
  const int n0 = direct ? 0 : groups, n1 = n0 + groups * ht * Q, n2 = n1 + groups * yt;
  const int n_units = n2 + p.T * yt;
  const int kt1 = p.d / 128, kt2 = p.dff / 128;
  if (!direct) {  // the first units: gathering
    while (true) {
      if (threadIdx.x == 0) sh.ticket = next;
      __syncthreads();
      const int u = sh.ticket;
      if (u >= n0) break;
      if (threadIdx.x == 0) next = atomicAdd(p.ticket, 1);
      gather_group(p, sh, u);
      __syncthreads();
      if (threadIdx.x == 0) red_release_add(p.xdone + u, 1);
    }
  }
  const int st1 = (kt1 + kStageKt - 1) / kStageKt, st2 = (kt2 + kStageKt - 1) / kStageKt;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    uint32_t it = 0, s = 0, phase = 1;
    bool ok = !(blockIdx.x == 0 && (p.withhold & 1u));
    while (ok) {
      const int u = __shfl_sync(0xFFFFFFFFu, next, 0);
      const bool work = u < n_units;
      if (lane == 0 && work) next = atomicAdd(p.ticket, 1);  // used after this unit's loads
      Unit un = {0, 0, 0, 0};
      int ks0 = 0, ks1 = 1;
      if (work && u < n1) {
        const int v = u - n0, w = v % (ht * Q);
        un = Unit{1, v / (ht * Q), w / Q, w % Q};
        ks0 = st1 * (un.q >> 1) / p.parts;
        ks1 = st1 * ((un.q >> 1) + 1) / p.parts;
      } else if (work && u < n2) {
        un = Unit{2, (u - n1) / yt, (u - n1) % yt, 0};
        ks1 = st2;
      } else if (work) {
        un = Unit{3, (u - n2) / yt, (u - n2) % yt, 0};
      }
      const bool loads = work && u < n2;
      const int e = loads ? sh.group[un.group].e : 0;
      const bool first = un.kind == 1;
      const bool wide = first ? p.wide1 : p.wide2;
      const int kt = first ? kt1 : kt2;
      const CUtensorMap* mw = first ? ((un.q & 1) ? &p.map3 : &p.map1) : &p.map2;
      const int wrow = (first ? e * p.dff : e * p.d) + 128 * un.tile;
      const uint8_t* sfa =
          (first ? ((un.q & 1) ? p.s3 : p.s1) + e * p.s1_bytes : p.s2 + e * p.s2_bytes) +
          static_cast<int64_t>(un.tile) * kt * kMxTileBytes;
      for (int ks = ks0; ks < ks1; ++ks) {
        if (it >= S) ok = warp_wait(empty(s), phase, abort_flag, p.err, 70, p.wait_ns);
        if (!ok) break;
        const int nkt = min(kStageKt, kt - kStageKt * ks);
        const uint32_t st = base + s * p.stage_bytes;
        if (elect_one()) {
          sh.meta[s] = StageMeta{un, ks, nkt, (ks == ks0 ? 1 : 0) | (ks == ks1 - 1 ? 2 : 0)};
          mbar_arrive(told(s));
          if (!loads) {
            mbar_arrive(full(s));
          } else if (wide) {
            mbar_arrive_expect_tx(full(s), kABytes + nkt * kMxTileBytes);
            tma_load_3d(st, mw, full(s), 0, wrow, 2 * ks);  // pieces past the row's end are zeros
          } else {
            const int pieces = (nkt + 1) / 2;
            mbar_arrive_expect_tx(full(s), pieces * (kABytes / 2) + nkt * kMxTileBytes);
            for (int c = 0; c < pieces; ++c)
              tma_load_2d(st + c * (kABytes / 2), mw, full(s), (2 * ks + c) * 128, wrow);
          }
          if (loads)
            bulk_load(st + kABytes + 2 * p.n * 128u, sfa + static_cast<int64_t>(ks) * kSfBytes,
                      nkt * kMxTileBytes, full(s));
        }
        __syncwarp();
        ++it;
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
      }
      if (!work) break;
    }
    if (lane == 0) sh.given = it;
  } else if (warp == 3) {
    // ---------------------------------------------------------------- loads of activations
    // apart from the weights' so that those run ahead while an h is not there yet
    uint32_t it = 0, s = 0, phase = 0;
    const uint32_t bbytes = p.n * 128u;
    const bool stop = blockIdx.x == 0 && (p.withhold & 2u);
    while (!stop && warp_wait(told(s), phase, abort_flag, p.err, 77, p.wait_ns)) {
      const StageMeta m = sh.meta[s];
      if (m.u.kind == 0 || m.u.kind == 3) {  // nothing to load
        if (elect_one()) mbar_arrive(full(s));
        __syncwarp();
        ++it;
        if (m.u.kind == 0) break;
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
        continue;
      }
      const bool first = m.u.kind == 1;
      const bool wide = first ? p.wide1 : p.wide2;
      const CUtensorMap* mx = first ? &p.mapx : &p.maph;
      const int xrow = first && direct ? 0 : m.u.group * p.cols * kTerms;
      const int64_t kt = first ? kt1 : kt2;
      const uint8_t* sfb = (first ? (direct ? p.xs : p.gs + m.u.group * kt * kMxTileBytes)
                                  : p.hs + m.u.group * kt * kMxTileBytes) +
                           static_cast<int64_t>(m.ks) * kSfBytes;
      const uint32_t stb = base + s * p.stage_bytes + kABytes, ssb = stb + 2 * bbytes + kSfBytes;
      if (m.flags & 1) {
        // a y unit waits for all h of its group (four 32-row quarters per tile), an h unit for
        // its gathered tokens
        const int32_t* flag = first ? (direct ? nullptr : p.xdone + m.u.group) : p.done1 + m.u.group;
        const bool there = !flag || wait_count(flag, first ? 1 : 4 * ht, abort_flag, p.err, 71, p.wait_ns);
        if (!__all_sync(0xFFFFFFFFu, there)) break;
        fence_proxy_async_global();
      }
      if (elect_one()) {
        if (wide) {
          mbar_arrive_expect_tx(full(s), 2 * bbytes + m.nkt * kMxTileBytes);
          tma_load_3d(stb, mx, full(s), 0, xrow, 2 * m.ks);
        } else {
          const int pieces = (m.nkt + 1) / 2;
          mbar_arrive_expect_tx(full(s), pieces * bbytes + m.nkt * kMxTileBytes);
          for (int c = 0; c < pieces; ++c)
            tma_load_2d(stb + c * bbytes, mx, full(s), (2 * m.ks + c) * 128, xrow);
        }
        bulk_load(ssb, sfb, m.nkt * kMxTileBytes, full(s));
      }
      __syncwarp();
      ++it;
      if (++s == S) {
        s = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) sh.joined = it;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    uint32_t it = 0, s = 0, phase = 0, units = 0;
    const uint32_t idesc = idesc_mxf4(128, p.n);
    const uint32_t bbytes = p.n * 128u;
    while (warp_wait(full(s), phase, abort_flag, p.err, 73, p.wait_ns)) {
      ++it;
      tc_fence_after();
      const StageMeta m = sh.meta[s];
      if (m.u.kind == 0) {  // no more work: every group gets that as its next unit
        for (int i = 0; i < kGroups; ++i, ++units) {
          const uint32_t a = units % kGroups;
          if (units >= kGroups &&
              !warp_wait(tempty(a), (units / kGroups - 1) & 1, abort_flag, p.err, 74, p.wait_ns))
            break;
          if (elect_one()) {
            sh.acc_unit[a] = m.u;
            mbar_arrive(tfull(a));
            mbar_arrive(tfull(a));
          }
          __syncwarp();
        }
        break;
      }
      const uint32_t acc = units % kGroups, tacc = tmem + acc * kAccCols;
      if ((m.flags & 1) && units >= kGroups) {
        if (!warp_wait(tempty(acc), (units / kGroups - 1) & 1, abort_flag, p.err, 74, p.wait_ns)) break;
        tc_fence_after();
      }
      const uint32_t st = base + s * p.stage_bytes, stb = st + kABytes;
      const uint32_t ssa = stb + 2 * bbytes, ssb = ssa + kSfBytes;
      const uint32_t tsf = tmem + kSfCol0 + s * kSfCols;
      if (m.u.kind == 3) {  // handed on without MMAs
        if (elect_one()) {
          mbar_arrive(empty(s));
          sh.acc_unit[acc] = m.u;
          mbar_arrive(tfull(acc));
          mbar_arrive(tfull(acc));
        }
      } else if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kStageKt; ++i) {
          if (i < m.nkt) {
            tmem_cp_scales(tsf + 4 * i, ssa + i * kMxTileBytes);
            tmem_cp_scales(tsf + 4 * kStageKt + 4 * i, ssb + i * kMxTileBytes);
          }
        }
        const uint64_t da = smem_desc_sw128(st, 16, 1024), db = smem_desc_sw128(stb, 16, 1024);
#pragma unroll
        for (int j = 0; j < 2 * kStageKt; ++j) {
          if (j < 2 * m.nkt) {
            const uint32_t id = (j & 1) * 2;
            umma_mxf4(tacc, da + (j >> 2) * (kABytes / 2 / 16) + 2 * (j & 3),
                      db + (j >> 2) * (bbytes / 16) + 2 * (j & 3), idesc | (id << 4) | (id << 29),
                      tsf + 4 * (j >> 1), tsf + 4 * kStageKt + 4 * (j >> 1),
                      !(m.flags & 1) || j > 0);
          }
        }
        umma_commit(empty(s));
        if (m.flags & 2) {
          sh.acc_unit[acc] = m.u;
          umma_commit(tfull(acc));
          mbar_arrive(tfull(acc));
        }
      }
      __syncwarp();
      if (m.flags & 2) ++units;
      if (++s == S) {
        s = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
    if (lane == 0) sh.landed = it;
    if (elect_one()) umma_commit(drain);  // every MMA issued is complete before TMEM is freed
    mbar_wait(drain, 0, nullptr, p.err, 75, p.wait_ns);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- finishing units
    const int qd = warp & 3;             // rows 32 qd .. of the tile
    const uint32_t acc = (warp >> 2) - 1;  // this group's accumulator
    for (uint32_t i = 0;; ++i) {
      // one answer for the warp: the tcgen05.ld below is .sync.aligned
      if (!warp_wait(tfull(acc), i & 1, abort_flag, p.err, 76, p.wait_ns)) break;
      const Unit un = sh.acc_unit[acc];
      if (un.kind == 0) break;
      if (un.kind == 3) {
        // 32 columns of a token, in slot order; the units of its experts are all older.  (Combining a
        // token in the unit of its last expert left most of them to the last few units: a tail of 5 us
        // at 32 tokens over 64 experts.)
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty(acc));
        const int t = un.group, col = 128 * un.tile + 32 * qd + lane;
        float o = 0.0f;
        bool ok = true;
#pragma unroll 1
        for (int jb = 0; ok && jb < p.k; jb += 8) {
          float v[8];
          ok = get_sums([&](int i) { return p.y + static_cast<int64_t>(row_of(sh, t, jb + i)) * p.d + col; },
                        min(8, p.k - jb), v, abort_flag, p.err, 79, p.wait_ns);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (jb + j < p.k) o = fmaf(sh.gate[t][jb + j], v[j], o);
        }
        if (!ok) break;
        p.out[static_cast<int64_t>(t) * p.d + col] = bf16_bits(o);
        continue;
      }
      tc_fence_after();
      const uint32_t tacc = tmem + acc * kAccCols + (static_cast<uint32_t>(32 * qd) << 16);
      float v[kMaxN];
#pragma unroll
      for (int c = 0; c < kMaxN; c += 16) {
        float x[16];
        if (c < p.n) {
          tmem_ld16(tacc + c, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[c + j] = x[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(acc));
      const Group gr = sh.group[un.group];
      const auto active = [&](int c) { return direct ? ((gr.tokens >> c) & 1u) != 0u : c < gr.n; };
      const auto row_at = [&](int c) {
        return gr.row0 + (direct ? __popc(gr.tokens & ((1u << c) - 1u)) : c);
      };
      const auto sum = [&](int c) {  // the terms' products, the smallest first
        float a = v[c * kTerms + kTerms - 1];
#pragma unroll
        for (int r = kTerms - 2; r >= 0; --r) a += v[c * kTerms + r];
        return a;
      };
      // 32 columns of this K range's x W1 or x W3, or of y, per token
      const bool first = un.kind == 1;
      float* dst = first ? p.part + (static_cast<int64_t>(un.tile) * Q + un.q) * 128 + 32 * qd + lane
                         : p.y + 128 * un.tile + 32 * qd + lane;
      const int64_t row_stride = first ? static_cast<int64_t>(ht) * Q * 128 : p.d;
#pragma unroll
      for (int c = 0; c < kTok; ++c)
        if (active(c)) put_sum(dst + row_at(c) * row_stride, sum(c));
      if (first) {
        if (un.q != Q - 1) continue;
        // the last range of W3: the others' units are older, so running CTAs hold them.  h of a
        // 32-value block per token, in MXFP4 terms
        const int row_bytes = p.dff / 2;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok && c < p.cols; ++c) {
          if (!active(c)) continue;
          const float* src = dst + row_at(c) * row_stride - un.q * 128;
          float a = 0.0f, b = 0.0f;
#pragma unroll 1
          for (int q = 0; ok && q < Q; q += 8) {
            float v[8];
            ok = get_sums([&](int i) { return src + (q + i) * 128; }, min(8, Q - q), v, abort_flag,
                          p.err, 78, p.wait_ns);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              a += v[i];
              b += v[i + 1];
            }
          }
          float h = a / (1.0f + expf(-a)) * b;
          uint8_t* hq = p.hq + (static_cast<int64_t>(un.group) * p.cols + c) * kTerms * row_bytes +
                        64 * un.tile + 16 * qd + lane / 2;
          uint8_t* hs = p.hs + (static_cast<int64_t>(un.group) * ht + un.tile) * kMxTileBytes;
#pragma unroll 1
          for (int r = 0; r < kTerms; ++r, hq += row_bytes) {
            const uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
            const uint32_t s = term_scale(amax);
            const uint32_t mine = e2m1(s == 255u ? 0.0f : h * mx_inverse_scale(s));
            h = fmaf(-e2m1_value(mine), mx_scale(s), h);
            // eight lanes' codes in the first one's word
            uint32_t code = mine;
            code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 4;
            code |= __shfl_down_sync(0xFFFFFFFFu, code, 2) << 8;
            code |= __shfl_down_sync(0xFFFFFFFFu, code, 4) << 16;
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(hq) = code;
            if (lane == 0) hs[sf_at(c * kTerms + r, qd)] = static_cast<uint8_t>(s);
          }
        }
        if (!ok) break;
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release_add(p.done1 + un.group, 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // After an abort copies may still be in flight: they land before the CTA ends.  At most a ring of
  // fills (a slot is given out again only after its fill landed); where the activations' loader
  // left before it joined one, its arrival is made up for.
  if (threadIdx.x == 0)
    for (uint32_t f = sh.landed; f < sh.given; ++f) {
      if (f >= sh.joined) mbar_arrive(full(f % S));
      mbar_wait(full(f % S), (f / S) & 1, nullptr, p.err, 72, p.wait_ns);
    }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status_t check_few(int64_t T, int d, int E, int k, int dff) {
  if (T < 0 || d <= 0 || E <= 0 || k <= 0 || dff <= 0 || k > E) return MOE_ERR_INVALID_ARG;
  if (T > kMaxT || k > kMaxK || E > kMaxE || d % 128 != 0 || dff % 128 != 0 || d > 65536 ||
      dff > 65536 || static_cast<int64_t>(E) * d > INT32_MAX ||
      static_cast<int64_t>(E) * dff > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Map of `rows` rows of `inner` bytes, boxes of 128 bytes x box_rows, 128-byte swizzle.  `wide`:
// inner is a multiple of 128; the 128-byte pieces of a row are an outer dimension and a box
// holds two, so a stage is one copy.  (Issuing a copy takes its thread some 170 cycles: eight of
// them per 16 KB stage held the stream at 2 TB/s.)  Otherwise a box is one piece, zeros past the
// row's end.
CUtensorMap make_piece_map(const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                           bool wide, cudaError_t* st) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  CUtensorMap m = {};
  auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
  const cuuint64_t dims[3] = {wide ? 128 : inner, rows, inner / 128};
  const cuuint64_t strides[2] = {inner, 128};
  const cuuint32_t box[3] = {128, box_rows, 2};
  const cuuint32_t ones[3] = {1, 1, 1};
  if (!enc || enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, wide ? 3 : 2, const_cast<void*>(base), dims,
                  strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    *st = cudaErrorInvalidValue;
  return m;
}

// U pieces of 1024 values in flight: 4 for narrow routers, which would load tokens for pieces that
// they do not have, 8 for wide ones, which would wait for a second round of loads.  A whole call with
// U = 4 and 8, 256 experts of d_ff = 128, routers out of HBM: 8 tokens of d = 1024 14.07 and 14.26 us, of
// 2560 15.97 and 16.25; one token of 4096 15.35 and 14.48, of 7168 17.50 and 16.08, of 12288 21.02 and
// 18.62.
template <int TB>
cudaError_t launch_router(const RouterParams& p, int grid, cudaStream_t s) {
  const auto kern = p.d < 4096 ? few_router_kernel<TB, 4> : few_router_kernel<TB, 8>;
  return launch_pdl(kern, dim3(grid, p.router ? (p.T + TB - 1) / TB : 1), dim3(kRouterThreads), 0, s, p);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_bytes(int64_t T, int d, int E, int k, int d_ff) {
  if (check_few(T, d, E, k, d_ff) != MOE_OK) return 0;
  return few_layout(T, d, E, k, d_ff).total;
}

moe_status_t moe_forward_few_fp4(const moe_bf16_t* x, float* logits, const float* router,
                                 const uint8_t* W1q, const uint8_t* W3q, const uint8_t* W2q,
                                 const uint8_t* w1_scales, const uint8_t* w3_scales,
                                 const uint8_t* w2_scales, int64_t T, int d, int E, int k, int d_ff,
                                 moe_bf16_t* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status_t c = check_few(T, d, E, k, d_ff);
  if (c != MOE_OK) return c;
  if (T == 0) return MOE_OK;
  const void* req[] = {x, logits, W1q, W3q, W2q, w1_scales, w3_scales, w2_scales, out, ws};
  for (const void* q : req)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (router && !aligned16(router)) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return MOE_ERR_INVALID_ARG;
  const FewLayout L = few_layout(T, d, E, k, d_ff);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  const auto bytes = [&](size_t at) { return reinterpret_cast<uint8_t*>(w + at); };
  const auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(w + at); };

  RouterParams r = {};
  r.x = x;
  r.router = router;
  r.logits = logits;
  r.T = static_cast<int>(T);
  r.d = d;
  r.E = E;
  r.err = reinterpret_cast<DevErr*>(w + L.err);
  r.clear = ints(L.ticket);
  r.n_clear = static_cast<int64_t>((L.clear_end - L.ticket) / 4);
  r.places = reinterpret_cast<uint4*>(w + L.part);  // part and y lie side by side
  r.n_places = static_cast<int64_t>((L.total - L.part) / 16);
  r.xq = bytes(L.xq);
  r.xs = bytes(L.xs);

  ExpertParams p = {};
  cudaError_t st = cudaSuccess;
  p.logits = logits;
  p.T = r.T;
  p.d = d;
  p.E = E;
  p.k = k;
  p.dff = d_ff;
  p.cols = L.cols;
  p.n = (L.cols * kTerms + 15) / 16 * 16;
  p.parts = L.parts;
  p.stage_bytes = kABytes + 2 * p.n * 128 + 2 * kSfBytes;
  const size_t room = 232448 - 1024 - sizeof(Shared);
  p.stages = static_cast<int>(room / p.stage_bytes < kMaxStages ? room / p.stage_bytes : kMaxStages);
  p.s1 = w1_scales;
  p.s3 = w3_scales;
  p.s2 = w2_scales;
  p.s1_bytes = mx_scale_bytes(d_ff, d);
  p.s2_bytes = mx_scale_bytes(d, d_ff);
  p.xq = r.xq;
  p.xs = r.xs;
  p.gq = bytes(L.gq);
  p.gs = bytes(L.gs);
  p.hq = bytes(L.hq);
  p.hs = bytes(L.hs);
  p.part = reinterpret_cast<float*>(w + L.part);
  p.y = reinterpret_cast<float*>(w + L.y);
  p.out = out;
  p.ticket = ints(L.ticket);
  p.done1 = ints(L.done1);
  p.xdone = ints(L.xdone);
  p.err = r.err;
  p.wait_ns = wait_limit_ns();
  p.withhold = withheld_loaders();
  p.wide1 = d % 256 == 0;
  p.wide2 = d_ff % 256 == 0;
  const uint64_t rows = static_cast<uint64_t>(L.cols) * kTerms, groups = static_cast<uint64_t>(L.groups);
  p.map1 = make_piece_map(W1q, d / 2, static_cast<uint64_t>(E) * d_ff, 128, p.wide1, &st);
  p.map3 = make_piece_map(W3q, d / 2, static_cast<uint64_t>(E) * d_ff, 128, p.wide1, &st);
  p.map2 = make_piece_map(W2q, d_ff / 2, static_cast<uint64_t>(E) * d, 128, p.wide2, &st);
  p.mapx = make_piece_map(T <= kTok ? p.xq : p.gq, d / 2, T <= kTok ? rows : groups * rows, p.n,
                          p.wide1, &st);
  p.maph = make_piece_map(p.hq, d_ff / 2, groups * rows, p.n, p.wide2, &st);
  if (st != cudaSuccess) return MOE_ERR_CUDA;

  const int sms = num_sms_of_current_device();
  const int64_t conv = T * ((d + kRouterThreads * 8 - 1) / (kRouterThreads * 8));
  r.conv = static_cast<int>(conv < sms ? conv : sms);
  int rgrid = r.conv + (router ? (E + kRouterExperts - 1) / kRouterExperts : 0);
  const int64_t marking = r.n_places / (4 * kRouterThreads);  // CTAs of four stores a thread
  if (rgrid < 2 * sms && rgrid < marking) rgrid = static_cast<int>(marking < 2 * sms ? marking : 2 * sms);
  st = T <= 1   ? launch_router<1>(r, rgrid, stream)
       : T <= 4 ? launch_router<4>(r, rgrid, stream)
                : launch_router<8>(r, rgrid, stream);
  if (st != cudaSuccess) return MOE_ERR_CUDA;

  static std::atomic<unsigned long long> attr_set_mask{0ull};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit == 0ull || !(attr_set_mask.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(few_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             232448) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set_mask.fetch_or(bit, std::memory_order_release);
  }
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + sizeof(Shared);
  const int64_t units = T * k * (d_ff / 128 * 2 * L.parts + d / 128) + T * (d / 128);
  st = launch_pdl(few_experts_kernel, dim3(static_cast<unsigned>(units < sms ? units : sms)),
                  dim3(kThreads), smem, stream, p);
  return st == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
