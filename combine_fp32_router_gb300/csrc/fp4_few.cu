// The whole MoE layer for a few tokens (T <= 32) on MXFP4 experts, in two launches:
//   few_router_kernel  logits = x R^T in fp32 (unless the caller has them), x as fp16 with a
//                      power of two per token, counters cleared
//   few_experts_kernel top-k and gates, both expert products with SwiGLU between, the combine
//
// Bound by reading the chosen experts' weights once, 17/32 byte a value, so the kernel is a
// stream of weight tiles: a producer warp keeps a ring of 16 KB stages full (TMA codes, and
// the scale words and activations beside them), eight warps multiply.  Weights are the M
// operand of mma.sync m16n8k16 (E2M1 to fp16 is one exact conversion per pair), up to eight
// tokens of the expert the N operand: with one token in eight columns the tensor work is
// still far below the stream's time, and the fp16 activations cost nothing in accuracy (fp16
// has bf16's bits and three more; each token's power of two keeps its largest value at 2^14,
// so only values below 2^-28 of it lose bits).  A block's scale is applied to the fp32 partial
// sums of its 32 products.
//
// Work units are (8 tokens of an expert) x 16 columns of h (both projections), then x 32
// columns of y; CTAs take them from a counter in that order, so whoever waits for an h waits
// only for units that running CTAs hold.  Every sum's order is fixed by the sizes: results do
// not depend on the batch or on which CTA did what.
#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>

#include "fp4.cuh"
#include "internal.h"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kMaxT = kFewMaxTokens;
constexpr int kMaxRows = kMaxT * kMaxK;  // (token, slot) pairs
constexpr int kUnitH = 16;               // columns of h per unit
constexpr int kUnitY = 32;               // columns of y per unit
constexpr int kTok = 8;                  // tokens per unit
constexpr int kStageK = 1024;            // values of K per stage: 32 weight rows x 512 bytes
constexpr uint32_t kWBytes = 32 * kStageK / 2;
constexpr uint32_t kScBytes = 32 * 8 * 4;        // 32 rows x 8 words of 4 scales
constexpr uint32_t kActRow = kStageK * 2 + 64;   // + 64: rows on different banks
constexpr uint32_t kHsRow = kStageK / 16 * 4 + 16;
constexpr int kMaxStages = 8;
constexpr int kCons = 16;  // consumer warps: 8 words of scales (128 values) x 2 halves of 16 rows
constexpr int kParts = 8;  // partial sums of an output: one per word
constexpr int kEpi = 4;    // epilogue warps: unit i of a CTA is finished by warp i % kEpi
// warp 0 loads weights, warps 1..16 multiply, 17..20 finish units, 21 loads scales and activations
constexpr int kThreads = 32 * (1 + kCons + kEpi + 1);

struct FewLayout {
  size_t err, ticket, done1, done2, xs, x16, hs, h16, y, total;
};
FewLayout few_layout(int64_t T, int d, int k, int dff) {
  FewLayout L;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t r = at;
    at = (at + n + 255) / 256 * 256;
    return r;
  };
  const size_t P = static_cast<size_t>(T) * k;
  L.err = take(sizeof(DevErr));
  L.ticket = take(4);
  L.done1 = take(kMaxRows * 4);
  L.done2 = take(static_cast<size_t>(d / kUnitY) * 4);
  L.xs = take(T * 4);
  L.x16 = take(T * d * 2);
  L.hs = take(P * (dff / 16) * 4);
  L.h16 = take(P * dff * 2);
  L.y = take(P * d * 4);
  L.total = at;
  return L;
}

// Power of two that brings a largest magnitude (fp32 bits) into [2^14, 2^15), and its inverse;
// held where both are normal numbers.
__device__ __forceinline__ void f16_scale(uint32_t amax, float* mul, float* inv) {
  int e = static_cast<int>(amax >> 23) - 127;
  if (amax == 0u) e = 14;
  e = max(e, -112);
  *mul = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
  *inv = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
}

// ------------------------------------------------------------------------------ router
struct RouterParams {
  const uint16_t* x;
  const float* router;  // null: the logits are given
  float* logits;
  int T, d, E;
  DevErr* err;
  int32_t* clear;  // counters, contiguous
  int n_clear;
  float* xs;
  uint16_t* x16;
};

constexpr int kRouterExperts = 2;  // per CTA
constexpr int kRouterThreads = 256;

// CTA b: token b as fp16 (b < T), then the logits of experts 2 b and 2 b + 1: warp w sums the
// 128-value pieces w, w + 8, ... of d for every token, lanes then warps are added in a fixed
// order.
template <int TB>
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(RouterParams p) {
  griddep_wait();
  __shared__ float red[8][TB][kRouterExperts];
  __shared__ uint32_t amax_sh[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.n_clear; i += kRouterThreads) p.clear[i] = 0;
    if (threadIdx.x == 0) *p.err = DevErr{};
  }
  if (static_cast<int>(blockIdx.x) < p.T) {
    const uint16_t* xr = p.x + static_cast<int64_t>(blockIdx.x) * p.d;
    uint32_t amax = 0;
    for (int c = threadIdx.x * 8; c < p.d; c += kRouterThreads * 8) {
      const uint4 u = ld_v4(xr + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        amax = max(amax, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (lane == 0) amax_sh[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, amax_sh[i]);
    float mul, inv;
    f16_scale(amax, &mul, &inv);
    uint16_t* o = p.x16 + static_cast<int64_t>(blockIdx.x) * p.d;
    for (int c = threadIdx.x * 8; c < p.d; c += kRouterThreads * 8) {
      const uint4 u = ld_v4(xr + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 v = __floats2half2_rn(bf16lo(w[i]) * mul, bf16hi(w[i]) * mul);
        h[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      st_v4(o + c, make_uint4(h[0], h[1], h[2], h[3]));
    }
    if (threadIdx.x == 0) p.xs[blockIdx.x] = inv;
  }
  if (!p.router) return;
  const int e0 = blockIdx.x * kRouterExperts;
  if (e0 >= p.E) return;
  const int ne = min(kRouterExperts, p.E - e0);
  const float* r0 = p.router + static_cast<int64_t>(e0) * p.d;
  const float* r1 = r0 + (ne > 1 ? p.d : 0);
  float acc[TB][kRouterExperts];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t][0] = acc[t][1] = 0.0f;
  constexpr int U = TB <= 8 ? 7 : 2;  // pieces of the router in flight
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
      const int c = c0 + u * 1024 + lane * 4;
      if (c >= p.d) continue;
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (t < p.T) {
          const uint2 xv = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<int64_t>(t) * p.d + c));
          const float x0 = bf16lo(xv.x), x1 = bf16hi(xv.x), x2 = bf16lo(xv.y), x3 = bf16hi(xv.y);
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
  for (int i = threadIdx.x; i < p.T * ne; i += kRouterThreads) {
    const int t = i / ne, j = i % ne;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][t][j];
    p.logits[static_cast<int64_t>(t) * p.E + e0 + j] = v;
  }
}

// ------------------------------------------------------------------------------ experts
struct ExpertParams {
  const float* logits;
  int T, d, E, k, dff;
  int tok;            // token columns kept per stage: min(T, 8)
  int stages;
  uint32_t stage_bytes;
  const uint8_t *s1, *s3, *s2;
  int64_t s1_bytes, s2_bytes;  // scale bytes per expert
  const float* xs;
  const uint16_t* x16;
  float* hs;
  uint16_t* h16;
  float* y;
  uint16_t* out;
  int32_t *ticket, *done1, *done2;
  DevErr* err;
  uint64_t wait_ns;
  // W1 and W3: boxes of 16 rows (8 j + i, i < 4) of 128 bytes, W2: of 32 rows; where a row is a
  // whole number of 128-byte pieces (wide), a box holds four of them side by side
  CUtensorMap map1, map3, map2;
  int wide1, wide2;
};

// A unit's token group: expert, tokens (bits), first row of its h and y rows.
struct Group {
  int32_t e;
  uint32_t tokens;
  int32_t row0;
  int32_t n;
};
struct StageMeta {
  int32_t kind;  // 0: no more work, 1: h unit, 2: y unit
  int32_t group, tile, ks;
};

struct Shared {
  Group group[kMaxRows];
  uint32_t mask[kMaxE];
  int32_t base[kMaxE];  // first row of an expert's tokens
  float gate[kMaxT][kMaxK];
  uint16_t slot_e[kMaxT][kMaxK];
  StageMeta meta[kMaxStages];
  uint64_t bars[3 * kMaxStages + 2 * kEpi];
  StageMeta unit[kEpi];  // the unit whose partial sums a buffer holds
  int32_t groups;
  int32_t abort_flag;
};
// behind Shared: kEpi buffers of partial sums [word][token][32 rows]

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int x,
                                            int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
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
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
// byte i of a scale word as a factor (0 stands for 2^-127, which is 0 beside any other
// block; 255 is handled for the whole row)
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float(((w >> (8 * i)) & 0xFFu) << 23);
}

// One stage of one warp: word w of the scales, i.e. 4 blocks of 32 values, for one 16-row half
// (`rows`: its 16 x 128-byte box, `sc`: its words).  KIND 2: the activations' own factors (16
// values each) are applied to the two halves of a block.
template <int KIND>
__device__ __forceinline__ void multiply(uint32_t rows, uint32_t sc, uint32_t act, uint32_t hs,
                                         int w, int lane, int tok, float (&acc)[4],
                                         uint32_t (&bad)[2]) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t r0 = rows + g * 128 + 4 * t;
  const uint32_t b0 = act + min(g, tok - 1) * kActRow + (w * 128 + 8 * t) * 2;
  const uint32_t h0 = hs + min(2 * t, tok - 1) * kHsRow + w * 32;
  const uint32_t h1 = hs + min(2 * t + 1, tok - 1) * kHsRow + w * 32;
  // every shared-memory read of the stage first: a warp has little else to hide their latency
  uint32_t wv[4][2];
  uint4 x[4];
  float2 f0[4], f1[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t chunk = (((w & 1) * 4 + b) ^ g) << 4;
    wv[b][0] = lds32(r0 + chunk);
    wv[b][1] = lds32(r0 + 1024 + chunk);
    x[b] = lds128(b0 + b * 64);
    if constexpr (KIND == 2) {
      f0[b] = lds_f2(h0 + b * 8);
      f1[b] = lds_f2(h1 + b * 8);
    }
  }
  const uint32_t slo = lds32(sc + g * 4), shi = lds32(sc + (8 + g) * 4);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    uint32_t a[4], c[4];
    e2m1x8_to_half(wv[b][0], a);
    e2m1x8_to_half(wv[b][1], c);
    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    mma_f16(p, a[0], c[0], a[1], c[1], x[b].x, x[b].y);
    if constexpr (KIND == 2) {
      float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma_f16(q, a[2], c[2], a[3], c[3], x[b].z, x[b].w);
      p[0] = fmaf(q[0], f0[b].y, p[0] * f0[b].x);
      p[1] = fmaf(q[1], f1[b].y, p[1] * f1[b].x);
      p[2] = fmaf(q[2], f0[b].y, p[2] * f0[b].x);
      p[3] = fmaf(q[3], f1[b].y, p[3] * f1[b].x);
    } else {
      mma_f16(p, a[2], c[2], a[3], c[3], x[b].z, x[b].w);
    }
    acc[0] = fmaf(p[0], scale_of(slo, b), acc[0]);
    acc[1] = fmaf(p[1], scale_of(slo, b), acc[1]);
    acc[2] = fmaf(p[2], scale_of(shi, b), acc[2]);
    acc[3] = fmaf(p[3], scale_of(shi, b), acc[3]);
  }
  bad[0] |= __vcmpeq4(slo, 0xFFFFFFFFu);
  bad[1] |= __vcmpeq4(shi, 0xFFFFFFFFu);
}

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

__global__ void __launch_bounds__(kThreads, 1)
    few_experts_kernel(const __grid_constant__ ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Shared& sh = *reinterpret_cast<Shared*>(
      smem_raw + (base - raw) + static_cast<size_t>(p.stages) * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.stages;
  const auto full = [&](int s) { return smem_u32(&sh.bars[s]); };
  const auto empty = [&](int s) { return smem_u32(&sh.bars[kMaxStages + s]); };
  const auto told = [&](int s) { return smem_u32(&sh.bars[2 * kMaxStages + s]); };
  const auto rfull = [&](int i) { return smem_u32(&sh.bars[3 * kMaxStages + i]); };
  const auto rfree = [&](int i) { return smem_u32(&sh.bars[3 * kMaxStages + kEpi + i]); };
  float* red = reinterpret_cast<float*>(&sh + 1);
  const int red_floats = kParts * p.tok * 32;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&sh.abort_flag);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 33);  // the weights' producer with the bytes, 32 lanes' own copies
      mbar_init(empty(s), kCons);
      mbar_init(told(s), 1);   // the stage's meta is written
    }
    for (int i = 0; i < kEpi; ++i) {
      mbar_init(rfull(i), kCons);
      mbar_init(rfree(i), 1);
    }
    fence_mbar_init();
    sh.abort_flag = 0;
    tma_prefetch_desc(&p.map1);
    tma_prefetch_desc(&p.map3);
    tma_prefetch_desc(&p.map2);
  }
  for (int e = threadIdx.x; e < p.E; e += kThreads) sh.mask[e] = 0u;
  __syncthreads();
  griddep_wait();
  for (int t = warp; t < p.T; t += kThreads / 32) {
    if (p.E <= 256) route_token<8>(p, sh, t, lane);
    else route_token<32>(p, sh, t, lane);
  }
  __syncthreads();
  if (warp == 0) {  // groups of up to 8 tokens per chosen expert, in expert order
    int rows = 0, groups = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t m = e < p.E ? sh.mask[e] : 0u;
      const int n = __popc(m), ng = (n + kTok - 1) / kTok;
      int pn = n, pg = ng;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(0xFFFFFFFFu, pn, o), ug = __shfl_up_sync(0xFFFFFFFFu, pg, o);
        if (lane >= o) {
          pn += un;
          pg += ug;
        }
      }
      if (e < p.E) {
        int r = rows + pn - n, gi = groups + pg - ng;
        sh.base[e] = r;
        uint32_t left = m;
        while (left) {
          uint32_t take = 0;
          int c = 0;
          while (left && c < kTok) {
            take |= left & (0u - left);
            left &= left - 1u;
            ++c;
          }
          sh.group[gi++] = Group{e, take, r, c};
          r += c;
        }
      }
      rows += __shfl_sync(0xFFFFFFFFu, pn, 31);
      groups += __shfl_sync(0xFFFFFFFFu, pg, 31);
    }
    if (lane == 0) sh.groups = groups;
  }
  __syncthreads();
  const int groups = sh.groups;
  const int hu = p.dff / kUnitH, yu = p.d / kUnitY;
  const int n1 = groups * hu, n_units = n1 + groups * yu;
  const int kt1 = p.d / 128, kt2 = p.dff / 128;  // scale words per row

  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      uint32_t it = 0, s = 0, phase = 1;  // phase: parity of the empty barrier's last use
      bool ok = true;
      int next = atomicAdd(p.ticket, 1);
      while (true) {
        const int u = next;
        const bool work = u < n_units;
        if (work) next = atomicAdd(p.ticket, 1);  // used after this unit's loads
        const bool first = u < n1;
        const int v = first ? u : u - n1, per = first ? hu : yu;
        const int gi = v / per, tile = v % per;
        const int kt = work ? (first ? kt1 : kt2) : 1;
        const int e = work ? sh.group[gi].e : 0;
        const CUtensorMap* ma = first ? &p.map1 : &p.map2;
        const bool wide = first ? p.wide1 : p.wide2;
        const int y = first ? 4 * (tile & 1) : e * p.d + kUnitY * tile;
        const int z = e * (p.dff / 8) + 4 * (tile >> 1);
        for (int ks = 0; 8 * ks < kt; ++ks) {
          if (it >= static_cast<uint32_t>(S))
            ok = mbar_wait(empty(s), phase, abort_flag, p.err, 70, p.wait_ns);
          if (!ok) break;
          sh.meta[s] = StageMeta{work ? (first ? 1 : 2) : 0, gi, tile, ks};
          mbar_arrive(told(s));
          const uint32_t st = base + s * p.stage_bytes;
          const int boxes = work ? (min(8, kt - 8 * ks) + 1) / 2 : 0;
          if (!work) {
            mbar_arrive(full(s));
          } else if (wide) {
            mbar_arrive_expect_tx(full(s), kWBytes);  // pieces past the row's end are zeros
            if (first) {
              tma_load_4d(st, ma, full(s), 0, y, z, 4 * ks);
              tma_load_4d(st + kWBytes / 2, &p.map3, full(s), 0, y, z, 4 * ks);
            } else {
              tma_load_3d(st, ma, full(s), 0, y, 4 * ks);
            }
          } else {
            mbar_arrive_expect_tx(full(s), boxes * 4096);
            for (int c = 0; c < boxes; ++c) {
              const int x = ks * (kStageK / 2) + 128 * c;
              if (first) {
                tma_load_3d(st + 2048 * c, ma, full(s), x, y, z);
                tma_load_3d(st + kWBytes / 2 + 2048 * c, &p.map3, full(s), x, y, z);
              } else {
                tma_load_2d(st + 4096 * c, ma, full(s), x, y);
              }
            }
          }
          ++it;
          if (++s == static_cast<uint32_t>(S)) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok || !work) break;
      }
      // copies still in flight land before the CTA ends
      if (*abort_flag)
        for (uint32_t i = it > static_cast<uint32_t>(S) ? it - S : 0; i < it; ++i)
          mbar_wait(full(i % S), (i / S) & 1, nullptr, p.err, 72, p.wait_ns);
    }
  } else if (warp == kThreads / 32 - 1) {
    // ---------------------------------------------------------------- scales, activations
    uint32_t s = 0, phase = 0;
    while (true) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(told(s), phase, abort_flag, p.err, 76, p.wait_ns)))
        break;
      const StageMeta m = sh.meta[s];
      if (m.kind == 0) {
        mbar_arrive(full(s));
        break;
      }
      const bool first = m.kind == 1;
      const Group gr = sh.group[m.group];
      const int kt = first ? kt1 : kt2;
      const int words = min(8, kt - 8 * m.ks);
      const uint32_t sc = base + s * p.stage_bytes + kWBytes;
      const uint32_t act = sc + kScBytes, hsm = act + p.tok * kActRow;
      {
        // this lane's weight row
        const int r = first ? 32 * (m.tile >> 1) + 8 * ((lane & 15) >> 2) + 4 * (m.tile & 1) + (lane & 3)
                            : kUnitY * m.tile + lane;
        const uint8_t* sp =
            (first ? (lane < 16 ? p.s1 : p.s3) + gr.e * p.s1_bytes : p.s2 + gr.e * p.s2_bytes) +
            (static_cast<int64_t>(r >> 7) * kt + 8 * m.ks) * kMxTileBytes + (r & 31) * 16 +
            ((r >> 5) & 3) * 4;
        const uint32_t dst = sc + lane * 4;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < words) cp_async_4(dst + j * 128, sp + j * kMxTileBytes);
      }
      // a y unit's activations are there once all h units of its group are
      if (!first && m.ks == 0 &&
          !__all_sync(0xFFFFFFFFu, wait_count(p.done1 + m.group, hu, abort_flag, p.err, 71, p.wait_ns)))
        break;
      uint32_t left = gr.tokens;
      for (int i = 0; i < gr.n; ++i, left &= left - 1u) {
        const uint16_t* src =
            (first ? p.x16 + static_cast<int64_t>(__ffs(left) - 1) * p.d
                   : p.h16 + static_cast<int64_t>(gr.row0 + i) * p.dff) + m.ks * kStageK + lane * 8;
        const uint32_t dst = act + i * kActRow + lane * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j)  // a word of scales stands for 16 pieces of 16 bytes
          if (j * 32 + lane < words * 16) cp_async_16(dst + j * 512, src + j * 256);
      }
      if (!first) {
        // the factors of 16 values each: 32 bytes per word, two pieces of 16 bytes
        for (int i = lane; i < gr.n * 16; i += 32)
          if ((i & 15) < words * 2)
            cp_async_16(hsm + (i >> 4) * kHsRow + (i & 15) * 16,
                        p.hs + static_cast<int64_t>(gr.row0 + (i >> 4)) * (p.dff / 16) +
                            m.ks * (kStageK / 16) + (i & 15) * 4);
      }
      cp_async_arrive_noinc(full(s));
      if (++s == static_cast<uint32_t>(S)) {
        s = 0;
        phase ^= 1;
      }
    }
    cp_async_wait_all();
  } else if (warp <= kCons) {
    // ---------------------------------------------------------------- consumers
    const int w = (warp - 1) & 7, half = (warp - 1) >> 3, g = lane >> 2, tc = 2 * (lane & 3);
    float acc[4] = {};
    uint32_t bad[2] = {};
    uint32_t units = 0, s = 0, phase = 0;
    while (true) {
      if (!mbar_wait(full(s), phase, abort_flag, p.err, 73, p.wait_ns)) break;
      const StageMeta m = sh.meta[s];
      if (m.kind == 0) break;
      const uint32_t st = base + s * p.stage_bytes;
      const uint32_t sc = st + kWBytes, act = sc + kScBytes, hsm = act + p.tok * kActRow;
      const int kt = m.kind == 1 ? kt1 : kt2;
      if (8 * m.ks + w < kt) {
        const uint32_t scw = sc + (w * 32 + half * 16) * 4;
        // h: [W1 | W3] of four 16-row boxes each; y: four 32-row boxes
        if (m.kind == 1)
          multiply<1>(st + half * (kWBytes / 2) + (w >> 1) * 2048, scw, act, hsm, w, lane, p.tok, acc, bad);
        else
          multiply<2>(st + (w >> 1) * 4096 + half * 2048, scw, act, hsm, w, lane, p.tok, acc, bad);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
      if (++s == static_cast<uint32_t>(S)) {
        s = 0;
        phase ^= 1;
      }
      if (8 * (m.ks + 1) < kt) continue;

      // end of a unit: the partial sums go to the epilogue warp whose turn it is
      const int buf = units % kEpi;
      if (units >= kEpi &&
          !mbar_wait(rfree(buf), (units / kEpi - 1) & 1, abort_flag, p.err, 74, p.wait_ns))
        break;
      float* r = red + buf * red_floats + w * p.tok * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (bad[i >> 1]) acc[i] = __uint_as_float(0x7FC00000u);  // a NaN scale in the row
        const int n = tc + (i & 1);
        if (n < p.tok) r[n * 32 + 16 * half + 8 * (i >> 1) + g] = acc[i];
        acc[i] = 0.0f;
      }
      bad[0] = bad[1] = 0u;
      if (warp == 1 && lane == 0) sh.unit[buf] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(rfull(buf));
      ++units;
    }
    // no more units: each epilogue warp gets an empty one
    if (!*abort_flag && warp <= kEpi) {
      const uint32_t last = units + warp - 1;
      const int buf = last % kEpi;
      // all warps have written every unit that this one follows
      bool ok = true;
      if (last >= kEpi)
        ok = mbar_wait(rfree(buf), (last / kEpi - 1) & 1, abort_flag, p.err, 74, p.wait_ns);
      if (ok && lane == 0) {
        sh.unit[buf].kind = 0;
        for (int i = 0; i < kCons; ++i) mbar_arrive(rfull(buf));
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - 1 - kCons;
    const float* r = red + ew * red_floats;
    for (uint32_t i = 0;; ++i) {
      if (!mbar_wait(rfull(ew), i & 1, abort_flag, p.err, 75, p.wait_ns)) break;
      const StageMeta m = sh.unit[ew];
      if (m.kind == 0) break;
      const Group& gr = sh.group[m.group];
      if (m.kind == 1) {
        // two tokens at a time, 16 columns of h each: rows 0..15 are W1's sums, 16..31 W3's
        const int c = lane & 15;
        uint32_t tokens = gr.tokens;
        for (int n0 = 0; n0 < gr.n; n0 += 2) {
          const int n = n0 + (lane >> 4);
          float h = 0.0f;
          if (n < gr.n) {
            const float* rn = r + n * 32 + c;
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int v = 0; v < kParts; ++v) {
              a += rn[v * p.tok * 32];
              b += rn[v * p.tok * 32 + 16];
            }
            const uint32_t tk = (lane >> 4) ? tokens & (tokens - 1u) : tokens;
            const float xs = __ldg(p.xs + __ffs(tk) - 1);
            a *= xs;
            b *= xs;
            h = a / (1.0f + expf(-a)) * b;
          }
          tokens &= tokens - 1u;
          tokens &= tokens - 1u;
          uint32_t amax = __float_as_uint(h) & 0x7FFFFFFFu;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          float mul, inv;
          f16_scale(amax, &mul, &inv);
          if (n < gr.n) {
            const int64_t row = gr.row0 + n;
            p.h16[row * p.dff + 32 * (m.tile >> 1) + 8 * (c >> 2) + 4 * (m.tile & 1) + (c & 3)] =
                __half_as_ushort(__float2half_rn(h * mul));
            if (c == 0) p.hs[row * (p.dff / 16) + m.tile] = inv;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rfree(ew));
        __threadfence();
        __syncwarp();
        if (lane == 0) red_release_add(p.done1 + m.group, 1);
      } else {
        const int col = kUnitY * m.tile + lane;
        for (int n = 0; n < gr.n; ++n) {
          const float* rn = r + n * 32 + lane;
          float v = 0.0f;
#pragma unroll
          for (int i2 = 0; i2 < kParts; ++i2) v += rn[i2 * p.tok * 32];
          __stcg(p.y + static_cast<int64_t>(gr.row0 + n) * p.d + col, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rfree(ew));
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = atomicAdd(p.done2 + m.tile, gr.n) + gr.n == p.T * p.k;
        if (__shfl_sync(0xFFFFFFFFu, last, 0)) {
          // the last rows of these 32 columns: combine them, in slot order
          __threadfence();
          for (int t = 0; t < p.T; ++t) {
            float o = 0.0f;
            for (int j = 0; j < p.k; ++j)
              o = fmaf(sh.gate[t][j],
                       __ldcg(p.y + static_cast<int64_t>(row_of(sh, t, j)) * p.d + col), o);
            p.out[static_cast<int64_t>(t) * p.d + col] = bf16_bits(o);
          }
        }
      }
    }
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

// Map of weight rows for units of h (16 rows 8 j + i, i < 4: the half of a 32-row block that
// shares a factor of h) or of y (32 rows), 128-byte swizzle.  `pieces` (a row is a whole number
// of 128-byte pieces): the pieces are an outer dimension, and a box holds four of them, so a
// stage is one copy per matrix; issuing eight 2 KB boxes per stage instead took the producer
// 1700 cycles, over twice the stage's share of the memory time.  Otherwise a box is one piece,
// zeros past the row's end.
CUtensorMap make_weight_map(const void* base, uint64_t inner, uint64_t rows, bool h, bool pieces,
                            cudaError_t* st) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  CUtensorMap m = {};
  auto enc = reinterpret_cast<Encode>(tensor_map_encoder());
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4];
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  cuuint32_t n = 0;
  const auto dim = [&](uint64_t size, uint64_t stride, uint32_t b) {
    dims[n] = size;
    if (n) strides[n - 1] = stride;
    box[n++] = b;
  };
  dim(pieces ? 128 : inner, 1, 128);
  if (h) {
    dim(8, inner, 4);
    dim(rows / 8, 8 * inner, 4);
  } else {
    dim(rows, inner, 32);
  }
  if (pieces) dim(inner / 128, 128, 4);
  if (!enc || enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, n, const_cast<void*>(base), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    *st = cudaErrorInvalidValue;
  return m;
}

template <int TB>
cudaError_t launch_router(const RouterParams& p, int grid, cudaStream_t s) {
  return launch_pdl(few_router_kernel<TB>, dim3(grid), dim3(kRouterThreads), 0, s, p);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_bytes(int64_t T, int d, int E, int k, int d_ff) {
  if (check_few(T, d, E, k, d_ff) != MOE_OK) return 0;
  return few_layout(T, d, k, d_ff).total;
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
  const FewLayout L = few_layout(T, d, k, d_ff);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);

  RouterParams r = {};
  r.x = x;
  r.router = router;
  r.logits = logits;
  r.T = static_cast<int>(T);
  r.d = d;
  r.E = E;
  r.err = reinterpret_cast<DevErr*>(w + L.err);
  r.clear = reinterpret_cast<int32_t*>(w + L.ticket);
  r.n_clear = static_cast<int>((L.xs - L.ticket) / 4);
  r.xs = reinterpret_cast<float*>(w + L.xs);
  r.x16 = reinterpret_cast<uint16_t*>(w + L.x16);

  ExpertParams p = {};
  cudaError_t st = cudaSuccess;
  p.logits = logits;
  p.T = static_cast<int>(T);
  p.d = d;
  p.E = E;
  p.k = k;
  p.dff = d_ff;
  p.tok = static_cast<int>(T < kTok ? T : kTok);
  p.stage_bytes = static_cast<uint32_t>((kWBytes + kScBytes + p.tok * (kActRow + kHsRow) + 1023) / 1024 * 1024);
  const size_t red_bytes = static_cast<size_t>(kEpi) * kParts * p.tok * 32 * sizeof(float);
  const size_t room = 232448 - 1024 - sizeof(Shared) - red_bytes;
  p.stages = static_cast<int>(room / p.stage_bytes < kMaxStages ? room / p.stage_bytes : kMaxStages);
  p.s1 = w1_scales;
  p.s3 = w3_scales;
  p.s2 = w2_scales;
  p.s1_bytes = mx_scale_bytes(d_ff, d);
  p.s2_bytes = mx_scale_bytes(d, d_ff);
  p.xs = r.xs;
  p.x16 = r.x16;
  p.hs = reinterpret_cast<float*>(w + L.hs);
  p.h16 = reinterpret_cast<uint16_t*>(w + L.h16);
  p.y = reinterpret_cast<float*>(w + L.y);
  p.out = out;
  p.ticket = reinterpret_cast<int32_t*>(w + L.ticket);
  p.done1 = reinterpret_cast<int32_t*>(w + L.done1);
  p.done2 = reinterpret_cast<int32_t*>(w + L.done2);
  p.err = r.err;
  p.wait_ns = wait_limit_ns();
  p.wide1 = d % 256 == 0;
  p.wide2 = d_ff % 256 == 0;
  p.map1 = make_weight_map(W1q, d / 2, static_cast<uint64_t>(E) * d_ff, true, p.wide1, &st);
  p.map3 = make_weight_map(W3q, d / 2, static_cast<uint64_t>(E) * d_ff, true, p.wide1, &st);
  p.map2 = make_weight_map(W2q, d_ff / 2, static_cast<uint64_t>(E) * d, false, p.wide2, &st);
  if (st != cudaSuccess) return MOE_ERR_CUDA;

  int rgrid = router ? (E + kRouterExperts - 1) / kRouterExperts : 1;
  if (rgrid < T) rgrid = static_cast<int>(T);
  st = T <= 1   ? launch_router<1>(r, rgrid, stream)
       : T <= 4 ? launch_router<4>(r, rgrid, stream)
       : T <= 8 ? launch_router<8>(r, rgrid, stream)
                : launch_router<32>(r, rgrid, stream);
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
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + sizeof(Shared) + red_bytes;
  const int64_t units = T * k * (d_ff / kUnitH + d / kUnitY);
  const int sms = num_sms_of_current_device();
  st = launch_pdl(few_experts_kernel, dim3(static_cast<unsigned>(units < sms ? units : sms)),
                  dim3(kThreads), smem, stream, p);
  return st == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
