// The MXFP4 format of the 4-bit expert operators (OCP Microscaling Formats 1.0): blocks of 32
// consecutive values share a power-of-two scale (E8M0, one byte: 2^(s - 127)), the values are
// E2M1 numbers (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two per byte, the earlier one
// in the low nibble.
//
// A row of C values takes Kp / 2 bytes, Kp = C rounded up to a multiple of 128 (the rest is
// zero codes).  The scale bytes are kept in the order in which the tensor cores read them:
// tiles of 128 rows x 4 blocks (128 values) of 512 bytes, tile (r / 128, b / 4) in row-major
// order, and inside a tile byte (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4.  A tile goes to TMEM
// with one tcgen05.cp and lands as one 32-bit word (4 blocks) per row, row r in lane r % 32.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

constexpr int kMxBlock = 32;       // values per scale
constexpr int kMxTileRows = 128;   // rows of a scale tile
constexpr int kMxTileBytes = 512;  // 128 rows x 4 blocks

__host__ __device__ inline int64_t mx_cols(int64_t cols) { return (cols + 127) / 128 * 128; }
__host__ __device__ inline int64_t mx_scale_bytes(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * 128 * (mx_cols(cols) / 32);
}
// Byte of (row, block) in the scale array of a matrix with kt = Kp / 128 tiles per row.
__device__ __forceinline__ int64_t mx_scale_at(int64_t row, int block, int kt) {
  return ((row >> 7) * kt + (block >> 2)) * kMxTileBytes + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (block & 3);
}

// Scale byte of a block whose largest magnitude has the bit pattern `amax` (fp32, sign clear):
// floor(log2(amax)) - 2 puts the largest magnitude in [4, 8), where E2M1 ends at 6.  255 (NaN)
// when the block holds an infinity or a NaN: there is no scale for it, and its finite
// neighbours must not pass for results.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e < 2u ? 0u : e - 2u);
}
// 2^-(s - 127), exact for every s that mx_scale_byte gives (255: zero, so that the block's
// codes are defined)
__device__ __forceinline__ float mx_inverse_scale(uint32_t s) {
  return __uint_as_float(s == 255u ? 0u : (254u - s) << 23);
}
// 2^(s - 127) (s = 0 is the subnormal 2^-127; 255 is NaN)
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7FC00000u : s << 23));
}

// Four bytes of codes of eight values already divided by their scale (nearest, ties to even,
// saturating at 6)
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// One such code, and the value of one
__device__ __forceinline__ uint32_t e2m1(float v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "mov.b32 %0, {a, a, a, a};\n\t}"
      : "=r"(r)
      : "f"(v), "f"(0.0f));
  return r & 15u;
}
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m <= 4u ? 0.5f * static_cast<float>(m) : (m < 7u ? static_cast<float>(m) - 2.0f : 6.0f);
  return (code & 8u) ? -v : v;
}
// Eight codes (four bytes) -> four half2 pairs, exact
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 512 bytes of a scale tile -> 4 TMEM columns, the 32 lanes repeated in each lane quadrant
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr) {
  // no swizzle, 8-row groups of 128 bytes
  const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;"
      "\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// Instruction descriptor of kind::mxf4: E2M1 operands, both K-major, E8M0 scales, K = 64; the
// scale ids (bytes 0 or 2 of the scale word) are or-ed in per instruction.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27);
}

// One lane of a converged warp.  The warps that issue copies and MMAs run their loops as whole
// warps and elect a lane only around the issue itself: the operands then stay in uniform
// registers.  With the loops inside `if (lane == 0)` every tcgen05 or TMA instruction cost its
// thread 100 to 170 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// mbar_wait by a whole warp, with one answer for all of it
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          DevErr* err, int site, uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, err, site, limit_ns));
}

}  // namespace moe
