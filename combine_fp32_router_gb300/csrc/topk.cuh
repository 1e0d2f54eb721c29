// Top-k selection and gate of one token by one warp, shared by the routing kernels.
#pragma once

#include <cstdint>

namespace moe {

// Order key of a logit: an unsigned integer that sorts like the float (larger logit, larger
// key), with -0 folded into +0 so that the two compare equal (the lower expert index then
// wins the tie).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v == 0.0f) v = 0.0f;
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// Top-k and gate of one token, by one warp: k rounds of a warp arg-max (a max-reduction of
// the order keys, then a min-reduction of the expert indices holding that key, so ties go
// to the lower index; the winner is marked taken), then a softmax over the k selected logits
// in fp32, summed in slot order.  v[c] is the logit of expert lane + 32 c.  Lane j < k
// receives slot j's expert and gate.
template <int EPL>
__device__ __forceinline__ void topk_token(const float (&v)[EPL], int E, int k, int lane,
                                           int* sel_e_out, float* gate_out) {
  uint32_t key[EPL];
#pragma unroll
  for (int c = 0; c < EPL; ++c) key[c] = order_key(v[c]);
  uint32_t live = 0;  // bit c: expert lane + 32c exists and is not yet taken
#pragma unroll
  for (int c = 0; c < EPL; ++c)
    if (lane + 32 * c < E) live |= 1u << c;
  int sel_e = 0;
  float sel_v = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;  // a lane with no live expert offers 0, never above a live key
#pragma unroll
    for (int c = 0; c < EPL; ++c)
      if (((live >> c) & 1u) && key[c] > best) best = key[c];
    const uint32_t bk = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t mine = 0xFFFFFFFFu;
#pragma unroll
    for (int c = EPL - 1; c >= 0; --c)
      if (((live >> c) & 1u) && key[c] == bk) mine = static_cast<uint32_t>(lane + 32 * c);
    const uint32_t ew = __reduce_min_sync(0xFFFFFFFFu, mine);
    if ((ew & 31u) == static_cast<uint32_t>(lane)) live &= ~(1u << (ew >> 5));
    if (lane == j) {
      sel_e = static_cast<int>(ew);
      sel_v = order_value(bk);
    }
  }
  const float v0 = __shfl_sync(0xFFFFFFFFu, sel_v, 0);
  const float ex = (lane < k) ? expf(sel_v - v0) : 0.0f;
  float s = 0.0f;
  for (int j = 0; j < k; ++j) s += __shfl_sync(0xFFFFFFFFu, ex, j);
  *sel_e_out = sel_e;
  *gate_out = ex / s;
}

}  // namespace moe
