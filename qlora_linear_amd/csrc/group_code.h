// Device helpers shared by the kernels that write 4-bit codes of groups of values
// (w4_quant.hip, kv4_append.hip): rows as float32, a group's extrema, its scale.
#pragma once

#include "device_common.h"

namespace lnf4 {

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}

// The float32 quotient r / d for d = 7 or 15, r >= 0 finite: the product with the rounded
// reciprocal c and one correction by its exact remainder. The correctly rounded quotient
// for every such r (compared with the division for all 2^31 of them, subnormal ones too); the
// product alone moves one scale in 10^5 by a bf16 step where the quotient is next to a tie.
__device__ __forceinline__ float quotient_of(float r, float d, float c) {
  const float p = r * c;
  return __builtin_fmaf(__builtin_fmaf(-p, d, r), c, p);
}

// Minimum and maximum over the 4, 8 or 16 consecutive lanes of a group, by lane moves
// inside a row of 16: neighbours, then pairs, are exchanged; after that quads hold one
// value each and mirrors join them.
template <int CTRL>
__device__ __forceinline__ void join_extrema(float& lo, float& hi) {
  auto moved = [](float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  };
  lo = fminf(lo, moved(lo));
  hi = fmaxf(hi, moved(hi));
}
__device__ __forceinline__ void group_extrema(int group, float& lo, float& hi) {
  join_extrema<0xB1>(lo, hi);                     // quad_perm 1 0 3 2
  join_extrema<0x4E>(lo, hi);                     // quad_perm 2 3 0 1
  if (group >= 64) join_extrema<0x141>(lo, hi);   // row_half_mirror
  if (group >= 128) join_extrema<0x140>(lo, hi);  // row_mirror
}

}  // namespace lnf4
