// E4M3 with a power-of-two scale for each 128 columns of a row: the encoder of 8 values per
// lane, a group being 16 neighbouring lanes.
#pragma once

#include "mxq_blocks.h"
#include "mxq_moe.h"

namespace mxq {

// Eight values of a lane -> E4M3 bytes, and the group's scale 2^i: i = e - 8 for a largest magnitude
// of 2^e to 1.75 * 2^e (448 = 1.75 * 2^8), else e - 7. x / 2^i is exact wherever E4M3 can tell it
// from zero, and the conversion rounds it to nearest, ties to even.
__device__ __forceinline__ uint2 fp8_encode8(const float (&v)[8], float& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, as_u(v[i]) & 0x7FFFFFFFu);
  m = reduce32<16>(m, [](uint32_t a, uint32_t b) { return max(a, b); });
  const bool bad = m >= 0x7F800000u;  // NaN or Inf
  const int field = m == 0u ? 127 : max((int)((m + 0x1FFFFFu) >> 23) - 8, 1);
  const float down = as_f((uint32_t)(254 - (bad ? 127 : field)) << 23);
  scale = as_f(bad ? 0x7FC00000u : (uint32_t)field << 23);
  uint2 r;
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0] * down, v[1] * down, 0, false);
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * down, v[3] * down, (int)r.x, true);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4] * down, v[5] * down, 0, false);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] * down, v[7] * down, (int)r.y, true);
  return bad ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu) : r;
}

// The scale that a product or a gradient reads: 2^(exponent field - 127), NaN for 255.
__device__ __forceinline__ float fp8_scale(uint32_t bits) {
  const uint32_t field = bits >> 23 & 255u;
  return as_f(field == 255u ? 0x7FC00000u : field ? field << 23 : 0x00400000u);
}

}  // namespace mxq
