// E4M3 with a power-of-two scale for each 128 columns of a row: encoders with a
// group spread over neighbouring lanes.
#pragma once

#include "mxq_blocks.h"
#include "mxq_moe.h"

namespace mxq {

// The scale's exponent field for a group's largest magnitude bits (below 0x7F800000): 2^i, i = e - 8
// for a largest magnitude of 2^e to 1.75 * 2^e (448 = 1.75 * 2^8), else e - 7; 1 for zeros.
__device__ __forceinline__ uint32_t fp8_field(uint32_t amax) {
  return amax == 0u ? 127u : (uint32_t)max((int)((amax + 0x1FFFFFu) >> 23) - 8, 1);
}

// N values of a lane -> E4M3 bytes under the scale of the group, LANES neighbouring lanes. x / 2^i is
// exact wherever E4M3 can tell it from zero, and the conversion rounds it to nearest, ties to even.
template <int N, int LANES>
__device__ __forceinline__ void fp8_encode(const float (&v)[N], uint32_t (&q)[N / 4], uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, as_u(v[i]) & 0x7FFFFFFFu);
  m = reduce32<LANES>(m, [](uint32_t a, uint32_t b) { return max(a, b); });
  const bool bad = m >= 0x7F800000u;  // NaN or Inf
  const uint32_t field = bad ? 127u : fp8_field(m);
  const float down = as_f((254u - field) << 23);
  scale = bad ? 0x7FC00000u : field << 23;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * down, v[4 * i + 1] * down, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * down, v[4 * i + 3] * down, r, true);
    q[i] = bad ? 0x7F7F7F7Fu : (uint32_t)r;
  }
}

// Sixteen neighbouring values, as they lie in memory (bf16, fp32).
__device__ __forceinline__ uint4 fp8_encode16(const uint4 (&w)[2], uint32_t& scale, uint16_t) {
  const uint32_t d[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = as_f(d[i] << 16);
    v[2 * i + 1] = as_f(d[i] & 0xFFFF0000u);
  }
  uint32_t q[4];
  fp8_encode<16, 8>(v, q, scale);
  return make_uint4(q[0], q[1], q[2], q[3]);
}
__device__ __forceinline__ uint4 fp8_encode16(const uint4 (&w)[4], uint32_t& scale, float) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = as_f(w[i].x); v[4 * i + 1] = as_f(w[i].y); v[4 * i + 2] = as_f(w[i].z); v[4 * i + 3] = as_f(w[i].w);
  }
  uint32_t q[4];
  fp8_encode<16, 8>(v, q, scale);
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// The scale that a product or a gradient reads: 2^(exponent field - 127), NaN for 255.
__device__ __forceinline__ float fp8_scale(uint32_t bits) {
  const uint32_t field = bits >> 23 & 255u;
  return as_f(field == 255u ? 0x7FC00000u : field ? field << 23 : 0x00400000u);
}

}  // namespace mxq
