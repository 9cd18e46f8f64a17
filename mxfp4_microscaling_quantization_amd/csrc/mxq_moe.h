// Device-side building blocks of the operators around the experts' products: accesses at any
// address, reductions over groups of lanes and exponentials.
#pragma once

#include "mxq_device.h"
#include "mxq_moe_launch.h"

namespace mxq {

// 16 and 8 bytes anywhere: the memory system takes them from any address. Rows whose start is no multiple
// of 16 bytes move this way, a row's last elements one by one; past the caches, as whole rows do.
typedef nt_u32x4 any_u32x4 __attribute__((aligned(1)));
typedef nt_u32x2 any_u32x2 __attribute__((aligned(1)));
template <int BYTES>
__device__ __forceinline__ void load_any(void* v, const void* p) {
  static_assert(BYTES == 8 || BYTES % 16 == 0, "");
  if constexpr (BYTES == 8) {
    const nt_u32x2 x = __builtin_nontemporal_load(static_cast<const any_u32x2*>(p));
    __builtin_memcpy(v, &x, 8);
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const nt_u32x4 x = __builtin_nontemporal_load(static_cast<const any_u32x4*>(p) + i);
      __builtin_memcpy(static_cast<char*>(v) + 16 * i, &x, 16);
    }
  }
}
template <int BYTES>
__device__ __forceinline__ void store_any(void* p, const void* v) {
  static_assert(BYTES == 8 || BYTES % 16 == 0, "");
  if constexpr (BYTES == 8) {
    nt_u32x2 x;
    __builtin_memcpy(&x, v, 8);
    __builtin_nontemporal_store((any_u32x2)x, static_cast<any_u32x2*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      nt_u32x4 x;
      __builtin_memcpy(&x, static_cast<const char*>(v) + 16 * i, 16);
      __builtin_nontemporal_store((any_u32x4)x, static_cast<any_u32x4*>(p) + i);
    }
  }
}

constexpr int kHalfMirror = 0x141, kMirror = 0x140;  // lane i of 8 takes lane 7 - i, of 16 lane 15 - i

// The same lane of the other 16 of 32, of the other 32 of 64.
__device__ __forceinline__ uint32_t swap16(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return (threadIdx.x & 16) ? r[0] : r[1];
}
__device__ __forceinline__ uint32_t swap32(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return (threadIdx.x & 32) ? r[0] : r[1];
}

// v combined over groups of N neighbouring lanes (N = 8 to 64), the result in all of them. After
// the first two steps four lanes hold the same, so a mirrored lane stands for the one across.
template <int N, typename Op>
__device__ __forceinline__ uint32_t reduce32(uint32_t v, Op op) {
  static_assert(N >= 8 && N <= 64, "");
  v = op(v, dpp<kQuadSwap1>(v));
  v = op(v, dpp<kQuadSwap2>(v));
  v = op(v, dpp<kHalfMirror>(v));
  if constexpr (N >= 16) v = op(v, dpp<kMirror>(v));
  if constexpr (N >= 32) v = op(v, swap16(v));
  if constexpr (N >= 64) v = op(v, swap32(v));
  return v;
}
template <int N>
__device__ __forceinline__ float group_sum(float v) {
  return as_f(reduce32<N>(as_u(v), [](uint32_t a, uint32_t b) { return as_u(as_f(a) + as_f(b)); }));
}
template <int N>
__device__ __forceinline__ float group_max(float v) {  // NaN if any is
  return as_f(reduce32<N>(as_u(v), [](uint32_t a, uint32_t b) {
    return as_u(__builtin_elementwise_maximum(as_f(a), as_f(b)));
  }));
}

// exp(x) for x <= 0, to about 1.5e-7 relative: x log2(e) in two parts, so that the product's rounding
// does not grow with x. -Inf and far below: 0; NaN: NaN.
__device__ __forceinline__ float exp_f(float x) {
  constexpr float kHi = 1.44269502e+00f, kLo = 1.92596299e-08f;
  const float t = __builtin_elementwise_maximum(x, -200.0f);  // (e^-200 is below the least fp32)
  const float h = t * kHi, l = fmaf(t, kLo, fmaf(t, kHi, -h));
  return __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.0f);
}

}  // namespace mxq
