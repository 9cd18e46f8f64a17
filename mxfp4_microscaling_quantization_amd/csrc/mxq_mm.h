// Device-side building blocks of the matrix products: fragments of the 32x32 matrix
// instructions and the epilogue.
#pragma once

#include "mxq_device.h"
#include "mxq_mm_launch.h"
#include "mxq_mm_segments.h"

namespace mxq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Codes of the f8f6f4 matrix instructions' format fields.
constexpr int kE4M3 = 0, kE2M1 = 4;

// ---------------------------------------------------------------------------
// Fragments. A lane of a 32x32x64 instruction holds 32 elements of operand row
// (lane % 32): with h = lane / 32, E2M1 elements [32h, 32h + 32) in 16 bytes, and E4M3
// elements [16h, 16h + 16) and [32 + 16h, 48 + 16h) in 32 bytes (checked on the chip);
// the scale byte of lane half h multiplies elements [32h, 32h + 32).
// Result register i of a lane is row 8 (i / 4) + 4h + i % 4 of the first operand and
// row (lane % 32) of the second. The weight goes first, so a lane holds runs of four
// consecutive output columns of one output row.

__device__ __forceinline__ v8i widen(v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// Eight elements (a bf16 fragment of a 32x32x16 instruction) from E4M3 bytes or E2M1
// codes, times the scale: exact, E4M3 and E2M1 significands have at most 4 bits.
__device__ __forceinline__ bf16x8 bf16_from_e4m3(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ bf16x8 bf16_from_e2m1(uint32_t w, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------------------
// Activations and their derivatives in fp32. exp and the reciprocal are the hardware's
// (about 1e-7 relative).
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}
constexpr float kGeluA = 1.5957691216057308f;          // 2 sqrt(2/pi)
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;
// tanh(u) = 2 sigmoid(2u) - 1, so the tanh form of GELU is z sigmoid(2u).
__device__ __forceinline__ float gelu_f(float z) {
  const float w = z * fmaf(-kLog2e * kGeluB, z * z, -kLog2e * kGeluA);
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w));
}

__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActGelu: return gelu_f(z);
    case kActSilu: return z * sigmoid_f(z);
  }
  return z;
}

// ---------------------------------------------------------------------------
// Epilogue of V consecutive columns [n0, n0 + V) of one row: bias, z, activation,
// residual. V is 4 or 8 and n0 a multiple of V. Rows are `vec` when every row of d, z
// and the residual starts on a V-element boundary (n % V == 0), else element by element.
template <typename T>
struct Out;
template <>
struct Out<float> {
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};
template <>
struct Out<__bf16> {
  static __device__ __forceinline__ float get(const __bf16* p) { return (float)*p; }
  static __device__ __forceinline__ void put(__bf16* p, float v) { *p = (__bf16)v; }
};

// Buffers are 16-byte aligned, so a run of more than 16 bytes is not known to be aligned further.
template <typename T, int V>
constexpr int kRunAlign = sizeof(T) * V < 16 ? sizeof(T) * V : 16;
template <typename T, int V>
__device__ __forceinline__ void put_run(T* p, const float (&v)[V]) {
  T t[V];
#pragma unroll
  for (int i = 0; i < V; ++i) Out<T>::put(&t[i], v[i]);
  __builtin_memcpy(__builtin_assume_aligned(p, (kRunAlign<T, V>)), t, sizeof(T) * V);
}
template <typename T, int V>
__device__ __forceinline__ void get_run(const T* p, float (&v)[V]) {
  T t[V];
  __builtin_memcpy(t, __builtin_assume_aligned(p, (kRunAlign<T, V>)), sizeof(T) * V);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = Out<T>::get(&t[i]);
}

// Stores V values (n0 + i < n) at p[0..], adding a residual first.
template <typename T, int V>
__device__ __forceinline__ void store_run(T* p, const T* res, float (&v)[V], int64_t left, bool vec) {
  if (vec) {
    if (res) {
      float r[V];
      get_run<T, V>(res, r);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += r[i];
    }
    put_run<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) Out<T>::put(p + i, res ? v[i] + Out<T>::get(res + i) : v[i]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void epilogue_run(const MmEpilogue& ep, int64_t row, int group, int64_t n0,
                                             float (&z)[V]) {
  const int64_t left = ep.n - n0;
  if (left <= 0) return;
  const bool vec = ep.n % V == 0;
  if (ep.bias) {
    const int64_t at = (int64_t)group * ep.n + n0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left)
        z[i] += ep.bias_f32 ? static_cast<const float*>(ep.bias)[at + i]
                            : (float)static_cast<const __bf16*>(ep.bias)[at + i];
  }
  if (ep.z) store_run<T, V>(static_cast<T*>(ep.z) + row * ep.n + n0, nullptr, z, left, vec);
  if (ep.act == kActSwiglu) {
    float d[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) d[i] = z[2 * i] * sigmoid_f(z[2 * i]) * z[2 * i + 1];
    const int64_t at = row * (ep.n / 2) + n0 / 2;
    store_run<T, V / 2>(static_cast<T*>(ep.d) + at, ep.res ? static_cast<const T*>(ep.res) + at : nullptr, d,
                        left / 2, vec);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = act_f(z[i], ep.act);
    const int64_t at = row * ep.n + n0;
    store_run<T, V>(static_cast<T*>(ep.d) + at, ep.res ? static_cast<const T*>(ep.res) + at : nullptr, z, left,
                    vec);
  }
}

// The same for one lane that finishes V fixed columns of many rows from sums in LDS:
// bias, addresses and strides are set up once, U rows are in flight together, and the
// residual's next U are fetched before these are stored.
template <typename T, int V, int U>
struct RunEpilogue {
  float bias[V];
  int64_t at;      // of the next row's results in d (in z twice that where half of d's columns are left)
  int left, rows;  // columns; rows from the next one on
  bool vec, gated;
  T raw[U][V] = {};

  // Rows first, first + STEP, ... below first + `rows` of columns col...
  template <int STEP>
  __device__ __forceinline__ void start(const MmEpilogue& ep, int64_t col, int64_t first, int to_do) {
    gated = ep.act == kActSwiglu;
    at = first * row_step(ep) + (gated ? col / 2 : col);
    left = ep.n - col < V ? (int)(ep.n - col) : V;
    rows = left > 0 ? to_do : 0;
    vec = ep.n % V == 0;
    if (ep.res && vec) fetch<STEP>(ep, 0);
  }

  __device__ __forceinline__ void fetch_bias(const MmEpilogue& ep, int group, int64_t col) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = 0.0f;
      if (ep.bias && i < left) {
        const int64_t b = (int64_t)group * ep.n + col + i;
        bias[i] = ep.bias_f32 ? static_cast<const float*>(ep.bias)[b] : (float)static_cast<const __bf16*>(ep.bias)[b];
      }
    }
  }

  __device__ __forceinline__ int64_t row_step(const MmEpilogue& ep) const { return gated ? ep.n / 2 : ep.n; }

  // The residual's rows `from`, from + 1, ... of those to come.
  template <int STEP>
  __device__ __forceinline__ void fetch(const MmEpilogue& ep, int from) {
    const int64_t step = STEP * row_step(ep);
    const T* p = static_cast<const T*>(ep.res) + at + from * step;
#pragma unroll
    for (int k = 0; k < U; ++k)
      if ((from + k) * STEP < rows) {
        if (gated)
          __builtin_memcpy(raw[k], __builtin_assume_aligned(p + k * step, (kRunAlign<T, V / 2>)), sizeof(T) * V / 2);
        else
          __builtin_memcpy(raw[k], __builtin_assume_aligned(p + k * step, (kRunAlign<T, V>)), sizeof(T) * V);
      }
  }

  // The next N rows, whose sums get(k, z) fetches.
  template <int N, int STEP, typename F>
  __device__ __forceinline__ void finish(const MmEpilogue& ep, F&& get) {
    const int64_t step = STEP * row_step(ep);
#pragma unroll 1
    for (int u = 0; u < N; u += U) {
      float v[U][V];
#pragma unroll
      for (int k = 0; k < U; ++k) get(u + k, v[k]);
      if (ep.bias) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) v[k][i] += bias[i];
      }
      if (ep.z) {
        T* z = static_cast<T*>(ep.z) + (gated ? 2 * at : at);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (k * STEP < rows) store_run<T, V>(z + k * (STEP * ep.n), nullptr, v[k], left, vec);
      }
      if (gated) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < V / 2; ++i) v[k][i] = v[k][2 * i] * sigmoid_f(v[k][2 * i]) * v[k][2 * i + 1];
      } else {
        act_runs(v, ep.act);
      }
      const T* rest = nullptr;
      if (ep.res && vec) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i) v[k][i] += Out<T>::get(&raw[k][i]);  // (gated: half of them count)
        fetch<STEP>(ep, U);
      } else if (ep.res) {
        rest = static_cast<const T*>(ep.res) + at;
      }
      T* d = static_cast<T*>(ep.d) + at;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const T* from = rest ? rest + k * step : nullptr;
        if (k * STEP < rows) {
          if (gated) {
            float g[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) g[i] = v[k][i];
            store_run<T, V / 2>(d + k * step, from, g, left / 2, vec);
          } else {
            store_run<T, V>(d + k * step, from, v[k], left, vec);
          }
        }
      }
      at += U * step;
      rows -= U * STEP;
    }
  }

  // (one uniform branch around all elements: a branch in each cost 45 us of 310 at
  // 8192 x 14336 results)
  static __device__ __forceinline__ void act_runs(float (&v)[U][V], int act) {
    if (act == kActRelu) {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = v[k][i] < 0.0f ? 0.0f : v[k][i];
    } else if (act == kActGelu) {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = gelu_f(v[k][i]);
    } else if (act == kActSilu) {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] *= sigmoid_f(v[k][i]);
    }
  }
};

}  // namespace mxq
