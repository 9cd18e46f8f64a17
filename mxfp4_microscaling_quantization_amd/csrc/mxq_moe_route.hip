// The choice of experts: the k largest logits of every token with their softmax weights, and
// the gradient.
//
// A token has G lanes of a wave (8 to 64, by the number of experts), each of them V logits in
// registers. Every logit is a key that orders as mxq_route says: its value made an unsigned
// number that grows with it, above the expert's complement, so that no two keys are equal and
// of equal values the lower expert is larger; 0 stands for none. k times the largest key of
// the group is found and taken out. For bf16 a key is 32 bits wide, for fp32 64.
#include "mxq_moe.h"

namespace mxq {

namespace {

template <typename T>
struct KeyOf;
template <>
struct KeyOf<__bf16> {
  typedef uint32_t type;
};
template <>
struct KeyOf<float> {
  typedef uint64_t type;
};

// fp32 bits that grow with the value as unsigned numbers; NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = v != v ? 0x7FFFFFFFu : as_u(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return as_f(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

template <typename K>
__device__ __forceinline__ K make_key(float v, uint32_t e) {
  if (v == -__builtin_inff()) return 0;
  if constexpr (sizeof(K) == 4) return (ordered(v) & 0xFFFF0000u) | (0xFFFFu - e);
  else return (K)ordered(v) << 32 | (0xFFFFFFFFu - e);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  // (below zero the bits cut off are ones)
  return unordered(k & 0x80000000u ? k & 0xFFFF0000u : k | 0xFFFFu);
}
__device__ __forceinline__ float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_expert(uint32_t k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
__device__ __forceinline__ int key_expert(uint64_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

template <int G>
__device__ __forceinline__ uint32_t group_max_key(uint32_t k) {
  return reduce32<G>(k, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
// The values first, then the experts of those lanes whose value is the largest.
template <int G>
__device__ __forceinline__ uint64_t group_max_key(uint64_t k) {
  const uint32_t hi = group_max_key<G>((uint32_t)(k >> 32));
  const uint32_t lo = group_max_key<G>((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// Logit i of a lane: runs of 8 lie side by side over the lanes.
template <int G>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return (i >> 3) * (8 * G) + lane * 8 + (i & 7);
}

// The lane's V logits of a row, behind the last one -Inf. vec: rows start on 16 bytes and have a
// multiple of 8 logits.
template <typename T, int G, int V>
__device__ __forceinline__ void load_logits(const T* row, int lane, int experts, bool vec, float (&v)[V]) {
#pragma unroll
  for (int b = 0; b < V / 8; ++b) {
    const int e0 = expert_of<G>(lane, b * 8);
    T t[8];
    if (vec) {
      if (e0 < experts)
        __builtin_memcpy(t, __builtin_assume_aligned(row + e0, 16), sizeof(t));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[b * 8 + i] = e0 < experts ? (float)t[i] : -__builtin_inff();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[b * 8 + i] = e0 + i < experts ? (float)row[e0 + i] : -__builtin_inff();
    }
  }
}

template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_kernel(RouteLaunch p, bool vec) {
  typedef typename KeyOf<T>::type K;
  constexpr int kSlots = G >= 64 ? 1 : 64 / G;  // choices that a lane keeps
  const int lane = threadIdx.x % G;
  const int64_t at = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const int64_t token = at < p.tokens ? at : p.tokens - 1;
  float v[V];
  load_logits<T, G, V>(static_cast<const T*>(p.logits) + token * p.ld, lane, p.experts, vec, v);
  K key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = make_key<K>(v[i], (uint32_t)expert_of<G>(lane, i));
  K mine[kSlots];
  float best = 0.0f;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    mine[s] = 0;
#pragma unroll 1
    for (int r = 0; r < G && s * G + r < p.top_k; ++r) {
      K top = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = key[i] > top ? key[i] : top;
      top = group_max_key<G>(top);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] == top ? (K)0 : key[i];
      if (s == 0 && r == 0) best = key_value(top);
      if (lane == r) mine[s] = top;
    }
  }
  float sum = 0.0f, w[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    w[s] = mine[s] ? exp_f(key_value(mine[s]) - best) : 0.0f;
    if (p.renorm) sum += w[s];
  }
  if (!p.renorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[i] == -__builtin_inff() ? 0.0f : exp_f(v[i] - best);
  }
  sum = group_sum<G>(sum);
  if (at >= p.tokens) return;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = s * G + lane;
    if (j < p.top_k) {
      p.weights[token * p.top_k + j] = mine[s] ? w[s] / sum : 0.0f;
      p.chosen[token * p.top_k + j] = mine[s] ? key_expert(mine[s]) : -1;
    }
  }
}

template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteLaunch p, bool vec, bool vec_out) {
  const int lane = threadIdx.x % G;
  const int64_t at = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const int64_t token = at < p.tokens ? at : p.tokens - 1;
  float v[V];
  if (!p.renorm) load_logits<T, G, V>(static_cast<const T*>(p.logits) + token * p.ld, lane, p.experts, vec, v);
  // S, and every logit's sum of w dw (and of w, with renorm) over the choices of it
  float mean = 0.0f, part[V], share[V];
#pragma unroll
  for (int i = 0; i < V; ++i) part[i] = share[i] = 0.0f;
  for (int j = 0; j < p.top_k; ++j) {
    const int64_t c = token * p.top_k + j;
    const int e = p.chosen[c];
    if ((uint32_t)e >= (uint32_t)p.experts) continue;
    const float w = p.weights[c], x = w * p.dw[c];
    mean += x;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<G>(lane, i) == e) {
        part[i] += x;
        share[i] += w;
      }
  }
  if (!p.renorm) {
    float best = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) best = __builtin_elementwise_maximum(best, v[i]);
    best = group_max<G>(best);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      share[i] = v[i] == -__builtin_inff() ? 0.0f : exp_f(v[i] - best);
      sum += share[i];
    }
    sum = group_sum<G>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // (0: every logit is -Inf)
#pragma unroll
    for (int i = 0; i < V; ++i) share[i] *= inv;
  }
  if (at >= p.tokens) return;
  T* row = static_cast<T*>(p.dlogits) + token * p.experts;
#pragma unroll
  for (int b = 0; b < V / 8; ++b) {
    const int e0 = expert_of<G>(lane, b * 8);
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (T)fmaf(-mean, share[b * 8 + i], part[b * 8 + i]);
    if (vec_out) {
      if (e0 < p.experts) __builtin_memcpy(__builtin_assume_aligned(row + e0, 16), t, sizeof(t));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < p.experts) row[e0 + i] = t[i];
    }
  }
}

bool whole(const void* p, int64_t ld, int experts, int size) {
  return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0 && experts % 8 == 0;
}

template <typename T, int G, int V>
hipError_t launch_g(const RouteLaunch& a, bool grad, hipStream_t st) {
  const dim3 grid((uint32_t)((a.tokens + 256 / G - 1) / (256 / G)));
  const bool vec = whole(a.logits, a.ld, a.experts, sizeof(T));
  if (grad)
    route_grad_kernel<T, G, V><<<grid, 256, 0, st>>>(a, vec, whole(a.dlogits, a.experts, a.experts, sizeof(T)));
  else
    route_kernel<T, G, V><<<grid, 256, 0, st>>>(a, vec);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const RouteLaunch& a, bool grad, hipStream_t st) {
  if (a.experts <= 64) return launch_g<T, 8, 8>(a, grad, st);
  if (a.experts <= 128) return launch_g<T, 16, 8>(a, grad, st);
  if (a.experts <= 256) return launch_g<T, 32, 8>(a, grad, st);
  if (a.experts <= 512) return launch_g<T, 64, 8>(a, grad, st);
  if (a.experts <= 1024) return launch_g<T, 64, 16>(a, grad, st);
  if (a.experts <= 2048) return launch_g<T, 64, 32>(a, grad, st);
  return launch_g<T, 64, 64>(a, grad, st);
}

}  // namespace

hipError_t launch_route(const RouteLaunch& a, hipStream_t st) {
  return a.f32 ? launch_t<float>(a, false, st) : launch_t<__bf16>(a, false, st);
}
hipError_t launch_route_grad(const RouteLaunch& a, hipStream_t st) {
  return a.f32 ? launch_t<float>(a, true, st) : launch_t<__bf16>(a, true, st);
}

}  // namespace mxq
