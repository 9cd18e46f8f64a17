// The choice of experts: the k largest logits of every token with their softmax weights, and
// the gradient.
//
// A token has G lanes of a wave (8 to 64, by the number of experts), each of them V logits in
// registers. Bound by the vector ALU's issue (four cycles of a SIMD for an instruction of a
// wave), so what counts is instructions: every lane keeps its four largest logits in order,
// the k rounds look at the first of each lane only, and the wave goes through all logits again
// only when a lane has given away its four. 65536 tokens of 256 bf16 logits, 8 chosen, half of
// the experts masked: 11.4 us of calls in a row (12.7 in a kernel trace) with 350 instructions for four
// tokens (264 and 12 for each choice, about); looking through all logits in every round 20.6 with 616. The
// same, none masked, fp32: 24.2 us (32768 tokens 14.9); with the softmax over all experts bf16 15.5, fp32 28.8. The
// gradient there in bf16: over all experts (67 MB) 16.1 us, 4 TB/s, over the chosen (40 MB) 9.6.
#include "mxq_moe.h"

namespace mxq {

namespace {

// Logits as unsigned numbers in the order that counts: the sign and magnitude bits become a
// two's complement number (-0 and +0 the same) and its top bit is turned. NaN is above all.
// -Inf is 0x00800000 (bf16: in the upper half of the word); 0 is no logit.
constexpr uint32_t kNegInf = 0x00800000u;

__device__ __forceinline__ uint32_t ordered(uint32_t bits) {
  const uint32_t s = (uint32_t)((int32_t)bits >> 31);
  return (((bits & 0x7FFFFFFFu) ^ s) - s) ^ 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  const int32_t c = (int32_t)(o ^ 0x80000000u);
  return as_f(c < 0 ? (uint32_t)-c | 0x80000000u : (uint32_t)c);
}

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Logit i of a lane: runs of 4 lie side by side over the lanes. (Runs of 8 leave a lane without a share
// in some groups of experts, and where a token may choose from some groups only, the others' lanes
// give away more than four: 65536 tokens of 256 experts, half of them masked, 14.7 us.)
constexpr int kRun = 4;
template <int G>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return (i / kRun) * (kRun * G) + lane * kRun + i % kRun;
}

// The bits of the lane's V logits of a row, behind the last one -Inf. Rows start on any element
// (the memory system takes such accesses); a run that the row's end cuts comes element by element.
template <typename T, int G, int V>
struct Logits {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kWords = kF32 ? V : V / 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* row, int lane, int experts) {
    constexpr int kRunWords = kF32 ? kRun : kRun / 2;
#pragma unroll
    for (int b = 0; b < V / kRun; ++b) {
      const int e0 = expert_of<G>(lane, b * kRun);
      uint32_t t[kRunWords];
      if (e0 + kRun <= experts) {
        __builtin_memcpy(t, row + e0, sizeof(t));
      } else {
        T x[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) x[i] = row[e0 + i < experts ? e0 + i : experts - 1];
#pragma unroll
        for (int i = 0; i < kRun; ++i) x[i] = e0 + i < experts ? x[i] : (T)-__builtin_inff();
        __builtin_memcpy(t, x, sizeof(t));
      }
#pragma unroll
      for (int i = 0; i < kRunWords; ++i) w[b * kRunWords + i] = t[i];
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (kF32) return as_f(w[i]);
    else return as_f(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // (fp32: `ordered`. bf16: two at a time, 16 bits each)
  __device__ __forceinline__ void order() {
    typedef short s2 __attribute__((ext_vector_type(2)));
    typedef unsigned short u2 __attribute__((ext_vector_type(2)));
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kF32) {
        most = max(most, w[i] & 0x7FFFFFFFu);
      } else {
        const u2 a = __builtin_bit_cast(u2, w[i] & 0x7FFF7FFFu), b = __builtin_bit_cast(u2, most);
        most = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
      }
    }
    const bool nan = kF32 ? most > 0x7F800000u : (most & 0xFFFFu) > 0x7F80u || most > 0x7F80FFFFu;
    const bool any = __any(nan);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t was = w[i];
      if constexpr (kF32) {
        w[i] = ordered(was);
        if (any && (was & 0x7FFFFFFFu) > 0x7F800000u) w[i] = 0xFFFFFFFFu;
      } else {
        const s2 s = __builtin_bit_cast(s2, was) >> 15;
        const s2 c = __builtin_bit_cast(s2, (was & 0x7FFF7FFFu) ^ __builtin_bit_cast(uint32_t, s)) - s;
        w[i] = __builtin_bit_cast(uint32_t, c) ^ 0x80008000u;
        if (any) {
          if ((was & 0x7FFFu) > 0x7F80u) w[i] |= 0xFFFFu;
          if ((was & 0x7FFF0000u) > 0x7F800000u) w[i] |= 0xFFFF0000u;
        }
      }
    }
  }
};

// A lane's four largest logits, in falling order.
//
// bf16: a logit and its expert in one word, the expert's complement below the logit, so that no two
// words are equal and of equal logits the lower expert is larger.
struct TopBf16 {
  struct Choice {
    uint32_t k;
    __device__ __forceinline__ uint32_t order() const { return k & 0xFFFF0000u; }
    __device__ __forceinline__ int expert() const { return (int)(0xFFFFu - (k & 0xFFFFu)); }
  };
  uint32_t m[4];
  uint32_t last = 0;  // the round's choice

  __device__ __forceinline__ void clear() { m[0] = m[1] = m[2] = m[3] = 0; }
  __device__ __forceinline__ void insert(uint32_t x) {
    m[3] = med3(m[2], m[3], x);
    m[2] = med3(m[1], m[2], x);
    m[1] = med3(m[0], m[1], x);
    m[0] = max(m[0], x);
  }
  template <typename L, int G, int V>
  __device__ __forceinline__ void fill(const L& l, int lane, bool again) {
    clear();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t low = 0xFFFFu - (uint32_t)expert_of<G>(lane, i);
      const uint32_t x = i & 1 ? (l.w[i / 2] & 0xFFFF0000u) | low : l.w[i / 2] << 16 | low;
      insert(again && x >= last ? 0u : x);
    }
  }
  template <int G>
  __device__ __forceinline__ void choose() {
    last = reduce32<G>(m[0], [](uint32_t a, uint32_t b) { return max(a, b); });
    const bool mine = m[0] == last;
    m[0] = mine ? m[1] : m[0];
    m[1] = mine ? m[2] : m[1];
    m[2] = mine ? m[3] : m[2];
    m[3] = mine ? 0u : m[3];
  }
  __device__ __forceinline__ Choice choice() const { return Choice{last}; }
};

// fp32: the logits, and beside each its expert. Equal ones stay in the order in which they come, which
// is that of their experts.
struct TopF32 {
  struct Choice {
    uint32_t o;
    int e;
    __device__ __forceinline__ uint32_t order() const { return o; }
    __device__ __forceinline__ int expert() const { return e; }
  };
  uint32_t m[4];
  int e[4];
  uint32_t last = 0;
  int last_e = 0;

  template <typename L, int G, int V>
  __device__ __forceinline__ void fill(const L& l, int lane, bool again) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = 0;
      e[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = expert_of<G>(lane, i);
      uint32_t x = l.w[i];
      if (again && (x > last || (x == last && at <= last_e))) x = 0;
      const bool c0 = x > m[0], c1 = x > m[1], c2 = x > m[2], c3 = x > m[3];
      e[3] = c2 ? e[2] : c3 ? at : e[3];
      e[2] = c1 ? e[1] : c2 ? at : e[2];
      e[1] = c0 ? e[0] : c1 ? at : e[1];
      e[0] = c0 ? at : e[0];
      m[3] = med3(m[2], m[3], x);
      m[2] = med3(m[1], m[2], x);
      m[1] = med3(m[0], m[1], x);
      m[0] = max(m[0], x);
    }
  }
  template <int G>
  __device__ __forceinline__ void choose() {
    last = reduce32<G>(m[0], [](uint32_t a, uint32_t b) { return max(a, b); });
    const uint32_t at = m[0] == last ? (uint32_t)e[0] : 0xFFFFFFFFu;
    last_e = (int)reduce32<G>(at, [](uint32_t a, uint32_t b) { return min(a, b); });
    const bool mine = at == (uint32_t)last_e;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      m[i] = mine ? m[i + 1] : m[i];
      e[i] = mine ? e[i + 1] : e[i];
    }
    m[3] = mine ? 0u : m[3];
  }
  __device__ __forceinline__ Choice choice() const { return Choice{last, last_e}; }
};

template <typename T>
struct TopOf {
  typedef TopBf16 type;
};
template <>
struct TopOf<float> {
  typedef TopF32 type;
};

template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_kernel(RouteLaunch p) {
  constexpr int kSlots = G >= 64 ? 1 : 64 / G;  // choices that a lane keeps
  const int lane = threadIdx.x % G;
  const int64_t at = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const int64_t token = at < p.tokens ? at : p.tokens - 1;
  typedef Logits<T, G, V> L;
  L l;
  l.load(static_cast<const T*>(p.logits) + token * p.ld, lane, p.experts);
  L o = l;
  o.order();
  typedef typename TopOf<T>::type Top;
  Top top;
  top.template fill<L, G, V>(o, lane, false);
  typename Top::Choice mine[kSlots] = {};
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
#pragma unroll 1
    for (int r = 0; r < G && s * G + r < p.top_k; ++r) {
      if (__any(top.m[0] == 0)) top.template fill<L, G, V>(o, lane, true);
      top.template choose<G>();
      if (lane == r) mine[s] = top.choice();
    }
  }
  const float best = unordered(__shfl(mine[0].order(), 0, G));
  float sum = 0.0f, w[kSlots];
  int expert[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (s * G >= p.top_k) break;  // (most calls have no more choices than lanes)
    const bool none = mine[s].order() <= kNegInf;  // -Inf, or no logit
    expert[s] = none ? -1 : mine[s].expert();
    w[s] = none ? 0.0f : exp_f(unordered(mine[s].order()) - best);
    if (p.renorm) sum += w[s];
  }
  if (!p.renorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = l.value(i);
      sum += v == -__builtin_inff() ? 0.0f : exp_f(v - best);
    }
  }
  const float inv = __builtin_amdgcn_rcpf(group_sum<G>(sum));
  if (at >= p.tokens) return;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (s * G >= p.top_k) break;
    const int j = s * G + lane;
    if (j < p.top_k) {
      p.weights[token * p.top_k + j] = expert[s] < 0 ? 0.0f : w[s] * inv;
      p.chosen[token * p.top_k + j] = expert[s];
    }
  }
}

// The terms w dw go to their logits through LDS: every lane clears the places of its logits, the
// lanes that hold a choice add it at its expert's place, every lane takes its logits' sums back. All
// of it inside a wave. With renorm, S w is part of the term.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteLaunch p) {
  constexpr int kSlots = G >= 64 ? 1 : 64 / G;
  __shared__ __attribute__((aligned(16))) float places[256 / G][G * V];
  const int lane = threadIdx.x % G;
  const int64_t at = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const int64_t token = at < p.tokens ? at : p.tokens - 1;
  float* place = places[threadIdx.x / G];
  typedef Logits<T, G, V> L;
  L l;
  if (!p.renorm) l.load(static_cast<const T*>(p.logits) + token * p.ld, lane, p.experts);
  // choice j belongs to lane j % G: its expert, its weight, and w dw
  int e[kSlots];
  float w[kSlots], x[kSlots], mean = 0.0f;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = s * G + lane;
    e[s] = -1;
    w[s] = x[s] = 0.0f;
    if (j < p.top_k) {
      const int64_t c = token * p.top_k + j;
      const int chosen = p.chosen[c];
      const float weight = p.weights[c], dw = p.dw[c];
      if ((uint32_t)chosen < (uint32_t)p.experts) {
        e[s] = chosen;
        w[s] = weight;
        x[s] = weight * dw;
      }
    }
    mean += x[s];
  }
  mean = group_sum<G>(mean);
#pragma unroll
  for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(place + expert_of<G>(lane, i)) = make_float4(0, 0, 0, 0);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int s = 0; s < kSlots; ++s)
    if (e[s] >= 0) atomicAdd(place + e[s], p.renorm ? fmaf(-mean, w[s], x[s]) : x[s]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float part[V];
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(place + expert_of<G>(lane, i));
    part[i] = q.x; part[i + 1] = q.y; part[i + 2] = q.z; part[i + 3] = q.w;
  }
  if (!p.renorm) {
    float best = -__builtin_inff(), sum = 0.0f, share[V];
#pragma unroll
    for (int i = 0; i < V; ++i) best = __builtin_elementwise_maximum(best, l.value(i));
    best = group_max<G>(best);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      share[i] = l.value(i) == -__builtin_inff() ? 0.0f : exp_f(l.value(i) - best);
      sum += share[i];
    }
    sum = group_sum<G>(sum);
    const float scale = sum == 0.0f ? 0.0f : -mean * __builtin_amdgcn_rcpf(sum);  // (0: every logit is -Inf)
#pragma unroll
    for (int i = 0; i < V; ++i) part[i] = fmaf(scale, share[i], part[i]);
  }
  if (at >= p.tokens) return;
  T* row = static_cast<T*>(p.dlogits) + token * p.experts;
#pragma unroll
  for (int b = 0; b < V / kRun; ++b) {
    const int e0 = expert_of<G>(lane, b * kRun);
    T t[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) t[i] = (T)part[b * kRun + i];
    if (e0 + kRun <= p.experts) {
      __builtin_memcpy(row + e0, t, sizeof(t));
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (e0 + i < p.experts) row[e0 + i] = t[i];
    }
  }
}

template <typename T, int G, int V>
hipError_t launch_g(const RouteLaunch& all, bool grad, hipStream_t st) {
  return by_slabs(all.tokens, G, [&](int64_t t0, int64_t tokens) {
    RouteLaunch a = all;
    a.tokens = tokens;
    if (a.logits) a.logits = static_cast<const T*>(all.logits) + t0 * all.ld;
    a.weights += t0 * all.top_k;
    a.chosen += t0 * all.top_k;
    const dim3 grid((uint32_t)((tokens + 256 / G - 1) / (256 / G)));
    if (grad) {
      a.dw += t0 * all.top_k;
      a.dlogits = static_cast<T*>(all.dlogits) + t0 * all.experts;
      route_grad_kernel<T, G, V><<<grid, 256, 0, st>>>(a);
    } else {
      route_kernel<T, G, V><<<grid, 256, 0, st>>>(a);
    }
  });
}

// Lanes of a token: few leave more logits to a lane, which then more often gives away its four; many
// take more steps to compare the lanes. (65536 tokens of 256 bf16 logits: 8 lanes 12.8 us, 16 11.6, 32
// 16.3; 32768 of fp32: 28.9, 15.2 and 14.4.)
template <typename T>
hipError_t launch_t(const RouteLaunch& a, bool grad, hipStream_t st) {
  if (a.experts <= 64) return launch_g<T, 8, 8>(a, grad, st);
  if (a.experts <= 128) return launch_g<T, 8, 16>(a, grad, st);
  if (a.experts <= 256) return launch_g<T, 16, 16>(a, grad, st);
  if (a.experts <= 512) return launch_g<T, 32, 16>(a, grad, st);
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
