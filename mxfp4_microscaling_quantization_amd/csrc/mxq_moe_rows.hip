// Tokens' rows to the rows of their experts and back: dispatch, combine and combine's gradient.
//
// All three go by tokens. A workgroup owns a token, or a part of its columns where there are
// few tokens: the token's own row moves once, and the rows of its assignments are found by the
// positions, which are the same for the whole workgroup. Bound by memory.
#include "mxq_blocks.h"
#include "mxq_moe.h"
#include "mxq_moe_fp8.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;

// The row of an assignment, or -1.
__device__ __forceinline__ int row_at(const RowsLaunch& p, int64_t a) {
  const int r = p.positions[a];
  return (uint32_t)r < (uint64_t)p.rows ? r : -1;
}

// Rows as they are, in units U of 16 bytes, of 4, or of an element.
template <typename U>
__global__ __launch_bounds__(kThreads) void dispatch_copy_kernel(RowsLaunch p, int64_t ld, int units, int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int tile = blockIdx.x % tiles;
  const U* x = static_cast<const U*>(p.x) + token * ld;
  for (int c = tile * kThreads + threadIdx.x; c < units; c += tiles * kThreads) {
    const U v = x[c];
    for (int j = 0; j < p.top_k; ++j) {
      const int r = row_at(p, token * p.top_k + j);
      if (r >= 0) static_cast<U*>(p.out)[(int64_t)r * units + c] = v;
    }
  }
}

// Rows as MXFP4 or FP8: 8 elements of a thread, so a block of 32 is a quad of lanes and a group of
// 128 sixteen of them; encoded once, stored for every assignment.
template <typename T, bool FP8>
__global__ __launch_bounds__(kThreads) void dispatch_quantize_kernel(RowsLaunch p, int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int tile = blockIdx.x % tiles, chunks = (int)(p.width / 8);
  const T* x = static_cast<const T*>(p.x) + token * p.ldx;
  for (int c0 = tile * kThreads; c0 < chunks; c0 += tiles * kThreads) {
    const int c = c0 + threadIdx.x;
    Raw<T> raw;
    if (c < chunks) load_raw(x, (size_t)c * 8, raw);
    else zero_raw(raw);
    uint32_t byte = 0, code = 0;
    uint2 code8 = make_uint2(0, 0);
    float scale = 0.0f;
    if constexpr (FP8) {
      float v[8];
      to_f32(raw, v);
      code8 = fp8_encode8(v, scale);
    } else if constexpr (sizeof(T) == 2) {
      code = mx_encode8_bf16(raw.w, byte);
    } else {
      float v[8];
      to_f32(raw, v);
      code = mx_encode8<false, 0>(v, nullptr, byte);
    }
    if (c < chunks)
      for (int j = 0; j < p.top_k; ++j) {
        const int r = row_at(p, token * p.top_k + j);
        if (r < 0) continue;
        if constexpr (FP8) {
          static_cast<uint2*>(p.out)[(int64_t)r * chunks + c] = code8;
          if (c % 16 == 0) static_cast<float*>(p.scales)[(int64_t)r * (chunks / 16) + c / 16] = scale;
        } else {
          static_cast<uint32_t*>(p.out)[(int64_t)r * chunks + c] = code;
          if (c % 4 == 0) static_cast<uint8_t*>(p.scales)[(int64_t)r * (chunks / 4) + c / 4] = (uint8_t)byte;
        }
      }
  }
}

// V neighbouring elements, whole: rows start on 16 bytes (V = 8), or one.
template <typename T, int V>
struct Piece {
  T v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) v[0] = *p;
    else __builtin_memcpy(v, __builtin_assume_aligned(p, 16), sizeof(v));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 1) *p = v[0];
    else __builtin_memcpy(__builtin_assume_aligned(p, 16), v, sizeof(v));
  }
};

template <typename Y, typename O, int V>
__global__ __launch_bounds__(kThreads) void combine_kernel(RowsLaunch p, int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int tile = blockIdx.x % tiles, width = (int)p.width;
  for (int c = (tile * kThreads + threadIdx.x) * V; c < width; c += tiles * kThreads * V) {
    float sum[V] = {};
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t a = token * p.top_k + j;
      const int r = row_at(p, a);
      if (r < 0) continue;
      const float w = p.weights ? p.weights[a] : 1.0f;
      Piece<Y, V> y;
      y.load(static_cast<const Y*>(p.x) + (int64_t)r * width + c);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = fmaf(w, (float)y.v[i], sum[i]);
    }
    if (p.res) {
      Piece<O, V> res;
      res.load(static_cast<const O*>(p.res) + token * width + c);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += (float)res.v[i];
    }
    Piece<O, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = (O)sum[i];
    o.store(static_cast<O*>(p.out) + token * width + c);
  }
}

// A workgroup: one token, its assignments one after the other (a row's gradient is written over the
// row itself where dy is y: the same thread reads and writes every element).
template <typename G, typename Y, int V, bool DW>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(RowsLaunch p) {
  __shared__ float parts[kThreads / 64];
  const int64_t token = blockIdx.x;
  const int width = (int)p.width;
  const G* g = static_cast<const G*>(p.x) + token * width;
  for (int j = 0; j < p.top_k; ++j) {
    const int64_t a = token * p.top_k + j;
    const int r = row_at(p, a);
    float dot = 0.0f;
    if (r >= 0) {
      const float w = p.weights ? p.weights[a] : 1.0f;
      for (int c = threadIdx.x * V; c < width; c += kThreads * V) {
        Piece<G, V> gv;
        gv.load(g + c);
        Piece<Y, V> o;
        if constexpr (DW) {
          o.load(static_cast<const Y*>(p.res) + (int64_t)r * width + c);
#pragma unroll
          for (int i = 0; i < V; ++i) dot = fmaf((float)gv.v[i], (float)o.v[i], dot);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = (Y)(w * (float)gv.v[i]);
        o.store(static_cast<Y*>(p.out) + (int64_t)r * width + c);
      }
    }
    if constexpr (DW) {
      dot = group_sum<64>(dot);
      if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = dot;
      __syncthreads();
      if (threadIdx.x == 0) p.dw[a] = (parts[0] + parts[1]) + (parts[2] + parts[3]);
      __syncthreads();
    }
  }
}

// Column parts of a token: one where there are enough tokens for the chip.
int tiles_of_token(int64_t tokens, int64_t units) {
  const int64_t most = (units + kThreads - 1) / kThreads;
  return (int)(tokens >= 2048 ? 1 : most);
}

template <typename U>
void launch_copy(const RowsLaunch& a, int64_t size, hipStream_t st) {
  const int64_t units = a.width * size / (int64_t)sizeof(U);
  const int tiles = tiles_of_token(a.tokens, units);
  dispatch_copy_kernel<U><<<dim3((uint32_t)(a.tokens * tiles)), kThreads, 0, st>>>(
      a, a.ldx * size / (int64_t)sizeof(U), (int)units, tiles);
}

template <typename Y, typename O>
void launch_combine_t(const RowsLaunch& a, hipStream_t st) {
  const bool vec = a.width % 8 == 0;
  const int tiles = tiles_of_token(a.tokens, vec ? a.width / 8 : a.width);
  const dim3 grid((uint32_t)(a.tokens * tiles));
  if (vec) combine_kernel<Y, O, 8><<<grid, kThreads, 0, st>>>(a, tiles);
  else combine_kernel<Y, O, 1><<<grid, kThreads, 0, st>>>(a, tiles);
}

template <typename G, typename Y, int V>
void launch_combine_grad_v(const RowsLaunch& a, hipStream_t st) {
  if (a.dw) combine_grad_kernel<G, Y, V, true><<<dim3((uint32_t)a.tokens), kThreads, 0, st>>>(a);
  else combine_grad_kernel<G, Y, V, false><<<dim3((uint32_t)a.tokens), kThreads, 0, st>>>(a);
}
template <typename G, typename Y>
void launch_combine_grad_t(const RowsLaunch& a, hipStream_t st) {
  if (a.width % 8 == 0) launch_combine_grad_v<G, Y, 8>(a, st);
  else launch_combine_grad_v<G, Y, 1>(a, st);
}

}  // namespace

hipError_t launch_dispatch(const RowsLaunch& a, hipStream_t st) {
  const int64_t size = a.x_f32 ? 4 : 2;
  if (a.fmt == 0) {
    const uint64_t all = (uintptr_t)a.x | (uint64_t)(a.ldx * size) | (uint64_t)(a.width * size);
    if (all % 16 == 0) launch_copy<uint4>(a, size, st);
    else if (all % 4 == 0) launch_copy<uint32_t>(a, size, st);
    else launch_copy<uint16_t>(a, size, st);
  } else {
    const int tiles = tiles_of_token(a.tokens, a.width / 8);
    const dim3 grid((uint32_t)(a.tokens * tiles));
    if (a.fmt == 1) {
      if (a.x_f32) dispatch_quantize_kernel<float, false><<<grid, kThreads, 0, st>>>(a, tiles);
      else dispatch_quantize_kernel<uint16_t, false><<<grid, kThreads, 0, st>>>(a, tiles);
    } else {
      if (a.x_f32) dispatch_quantize_kernel<float, true><<<grid, kThreads, 0, st>>>(a, tiles);
      else dispatch_quantize_kernel<uint16_t, true><<<grid, kThreads, 0, st>>>(a, tiles);
    }
  }
  return hipGetLastError();
}

hipError_t launch_combine(const RowsLaunch& a, hipStream_t st) {
  if (a.x_f32) a.out_f32 ? launch_combine_t<float, float>(a, st) : launch_combine_t<float, __bf16>(a, st);
  else a.out_f32 ? launch_combine_t<__bf16, float>(a, st) : launch_combine_t<__bf16, __bf16>(a, st);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const RowsLaunch& a, hipStream_t st) {
  if (a.x_f32) a.out_f32 ? launch_combine_grad_t<float, float>(a, st) : launch_combine_grad_t<float, __bf16>(a, st);
  else a.out_f32 ? launch_combine_grad_t<__bf16, float>(a, st) : launch_combine_grad_t<__bf16, __bf16>(a, st);
  return hipGetLastError();
}

}  // namespace mxq
