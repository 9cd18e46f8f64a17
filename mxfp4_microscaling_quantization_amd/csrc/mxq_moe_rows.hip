// Tokens' rows to the rows of their experts and back: dispatch, combine and combine's gradient.
//
// All three go by tokens. A workgroup owns a token or a part of its columns: the token's own row moves
// once, and the rows of its assignments are found by the positions, which are the same for the whole
// workgroup. Bound by memory; a 1 GiB copy runs at 5.1 TB/s on the card the times below are from.
#include "mxq_blocks.h"
#include "mxq_moe.h"
#include "mxq_moe_fp8.h"

namespace mxq {

namespace {

// The row of an assignment, or -1.
__device__ __forceinline__ int row_at(const RowsLaunch& p, int64_t a) {
  const int r = p.positions[a];
  return (uint32_t)r < (uint64_t)p.rows ? r : -1;
}

// Rows as they are, 16 bytes of a thread. WHOLE: rows start on 16 bytes and hold whole 16s; otherwise
// they start anywhere, and a row's last bytes go two by two. (16384 tokens' 8 rows of 7168 bf16, 2.1 GB:
// 395 us, 5.3 TB/s, with 256 threads 454; 2 rows of 4097 bf16, 0.4 GB: 82 us, with 128 threads 91, stores
// through the caches 87, element by element 146.) A row of less than 2 KiB leaves threads without work:
// 65536 tokens' 4 rows of 128 bf16 39.6 us, 2.1 TB/s, of 256 50.2 and 3.3, of 512 65.3 and 5.1.
template <bool WHOLE>
constexpr int kCopyThreads = WHOLE ? 128 : 256;
template <bool WHOLE>
__global__ __launch_bounds__(kCopyThreads<WHOLE>) void dispatch_copy_kernel(RowsLaunch p, int64_t ld, int bytes,
                                                                            int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int c = ((int)(blockIdx.x % tiles) * kCopyThreads<WHOLE> + threadIdx.x) * 16, pairs = (bytes - c) / 2;
  if (c >= bytes) return;
  const char* x = static_cast<const char*>(p.x) + token * ld + c;
  nt_u32x4 v;
  uint16_t last[7];
  if (WHOLE) {
    v = __builtin_nontemporal_load(reinterpret_cast<const nt_u32x4*>(x));
  } else if (pairs >= 8) {
    load_any<16>(&v, x);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i) last[i] = i < pairs ? reinterpret_cast<const uint16_t*>(x)[i] : 0;
  }
  for (int j = 0; j < p.top_k; ++j) {
    const int r = row_at(p, token * p.top_k + j);
    if (r < 0) continue;
    char* out = static_cast<char*>(p.out) + (int64_t)r * bytes + c;
    if (WHOLE) {
      __builtin_nontemporal_store(v, reinterpret_cast<nt_u32x4*>(out));
    } else if (pairs >= 8) {
      store_any<16>(out, &v);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < pairs) reinterpret_cast<uint16_t*>(out)[i] = last[i];
    }
  }
}

// The bits of N elements of a row that starts on 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void load_span(const T* p, uint4 (&w)[N * sizeof(T) / 16]) {
#pragma unroll
  for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
}

// A block of 32 values -> 16 bytes of codes and the block's byte: mx_encode8's steps with the whole
// block in one lane.
__device__ __forceinline__ uint4 mx_encode32(const uint4 (&w)[4], uint32_t& byte, uint16_t) {
  uint32_t m = 0, d[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d[4 * i] = w[i].x; d[4 * i + 1] = w[i].y; d[4 * i + 2] = w[i].z; d[4 * i + 3] = w[i].w;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, max(d[i] & 0x7FFFu, (d[i] >> 16) & 0x7FFFu));
  const uint32_t ea = m >> 7;
  byte = ea >= 255u ? 255u : (ea > 2u ? ea - 2u : 0u);
  const float scale = e8m0_operand(min(byte, 254u));
  if (byte == 255u) return make_uint4(0, 0, 0, 0);
  return make_uint4(fp4x8_from_bf16(d, scale), fp4x8_from_bf16(d + 4, scale), fp4x8_from_bf16(d + 8, scale),
                    fp4x8_from_bf16(d + 12, scale));
}
__device__ __forceinline__ uint4 mx_encode32(const uint4 (&w)[8], uint32_t& byte, float) {
  uint32_t m = 0;
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[4 * i] = as_f(w[i].x); v[4 * i + 1] = as_f(w[i].y); v[4 * i + 2] = as_f(w[i].z); v[4 * i + 3] = as_f(w[i].w);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, as_u(v[i]) & 0x7FFFFFFFu);
  byte = mx_byte<0>(m);
  const float scale = e8m0_operand(min(byte, 252u));
  if (byte == 255u) return make_uint4(0, 0, 0, 0);
  return make_uint4(fp4x8_from_f32(v, scale), fp4x8_from_f32(v + 8, scale), fp4x8_from_f32(v + 16, scale),
                    fp4x8_from_f32(v + 24, scale));
}

// Rows as MXFP4 or FP8, encoded once and stored for every assignment, 16 bytes of codes of a thread: a
// block of 32 for MXFP4, 16 elements of a group of 128 for FP8. A workgroup takes a whole token, so that
// the lines of scales, which no store fills, are put together in one L2. (16384 tokens' 8 rows of 7168
// bf16 in MXFP4, 0.73 GB: 136 to 145 us, 5 to 5.4 TB/s; waves for each part of a token 159, codes through
// the caches 154, 8 elements of a thread 211. FP8, 1.2 GB: 217 to 232 us; 248, and 291.)
constexpr int kQuantThreads = 256;
template <typename T, bool FP8>
__global__ __launch_bounds__(kQuantThreads) void dispatch_quantize_kernel(RowsLaunch p, int tiles) {
  constexpr int N = FP8 ? 16 : 32;
  const int64_t token = blockIdx.x / tiles;
  const int spans = (int)p.width / N;
  const T* x = static_cast<const T*>(p.x) + token * p.ldx;
  for (int c0 = (int)(blockIdx.x % tiles) * blockDim.x; c0 < spans; c0 += tiles * blockDim.x) {
    const int c = c0 + threadIdx.x;
    uint4 w[N * sizeof(T) / 16] = {}, code;
    uint32_t scale = 0;
    if (c < spans) load_span<T, N>(x + c * N, w);
    if constexpr (FP8) code = fp8_encode16(w, scale, T());
    else code = mx_encode32(w, scale, T());
    if (c >= spans) continue;
    for (int j = 0; j < p.top_k; ++j) {
      const int r = row_at(p, token * p.top_k + j);
      if (r < 0) continue;
      const int64_t at = (int64_t)r * spans + c;
      store_nt(static_cast<uint4*>(p.out) + at, code);
      if constexpr (FP8) {
        if (c % 8 == 0) static_cast<uint32_t*>(p.scales)[at / 8] = scale;
      } else {
        static_cast<uint8_t*>(p.scales)[at] = (uint8_t)scale;
      }
    }
  }
}

// Eight neighbouring elements of a row, read or written once. WHOLE: rows start on 16 bytes and hold
// whole eights; otherwise they start on any element, and the last elements of a row go one by one.
template <typename T, bool WHOLE>
struct Eight {
  T v[8];
  __device__ __forceinline__ void load(const T* p, int left) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
        const uint4 x = load_nt(reinterpret_cast<const uint4*>(p) + i);
        __builtin_memcpy(v + i * 16 / sizeof(T), &x, 16);
      }
    } else if (left >= 8) {
      load_any<sizeof(v)>(v, p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : (T)0.0f;
    }
  }
  __device__ __forceinline__ void store(T* p, int left) const {
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
        uint4 x;
        __builtin_memcpy(&x, v + i * 16 / sizeof(T), 16);
        store_nt(reinterpret_cast<uint4*>(p) + i, x);
      }
    } else if (left >= 8) {
      store_any<sizeof(v)>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = v[i];
    }
  }
};

// sum += the rows of U assignments from `first` on, in order, their loads in flight together.
template <typename Y, bool WHOLE, int U>
__device__ __forceinline__ void add_rows(const RowsLaunch& p, int64_t first, int c, float (&sum)[8]) {
  const int width = (int)p.width;
  int r[U];
  Eight<Y, WHOLE> y[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r[u] = row_at(p, first + u);
    y[u].load(static_cast<const Y*>(p.x) + (int64_t)(r[u] < 0 ? 0 : r[u]) * width + c, width - c);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (r[u] < 0) continue;  // (the same for the whole workgroup)
    const float w = p.weights ? p.weights[first + u] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, (float)y[u].v[i], sum[i]);
  }
}

// A wave: 512 columns of a token. (16384 tokens, 8 rows of 7168 bf16 each to fp32, 2.3 GB: 393 us, 5.9
// TB/s; a workgroup for a whole token, row after row, 474; stores through the caches 420. 4 rows of 4097
// columns to bf16 in pieces of 16 bytes that start anywhere 147, by elements 397.)
template <typename Y, typename O, bool WHOLE>
__global__ __launch_bounds__(64) void combine_kernel(RowsLaunch p, int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int width = (int)p.width, c = ((int)(blockIdx.x % tiles) * 64 + threadIdx.x) * 8;
  if (c >= width) return;
  float sum[8] = {};
  if (p.rows > 0) {
    int64_t a = token * p.top_k;
    int left = p.top_k;
    for (; left >= 8; left -= 8, a += 8) add_rows<Y, WHOLE, 8>(p, a, c, sum);
    if (left & 4) add_rows<Y, WHOLE, 4>(p, a, c, sum), a += 4;
    if (left & 2) add_rows<Y, WHOLE, 2>(p, a, c, sum), a += 2;
    if (left & 1) add_rows<Y, WHOLE, 1>(p, a, c, sum);
  }
  if (p.res) {
    Eight<O, WHOLE> res;
    res.load(static_cast<const O*>(p.res) + token * width + c, width - c);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += (float)res.v[i];
  }
  Eight<O, WHOLE> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = (O)sum[i];
  o.store(static_cast<O*>(p.out) + token * width + c, width - c);
}

constexpr int kGradThreads = 512, kGradRows = 8;

// U assignments of a token from `first` on: their rows' gradients, and the weights'. A row's gradient
// may be written over the row itself: the same thread reads and writes every element.
template <typename G, typename Y, bool WHOLE, int U>
__device__ __forceinline__ void grad_rows(const RowsLaunch& p, int64_t first, const G* g, float (*parts)[kGradRows]) {
  const int width = (int)p.width;
  int r[U];
  float w[U], dot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r[u] = row_at(p, first + u);
    w[u] = p.weights ? p.weights[first + u] : 1.0f;
    dot[u] = 0.0f;
  }
  if (p.rows > 0) {
    for (int c = threadIdx.x * 8; c < width; c += blockDim.x * 8) {
      Eight<G, WHOLE> gv;
      Eight<Y, WHOLE> y[U];
      gv.load(g + c, width - c);
#pragma unroll
      for (int u = 0; u < U; ++u)
        y[u].load(static_cast<const Y*>(p.res) + (int64_t)(r[u] < 0 ? 0 : r[u]) * width + c, width - c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r[u] < 0) continue;
        Eight<Y, WHOLE> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[u] = fmaf((float)gv.v[i], (float)y[u].v[i], dot[u]);
          o.v[i] = (Y)(w[u] * (float)gv.v[i]);
        }
        o.store(static_cast<Y*>(p.out) + (int64_t)r[u] * width + c, width - c);
      }
    }
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    dot[u] = group_sum<64>(dot[u]);
    if (lane == 0) parts[wave][u] = dot[u];
  }
  __syncthreads();
  if (threadIdx.x < U) {
    float sum = parts[0][threadIdx.x];
    for (int i = 1; i < (int)blockDim.x / 64; ++i) sum += parts[i][threadIdx.x];
    p.dw[first + threadIdx.x] = sum;
  }
  __syncthreads();
}

// A workgroup: one token, up to eight waves side by side. (16384 tokens, 4 rows of 4096 bf16 each from
// fp32, 1.34 GB: 235 us, 5.7 TB/s; four waves 241, two 255, one 269; row after row 295.)
template <typename G, typename Y, bool WHOLE>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(RowsLaunch p) {
  __shared__ float parts[kGradThreads / 64][kGradRows];
  const int64_t token = blockIdx.x;
  const G* g = static_cast<const G*>(p.x) + token * (int)p.width;
  int64_t a = token * p.top_k;
  int left = p.top_k;
  for (; left >= 8; left -= 8, a += 8) grad_rows<G, Y, WHOLE, 8>(p, a, g, parts);
  if (left & 4) grad_rows<G, Y, WHOLE, 4>(p, a, g, parts), a += 4;
  if (left & 2) grad_rows<G, Y, WHOLE, 2>(p, a, g, parts), a += 2;
  if (left & 1) grad_rows<G, Y, WHOLE, 1>(p, a, g, parts);
}

// The rows' gradients alone: a part of a token's columns, weighted for each of its assignments. (14368
// tokens, 5 rows of 2200 bf16 from fp32, 0.44 GB: 99 us; parts of 512 columns 106, of 2048 120, a token in
// a workgroup 115. Narrow rows leave threads without work: 65536 tokens, 4 rows of 128 bf16 from fp32, 59.5 us, 1.7
// TB/s, of 256 71.0 and 2.8, of 512 87.3 and 4.6.)
constexpr int kWeightThreads = 128;
template <typename G, typename Y, bool WHOLE>
__global__ __launch_bounds__(kWeightThreads) void combine_grad_rows_kernel(RowsLaunch p, int tiles) {
  const int64_t token = blockIdx.x / tiles;
  const int width = (int)p.width, c = ((int)(blockIdx.x % tiles) * kWeightThreads + threadIdx.x) * 8;
  if (c >= width) return;
  Eight<G, WHOLE> g;
  g.load(static_cast<const G*>(p.x) + token * width + c, width - c);
  for (int j = 0; j < p.top_k; ++j) {
    const int64_t a = token * p.top_k + j;
    const int r = row_at(p, a);
    if (r < 0) continue;
    const float w = p.weights ? p.weights[a] : 1.0f;
    Eight<Y, WHOLE> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = (Y)(w * (float)g.v[i]);
    o.store(static_cast<Y*>(p.out) + (int64_t)r * width + c, width - c);
  }
}

// The launch for tokens t0 to t0 + tokens, with the pointers to the tokens' data moved on; `x` and `out`:
// bytes of a token there (0 where they are the experts' rows), `res` likewise.
RowsLaunch slab(const RowsLaunch& all, int64_t t0, int64_t tokens, int64_t x, int64_t res, int64_t out) {
  RowsLaunch a = all;
  a.tokens = tokens;
  a.x = static_cast<const char*>(all.x) + t0 * x;
  if (all.res) a.res = static_cast<const char*>(all.res) + t0 * res;
  a.out = static_cast<char*>(all.out) + t0 * out;
  a.positions += t0 * all.top_k;
  if (all.weights) a.weights += t0 * all.top_k;
  if (all.dw) a.dw += t0 * all.top_k;
  return a;
}

template <bool WHOLE>
hipError_t launch_copy(const RowsLaunch& all, int64_t ld, int64_t bytes, hipStream_t st) {
  constexpr int kThreads = kCopyThreads<WHOLE>;
  const int tiles = (int)((bytes + kThreads * 16 - 1) / (kThreads * 16));
  return by_slabs(all.tokens, (int64_t)tiles * kThreads, [&](int64_t t0, int64_t tokens) {
    const RowsLaunch a = slab(all, t0, tokens, ld, 0, 0);
    dispatch_copy_kernel<WHOLE><<<dim3((uint32_t)(tokens * tiles)), kThreads, 0, st>>>(a, ld, (int)bytes, tiles);
  });
}

template <typename T, bool FP8>
hipError_t launch_quantize(const RowsLaunch& all, hipStream_t st) {
  const int64_t waves = (all.width / (FP8 ? 16 : 32) + 63) / 64;
  // Few tokens: a wave for each part, so that one token's parts run side by side. (us, such waves and a whole
  // token in a workgroup, 8 rows of 7168 bf16: FP8 64 tokens 3.9 and 5.8, 256 5.0 and 6.3, 512 7.5 and 7.8, 1024
  // 14.8 and 13.9, 1500 20.2 and 19.4; MXFP4 64 tokens 3.7 and 4.0, 512 5.4 and 5.1, 1024 9.2 and 8.8, 4096 31.6
  // and 29.4. Rows of 2048: alike up to 512, FP8 1024 5.3 and 5.0.)
  const bool few = all.tokens < 1024;
  const int threads = few ? 64 : 64 * (int)(waves < kQuantThreads / 64 ? waves : kQuantThreads / 64);
  const int tiles = few ? (int)waves : 1;
  return by_slabs(all.tokens, (int64_t)tiles * threads, [&](int64_t t0, int64_t tokens) {
    const RowsLaunch a = slab(all, t0, tokens, all.ldx * (int64_t)sizeof(T), 0, 0);
    dispatch_quantize_kernel<T, FP8><<<dim3((uint32_t)(tokens * tiles)), threads, 0, st>>>(a, tiles);
  });
}

template <typename Y, typename O>
hipError_t launch_combine_t(const RowsLaunch& all, hipStream_t st) {
  const int tiles = (int)((all.width + 511) / 512);
  return by_slabs(all.tokens, (int64_t)tiles * 64, [&](int64_t t0, int64_t tokens) {
    const int64_t row = all.width * (int64_t)sizeof(O);
    const RowsLaunch a = slab(all, t0, tokens, 0, row, row);
    const dim3 grid((uint32_t)(tokens * tiles));
    if (a.width % 8 == 0) combine_kernel<Y, O, true><<<grid, 64, 0, st>>>(a, tiles);
    else combine_kernel<Y, O, false><<<grid, 64, 0, st>>>(a, tiles);
  });
}

template <typename G, typename Y, bool WHOLE>
hipError_t launch_combine_grad_v(const RowsLaunch& all, hipStream_t st) {
  const int64_t waves = (all.width + 511) / 512, row = all.width * (int64_t)sizeof(G);
  if (!all.dw) {
    const int tiles = (int)((all.width + kWeightThreads * 8 - 1) / (kWeightThreads * 8));
    return by_slabs(all.tokens, (int64_t)tiles * kWeightThreads, [&](int64_t t0, int64_t tokens) {
      const RowsLaunch a = slab(all, t0, tokens, row, 0, 0);
      combine_grad_rows_kernel<G, Y, WHOLE><<<dim3((uint32_t)(tokens * tiles)), kWeightThreads, 0, st>>>(a, tiles);
    });
  }
  const int threads = 64 * (int)(waves < kGradThreads / 64 ? waves : kGradThreads / 64);
  return by_slabs(all.tokens, threads, [&](int64_t t0, int64_t tokens) {
    const RowsLaunch a = slab(all, t0, tokens, row, 0, 0);
    combine_grad_kernel<G, Y, WHOLE><<<dim3((uint32_t)tokens), threads, 0, st>>>(a);
  });
}
template <typename G, typename Y>
hipError_t launch_combine_grad_t(const RowsLaunch& a, hipStream_t st) {
  return a.width % 8 == 0 ? launch_combine_grad_v<G, Y, true>(a, st) : launch_combine_grad_v<G, Y, false>(a, st);
}

}  // namespace

hipError_t launch_dispatch(const RowsLaunch& a, hipStream_t st) {
  if (a.fmt == 0) {
    const int64_t size = a.x_f32 ? 4 : 2, bytes = a.width * size, ld = a.ldx * size;
    const bool whole = ((uint64_t)(uintptr_t)a.x | (uint64_t)(ld | bytes)) % 16 == 0;
    return whole ? launch_copy<true>(a, ld, bytes, st) : launch_copy<false>(a, ld, bytes, st);
  }
  if (a.fmt == 1) return a.x_f32 ? launch_quantize<float, false>(a, st) : launch_quantize<uint16_t, false>(a, st);
  return a.x_f32 ? launch_quantize<float, true>(a, st) : launch_quantize<uint16_t, true>(a, st);
}

hipError_t launch_combine(const RowsLaunch& a, hipStream_t st) {
  if (a.x_f32) return a.out_f32 ? launch_combine_t<float, float>(a, st) : launch_combine_t<float, __bf16>(a, st);
  return a.out_f32 ? launch_combine_t<__bf16, float>(a, st) : launch_combine_t<__bf16, __bf16>(a, st);
}

hipError_t launch_combine_grad(const RowsLaunch& a, hipStream_t st) {
  if (a.x_f32) return a.out_f32 ? launch_combine_grad_t<float, float>(a, st) : launch_combine_grad_t<float, __bf16>(a, st);
  return a.out_f32 ? launch_combine_grad_t<__bf16, float>(a, st) : launch_combine_grad_t<__bf16, __bf16>(a, st);
}

}  // namespace mxq
