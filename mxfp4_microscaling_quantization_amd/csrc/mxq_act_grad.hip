// The gradient of the products' epilogue: dz = act'(z) dy and its column sums per
// group of rows (the bias gradient).
#include "mxq_mm.h"

namespace mxq {

namespace {

constexpr int kCols = 512;  // columns of a workgroup: 64 lanes of 8

// act'(z) and, for SWIGLU, both halves of a pair (gate g, up u). Far from zero s is 0 or 1 exactly
// (for gelu from |z| = 11 on, for silu's from 89 on) and so is the slope: the polynomials that s
// (1 - s) holds down there take z clamped, or they would be infinite and their products with
// zero NaN. s itself takes z as it is, so NaN stays NaN.
constexpr float kGeluFar = 16.0f, kSiluFar = 128.0f;
__device__ __forceinline__ float silu_slope(float z, float s) {
  return s * fmaf(__builtin_amdgcn_fmed3f(z, -kSiluFar, kSiluFar), 1.0f - s, 1.0f);
}

__device__ __forceinline__ float act_grad_f(float dy, float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.0f ? dy : 0.0f;
    case kActGelu: {
      // d/dz [z s(w)], w = A z + B z^3: s + z s (1 - s) (A + 3 B z^2)
      const float near = __builtin_amdgcn_fmed3f(z, -kGeluFar, kGeluFar), zz = near * near;
      const float s = sigmoid_f(z * fmaf(kGeluB, zz, kGeluA));
      return dy * fmaf(near * s * (1.0f - s), fmaf(3.0f * kGeluB, zz, kGeluA), s);
    }
    case kActSilu: return dy * silu_slope(z, sigmoid_f(z));
  }
  return dy;
}

// V elements of a row, as they lie in memory: whole (VEC: every row starts on V elements; data
// read once, so non-temporal) or one by one, those past the row's end as zeros.
template <typename T, int V, bool VEC>
struct Run {
  T v[V];
  __device__ __forceinline__ void load(const T* p, int64_t left) {
    if constexpr (VEC) {
      if constexpr (sizeof(v) == 8) {
        const uint2 x = load_nt(reinterpret_cast<const uint2*>(p));
        __builtin_memcpy(v, &x, 8);
      } else {
#pragma unroll
        for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
          const uint4 x = load_nt(reinterpret_cast<const uint4*>(p) + i);
          __builtin_memcpy(v + i * 16 / sizeof(T), &x, 16);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < left ? p[i] : (T)0.0f;
    }
  }
  __device__ __forceinline__ void store(T* p, int64_t left) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
        uint4 x;
        __builtin_memcpy(&x, v + i * 16 / sizeof(T), 16);
        store_nt(reinterpret_cast<uint4*>(p) + i, x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) p[i] = v[i];
    }
  }
};

// One workgroup: up to p.block_rows rows of one group, 512 columns. Its waves take every
// fourth row, four of them in flight: their loads go ahead of the first one's arithmetic.
// The sums of the four waves are added in order through LDS.
// Bound by memory: 65536 x 4096 bf16 swiglu with its sums moves 1.34 GB in 255 us, 5.3 TB/s, what a
// plain stream that reads twice what it writes reaches here.
template <typename T, bool SUM, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradLaunch p, int col_tiles) {
  __shared__ float sums[4][kCols];
  constexpr int U = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int block = blockIdx.x / col_tiles, col_tile = blockIdx.x % col_tiles;
  Segment s{0, 0, p.rows, block};
  if (p.offsets && !find_segment(p.offsets, p.groups, p.rows, p.block_rows, block, s)) return;
  const int64_t first = (int64_t)s.tile * p.block_rows;
  const int count = (int)(s.count - first < p.block_rows ? s.count - first : p.block_rows);
  const int64_t col = (int64_t)col_tile * kCols + lane * 8, left = p.n - col;
  float sum[8] = {};
  if (left > 0) {
    const int64_t dn = GATED ? p.n / 2 : p.n;
    const T* z = static_cast<const T*>(p.z) + (s.begin + first) * p.n + col;
    const T* dy = static_cast<const T*>(p.dy) + (s.begin + first) * dn + (GATED ? col / 2 : col);
    T* dz = static_cast<T*>(p.dz) + (s.begin + first) * p.n + col;
    for (int r0 = wave; r0 < count; r0 += 4 * U) {
      Run<T, 8, VEC> zr[U];
      Run<T, GATED ? 4 : 8, VEC> dr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r0 + 4 * u < count ? r0 + 4 * u : count - 1;
        zr[u].load(z + row * p.n, left);
        dr[u].load(dy + row * dn, GATED ? left / 2 : left);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + 4 * u >= count) break;
        float v[8];
        if constexpr (GATED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float g = (float)zr[u].v[2 * i], up = (float)zr[u].v[2 * i + 1], d = (float)dr[u].v[i];
            const float sg = sigmoid_f(g);
            v[2 * i] = d * up * silu_slope(g, sg);
            v[2 * i + 1] = d * (g * sg);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = act_grad_f((float)dr[u].v[i], (float)zr[u].v[i], p.act);
        }
        Run<T, 8, VEC> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (SUM) sum[i] += v[i];
          o.v[i] = (T)v[i];
        }
        o.store(dz + (int64_t)(r0 + 4 * u) * p.n, left);
      }
    }
  }
  if constexpr (SUM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[wave][lane * 8 + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += 256) {
      const int64_t at = (int64_t)col_tile * kCols + c;
      if (at < p.n) p.partials[(int64_t)block * p.n + at] = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
    }
  }
}

// db[g] = the partial sums of the group's row blocks. A column has kLanes threads, each with
// every kLanes-th block in order; their sums are added in order. (A group with a third of
// the rows has hundreds of blocks: one thread after them all was the longest part.)
constexpr int kLanes = 4;

__global__ __launch_bounds__(64 * kLanes) void act_grad_sum_kernel(ActGradLaunch p, int col_tiles) {
  __shared__ float sums[kLanes][64];
  const int g = blockIdx.x / col_tiles, lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t col = (int64_t)(blockIdx.x % col_tiles) * 64 + lane;
  const int each = p.block_rows;
  int first = 0, blocks = (int)((p.rows + each - 1) / each);
  // (malformed offsets stay inside the workspace)
  if (p.offsets) blocks = tiles_of(p.offsets, g, p.rows, each, (int)act_grad_blocks(p.rows, p.groups, each), first);
  float sum = 0.0f;
  if (col < p.n) {
    const float* q = p.partials + (int64_t)first * p.n + col;
#pragma unroll 8
    for (int b = part; b < blocks; b += kLanes) sum += q[(int64_t)b * p.n];
  }
  sums[part][lane] = sum;
  __syncthreads();
  if (part == 0 && col < p.n) {
    for (int i = 1; i < kLanes; ++i) sum += sums[i][lane];
    p.db[(int64_t)g * p.n + col] = sum;
  }
}

template <typename T, bool SUM, bool GATED>
void launch_rows(const ActGradLaunch& a, dim3 grid, int col_tiles, hipStream_t st) {
  if (a.n % 8 == 0)
    act_grad_kernel<T, SUM, GATED, true><<<grid, 256, 0, st>>>(a, col_tiles);
  else
    act_grad_kernel<T, SUM, GATED, false><<<grid, 256, 0, st>>>(a, col_tiles);
}

template <typename T>
hipError_t launch_t(ActGradLaunch a, hipStream_t st) {
  const int64_t col_tiles = (a.n + kCols - 1) / kCols, blocks = act_grad_blocks(a.rows, a.groups, a.block_rows);
  // one block of rows: its sums are the bias gradient
  const bool direct = a.db && !a.offsets && blocks == 1;
  if (direct) a.partials = a.db;
  if (blocks > 0) {
    const dim3 grid((uint32_t)(blocks * col_tiles));
    const bool gated = a.act == kActSwiglu;
    if (a.db && gated)
      launch_rows<T, true, true>(a, grid, (int)col_tiles, st);
    else if (a.db)
      launch_rows<T, true, false>(a, grid, (int)col_tiles, st);
    else if (gated)
      launch_rows<T, false, true>(a, grid, (int)col_tiles, st);
    else
      launch_rows<T, false, false>(a, grid, (int)col_tiles, st);
  }
  if (a.db && !direct) {
    const int64_t sum_tiles = (a.n + 63) / 64;
    act_grad_sum_kernel<<<dim3((uint32_t)(a.groups * sum_tiles)), 64 * kLanes, 0, st>>>(a, (int)sum_tiles);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_grad(const ActGradLaunch& a, hipStream_t st) {
  return a.f32 ? launch_t<float>(a, st) : launch_t<__bf16>(a, st);
}

}  // namespace mxq
