// The gradient of the products' epilogue: dz = act'(z) dy and its column sums per
// group of rows (the bias gradient).
#include "mxq_mm.h"

namespace mxq {

namespace {

constexpr int kCols = 512;  // columns of a workgroup: 64 lanes of 8

// act'(z) and, for SWIGLU, both halves of a pair (gate g, up u).
__device__ __forceinline__ float act_grad_f(float dy, float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.0f ? dy : 0.0f;
    case kActGelu: {
      // d/dz [z s(w)], w = A z + B z^3: s + z s (1 - s) (A + 3 B z^2)
      const float zz = z * z, s = sigmoid_f(z * fmaf(kGeluB, zz, kGeluA));
      return dy * fmaf(z * s * (1.0f - s), fmaf(3.0f * kGeluB, zz, kGeluA), s);
    }
    case kActSilu: {
      const float s = sigmoid_f(z);
      return dy * (s * fmaf(z, 1.0f - s, 1.0f));
    }
  }
  return dy;
}

template <typename T>
__device__ __forceinline__ void load_run(const T* p, float (&v)[8], int64_t left, bool vec) {
  if (vec) {
    get_run<T, 8>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? Out<T>::get(p + i) : 0.0f;
  }
}

// One workgroup: up to 64 rows of one group, 512 columns. Its waves take every fourth
// row; the sums of the four waves are added in order through LDS.
template <typename T, bool SUM>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradLaunch p, int col_tiles) {
  __shared__ float sums[4][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int block = blockIdx.x / col_tiles, col_tile = blockIdx.x % col_tiles;
  Segment s{0, 0, p.rows, block};
  if (p.offsets && !find_segment(p.offsets, p.groups, p.rows, kActGradRows, block, s)) return;
  const int64_t first = (int64_t)s.tile * kActGradRows;
  const int count = (int)(s.count - first < kActGradRows ? s.count - first : kActGradRows);
  const int64_t col = (int64_t)col_tile * kCols + lane * 8, left = p.n - col;
  const bool vec = p.n % 8 == 0, gated = p.act == kActSwiglu;
  float sum[8] = {};
  if (left > 0) {
    // four rows of a wave in flight: their loads go ahead of the first one's arithmetic
    for (int r0 = wave; r0 < count; r0 += 16) {
      float z[4][8], dy[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t row = s.begin + first + (r0 + 4 * u < count ? r0 + 4 * u : count - 1);
        load_run<T>(static_cast<const T*>(p.z) + row * p.n + col, z[u], left, vec);
        if (gated) {
          const T* q = static_cast<const T*>(p.dy) + row * (p.n / 2) + col / 2;
          float g[4];
          if (vec) {
            get_run<T, 4>(q, g);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = 2 * i < left ? Out<T>::get(q + i) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) dy[u][2 * i] = g[i];
        } else {
          load_run<T>(static_cast<const T*>(p.dy) + row * p.n + col, dy[u], left, vec);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r0 + 4 * u >= count) break;
        float dz[8];
        if (gated) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float g = z[u][2 * i], sg = sigmoid_f(g), d = dy[u][2 * i];
            dz[2 * i] = d * z[u][2 * i + 1] * (sg * fmaf(g, 1.0f - sg, 1.0f));
            dz[2 * i + 1] = d * (g * sg);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dz[i] = act_grad_f(dy[u][i], z[u][i], p.act);
        }
        if (SUM) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += dz[i];
        }
        store_run<T, 8>(static_cast<T*>(p.dz) + (s.begin + first + r0 + 4 * u) * p.n + col, nullptr, dz, left, vec);
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
constexpr int kLanes = 16;

__global__ __launch_bounds__(64 * kLanes) void act_grad_sum_kernel(ActGradLaunch p, int col_tiles) {
  __shared__ float sums[kLanes][64];
  const int g = blockIdx.x / col_tiles, lane = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int64_t col = (int64_t)(blockIdx.x % col_tiles) * 64 + lane;
  int first = 0, blocks = (int)((p.rows + kActGradRows - 1) / kActGradRows);
  if (p.offsets) {
    first = segment_tiles(p.offsets, g, p.rows, kActGradRows);
    const int64_t c = clamp_row(p.offsets[g + 1], p.rows) - clamp_row(p.offsets[g], p.rows);
    blocks = c > 0 ? (int)((c + kActGradRows - 1) / kActGradRows) : 0;
    // malformed offsets stay inside the workspace
    const int most = (int)act_grad_blocks(p.rows, p.groups);
    blocks = first >= most ? 0 : first + blocks > most ? most - first : blocks;
  }
  float sum = 0.0f;
  if (col < p.n) {
    const float* q = p.partials + (int64_t)first * p.n + col;
#pragma unroll 4
    for (int b = part; b < blocks; b += kLanes) sum += q[(int64_t)b * p.n];
  }
  sums[part][lane] = sum;
  __syncthreads();
  if (part == 0 && col < p.n) {
    for (int i = 1; i < kLanes; ++i) sum += sums[i][lane];
    p.db[(int64_t)g * p.n + col] = sum;
  }
}

template <typename T>
hipError_t launch_t(const ActGradLaunch& a, hipStream_t st) {
  const int64_t col_tiles = (a.n + kCols - 1) / kCols, blocks = act_grad_blocks(a.rows, a.groups);
  if (blocks > 0) {
    const dim3 grid((uint32_t)(blocks * col_tiles));
    if (a.db)
      act_grad_kernel<T, true><<<grid, 256, 0, st>>>(a, (int)col_tiles);
    else
      act_grad_kernel<T, false><<<grid, 256, 0, st>>>(a, (int)col_tiles);
  }
  if (a.db) {
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
