// The gradient of the products' epilogue: dz = act'(z) dy and its column sums per
// group of rows (the bias gradient), from z as it was or as it was kept in FP8.
#include "mxq_mm.h"
#include "mxq_moe_fp8.h"

namespace mxq {

namespace {

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
// read once, so non-temporal), or rows that start on any element (the memory system takes such
// accesses) with the last elements one by one, those past the row's end as zeros. Stores of 16 and 8
// bytes of a lane write whole lines and go past the caches (65536 x 4096 bf16 swiglu from FP8 with h 269
// us, through them 280), and so do rows that share lines (16384 x 4098 119 us, through them 148); fp32's
// two pieces of 16 of whole rows, each of which writes half of every line, do not (mxq_act_grad, us through the
// caches and past them: 16384 x 4096 silu 192 and 228, 65536 x 4096 gelu 650 and 851, swiglu with sums 555 and
// 624, 4096 x 4096 gelu 42.0 and 46.1).
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
    } else if (left >= V) {
      __builtin_memcpy(v, p, sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < left ? p[i] : (T)0.0f;
    }
  }
  __device__ __forceinline__ void store(T* p, int64_t left) const {
    if constexpr (VEC && sizeof(v) == 16) {
      uint4 x;
      __builtin_memcpy(&x, v, 16);
      store_nt(reinterpret_cast<uint4*>(p), x);
    } else if constexpr (VEC && sizeof(v) == 8) {
      uint2 x;
      __builtin_memcpy(&x, v, 8);
      store_nt(reinterpret_cast<uint2*>(p), x);
    } else if constexpr (VEC) {
      __builtin_memcpy(__builtin_assume_aligned(p, sizeof(v) < 16 ? sizeof(v) : 16), v, sizeof(v));
    } else if (left >= V) {
      store_any<sizeof(v)>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) p[i] = v[i];
    }
  }
};

// V neighbouring values of z: as they are, or E4M3 under the scale of their 128 columns. `From`: row and
// column of a block's first values of the lane. z as it is starts from there, so that without a gate a
// row's offset serves dy as well.
template <typename T, int V, bool VEC>
struct ZRun {
  static constexpr bool kInOrder = true;
  struct From {
    const T* z;
    __device__ __forceinline__ From(const ActGradLaunch& p, int64_t row, int64_t col)
        : z(static_cast<const T*>(p.z) + row * p.n + col) {}
  };
  Run<T, V, VEC> run;
  __device__ __forceinline__ void load(const ActGradLaunch& p, const From& from, int64_t row, int64_t left) {
    run.load(from.z + row * p.n, left);
  }
  __device__ __forceinline__ void values(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)run.v[i];
  }
};
template <int V, bool VEC>
struct ZRun8 {
  static constexpr bool kInOrder = false;
  struct From {
    int64_t first, col;
    __device__ __forceinline__ From(const ActGradLaunch&, int64_t row, int64_t c) : first(row), col(c) {}
  };
  uint32_t q[V / 4], scale;
  __device__ __forceinline__ void load(const ActGradLaunch& p, const From& from, int64_t r, int64_t left) {
    const int64_t row = from.first + r, col = from.col;
    const uint8_t* z = static_cast<const uint8_t*>(p.z) + row * p.n + col;
    scale = as_u(p.z_scales[row * ((p.n + 127) / 128) + col / 128]);
    if constexpr (VEC && V == 8) {
      const uint2 x = load_nt(reinterpret_cast<const uint2*>(z));
      __builtin_memcpy(q, &x, 8);
    } else if constexpr (VEC) {
      q[0] = load_nt(reinterpret_cast<const uint32_t*>(z));
    } else if (left >= V) {
      __builtin_memcpy(q, z, V);
    } else {
      uint8_t b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = i < left ? z[i] : 0;
      __builtin_memcpy(q, b, V);
    }
  }
  __device__ __forceinline__ void values(float (&v)[V]) const {
    const float s = fp8_scale(scale);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
      v[4 * i] = a.x * s; v[4 * i + 1] = a.y * s; v[4 * i + 2] = b.x * s; v[4 * i + 3] = b.y * s;
    }
  }
};

// One workgroup: up to p.block_rows rows of one group, V columns of a lane. Its waves take every
// fourth row, U of them in flight: their loads go ahead of the first one's arithmetic.
// The sums of the four waves are added in order through LDS. H: act(z) goes out as well.
template <typename T, typename Z, int V, bool SUM, bool GATED, bool VEC, bool H, int U>
__device__ __forceinline__ void grad_block(const ActGradLaunch& p, int col_tiles) {
  constexpr int kCols = 64 * V, D = GATED ? V / 2 : V;  // D: a lane's values of dy
  __shared__ float sums[4][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int block = blockIdx.x / col_tiles, col_tile = blockIdx.x % col_tiles;
  Segment s{0, 0, p.rows, block};
  if (p.offsets && !find_segment(p.offsets, p.groups, p.rows, p.block_rows, block, s)) return;
  const int64_t first = (int64_t)s.tile * p.block_rows;
  const int count = (int)(s.count - first < p.block_rows ? s.count - first : p.block_rows);
  const int64_t col = (int64_t)col_tile * kCols + lane * V, left = p.n - col;
  float sum[V] = {};
  if (left > 0) {
    const int64_t dn = GATED ? p.n / 2 : p.n;
    const typename Z::From z_from(p, s.begin + first, col);
    const int64_t from = (s.begin + first) * dn + (GATED ? col / 2 : col);
    const T* dy = static_cast<const T*>(p.dy) + from;
    T* dz = static_cast<T*>(p.dz) + (s.begin + first) * p.n + col;
    T* h = H ? static_cast<T*>(p.h) + from : nullptr;
    for (int r0 = wave; r0 < count; r0 += 4 * U) {
      Z zr[U];
      Run<T, D, VEC> dr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = r0 + 4 * u < count ? r0 + 4 * u : count - 1;
        zr[u].load(p, z_from, row, left);
        dr[u].load(dy + row * dn, GATED ? left / 2 : left);
        // No load passes another row's: left to itself the compiler puts z of the first row behind all others in
        // bf16, and its arithmetic waits for every row (700 x 2048 gelu 5.9 us, in order 5.3).
        if constexpr (Z::kInOrder) __builtin_amdgcn_sched_barrier(0x7);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + 4 * u >= count) break;
        float z[V], v[V];
        Run<T, D, VEC> ho;
        zr[u].values(z);
        if constexpr (GATED) {
#pragma unroll
          for (int i = 0; i < D; ++i) {
            const float g = z[2 * i], up = z[2 * i + 1], d = (float)dr[u].v[i];
            const float sg = sigmoid_f(g);
            v[2 * i] = d * up * silu_slope(g, sg);
            v[2 * i + 1] = d * (g * sg);
            if constexpr (H) ho.v[i] = (T)(g * sg * up);
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = act_grad_f((float)dr[u].v[i], z[i], p.act);
          if constexpr (H) {
#pragma unroll
            for (int i = 0; i < V; ++i) ho.v[i] = (T)act_f(z[i], p.act);
          }
        }
        Run<T, V, VEC> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (SUM) sum[i] += v[i];
          o.v[i] = (T)v[i];
        }
        o.store(dz + (int64_t)(r0 + 4 * u) * p.n, left);
        if constexpr (H) ho.store(h + (int64_t)(r0 + 4 * u) * dn, GATED ? left / 2 : left);
      }
    }
  }
  if constexpr (SUM) {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][lane * V + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += 256) {
      const int64_t at = (int64_t)col_tile * kCols + c;
      if (at < p.n) p.partials[(int64_t)block * p.n + at] = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
    }
  }
}

// Bound by memory: 65536 x 4096 bf16 swiglu with its sums moves 1.34 GB in 255 us, 5.3 TB/s, what a
// plain stream that reads twice what it writes reaches here.
template <typename T, bool SUM, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradLaunch p, int col_tiles) {
  grad_block<T, ZRun<T, 8, VEC>, 8, SUM, GATED, VEC, false, 4>(p, col_tiles);
}

// Eight rows of a wave in flight: 65536 x 4096 bf16 swiglu from FP8, 64 experts, with its sums and h, 1.35
// GB, 269 us, 5.0 TB/s, with four 278 (without h, 1.08 GB, 205 and 213; fp32 with h 450 and 467). Blocks of 16
// rows, which act_grad_rows gives smaller matrices, have but four for a wave: the other loads are of its last
// row again, for nothing, and four in flight would take less there (4096 x 4096 bf16 with h 27.8 us, four 24.3;
// 16384 x 1024 27.8 and 24.3, fp32 38.5 and 34.9; 4096 x 14336 gelu without h 77.9 and 63.7). Rows that start
// anywhere: four (16384 x 4098 119 us, eight 123). 16 bytes of a lane's dz: 8 columns in bf16, 4 in fp32 (16384 x
// 4096 fp32 with h 132 us, 8 columns 150).
template <typename T>
constexpr int kFp8Run = 16 / sizeof(T);
template <typename T, bool SUM, bool GATED, bool VEC, bool H>
__global__ __launch_bounds__(256) void fp8_act_grad_kernel(ActGradLaunch p, int col_tiles) {
  grad_block<T, ZRun8<kFp8Run<T>, VEC>, kFp8Run<T>, SUM, GATED, VEC, H, VEC ? 8 : 4>(p, col_tiles);
}

// db[g] = the partial sums of the group's row blocks. A column has kLanes threads, each with
// every kLanes-th block in order; their sums are added in order. (A group with a third of
// the rows has hundreds of blocks: one thread after them all was the longest part.)
// Narrow matrices of many rows have few threads for thousands of blocks, which then take as long as
// their loads one batch after the other: kAhead in flight, added in order (gradient from FP8, rows and
// sums, 65536 x 256 44 us, with 32 in flight 49, with 8 76; 36327 x 512 36, 37 and 51).
constexpr int kLanes = 4, kAhead = 64;

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
    int b = part;
    for (; b + (kAhead - 1) * kLanes < blocks; b += kAhead * kLanes) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = q[(int64_t)(b + i * kLanes) * p.n];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) sum += v[i];
    }
#pragma unroll 8
    for (; b < blocks; b += kLanes) sum += q[(int64_t)b * p.n];
  }
  sums[part][lane] = sum;
  __syncthreads();
  if (part == 0 && col < p.n) {
    for (int i = 1; i < kLanes; ++i) sum += sums[i][lane];
    p.db[(int64_t)g * p.n + col] = sum;
  }
}

template <typename T, bool SUM, bool GATED>
struct Rows {
  static constexpr int kRun = 8;
  static void launch(const ActGradLaunch& a, dim3 grid, int col_tiles, hipStream_t st) {
    if (a.n % 8 == 0)
      act_grad_kernel<T, SUM, GATED, true><<<grid, 256, 0, st>>>(a, col_tiles);
    else
      act_grad_kernel<T, SUM, GATED, false><<<grid, 256, 0, st>>>(a, col_tiles);
  }
};
template <typename T, bool SUM, bool GATED>
struct Fp8Rows {
  static constexpr int kRun = kFp8Run<T>;
  template <bool VEC>
  static void launch_v(const ActGradLaunch& a, dim3 grid, int col_tiles, hipStream_t st) {
    if (a.h)
      fp8_act_grad_kernel<T, SUM, GATED, VEC, true><<<grid, 256, 0, st>>>(a, col_tiles);
    else
      fp8_act_grad_kernel<T, SUM, GATED, VEC, false><<<grid, 256, 0, st>>>(a, col_tiles);
  }
  static void launch(const ActGradLaunch& a, dim3 grid, int col_tiles, hipStream_t st) {
    if (a.n % 8 == 0) launch_v<true>(a, grid, col_tiles, st);
    else launch_v<false>(a, grid, col_tiles, st);
  }
};

template <template <typename, bool, bool> class Kernel, typename T>
hipError_t launch_t(ActGradLaunch a, hipStream_t st) {
  constexpr int kCols = 64 * Kernel<T, true, true>::kRun;
  const int64_t col_tiles = (a.n + kCols - 1) / kCols, blocks = act_grad_blocks(a.rows, a.groups, a.block_rows);
  // one block of rows: its sums are the bias gradient
  const bool direct = a.db && !a.offsets && blocks == 1;
  if (direct) a.partials = a.db;
  if (blocks > 0) {
    const dim3 grid((uint32_t)(blocks * col_tiles));
    const bool gated = a.act == kActSwiglu;
    if (a.db && gated)
      Kernel<T, true, true>::launch(a, grid, (int)col_tiles, st);
    else if (a.db)
      Kernel<T, true, false>::launch(a, grid, (int)col_tiles, st);
    else if (gated)
      Kernel<T, false, true>::launch(a, grid, (int)col_tiles, st);
    else
      Kernel<T, false, false>::launch(a, grid, (int)col_tiles, st);
  }
  if (a.db && !direct) {
    const int64_t sum_tiles = (a.n + 63) / 64;
    act_grad_sum_kernel<<<dim3((uint32_t)(a.groups * sum_tiles)), 64 * kLanes, 0, st>>>(a, (int)sum_tiles);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_grad(const ActGradLaunch& a, hipStream_t st) {
  return a.f32 ? launch_t<Rows, float>(a, st) : launch_t<Rows, __bf16>(a, st);
}
hipError_t launch_fp8_act_grad(const ActGradLaunch& a, hipStream_t st) {
  return a.f32 ? launch_t<Fp8Rows, float>(a, st) : launch_t<Fp8Rows, __bf16>(a, st);
}

}  // namespace mxq
