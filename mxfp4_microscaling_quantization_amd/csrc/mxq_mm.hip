// Matrix products on MXFP4 / FP8 operands, dense and grouped by expert, and the
// weight gradient over experts' token segments. This file's kernels take one 32x32
// tile of the result per wave, fragments straight from global memory.
#include "mxq_mm.h"

namespace mxq {

namespace {

// The 32 elements of one lane half: [k0, k0 + 32) of a row (all inside k or all past it).
template <bool FP8>
__device__ __forceinline__ void load_block(const uint8_t* row, const void* scales, int64_t srow, int64_t k, int64_t k0,
                                           uint32_t (&w)[8], uint32_t& byte) {
  const bool in = k0 < k;
  const int64_t at = in ? k0 : 0;
  const v4i* p = reinterpret_cast<const v4i*>(row + (FP8 ? at : at / 2));
  const v4i lo = p[0];
  v4i hi = {};
  if constexpr (FP8) {
    hi = p[1];
    byte = (as_u(static_cast<const float*>(scales)[srow * (k / 128) + at / 128]) >> 23) & 255u;
  } else {
    byte = static_cast<const uint8_t*>(scales)[srow * (k / 32) + at / 32];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = in ? (uint32_t)lo[i] : 0u;
    w[4 + i] = in ? (uint32_t)hi[i] : 0u;
  }
  byte = in ? byte : 127u;
}

template <bool FP8>
__device__ __forceinline__ bf16x8 bf16_run(const uint32_t (&w)[8], int j, float scale) {
  return FP8 ? bf16_from_e4m3(w[2 * j], w[2 * j + 1], scale) : bf16_from_e2m1(w[j], scale);
}

template <bool A8, bool B8>
__device__ __forceinline__ f32x16 multiply_blocks(const uint32_t (&a)[8], uint32_t sa, const uint32_t (&b)[8],
                                                  uint32_t sb, f32x16 c) {
  if constexpr (!A8 && !B8) {
    const v8i fa = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const v8i fb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb, fa, c, kE2M1, kE2M1, 0, (int)sb, 0, (int)sa);
  } else {
    const float fa = e8m0_operand(sa), fb = e8m0_operand(sb);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16_run<B8>(b, j, fb), bf16_run<A8>(a, j, fa), c, 0, 0, 0);
    return c;
  }
}

// One wave per 32x32 tile; consecutive workgroups walk the columns of one row tile.
template <bool A8, bool B8, typename T>
__global__ __launch_bounds__(64) void mm_wave_kernel(MmLaunch p, int col_tiles) {
  const int lane = threadIdx.x, r = lane & 31, h = lane >> 5;
  const int row_tile = blockIdx.x / col_tiles, col_tile = blockIdx.x % col_tiles;
  Segment s{0, 0, p.rows, row_tile};
  if (p.offsets && !find_segment(p.offsets, p.groups, p.rows, 32, row_tile, s)) return;
  const int64_t i = (int64_t)s.tile * 32 + r;
  const int64_t row = s.begin + (i < s.count ? i : s.count - 1);
  const int64_t j = (int64_t)col_tile * 32 + r;
  const int64_t brow = (int64_t)s.expert * p.n + (j < p.n ? j : p.n - 1);
  const uint8_t* a = p.a + row * (A8 ? p.k : p.k / 2);
  const uint8_t* b = p.b + brow * (B8 ? p.k : p.k / 2);
  f32x16 c = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += 64) {
    uint32_t wa[8], wb[8], sa, sb;
    load_block<A8>(a, p.a_scales, row, p.k, k0 + 32 * h, wa, sa);
    load_block<B8>(b, p.b_scales, brow, p.k, k0 + 32 * h, wb, sb);
    c = multiply_blocks<A8, B8>(wa, sa, wb, sb, c);
  }
  if (i >= s.count) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float z[4] = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
    epilogue_run<T, 4>(p.ep, row, s.expert, (int64_t)col_tile * 32 + 8 * q + 4 * h, z);
  }
}

template <bool A8, bool B8>
hipError_t launch_wave(const MmLaunch& a, hipStream_t st) {
  const int64_t col_tiles = (a.n + 31) / 32;
  const int64_t row_tiles =
      a.offsets ? a.rows / 32 + (a.rows < a.groups ? a.rows : a.groups) : (a.rows + 31) / 32;
  const dim3 grid((uint32_t)(row_tiles * col_tiles));
  if (a.ep.out_f32)
    mm_wave_kernel<A8, B8, float><<<grid, 64, 0, st>>>(a, (int)col_tiles);
  else
    mm_wave_kernel<A8, B8, __bf16><<<grid, 64, 0, st>>>(a, (int)col_tiles);
  return hipGetLastError();
}

// The 32 tokens [t, t + 32) of a column, those from `end` on as zeros. A token lies at
// any byte, so the words are loaded unaligned; only whole blocks are loaded that way.
__device__ __forceinline__ void load_tokens(const uint8_t* col, int64_t t, int64_t end, uint32_t (&w)[8]) {
  if (t + 32 <= end) {
    __builtin_memcpy(w, col + t, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t + 4 * i + j < end) w[i] |= (uint32_t)col[t + 4 * i + j] << (8 * j);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(64) void wgrad_wave_kernel(WgradLaunch p, int col_tiles, int row_tiles) {
  const int lane = threadIdx.x, r = lane & 31, h = lane >> 5;
  const int col_tile = blockIdx.x % col_tiles, row_tile = blockIdx.x / col_tiles % row_tiles;
  const int e = blockIdx.x / (col_tiles * row_tiles);
  // the expert's first group: all groups of the experts before it
  int slots = 0;
  for (int o = lane; o < e; o += 64) {
    const int64_t c = clamp_row(p.offsets[o + 1], p.rows) - clamp_row(p.offsets[o], p.rows);
    slots += c > 0 ? (int)((c + 127) / 128) : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) slots += __shfl_xor(slots, d);
  const int64_t begin = clamp_row(p.offsets[e], p.rows), end = clamp_row(p.offsets[e + 1], p.rows);
  const int64_t i = (int64_t)row_tile * 32 + r, j = (int64_t)col_tile * 32 + r;
  const int64_t yi = i < p.n ? i : p.n - 1, xj = j < p.k ? j : p.k - 1;
  const int64_t last = (p.rows + 127 * (int64_t)p.experts) / 128 - 1;  // malformed offsets stay in the scales
  f32x16 c = {};
  for (int64_t t = begin; t < end; t += 128) {
    const int64_t g = slots + (t - begin) / 128, slot = g < last ? g : last;
    const uint32_t sy = (as_u(p.y_scales[yi * p.ld_ys + slot]) >> 23) & 255u;
    const uint32_t sx = (as_u(p.x_scales[xj * p.ld_xs + slot]) >> 23) & 255u;
    const int64_t stop = t + 128 < end ? t + 128 : end;
    for (int64_t u = t; u < stop; u += 64) {
      uint32_t wy[8], wx[8];
      load_tokens(p.y + yi * p.ld_y, u + 32 * h, stop, wy);
      load_tokens(p.x + xj * p.ld_x, u + 32 * h, stop, wx);
      c = multiply_blocks<true, true>(wy, sy, wx, sx, c);
    }
  }
  if (i >= p.n) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t j0 = (int64_t)col_tile * 32 + 8 * q + 4 * h;
    if (j0 >= p.k) break;
    float v[4] = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
    const int64_t at = ((int64_t)e * p.n + i) * p.k + j0;
    store_run<T, 4>(static_cast<T*>(p.d) + at, p.add ? static_cast<const T*>(p.add) + at : nullptr, v, p.k - j0,
                    p.k % 4 == 0);
  }
}

}  // namespace

hipError_t launch_gemm(const MmLaunch& a, hipStream_t st) {
  if (a.rows > 32) return launch_gemm_tiles(a, a.rows >= 200, st);
  if (a.a_fmt && a.b_fmt) return launch_wave<true, true>(a, st);
  if (a.a_fmt) return launch_wave<true, false>(a, st);
  return launch_wave<false, false>(a, st);
}

hipError_t launch_grouped_wgrad(const WgradLaunch& a, hipStream_t st) {
  const int64_t col_tiles = (a.k + 31) / 32, row_tiles = (a.n + 31) / 32;
  const dim3 grid((uint32_t)(col_tiles * row_tiles * a.experts));
  if (a.out_f32)
    wgrad_wave_kernel<float><<<grid, 64, 0, st>>>(a, (int)col_tiles, (int)row_tiles);
  else
    wgrad_wave_kernel<__bf16><<<grid, 64, 0, st>>>(a, (int)col_tiles, (int)row_tiles);
  return hipGetLastError();
}

}  // namespace mxq
