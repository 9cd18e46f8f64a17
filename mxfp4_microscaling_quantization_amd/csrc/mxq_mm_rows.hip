// Matrix products on MXFP4 / FP8 operands for few rows (of a call, or of each expert):
// the weight streams from memory to the matrix cores once, with no stop in LDS.
#include "mxq_mm.h"

namespace mxq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A 16x16x128 instruction: lane l holds elements [32 g, 32 g + 32) of operand row l % 16,
// g = l / 16, and result rows 4 g .. 4 g + 3 of the first operand (the weight's, so four
// consecutive columns) against row l % 16 of the second. A chunk is 256 elements of a
// row, two steps of 128.
template <bool FP8>
struct Part {
  v4i w[2][FP8 ? 2 : 1];
  uint32_t scale[2];  // MXFP4: the low byte is this lane's block; FP8: the fp32 scale's bits
};

template <bool FP8>
__device__ __forceinline__ void load_part(Part<FP8>& p, const uint8_t* row, const uint8_t* scales, int64_t k, int c,
                                          int g) {
  if ((int64_t)(c + 1) * 256 <= k) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t at = (int64_t)c * 256 + s * 128 + 32 * g;
      const v4i* q = reinterpret_cast<const v4i*>(row + (FP8 ? at : at / 2));
#pragma unroll
      for (int i = 0; i < (FP8 ? 2 : 1); ++i) p.w[s][i] = q[i];
    }
    // a row's eight bytes of scales, the same in its four lanes (block bytes start anywhere)
    uint32_t raw[2];
    __builtin_memcpy(raw, scales + (int64_t)c * 8, 8);
#pragma unroll
    for (int s = 0; s < 2; ++s) p.scale[s] = FP8 ? raw[s] : raw[s] >> (8 * g);
    return;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t at = (int64_t)c * 256 + s * 128 + 32 * g;
    const bool in = at < k;  // an MXFP4 row may end in any block; a lane's are whole
    const int64_t from = in ? at : 0;
    const v4i* q = reinterpret_cast<const v4i*>(row + (FP8 ? from : from / 2));
#pragma unroll
    for (int i = 0; i < (FP8 ? 2 : 1); ++i) {
      const v4i v = q[i];
      p.w[s][i] = in ? v : v4i{0, 0, 0, 0};
    }
    if constexpr (FP8)
      p.scale[s] = in ? reinterpret_cast<const uint32_t*>(scales)[from / 128] : 0x3F800000u;
    else
      p.scale[s] = in ? scales[from / 32] : 127u;
  }
}

template <bool FP8>
__device__ __forceinline__ bf16x8 bf16_part(const Part<FP8>& p, int s, int j, float scale) {
  if constexpr (FP8)
    return bf16_from_e4m3((uint32_t)p.w[s][j / 2][2 * (j % 2)], (uint32_t)p.w[s][j / 2][2 * (j % 2) + 1], scale);
  else
    return bf16_from_e2m1((uint32_t)p.w[s][0][j], scale);
}

template <bool FP8>
__device__ __forceinline__ float scale_part(const Part<FP8>& p, int s) {
  return e8m0_operand((FP8 ? p.scale[s] >> 23 : p.scale[s]) & 255u);
}

// One workgroup: 16 MT rows of one segment, 16 NT columns. Its W waves share the chunks
// out in turn, D of a wave in flight together, and their sums are added in wave order
// through LDS (so equal inputs give equal bits).
// Bound by the weight's bytes where there are many (8 rows for each of 64 experts of 4096 x 7168:
// 1.0 GB in 201 us, 5.0 TB/s; 512 rows of which about 50 of them have any: 0.8 GB in 175 us), by a
// wave's latencies and the launch where there are few (one row of 4096 x 14336: 31 MB in 9 us).
template <bool A8, bool B8, int MT, int NT, int W, int D, typename T>
__global__ __launch_bounds__(64 * W, 1) void mm_rows_kernel(MmLaunch p, int col_tiles) {
  __shared__ float sums[W][MT * 16][NT * 16 + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int row_tile, col_tile;
  Segment s{0, 0, p.rows, 0};
  if (p.offsets) {
    // the row tiles of an expert follow each other for one column tile, so that its weight
    // rows are read together
    row_tile = blockIdx.x / col_tiles;
    col_tile = blockIdx.x % col_tiles;
    if (!find_segment(p.offsets, p.groups, p.rows, 16 * MT, row_tile, s)) return;
  } else {
    const int row_tiles = (int)((p.rows + 16 * MT - 1) / (16 * MT));
    s.tile = blockIdx.x % row_tiles;
    col_tile = blockIdx.x / row_tiles;
  }
  const int64_t first = s.begin + (int64_t)s.tile * 16 * MT;
  const int rows = (int)(s.count - (int64_t)s.tile * 16 * MT < 16 * MT ? s.count - (int64_t)s.tile * 16 * MT : 16 * MT);
  const int64_t abytes = A8 ? p.k : p.k / 2, bbytes = B8 ? p.k : p.k / 2;
  const int64_t asbytes = A8 ? p.k / 128 * 4 : p.k / 32, bsbytes = B8 ? p.k / 128 * 4 : p.k / 32;
  const uint8_t *a[MT], *b[NT], *as[MT], *bs[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = first + (16 * i + r < rows ? 16 * i + r : rows - 1);
    a[i] = p.a + row * abytes;
    as[i] = static_cast<const uint8_t*>(p.a_scales) + row * asbytes;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t col = (int64_t)col_tile * 16 * NT + 16 * j + r;
    const int64_t row = (int64_t)s.expert * p.n + (col < p.n ? col : p.n - 1);
    b[j] = p.b + row * bbytes;
    bs[j] = static_cast<const uint8_t*>(p.b_scales) + row * bsbytes;
  }
  const int chunks = (int)((p.k + 255) / 256);
  f32x4 c[MT][NT] = {};
  for (int base = wave; base < chunks; base += W * D) {
    Part<A8> pa[D][MT];
    Part<B8> pb[D][NT];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int at = base + W * d;
      if (at >= chunks) break;
#pragma unroll
      for (int j = 0; j < NT; ++j) load_part<B8>(pb[d][j], b[j], bs[j], p.k, at, g);
#pragma unroll
      for (int i = 0; i < MT; ++i) load_part<A8>(pa[d][i], a[i], as[i], p.k, at, g);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (base + W * d >= chunks) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if constexpr (!A8 && !B8) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              c[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  widen(pb[d][j].w[t][0]), widen(pa[d][i].w[t][0]), c[i][j], kE2M1, kE2M1, 0, (int)pb[d][j].scale[t], 0,
                  (int)pa[d][i].scale[t]);
        } else {
          // exact: both widened to bf16, 32 elements an instruction
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            bf16x8 wa[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) wa[i] = bf16_part<A8>(pa[d][i], t, q, scale_part<A8>(pa[d][i], t));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const bf16x8 wb = bf16_part<B8>(pb[d][j], t, q, scale_part<B8>(pb[d][j], t));
#pragma unroll
              for (int i = 0; i < MT; ++i)
                c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, wa[i], c[i][j], 0, 0, 0);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(&sums[wave][16 * i + r][16 * j + 4 * g]) = c[i][j];
  __syncthreads();
  for (int at = threadIdx.x; at < MT * 16 * NT * 4; at += 64 * W) {
    const int row = at / (NT * 4), col = at % (NT * 4) * 4;
    if (row >= rows) break;
    float z[4] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int v = 0; v < 4; ++v) z[v] += sums[w][row][col + v];
    epilogue_run<T, 4>(p.ep, first + row, s.expert, (int64_t)col_tile * 16 * NT + col, z);
  }
}

template <bool A8, bool B8, int MT, int NT, int W, int D>
hipError_t launch_waves(const MmLaunch& a, hipStream_t st) {
  const int64_t col_tiles = (a.n + 16 * NT - 1) / (16 * NT);
  const int64_t row_tiles = a.offsets ? most_tiles(a.rows, a.groups, 16 * MT) : (a.rows + 16 * MT - 1) / (16 * MT);
  const dim3 grid((uint32_t)(row_tiles * col_tiles));
  if (a.ep.out_f32)
    mm_rows_kernel<A8, B8, MT, NT, W, D, float><<<grid, 64 * W, 0, st>>>(a, (int)col_tiles);
  else if constexpr (A8 && B8 && MT == 2)
    return hipErrorInvalidValue;  // launch_gemm sends these to the tiles
  else
    mm_rows_kernel<A8, B8, MT, NT, W, D, __bf16><<<grid, 64 * W, 0, st>>>(a, (int)col_tiles);
  return hipGetLastError();
}

// Up to 16 rows. Where 16-column workgroups leave CUs idle, many waves split a long k; where
// they fill the chip several times over, wider ones read A's rows for more columns and
// pass over the chip fewer times (us, MXFP4, one row of n x k; 16 columns and 4, 8, 16 waves:
// 4096 x 14336 16.3, 12.2, 10.5; 4096 x 4096 5.9, 5.3, 5.6; 16 columns and 4 waves, 32 and 8,
// 64 and 4: 14336 x 4096 11.0, 10.1, 13.8; 28672 x 4096 19.8, 17.8, 17.0; 64 experts of
// 4096 x 7168 for 512 rows 238, 206, 184.5).
// More rows: 32 x 32 results, so that a row of A is read for 32 columns
// (64 rows of 4096 x 4096: 9.0 us; 32 x 16 results 12.5, 64 x 32 11.3).
template <bool A8, bool B8>
hipError_t launch_rows(const MmLaunch& a, bool few, hipStream_t st) {
  if (!few) return launch_waves<A8, B8, 2, 2, 8, 2>(a, st);
  const int64_t tiles = (a.n + 15) / 16 * (a.offsets ? (a.rows < a.groups ? a.rows : a.groups) : 1);
  if (tiles >= 1536) return launch_waves<A8, B8, 1, 4, 4, 1>(a, st);
  if (tiles >= 768) return launch_waves<A8, B8, 1, 2, 8, 1>(a, st);
  if (a.k > 8192) return launch_waves<A8, B8, 1, 1, 16, 2>(a, st);
  return launch_waves<A8, B8, 1, 1, 8, 2>(a, st);
}

}  // namespace

hipError_t launch_gemm_rows(const MmLaunch& a, bool few, hipStream_t st) {
  if (a.a_fmt && a.b_fmt) return launch_rows<true, true>(a, few, st);
  if (a.a_fmt) return launch_rows<true, false>(a, few, st);
  return launch_rows<false, false>(a, few, st);
}

}  // namespace mxq
