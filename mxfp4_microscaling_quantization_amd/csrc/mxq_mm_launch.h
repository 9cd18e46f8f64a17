// Host-side launch interface of the matrix products and the epilogue's gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

struct MmEpilogue {
  const void* bias;  // [groups, n] or null
  const void* res;   // as d, or null
  void* d;           // [rows, n], or [rows, n / 2] for kActSwiglu
  void* z;           // [rows, n] or null
  int64_t n;
  int act;
  int bias_f32, out_f32;
};

// One product. Dense: groups == 1 and offsets == null; grouped: `rows` tokens of
// `groups` experts. fmt 0: MXFP4, 1: FP8.
struct MmLaunch {
  const uint8_t *a, *b;
  const void *a_scales, *b_scales;
  int a_fmt, b_fmt;
  int64_t rows, n, k;
  const int64_t* offsets;
  int groups;
  MmEpilogue ep;
  int64_t ld_a, ld_b, ld_as, ld_bs;  // weight gradient only: row pitches of codes and scales
};

// Few rows: 16 (few) or 32 rows of a workgroup, the weight straight from memory.
hipError_t launch_gemm_rows(const MmLaunch& a, bool few, hipStream_t st);
// The tiled kernel: `side` x `side` results of a workgroup (64, 128 or 256).
hipError_t launch_gemm_tiles(const MmLaunch& a, int side, hipStream_t st);
// The side for `each` results of rows x cols, the rows those of `experts` (0: of one matrix), each of
// which has a row tile at least and half of one over on average. Tiles of 64 while all of them run at once, two on each of the 256 CUs (MXFP4 / FP8, k 4096, 64 and 128, us:
// 256 x 4096 results 11.0 and 15.1 / 12.8 and 20.4, 512 x 4096 13.8 and 15.8 / 18.1 and 21.8,
// 256 x 14336 25.7 and 17.6 / 33.8 and 24.0). A tile of 256 takes about 2.2 times one of 128's time
// for four times its results, and 256 of either run at once (MXFP4, k 4096, 256 and 128, us:
// 1024 x 4096 results 32.0 and 17.9, 2048 x 4096 33.3 and 31.5, 4096 x 4096 40.0 and 58.2).
int tile_side(int64_t rows, int64_t cols, int64_t experts, int64_t each);
hipError_t launch_gemm(const MmLaunch& a, hipStream_t st);

// The weight gradient of every expert: a = dY's FP8 columns [n, ld_a], b = X's [k, ld_b],
// contracted over the tokens of each segment; ep.d [groups * n, k], ep.n = k.
hipError_t launch_grouped_wgrad(const MmLaunch& a, hipStream_t st);

struct ActGradLaunch {
  const void *dy, *z;
  int f32;
  int64_t rows, n;
  int act;
  const int64_t* offsets;
  int groups;
  void* dz;
  float* db;
  float* partials;
  int block_rows;
  const float* z_scales;  // z in FP8 only: [rows, ceil(n / 128)]
  void* h;                // z in FP8 only: act(z), or null
};

// Rows that one workgroup of the activation gradient sums: all of up to 64, whose sums then
// need no second launch, else few where there would be fewer workgroups of many than the chip
// holds. (us with the binding, one launch, and blocks of 16 rows with their sums. Outputs that the
// call makes: 1336 fp32 gelu, 17 rows 11.4 and 14.0, 48 rows 11.5 and 14.2, 64 rows 13.4 and 14.3;
// 4096 bf16 swiglu, 64 rows 11.7 and 14.4. Outputs given: 4096 bf16 swiglu, 64 rows 7.5 and 10.2;
// 1336 fp32 gelu, 17 rows 7.3 and 10.2, 32 rows 9.4 and 10.1, and past about 36 rows the other way,
// 64 rows 16.0 and 10.2; 14336 bf16 gelu, 32 rows 7.8 and 10.2, 64 rows 13.9 and 10.2.)
constexpr int act_grad_rows(int64_t rows, int64_t n) {
  return rows <= 64 ? 64 : rows * ((n + 511) / 512) < 128 * 1024 ? 16 : 128;
}
// The row blocks that any split of the rows into groups has at most.
constexpr int64_t act_grad_blocks(int64_t rows, int64_t groups, int64_t each) {
  return (rows + (each - 1) * groups) / each;
}
hipError_t launch_act_grad(const ActGradLaunch& a, hipStream_t st);
hipError_t launch_fp8_act_grad(const ActGradLaunch& a, hipStream_t st);

}  // namespace mxq
