// Host-side launch interface of the operators around the experts' products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// launch(first token, tokens) for runs of tokens that one launch holds: grids count threads in 32 bits.
template <typename F>
hipError_t by_slabs(int64_t tokens, int64_t threads_of_token, F&& launch) {
  const int64_t most = ((int64_t)1 << 31) / threads_of_token;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    launch(t0, tokens - t0 < most ? tokens - t0 : most);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

struct RouteLaunch {
  const void* logits;  // [tokens, experts], row stride ld
  int f32;
  int64_t tokens, ld;
  int experts, top_k, renorm;
  float* weights;  // [tokens, top_k]
  int32_t* chosen;
  const float* dw;  // gradient only
  void* dlogits;    // gradient only: [tokens, experts]
};
hipError_t launch_route(const RouteLaunch& a, hipStream_t st);
hipError_t launch_route_grad(const RouteLaunch& a, hipStream_t st);

struct SortLaunch {
  const int32_t* experts;  // [count]
  int64_t count;
  int n_experts;
  int64_t* offsets;
  int32_t *positions, *order;
  int32_t* counts;  // workspace [blocks, n_experts], then [n_experts]
};
// Up to this many assignments one workgroup does everything in one launch (256 experts, us: 4096
// assignments 6.6, 6144 8.5 and 11.4 in three launches, 8192 10.0 and 11.4, 12288 13.4 and 11.4).
constexpr int64_t kSortOne = 8192;
// Assignments of a block otherwise: as many as keep the table of counts at 1024 blocks at most.
constexpr int64_t sort_chunk(int64_t count) {
  return count <= 1024 * 2048 ? 2048 : (count + 1023) / 1024 + 255 & ~(int64_t)255;
}
constexpr int64_t sort_blocks(int64_t count) { return (count + sort_chunk(count) - 1) / sort_chunk(count); }
// Two launches, every block summing up the table of counts for itself, while all of them together read
// up to 64 MiB of it; else three. (Two and three launches, us of the kernels: 33600 assignments to 256
// experts 10.2 and 11.6, 131072 10.1 and 12.0, 524288 14.5 and 13.8, but with the launches' own time
// 14.7 and 16.6; 524288 to 64 experts 10.7 and 12.2, to 512 19.5 and 15.1.)
constexpr bool sort_in_two(int64_t count, int64_t experts) {
  return experts <= 512 && sort_blocks(count) * sort_blocks(count) * experts <= (int64_t)1 << 24;
}
constexpr int64_t sort_workspace(int64_t count, int64_t experts) {
  return count <= kSortOne ? 0 : (sort_blocks(count) + 1) * experts * 4;
}
hipError_t launch_expert_sort(const SortLaunch& a, hipStream_t st);

// dispatch and combine: rows of tokens and rows of experts.
struct RowsLaunch {
  const void* x;  // dispatch: tokens; combine: experts' rows; gradient: of the tokens
  int x_f32;
  int64_t ldx;  // dispatch only
  int64_t tokens, width, rows;
  const int32_t* positions;
  int top_k;
  int fmt;  // dispatch only
  const float* weights;
  const void* res;  // combine: residual; gradient: experts' rows
  void* out;        // dispatch, gradient: experts' rows; combine: tokens
  int out_f32;
  void* scales;  // dispatch only
  float* dw;     // gradient only
};
hipError_t launch_dispatch(const RowsLaunch& a, hipStream_t st);
hipError_t launch_combine(const RowsLaunch& a, hipStream_t st);
hipError_t launch_combine_grad(const RowsLaunch& a, hipStream_t st);

hipError_t launch_fp8_quantize(const void* x, int f32, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q8,
                               float* scales, hipStream_t st);

}  // namespace mxq
