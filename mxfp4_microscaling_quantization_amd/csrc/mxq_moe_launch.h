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
// Up to this many assignments one workgroup does everything in one launch, without a workspace. (One
// launch and the two or, past 512 experts, three that would do it otherwise, us of calls in a row. 64 experts:
// 4096 assignments 5.4 and 7.5, 6144 7.1 and 7.4, 8192 8.4 and 7.6, 12288 11.2 and 7.7. 256: 6.1 and 7.9, 8.1 and
// 8.2, 9.5 and 8.2, 13.0 and 8.6. 512: 6.9 and 8.8, 9.0 and 9.0, 10.5 and 9.2, 14.2 and 9.6. 1024, where the
// workgroup has two waves instead of 16: 1024 assignments 10.4 and 12.1, 2048 16.1 and 13.7, 8192 50.3 and 13.7.
// So between 6144 and the limit a call of up to 512 experts takes up to 1.3 us more than it need, and one of
// more experts loses from between 1024 and 2048 on. The limit is older than the two launches; callers may give no
// workspace up to it.)
constexpr int64_t kSortOne = 8192;
// Assignments of a block otherwise: as many as keep the table of counts at 1024 blocks at most.
constexpr int64_t sort_chunk(int64_t count) {
  return count <= 1024 * 2048 ? 2048 : (count + 1023) / 1024 + 255 & ~(int64_t)255;
}
constexpr int64_t sort_blocks(int64_t count) { return (count + sort_chunk(count) - 1) / sort_chunk(count); }
// Two launches, every block summing up the table of counts for itself, while all of them together read
// up to 64 MiB of it; else three. (Two and three launches, us of calls in a row from C. 256 experts: 131072
// assignments 9.6 and 11.4, 262144 11.1 and 11.9, 524288, the last size of two, 14.5 and 13.6, 655360 22.2 and
// 18.1, 1048576 28.3 and 21.1. 64: 524288 10.1 and 12.0, 1048576, the last, 16.8 and 18.0, 2097152 31.3 and
// 27.8. 512: 131072 11.2 and 12.4, 262144 13.9 and 13.1, and past the last size 524288 20.4 and 15.1. Through the
// Python binding, where the host's time for a third launch counts, 524288 to 256 experts 14.1 and 17.2.)
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
