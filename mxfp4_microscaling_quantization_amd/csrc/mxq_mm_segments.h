// The walk over experts' token segments. Expert e owns rows [offsets[e], offsets[e + 1]),
// clamped to [0, rows]. Offsets come from the device and may be malformed (segments that
// overlap, thousands of times over): sums of tiles saturate, so that no number formed
// from them leaves its range, and every tile lies inside its own expert's rows.
#pragma once

#include <stdint.h>

namespace mxq {

struct Segment {
  int expert;
  int64_t begin;  // first row of the expert
  int64_t count;  // its rows
  int tile;       // which of the expert's tiles
};

// Well-formed offsets give fewer than 2^31 / 16 + 4096 tiles. Two saturated sums add up within 32 bits.
constexpr int kMostTiles = (1 << 30) - 1;

// Tiles that any split of the rows into groups has at most.
constexpr int64_t most_tiles(int64_t rows, int64_t groups, int64_t step) {
  return rows / step + (rows < groups ? rows : groups);
}

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t rows) {
  return v < 0 ? 0 : v > rows ? rows : v;
}

__device__ __forceinline__ int add_tiles(int a, int b) {
  const int sum = a + b;
  return sum < kMostTiles ? sum : kMostTiles;
}

// Tiles of `step` rows over all segments, in expert order: their number.
__device__ __forceinline__ int segment_tiles(const int64_t* offsets, int experts, int64_t rows, int step) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  for (int e = lane; e < experts; e += 64) {
    const int64_t c = clamp_row(offsets[e + 1], rows) - clamp_row(offsets[e], rows);
    sum = add_tiles(sum, c > 0 ? (int)((c + step - 1) / step) : 0);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum = add_tiles(sum, __shfl_xor(sum, d));
  return __builtin_amdgcn_readfirstlane(sum);
}

// The segment that holds tile `index` (below kMostTiles); false past the last one. Every wave
// of a workgroup finds it for itself: 64 experts a turn, an inclusive scan over the lanes.
__device__ __forceinline__ bool find_segment(const int64_t* offsets, int experts, int64_t rows, int step, int index,
                                             Segment& s) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int64_t begin = 0, count = 0;
    if (e < experts) {
      begin = clamp_row(offsets[e], rows);
      count = clamp_row(offsets[e + 1], rows) - begin;
      if (count < 0) count = 0;
    }
    int inc = (int)((count + step - 1) / step);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(inc, d);
      if (lane >= d) inc = add_tiles(inc, up);
    }
    const unsigned long long past = __ballot(inc > index - before);
    if (past) {
      const int at = __builtin_ctzll(past);
      s.expert = e0 + at;
      // rows < 2^31
      s.begin = (uint32_t)__builtin_amdgcn_readlane((int)begin, at);
      s.count = (uint32_t)__builtin_amdgcn_readlane((int)count, at);
      // (the sums up to the expert before are at most `index`, so not saturated)
      s.tile = index - before - (at ? __builtin_amdgcn_readlane(inc, at - 1) : 0);
      return true;
    }
    before = add_tiles(before, __builtin_amdgcn_readlane(inc, 63));
  }
  return false;
}

// The tiles of segment g, [first, first + the result) of the first `most`: all of them for
// well-formed offsets.
__device__ __forceinline__ int tiles_of(const int64_t* offsets, int g, int64_t rows, int step, int most, int& first) {
  first = segment_tiles(offsets, g, rows, step);
  const int64_t c = clamp_row(offsets[g + 1], rows) - clamp_row(offsets[g], rows);
  const int tiles = c > 0 ? (int)((c + step - 1) / step) : 0;
  return first >= most ? 0 : tiles < most - first ? tiles : most - first;
}

}  // namespace mxq
