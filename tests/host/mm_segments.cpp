// The walk over experts' segments (csrc/mxq_mm_segments.h) on the CPU: one thread a lane of a
// wave, cross-lane operations by a barrier. Reads from stdin
//   rows step groups most indexes, offsets[groups + 1], index[indexes]
// and prints the number of tiles, then for each index "found expert begin count tile", then
// for each segment "first tiles" of tiles_of.
#include <pthread.h>
#include <stdint.h>
#include <stdio.h>

#include <vector>

struct Index { unsigned x; };
static thread_local Index threadIdx;
static pthread_barrier_t barrier;
static int64_t shared[64];

static int64_t from_lane(int64_t v, int lane) {
  shared[threadIdx.x] = v;
  pthread_barrier_wait(&barrier);
  const int64_t got = shared[lane & 63];
  pthread_barrier_wait(&barrier);
  return got;
}
static int __shfl_xor(int v, int d) { return (int)from_lane(v, (int)threadIdx.x ^ d); }
static int __shfl_up(int v, int d) {
  const int lane = (int)threadIdx.x;
  return (int)from_lane(v, lane >= d ? lane - d : lane);
}
static unsigned long long __ballot(bool b) {
  shared[threadIdx.x] = b;
  pthread_barrier_wait(&barrier);
  unsigned long long bits = 0;
  for (int i = 0; i < 64; ++i) bits |= (unsigned long long)shared[i] << i;
  pthread_barrier_wait(&barrier);
  return bits;
}
static int read_lane(int v, int lane) { return (int)from_lane(v, lane); }
static int read_first(int v) { return (int)from_lane(v, 0); }
#define __builtin_amdgcn_readlane read_lane
#define __builtin_amdgcn_readfirstlane read_first
#define __device__
#define __forceinline__ inline
#include "mxq_mm_segments.h"

static int64_t rows, step, groups, most, indexes;
static std::vector<int64_t> offsets, index_;

static void* lane_main(void* arg) {
  threadIdx.x = (unsigned)(intptr_t)arg;
  const bool print = threadIdx.x == 0;
  const int tiles = mxq::segment_tiles(offsets.data(), (int)groups, rows, (int)step);
  if (print) printf("%d\n", tiles);
  for (int64_t i : index_) {
    mxq::Segment s{-1, -1, -1, -1};
    const bool found = mxq::find_segment(offsets.data(), (int)groups, rows, (int)step, (int)i, s);
    if (print) printf("%d %d %lld %lld %d\n", found, s.expert, (long long)s.begin, (long long)s.count, s.tile);
  }
  for (int64_t g = 0; g < groups; g += groups > 200 ? 97 : 1) {
    int first = 0;
    const int n = mxq::tiles_of(offsets.data(), (int)g, rows, (int)step, (int)most, first);
    if (print) printf("%lld %d %d\n", (long long)g, first, n);
  }
  return nullptr;
}

int main() {
  long long v[5];
  for (long long& x : v)
    if (scanf("%lld", &x) != 1) return 2;
  rows = v[0], step = v[1], groups = v[2], most = v[3], indexes = v[4];
  for (int64_t i = 0; i < groups + 1 + indexes; ++i) {
    long long x;
    if (scanf("%lld", &x) != 1) return 2;
    (i <= groups ? offsets : index_).push_back(x);
  }
  pthread_barrier_init(&barrier, nullptr, 64);
  pthread_t t[64];
  for (intptr_t i = 0; i < 64; ++i)
    if (pthread_create(&t[i], nullptr, lane_main, (void*)i)) return 3;
  for (pthread_t& x : t) pthread_join(x, nullptr);
  return 0;
}
