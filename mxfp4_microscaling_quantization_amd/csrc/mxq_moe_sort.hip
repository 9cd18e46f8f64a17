// The rows of every expert: a stable counting sort of the assignments by expert.
//
// Launches joined by a table of counts [blocks, experts]: every block counts the experts of its
// assignments; every block numbers its assignments from the sums of the counts. The sums are
// formed by each block for itself while the table is small, else by a launch between, in which a
// thread per expert turns a part of its column into sums over the blocks before and leaves the
// total. Up to kSortOne assignments a single workgroup does all of it.
//
// Numbers inside a block: a wave owns a contiguous part, with a counter per expert in LDS that
// starts at the expert's rows before that part. Of 64 assignments at a time, each finds the
// lanes with its own expert (one ballot per bit of the expert), takes the counter plus the
// number of such lanes below itself, and the last of them moves the counter on. No order
// depends on timing: the only atomics add whole numbers.
//
// 524288 assignments to 256 experts move 6.3 MB and take 14.1 us, in a kernel trace 3.5 the counting and 11.6
// the numbering (three launches with a quarter of the loads in flight and half of the waves took 23). What
// the numbering does first is wait: each of its 256 workgroups reads the whole table, 64 MiB of L2 reads in
// all, 64 loads of a thread in four batches, and then, behind a barrier, its assignments, of which two of a
// lane's four turns are empty. To 4096 experts it takes 56 us, 47 of them numbering with two waves of a
// workgroup for 4096 counters each.
#include "mxq_moe.h"

namespace mxq {

namespace {

constexpr int kTurns = 4;           // assignments of a lane in flight
constexpr int kStep = 64 * kTurns;  // of a wave

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// table[0..n) becomes its exclusive sums; returns the total. One wave: a lane has n / 64 neighbouring
// entries.
__device__ __forceinline__ int scan_table(int* table, int n) {
  const int each = (n + 63) / 64, first = lane_id() * each, last = first + each < n ? first + each : n;
  int sum = 0;
  for (int e = first; e < last; ++e) sum += table[e];
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(inc, d);
    if (lane_id() >= d) inc += up;
  }
  int before = inc - sum;
  for (int e = first; e < last; ++e) {
    const int c = table[e];
    table[e] = before;
    before += c;
  }
  return __builtin_amdgcn_readlane(inc, 63);
}

// The experts of kStep assignments from i0 on; behind `end` and where there is none: n.
__device__ __forceinline__ void fetch(const SortLaunch& p, int64_t i0, int64_t end, int (&e)[kTurns]) {
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int64_t i = i0 + t * 64 + lane_id();
    e[t] = i < end ? p.experts[i] : -1;
  }
#pragma unroll
  for (int t = 0; t < kTurns; ++t) e[t] = (uint32_t)e[t] < (uint32_t)p.n_experts ? e[t] : p.n_experts;
}

__device__ __forceinline__ void count(const SortLaunch& p, const int (&e)[kTurns], int* counter) {
#pragma unroll
  for (int t = 0; t < kTurns; ++t)
    if (e[t] < p.n_experts) atomicAdd(&counter[e[t]], 1);
}

// counter[e]: the row of the next assignment of expert e.
__device__ __forceinline__ void number(const SortLaunch& p, int64_t i0, int64_t end, const int (&e)[kTurns],
                                       int* counter, int bits) {
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int64_t i = i0 + t * 64 + lane_id();
    const bool has = e[t] < p.n_experts;
    unsigned long long same = __ballot(has);
    if (!same && i0 + t * 64 >= end) break;
    for (int b = 0; b < bits; ++b) {
      const bool on = (e[t] >> b) & 1;
      const unsigned long long one = __ballot(on);
      same &= on ? one : ~one;
    }
    int row = -1;
    if (has) {
      const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
      row = counter[e[t]] + below;
      if (same >> lane_id() == 1ull) counter[e[t]] = row + 1;  // the last lane of this expert
      p.order[row] = (int)i;
    }
    if (i < end) p.positions[i] = row;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the counters, for the next 64
  }
}

// One block's assignments [first, last) by W waves. lds: counters [W][n]. A wave's part is whole 64s.
template <int W>
struct Block {
  int64_t begin, end;
  int e[kTurns];
  int* counter;

  __device__ __forceinline__ void count_all(const SortLaunch& p, int64_t first, int64_t last, int* lds) {
    const int wave = threadIdx.x >> 6;
    const int64_t each = ((last - first + W - 1) / W + 63) & ~(int64_t)63;
    begin = first + wave * each < last ? first + wave * each : last;
    end = begin + each < last ? begin + each : last;
    counter = lds + wave * p.n_experts;
    fetch(p, begin, end, e);
    for (int i = threadIdx.x; i < W * p.n_experts; i += 64 * W) lds[i] = 0;
    __syncthreads();
    count(p, e, counter);
    for (int64_t i = begin + kStep; i < end; i += kStep) {
      int more[kTurns];
      fetch(p, i, end, more);
      count(p, more, counter);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void number_all(const SortLaunch& p) {
    const int bits = 32 - __clz(p.n_experts - 1 | 1);
    number(p, begin, end, e, counter, bits);
    for (int64_t i = begin + kStep; i < end; i += kStep) {
      int more[kTurns];
      fetch(p, i, end, more);
      number(p, i, end, more, counter, bits);
    }
  }
};

// The waves' counts of expert e become its rows before each wave's part, from `row` on.
template <int W>
__device__ __forceinline__ void start_counters(int* lds, int n, int e, int row) {
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int c = lds[w * n + e];
    lds[w * n + e] = row;
    row += c;
  }
}

// The rows without an assignment among rows [first, last).
__device__ __forceinline__ void no_rows(const SortLaunch& p, int64_t first, int64_t last, int64_t used) {
  if (first < used) first = used;
  for (int64_t i = first + threadIdx.x; i < last; i += blockDim.x) p.order[i] = -1;
}

template <int W>
__global__ __launch_bounds__(64 * W) void sort_one_kernel(SortLaunch p) {
  extern __shared__ int lds[];  // counters [W][n_experts], table [n_experts + 1]
  const int n = p.n_experts;
  int* table = lds + W * n;
  Block<W> b;
  b.count_all(p, 0, p.count, lds);
  for (int e = threadIdx.x; e < n; e += 64 * W) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += lds[w * n + e];
    table[e] = sum;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int total = scan_table(table, n);
    if (lane_id() == 0) table[n] = total;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= n; e += 64 * W) {
    p.offsets[e] = table[e];
    if (e < n) start_counters<W>(lds, n, e, table[e]);
  }
  const int used = table[n];
  __syncthreads();
  b.number_all(p);
  no_rows(p, 0, p.count, used);
}

constexpr int kCountThreads = 256;
__global__ __launch_bounds__(kCountThreads) void sort_count_kernel(SortLaunch p, int64_t chunk) {
  extern __shared__ int lds[];
  const int n = p.n_experts, wave = threadIdx.x >> 6;
  const int64_t first = blockIdx.x * chunk, last = first + chunk < p.count ? first + chunk : p.count;
  int e[kTurns];
  fetch(p, first + wave * kStep, last, e);
  for (int i = threadIdx.x; i < n; i += kCountThreads) lds[i] = 0;
  __syncthreads();
  count(p, e, lds);
  for (int64_t i = first + wave * kStep + kCountThreads * kTurns; i < last; i += kCountThreads * kTurns) {
    fetch(p, i, last, e);
    count(p, e, lds);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kCountThreads) p.counts[(int64_t)blockIdx.x * n + i] = lds[i];
}

// Column e of the counts becomes the sums over the blocks before; row `blocks` the totals. A
// workgroup has 64 experts, its waves a run of blocks each, of which kHeld stay in registers.
constexpr int kScanWaves = 16, kHeld = 16;
__global__ __launch_bounds__(64 * kScanWaves) void sort_scan_kernel(SortLaunch p, int blocks) {
  __shared__ int part[kScanWaves][64];
  const int n = p.n_experts, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane_id();
  const int each = (blocks + kScanWaves - 1) / kScanWaves;
  const int first = wave * each;
  const int last = e >= n ? first : first + each < blocks ? first + each : blocks;  // (no blocks behind the last expert)
  int* column = p.counts + e;
  int held[kHeld], sum = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = first + i < last ? column[(int64_t)(first + i) * n] : 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) sum += held[i];
#pragma unroll 8
  for (int b = first + kHeld; b < last; ++b) sum += column[(int64_t)b * n];
  part[wave][lane_id()] = sum;
  __syncthreads();
  if (e >= n) return;
  int before = 0;
#pragma unroll
  for (int w = 0; w < kScanWaves; ++w) before += w < wave ? part[w][lane_id()] : 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (first + i < last) column[(int64_t)(first + i) * n] = before;
    before += held[i];
  }
#pragma unroll 8
  for (int b = first + kHeld; b < last; ++b) {
    const int c = column[(int64_t)b * n];
    column[(int64_t)b * n] = before;
    before += c;
  }
  if (wave == kScanWaves - 1) column[(int64_t)blocks * n] = before;
}

// What a block needs of the counts: table[e], all assignments of expert e, and base[e], those of the
// blocks before it, summed up by the block itself. The threads share out the rows of every expert.
template <int THREADS>
__device__ __forceinline__ void sum_counts(const SortLaunch& p, int blocks, int* table, int* base) {
  const int n = p.n_experts, parts = THREADS / n, part = threadIdx.x / n, e = threadIdx.x % n;
  for (int i = threadIdx.x; i < 2 * n; i += THREADS) table[i] = 0;  // (base lies behind table)
  __syncthreads();
  if (part < parts) {
    const int each = (blocks + parts - 1) / parts, first = part * each;
    const int last = first + each < blocks ? first + each : blocks;
    int all = 0, before = 0;
#pragma unroll 16
    for (int b = first; b < last; ++b) {
      const int c = p.counts[(int64_t)b * n + e];
      all += c;
      before += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&table[e], all);
    atomicAdd(&base[e], before);
  }
}

// SUM: the counts are as sort_count_kernel left them; otherwise as sort_scan_kernel did.
template <int W, bool SUM>
__global__ __launch_bounds__(64 * W) void sort_number_kernel(SortLaunch p, int64_t chunk, int blocks) {
  extern __shared__ int lds[];  // counters [W][n_experts], SUM: table and base [n_experts] each, else table [n_experts]
  __shared__ int rows;
  const int n = p.n_experts;
  int* table = lds + W * n;
  const int* mine = p.counts + (int64_t)blockIdx.x * n;
  int held = 0;
  if constexpr (SUM) {
    sum_counts<64 * W>(p, blocks, table, table + n);
  } else {
    held = threadIdx.x < n ? mine[threadIdx.x] : 0;  // (asked for early: most calls have no more experts than threads)
    for (int i = threadIdx.x; i < n; i += 64 * W) table[i] = p.counts[(int64_t)blocks * n + i];
  }
  const int64_t first = blockIdx.x * chunk, last = first + chunk < p.count ? first + chunk : p.count;
  Block<W> b;
  b.count_all(p, first, last, lds);
  if (threadIdx.x < 64) {
    const int total = scan_table(table, n);
    if (lane_id() == 0) rows = total;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += 64 * W) {
    if (blockIdx.x == 0) p.offsets[e] = table[e];
    start_counters<W>(lds, n, e, table[e] + (SUM ? table[n + e] : e < 64 * W ? held : mine[e]));
  }
  const int used = rows;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[n] = used;
  __syncthreads();
  b.number_all(p);
  no_rows(p, first, last, used);
}

}  // namespace

hipError_t launch_expert_sort(const SortLaunch& a, hipStream_t st) {
  if (a.count <= kSortOne) {
    // (the counters of the waves, and the table, within 64 KiB of LDS)
    if (a.n_experts <= 512)
      sort_one_kernel<16><<<1, 1024, (17 * a.n_experts + 1) * 4, st>>>(a);
    else
      sort_one_kernel<2><<<1, 128, (3 * a.n_experts + 1) * 4, st>>>(a);
    return hipGetLastError();
  }
  const int64_t chunk = sort_chunk(a.count);
  const int blocks = (int)sort_blocks(a.count);
  sort_count_kernel<<<blocks, kCountThreads, a.n_experts * 4, st>>>(a, chunk);
  if (sort_in_two(a.count, a.n_experts)) {
    sort_number_kernel<16, true><<<blocks, 1024, 18 * a.n_experts * 4, st>>>(a, chunk, blocks);
    return hipGetLastError();
  }
  sort_scan_kernel<<<(a.n_experts + 63) / 64, 64 * kScanWaves, 0, st>>>(a, blocks);
  if (a.n_experts <= 1024)
    sort_number_kernel<8, false><<<blocks, 512, 9 * a.n_experts * 4, st>>>(a, chunk, blocks);
  else
    sort_number_kernel<2, false><<<blocks, 128, 3 * a.n_experts * 4, st>>>(a, chunk, blocks);
  return hipGetLastError();
}

}  // namespace mxq
