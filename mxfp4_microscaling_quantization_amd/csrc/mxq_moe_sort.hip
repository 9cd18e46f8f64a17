// The rows of every expert: a stable counting sort of the assignments by expert.
//
// Three launches, joined by a table of counts [blocks, experts]: every block counts the
// experts of its assignments; one thread per expert turns its column into sums over the
// blocks before and leaves the total; every block then numbers its assignments. Up to kSortOne
// assignments a single workgroup does all of it.
//
// Numbers inside a block: a wave owns a contiguous part, with a counter per expert in LDS that
// starts at the expert's rows before that part. Of 64 assignments at a time, each finds the
// lanes with its own expert (one ballot per bit of the expert), takes the counter plus the
// number of such lanes below itself, and the last of them moves the counter on. No order
// depends on timing: the only atomics add whole numbers.
#include "mxq_moe.h"

namespace mxq {

namespace {

constexpr int kBlock = 256, kWaves = kBlock / 64;

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Exclusive sum over the lanes of a wave; total: over all of them.
__device__ __forceinline__ int wave_scan(int v, int& total) {
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(inc, d);
    if (lane_id() >= d) inc += up;
  }
  total = __builtin_amdgcn_readlane(inc, 63);
  return inc - v;
}

// One wave: table[0..n) becomes its exclusive sums; returns the total.
__device__ __forceinline__ int scan_table(int* table, int n) {
  int before = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int e = e0 + lane_id();
    int total;
    const int x = wave_scan(e < n ? table[e] : 0, total);
    if (e < n) table[e] = before + x;
    before += total;
  }
  return before;
}

// The part [begin, end) of wave w of W in the block's assignments [first, last), in whole 64.
struct Part {
  int64_t begin, end;
};
template <int W>
__device__ __forceinline__ Part wave_part(int64_t first, int64_t last, int w) {
  const int64_t each = ((last - first + W - 1) / W + 63) & ~(int64_t)63;
  const int64_t b = first + w * each, e = b + each;
  return Part{b < last ? b : last, e < last ? e : last};
}

__device__ __forceinline__ void count_part(const SortLaunch& p, Part part, int* counter) {
  for (int64_t i = part.begin + lane_id(); i < part.end; i += 64) {
    const uint32_t e = (uint32_t)p.experts[i];
    if (e < (uint32_t)p.n_experts) atomicAdd(&counter[e], 1);
  }
}

// counter[e]: the row of the part's next assignment of expert e.
__device__ __forceinline__ void number_part(const SortLaunch& p, Part part, int* counter, int bits) {
  for (int64_t i0 = part.begin; i0 < part.end; i0 += 64) {
    const int64_t i = i0 + lane_id();
    const uint32_t e = i < part.end ? (uint32_t)p.experts[i] : 0xFFFFFFFFu;
    const bool has = e < (uint32_t)p.n_experts;
    unsigned long long same = __ballot(has);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long one = __ballot((e >> b) & 1u);
      same &= (e >> b) & 1u ? one : ~one;
    }
    int row = -1;
    if (has) {
      const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
      const int base = counter[e];
      row = base + below;
      if (same >> lane_id() == 1ull) counter[e] = row + 1;  // the last lane of this expert
      p.order[row] = (int)i;
    }
    if (i < part.end) p.positions[i] = row;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the counters, for the next 64
  }
}

__device__ __forceinline__ int bits_of(int n_experts) { return 32 - __clz(n_experts - 1 | 1); }

// The rows without an assignment among rows [first, last).
__device__ __forceinline__ void no_rows(const SortLaunch& p, int64_t first, int64_t last, int64_t used) {
  if (first < used) first = used;
  for (int64_t i = first + threadIdx.x; i < last; i += blockDim.x) p.order[i] = -1;
}

template <int W>
__global__ __launch_bounds__(64 * W) void sort_one_kernel(SortLaunch p) {
  extern __shared__ int lds[];  // counters [W][n_experts], table [n_experts + 1]
  const int n = p.n_experts, wave = threadIdx.x >> 6;
  int* table = lds + W * n;
  for (int i = threadIdx.x; i < W * n; i += 64 * W) lds[i] = 0;
  __syncthreads();
  const Part part = wave_part<W>(0, p.count, wave);
  count_part(p, part, lds + wave * n);
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += 64 * W) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += lds[w * n + e];
    table[e] = sum;
  }
  __syncthreads();
  if (wave == 0) {
    const int total = scan_table(table, n);
    if (lane_id() == 0) table[n] = total;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= n; e += 64 * W) {
    int sum = table[e];
    p.offsets[e] = sum;
    if (e < n) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int c = lds[w * n + e];
        lds[w * n + e] = sum;
        sum += c;
      }
    }
  }
  const int used = table[n];
  __syncthreads();
  number_part(p, part, lds + wave * n, bits_of(n));
  no_rows(p, 0, p.count, used);
}

__global__ __launch_bounds__(kBlock) void sort_count_kernel(SortLaunch p, int64_t chunk) {
  extern __shared__ int lds[];
  const int n = p.n_experts;
  for (int i = threadIdx.x; i < n; i += kBlock) lds[i] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = first + chunk < p.count ? first + chunk : p.count;
  for (int64_t i = first + threadIdx.x; i < last; i += kBlock) {
    const uint32_t e = (uint32_t)p.experts[i];
    if (e < (uint32_t)n) atomicAdd(&lds[e], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBlock) p.counts[(int64_t)blockIdx.x * n + i] = lds[i];
}

// Column e of the counts becomes the sums over the blocks before; row `blocks` the totals. 64
// experts of a workgroup, whose waves take the blocks in kWaves runs.
__global__ __launch_bounds__(kBlock) void sort_scan_kernel(SortLaunch p, int blocks) {
  __shared__ int part[kWaves][64];
  const int n = p.n_experts, wave = threadIdx.x >> 6, e = blockIdx.x * 64 + lane_id();
  const int each = (blocks + kWaves - 1) / kWaves;
  const int first = wave * each, last = first + each < blocks ? first + each : blocks;
  int sum = 0;
  if (e < n) {
#pragma unroll 8
    for (int b = first; b < last; ++b) sum += p.counts[(int64_t)b * n + e];
  }
  part[wave][lane_id()] = sum;
  __syncthreads();
  if (e >= n) return;
  int before = 0;
  for (int w = 0; w < wave; ++w) before += part[w][lane_id()];
#pragma unroll 8
  for (int b = first; b < last; ++b) {
    const int c = p.counts[(int64_t)b * n + e];
    p.counts[(int64_t)b * n + e] = before;
    before += c;
  }
  if (wave == kWaves - 1) p.counts[(int64_t)blocks * n + e] = before;
}

template <int W>
__global__ __launch_bounds__(64 * W) void sort_number_kernel(SortLaunch p, int64_t chunk, int blocks) {
  extern __shared__ int lds[];  // counters [W][n_experts], table [n_experts + 1]
  const int n = p.n_experts, wave = threadIdx.x >> 6;
  int* table = lds + W * n;
  for (int i = threadIdx.x; i < W * n; i += 64 * W) lds[i] = 0;
  for (int i = threadIdx.x; i < n; i += 64 * W) table[i] = p.counts[(int64_t)blocks * n + i];
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, last = first + chunk < p.count ? first + chunk : p.count;
  const Part part = wave_part<W>(first, last, wave);
  count_part(p, part, lds + wave * n);
  if (wave == 0) {
    const int total = scan_table(table, n);
    if (lane_id() == 0) table[n] = total;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= n; e += 64 * W) {
    if (blockIdx.x == 0) p.offsets[e] = table[e];
    if (e < n) {
      int sum = table[e] + p.counts[(int64_t)blockIdx.x * n + e];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int c = lds[w * n + e];
        lds[w * n + e] = sum;
        sum += c;
      }
    }
  }
  __syncthreads();
  number_part(p, part, lds + wave * n, bits_of(n));
  no_rows(p, first, last, table[n]);
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
  const int blocks = (int)((a.count + chunk - 1) / chunk);
  sort_count_kernel<<<blocks, kBlock, a.n_experts * 4, st>>>(a, chunk);
  sort_scan_kernel<<<(a.n_experts + 63) / 64, kBlock, 0, st>>>(a, blocks);
  if (a.n_experts <= 2048)
    sort_number_kernel<4><<<blocks, 256, (5 * a.n_experts + 1) * 4, st>>>(a, chunk, blocks);
  else
    sort_number_kernel<2><<<blocks, 128, (3 * a.n_experts + 1) * 4, st>>>(a, chunk, blocks);
  return hipGetLastError();
}

}  // namespace mxq
