// Rows in FP8: E4M3 with a power-of-two scale for each 128 columns.
#include <algorithm>

#include "mxq_internal.h"
#include "mxq_moe_fp8.h"

namespace mxq {

namespace {

constexpr int kThreads = 256, kUnroll = 4;
constexpr uint32_t kChunks = kThreads * kUnroll;

struct Fp8Params {
  const void* x;
  int64_t ldx, cols;
  uint32_t chunks;  // of 8 elements; rows are counted as whole groups
  FastDiv cpr;      // chunks of a row
  uint8_t* q8;
  float* scales;
};

// A thread takes chunks base + 256 j, so a wave's loads and stores are contiguous and a group is 16
// neighbouring lanes. VEC: rows of x start on 16 bytes and cols is a multiple of 8; otherwise rows start
// anywhere (the memory system takes such accesses), and a row's last elements go one by one. Bound by
// memory: 65536 x 4096 bf16, 0.81 GB, 127 us, 6.4 TB/s (codes through the caches 136, 16 elements of a
// thread 133); 16384 x 4098 39 us, by elements 117.
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(Fp8Params p) {
  const uint32_t base = blockIdx.x * kChunks + threadIdx.x;
  const T* x = static_cast<const T*>(p.x);
  Raw<T> raw[kUnroll];
  int64_t row[kUnroll];
  int col[kUnroll], left[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t c = base + u * kThreads;
    const uint32_t r = fdiv(c, p.cpr);
    row[u] = r;
    col[u] = (int)(c - r * p.cpr.d) * 8;
    left[u] = c < p.chunks ? (int)p.cols - col[u] : 0;
    zero_raw(raw[u]);
    const size_t off = (size_t)(row[u] * p.ldx + col[u]);
    if constexpr (VEC) {
      if (left[u] > 0) load_raw(x, off, raw[u]);
    } else if (left[u] >= 8) {
      __builtin_memcpy(&raw[u], x + off, 8 * sizeof(T));
    } else {
      T t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = i < left[u] ? x[off + i] : (T)0;
      __builtin_memcpy(&raw[u], t, sizeof(t));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float v[8];
    uint32_t q[2], scale;
    to_f32(raw[u], v);
    fp8_encode<8, 16>(v, q, scale);
    uint8_t* to = p.q8 + row[u] * p.cols + col[u];
    if constexpr (VEC) {
      if (left[u] > 0) store_nt(reinterpret_cast<uint2*>(to), make_uint2(q[0], q[1]));
    } else if (left[u] >= 8) {
      store_any<8>(to, q);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left[u]) to[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
    }
    if (left[u] > 0 && col[u] % 128 == 0) p.scales[row[u] * (p.cpr.d / 16) + col[u] / 128] = as_f(scale);
  }
}

template <typename T>
hipError_t launch_t(const void* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q8, float* scales,
                    hipStream_t st) {
  const int64_t groups = (cols + 127) / 128, cpr = groups * 16;
  const bool vec = ((uintptr_t)x & 15) == 0 && ldx * (int64_t)sizeof(T) % 16 == 0 && cols % 8 == 0;
  const int64_t max_rows = std::max<int64_t>(1, ((int64_t)1 << 29) / cpr);
  for (int64_t r0 = 0; r0 < rows; r0 += max_rows) {
    const int64_t nr = std::min(max_rows, rows - r0);
    Fp8Params p;
    p.x = static_cast<const T*>(x) + r0 * ldx;
    p.ldx = ldx;
    p.cols = cols;
    p.chunks = (uint32_t)(nr * cpr);
    const FastDivHost fd = make_fastdiv((uint32_t)cpr);
    p.cpr = FastDiv{fd.d, fd.m, fd.s};
    p.q8 = q8 + r0 * cols;
    p.scales = scales + r0 * groups;
    const dim3 grid((p.chunks + kChunks - 1) / kChunks);
    if (vec) fp8_rows_kernel<T, true><<<grid, kThreads, 0, st>>>(p);
    else fp8_rows_kernel<T, false><<<grid, kThreads, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int f32, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q8,
                               float* scales, hipStream_t st) {
  return f32 ? launch_t<float>(x, rows, cols, ldx, q8, scales, st)
             : launch_t<uint16_t>(x, rows, cols, ldx, q8, scales, st);
}

}  // namespace mxq
