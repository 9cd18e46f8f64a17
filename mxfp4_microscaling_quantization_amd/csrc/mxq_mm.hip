// Choice of the matrix product's kernel.
#include "mxq_mm_launch.h"

namespace mxq {

// Which kernel. Few rows: the weight streams past them (rows kernel; an expert's share of
// the tokens stands for its rows). With 17 to 64 rows that holds while the 128-column tiles
// are few (64 rows of n x k, rows kernel and tiles, us: 4096 x 4096 9.0 and 13.6, 14336 x 4096
// 31.7 and 16.6). Otherwise tiles of 256 x 256 or 128 x 128: a large one takes about 2.2 times
// a small one's time for four times its results, and 256 run at once (MXFP4, k 4096, large
// and small, us: 1024 x 4096 results 32.0 and 17.9, 2048 x 4096 33.3 and 31.5, 4096 x 4096
// 40.0 and 58.2).
hipError_t launch_gemm(const MmLaunch& a, hipStream_t st) {
  const int64_t each = a.offsets ? (a.rows + a.groups - 1) / a.groups : a.rows;
  if (each <= 16 || (each <= 64 && a.n < 8192)) return launch_gemm_rows(a, each <= 16, st);
  auto rounds = [&](int64_t side) {
    const int64_t rows = a.offsets ? a.rows / side + a.groups / 2 + 1 : (a.rows + side - 1) / side;
    return (rows * ((a.n + side - 1) / side) + 255) / 256;
  };
  return launch_gemm_tiles(a, 22 * rounds(256) <= 10 * rounds(128), st);
}

}  // namespace mxq
