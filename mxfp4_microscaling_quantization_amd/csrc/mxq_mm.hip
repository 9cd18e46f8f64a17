// Choice of the matrix product's kernel.
#include "mxq_mm_launch.h"

namespace mxq {

// Which kernel. Few rows: the weight streams past them (rows kernel; an expert's share of
// the tokens stands for its rows). With 17 to 64 rows that holds while the 128-column tiles
// are few (64 rows of n x k, rows kernel and tiles, us: 4096 x 4096 9.0 and 13.6, 14336 x 4096
// 31.7 and 16.6). Otherwise tiles, see large_tiles.
hipError_t launch_gemm(const MmLaunch& a, hipStream_t st) {
  const int64_t each = a.offsets ? (a.rows + a.groups - 1) / a.groups : a.rows;
  if (each <= 16 || (each <= 64 && a.n < 8192)) return launch_gemm_rows(a, each <= 16, st);
  const bool large = a.offsets ? large_tiles(a.rows, a.n, a.groups / 2, 1) : large_tiles(a.rows - 1, a.n, 0, 1);
  return launch_gemm_tiles(a, large, st);
}

}  // namespace mxq
