// Choice of the matrix product's kernel.
#include "mxq_mm_launch.h"

namespace mxq {

// Which kernel. Few rows: the weight streams past them (rows kernel; an expert's share of
// the tokens stands for its rows). With 17 to 64 rows that holds while its workgroups of
// 32 x 32 results all run at once, one on each of the 256 CUs (MXFP4, k 4096, rows kernel and
// tiles, us: 64 x 4096 results 8.8 and 10.4, 64 x 6144 16.2 and 10.7, 32 x 8192 9.2 and 10.8),
// but not for FP8 products that may take the FP8 matrix instructions, which the rows kernel
// does without (64 x 4096: 16.2 and 11.8), and not for experts, whose rows are uneven (8
// experts, 384 tokens, 4096 x 4096: 62.6 and 19.7); for these tiles come in from 13 rows on
// average (64 experts of 4096 x 4096 with 8 uneven rows 127 and 106, with 16 177 and 123; of
// 2048 x 1024 with 8 19 and 30, with 16 25 and 30), from 17 where the tiles' product is the
// slower exact one (with 16: 272 and 301). The rows kernel has a workgroup for every
// tile; past what one launch can hold, the tiled kernel's workgroups walk over theirs.
hipError_t launch_gemm(const MmLaunch& a, hipStream_t st) {
  const int64_t each = a.offsets ? (a.rows + a.groups - 1) / a.groups : a.rows;
  const bool at_once = (a.rows + 31) / 32 * ((a.n + 31) / 32) <= 256;
  const bool exact = a.a_fmt && a.ep.out_f32, fp8 = a.a_fmt && a.b_fmt && !exact;
  const int64_t grid = (a.rows / 16 + (a.rows < a.groups ? a.rows : a.groups)) * ((a.n + 15) / 16);
  const bool few = each <= (a.offsets && !exact ? 12 : 16) && grid < 1 << 21;
  if (few || (each <= 64 && !a.offsets && at_once && !fp8)) return launch_gemm_rows(a, few, st);
  const int side = a.offsets ? tile_side(a.rows, a.n, a.groups, 1) : tile_side(a.rows - 1, a.n, 0, 1);
  return launch_gemm_tiles(a, side, st);
}

}  // namespace mxq
