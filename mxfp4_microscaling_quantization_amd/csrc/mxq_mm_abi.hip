// C ABI of the matrix products: argument validation and dispatch to the launchers.
// Declarations and the contract of every entry point are in include/mxq_gemm.h.
#include <stdint.h>

#include "../../include/mxq_gemm.h"
#include "mxq_internal.h"
#include "mxq_mm_launch.h"

using namespace mxq;

namespace {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;  // rows and columns
constexpr int64_t kMaxK = (int64_t)1 << 22;          // tile-relative byte offsets stay within 32 bits
constexpr int64_t kMaxLd = (int64_t)1 << 23;         // the same for columns of tokens
constexpr int64_t kMaxLdScales = ((int64_t)1 << 22) - 1;  // and for their scales: 256 rows within 2^32 bytes
constexpr int64_t kMaxGrid = (int64_t)1 << 30;       // results in tiles of 32 x 32: tiles are counted in 32 bits

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

mxq_status from_hip(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_EHIP; }

bool is_dtype(mxq_dtype t) { return t == MXQ_BF16 || t == MXQ_F32; }
bool is_act(mxq_act a) { return a >= MXQ_ACT_NONE && a <= MXQ_ACT_SWIGLU; }

mxq_status gemm_impl(const uint8_t* a, const void* a_scales, mxq_operand a_fmt, const uint8_t* b,
                     const void* b_scales, mxq_operand b_fmt, int64_t rows, int64_t n, int64_t k, bool grouped,
                     const int64_t* offsets, int64_t groups, const void* bias, mxq_dtype bias_dt, mxq_act act,
                     const void* residual, void* d, mxq_dtype d_dt, void* z, void* stream) {
  if ((a_fmt != MXQ_OPERAND_MXFP4 && a_fmt != MXQ_OPERAND_FP8) ||
      (b_fmt != MXQ_OPERAND_MXFP4 && b_fmt != MXQ_OPERAND_FP8) || !is_dtype(d_dt) || !is_act(act) ||
      (bias && !is_dtype(bias_dt)))
    return MXQ_EINVAL;
  if (rows < 0 || n < 0 || k < 0) return MXQ_EINVAL;
  if (grouped && (groups < 1 || groups > 4096)) return MXQ_EINVAL;
  if (b_fmt == MXQ_OPERAND_FP8 && a_fmt != MXQ_OPERAND_FP8) return MXQ_EUNSUPPORTED;
  if (rows == 0) return MXQ_OK;
  if (!a || !a_scales || !b || !b_scales || !d || (grouped && !offsets)) return MXQ_EINVAL;
  const int64_t block = a_fmt == MXQ_OPERAND_FP8 ? 128 : 32;
  if (n == 0 || k == 0 || k % block || k > kMaxK || n > kMaxDim || rows > kMaxDim) return MXQ_ESHAPE;
  if (act == MXQ_ACT_SWIGLU && n % 2) return MXQ_ESHAPE;
  if (rows > ((int64_t)1 << 40) / n || groups * n > ((int64_t)1 << 40) / k) return MXQ_ESHAPE;
  if ((rows / 32 + groups + 1) * ((n + 31) / 32) >= kMaxGrid) return MXQ_ESHAPE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(residual, 16) || !aligned(d, 16) || !aligned(z, 16))
    return MXQ_EALIGN;
  if ((a_fmt == MXQ_OPERAND_FP8 && !aligned(a_scales, 4)) || (b_fmt == MXQ_OPERAND_FP8 && !aligned(b_scales, 4)) ||
      (bias && !aligned(bias, bias_dt == MXQ_F32 ? 4 : 2)) || (grouped && !aligned(offsets, 8)))
    return MXQ_EALIGN;
  MmLaunch l{};
  l.a = a;
  l.b = b;
  l.a_scales = a_scales;
  l.b_scales = b_scales;
  l.a_fmt = a_fmt;
  l.b_fmt = b_fmt;
  l.rows = rows;
  l.n = n;
  l.k = k;
  l.offsets = offsets;
  l.groups = (int)groups;
  l.ep.bias = bias;
  l.ep.res = residual;
  l.ep.d = d;
  l.ep.z = z;
  l.ep.n = n;
  l.ep.act = (int)act;
  l.ep.bias_f32 = bias_dt == MXQ_F32;
  l.ep.out_f32 = d_dt == MXQ_F32;
  return from_hip(launch_gemm(l, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

mxq_status mxq_gemm(const uint8_t* a, const void* a_scales, mxq_operand a_fmt, const uint8_t* b,
                    const void* b_scales, mxq_operand b_fmt, int64_t m, int64_t n, int64_t k, const void* bias,
                    mxq_dtype bias_dt, mxq_act act, const void* residual, void* d, mxq_dtype d_dt, void* z,
                    void* stream) {
  return gemm_impl(a, a_scales, a_fmt, b, b_scales, b_fmt, m, n, k, false, nullptr, 1, bias, bias_dt, act, residual,
                   d, d_dt, z, stream);
}

mxq_status mxq_grouped_gemm(const uint8_t* a, const void* a_scales, mxq_operand a_fmt, const uint8_t* b,
                            const void* b_scales, mxq_operand b_fmt, int64_t rows, int64_t n, int64_t k,
                            const int64_t* offsets, int64_t n_experts, const void* bias, mxq_dtype bias_dt,
                            mxq_act act, const void* residual, void* d, mxq_dtype d_dt, void* z, void* stream) {
  return gemm_impl(a, a_scales, a_fmt, b, b_scales, b_fmt, rows, n, k, true, offsets, n_experts, bias, bias_dt, act,
                   residual, d, d_dt, z, stream);
}

mxq_status mxq_grouped_wgrad(const uint8_t* y, const float* y_scales, int64_t ld_y, int64_t ld_ys, const uint8_t* x,
                             const float* x_scales, int64_t ld_x, int64_t ld_xs, int64_t rows, int64_t n, int64_t k,
                             const int64_t* offsets, int64_t n_experts, const void* add, void* d, mxq_dtype d_dt,
                             void* stream) {
  if (!is_dtype(d_dt) || rows < 0 || n < 0 || k < 0) return MXQ_EINVAL;
  if (n_experts < 1 || n_experts > 4096) return MXQ_EINVAL;
  if (!offsets || !d || (rows > 0 && (!y || !y_scales || !x || !x_scales))) return MXQ_EINVAL;
  if (n == 0 || k == 0 || n > kMaxDim || k > kMaxDim || rows > kMaxDim) return MXQ_ESHAPE;
  if (n > ((int64_t)1 << 40) / k || n * k > ((int64_t)1 << 40) / n_experts) return MXQ_ESHAPE;
  if (ld_y < rows || ld_x < rows || ld_y > kMaxLd || ld_x > kMaxLd) return MXQ_ESHAPE;
  if (ld_ys > kMaxLdScales || ld_xs > kMaxLdScales) return MXQ_ESHAPE;
  if (rows > 0 && (ld_ys < rc_group_slots(rows, n_experts) || ld_xs < rc_group_slots(rows, n_experts)))
    return MXQ_ESHAPE;
  if (((n + 31) / 32) * ((k + 31) / 32) >= kMaxGrid / n_experts) return MXQ_ESHAPE;
  if (ld_y % 16 || ld_x % 16 || !aligned(y, 16) || !aligned(x, 16) || !aligned(y_scales, 4) ||
      !aligned(x_scales, 4) || !aligned(offsets, 8) || !aligned(add, 16) || !aligned(d, 16))
    return MXQ_EALIGN;
  MmLaunch l{};
  l.a = y;
  l.b = x;
  l.a_scales = y_scales;
  l.b_scales = x_scales;
  l.a_fmt = l.b_fmt = 1;
  l.rows = rows;
  l.n = n;
  l.k = k;
  l.offsets = offsets;
  l.groups = (int)n_experts;
  l.ld_a = ld_y;
  l.ld_b = ld_x;
  l.ld_as = ld_ys;
  l.ld_bs = ld_xs;
  l.ep.res = add;
  l.ep.d = d;
  l.ep.n = k;
  l.ep.out_f32 = d_dt == MXQ_F32;
  return from_hip(launch_grouped_wgrad(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_act_grad(const void* dy, const void* z, mxq_dtype dt, int64_t rows, int64_t n, mxq_act act,
                        const int64_t* offsets, int64_t n_experts, void* dz, float* db, void* workspace,
                        void* stream) {
  if (!is_dtype(dt) || !is_act(act) || rows < 0 || n < 0) return MXQ_EINVAL;
  if (offsets ? (n_experts < 1 || n_experts > 4096) : n_experts != 1) return MXQ_EINVAL;
  if (rows == 0 && !db) return MXQ_OK;
  if (rows > 0 && (!dy || !z || !dz || (db && !workspace))) return MXQ_EINVAL;
  if (n == 0 || n > kMaxDim || rows > kMaxDim || rows > ((int64_t)1 << 40) / n) return MXQ_ESHAPE;
  if (act == MXQ_ACT_SWIGLU && n % 2) return MXQ_ESHAPE;
  // the grids enumerate row blocks x column tiles and groups x column tiles
  if (act_grad_blocks(rows, n_experts, act_grad_rows(rows, n)) * ((n + 511) / 512) >= kMaxGrid / 64 ||
      n_experts * ((n + 63) / 64) >= kMaxGrid / 256)
    return MXQ_ESHAPE;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16) || !aligned(db, 16) || !aligned(workspace, 16) ||
      !aligned(offsets, 8))
    return MXQ_EALIGN;
  ActGradLaunch l{};
  l.dy = dy;
  l.z = z;
  l.f32 = dt == MXQ_F32;
  l.rows = rows;
  l.n = n;
  l.act = (int)act;
  l.offsets = offsets;
  l.groups = (int)n_experts;
  l.dz = dz;
  l.db = db;
  l.partials = static_cast<float*>(workspace);
  l.block_rows = act_grad_rows(rows, n);
  return from_hip(launch_act_grad(l, reinterpret_cast<hipStream_t>(stream)));
}

int64_t mxq_act_grad_workspace(int64_t rows, int64_t n, int64_t n_experts) {
  if (rows <= 0 || n <= 0 || n_experts < 1 || rows > kMaxDim || n > kMaxDim || n_experts > 4096) return 0;
  return act_grad_blocks(rows, n_experts, act_grad_rows(rows, n)) * n * 4;
}

}  // extern "C"
