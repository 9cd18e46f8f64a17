// C ABI of the operators around the experts' products: argument validation and dispatch to
// the launchers. Declarations and the contract of every entry point are in include/mxq_moe.h.
#include <stdint.h>

#include "../../include/mxq_moe.h"
#include "mxq_mm_launch.h"
#include "mxq_moe_launch.h"

using namespace mxq;

namespace {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;  // tokens, rows, assignments
constexpr int64_t kMaxWidth = (int64_t)1 << 22;      // column offsets stay within 32 bits
constexpr int64_t kMaxExperts = 4096, kMaxTopK = 64;
constexpr int64_t kMaxGrid = (int64_t)1 << 30;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
mxq_status from_hip(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_EHIP; }
bool is_dtype(mxq_dtype t) { return t == MXQ_BF16 || t == MXQ_F32; }
int64_t size_of(mxq_dtype t) { return t == MXQ_F32 ? 4 : 2; }

// Tokens, their choices and the rows of width `width`: what dispatch and combine share.
mxq_status check_rows(int64_t tokens, int64_t top_k, int64_t rows, int64_t width) {
  if (tokens < 0 || rows < 0 || width < 0) return MXQ_EINVAL;
  if (top_k < 1 || top_k > kMaxTopK) return MXQ_EINVAL;
  if (tokens > kMaxDim / top_k || rows > kMaxDim || width == 0 || width > kMaxWidth) return MXQ_ESHAPE;
  if (tokens > ((int64_t)1 << 40) / width || rows > ((int64_t)1 << 40) / width) return MXQ_ESHAPE;
  return MXQ_OK;
}

}  // namespace

extern "C" {

mxq_status mxq_route(const void* logits, mxq_dtype dt, int64_t tokens, int64_t n_experts, int64_t ld, int64_t top_k,
                     int renorm, float* weights, int32_t* experts, void* stream) {
  if (!is_dtype(dt) || tokens < 0 || (renorm != 0 && renorm != 1)) return MXQ_EINVAL;
  if (n_experts < 1 || n_experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > n_experts)
    return MXQ_EINVAL;
  if (tokens == 0) return MXQ_OK;
  if (!logits || !weights || !experts) return MXQ_EINVAL;
  if (ld < n_experts || tokens > kMaxDim / top_k || tokens > ((int64_t)1 << 40) / ld) return MXQ_ESHAPE;
  if (!aligned(logits, size_of(dt)) || !aligned(weights, 4) || !aligned(experts, 4)) return MXQ_EALIGN;
  RouteLaunch l{};
  l.logits = logits;
  l.f32 = dt == MXQ_F32;
  l.tokens = tokens;
  l.ld = ld;
  l.experts = (int)n_experts;
  l.top_k = (int)top_k;
  l.renorm = renorm;
  l.weights = weights;
  l.chosen = experts;
  return from_hip(launch_route(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_route_grad(const float* dw, const float* weights, const int32_t* experts, const void* logits,
                          mxq_dtype dt, int64_t tokens, int64_t n_experts, int64_t ld, int64_t top_k, int renorm,
                          void* dlogits, void* stream) {
  if (!is_dtype(dt) || tokens < 0 || (renorm != 0 && renorm != 1)) return MXQ_EINVAL;
  if (n_experts < 1 || n_experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > n_experts)
    return MXQ_EINVAL;
  if (tokens == 0) return MXQ_OK;
  if (!dw || !weights || !experts || !dlogits || (!renorm && !logits)) return MXQ_EINVAL;
  if (renorm) ld = n_experts;
  if (ld < n_experts || tokens > kMaxDim / top_k || tokens > ((int64_t)1 << 40) / ld) return MXQ_ESHAPE;
  if ((!renorm && !aligned(logits, size_of(dt))) || !aligned(dw, 4) || !aligned(weights, 4) || !aligned(experts, 4) ||
      !aligned(dlogits, size_of(dt)))
    return MXQ_EALIGN;
  RouteLaunch l{};
  l.logits = logits;
  l.f32 = dt == MXQ_F32;
  l.tokens = tokens;
  l.ld = ld;
  l.experts = (int)n_experts;
  l.top_k = (int)top_k;
  l.renorm = renorm;
  l.weights = const_cast<float*>(weights);
  l.chosen = const_cast<int32_t*>(experts);
  l.dw = dw;
  l.dlogits = dlogits;
  return from_hip(launch_route_grad(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_expert_sort(const int32_t* experts, int64_t count, int64_t n_experts, int64_t* offsets,
                           int32_t* positions, int32_t* order, void* workspace, void* stream) {
  if (count < 0 || n_experts < 1 || n_experts > kMaxExperts) return MXQ_EINVAL;
  if (!offsets || (count > 0 && (!experts || !positions || !order))) return MXQ_EINVAL;
  if (count > kMaxDim) return MXQ_ESHAPE;
  if (sort_workspace(count, n_experts) > 0 && !workspace) return MXQ_EINVAL;
  if (!aligned(experts, 4) || !aligned(offsets, 8) || !aligned(positions, 4) || !aligned(order, 4) ||
      !aligned(workspace, 16))
    return MXQ_EALIGN;
  SortLaunch l{};
  l.experts = experts;
  l.count = count;
  l.n_experts = (int)n_experts;
  l.offsets = offsets;
  l.positions = positions;
  l.order = order;
  l.counts = static_cast<int32_t*>(workspace);
  return from_hip(launch_expert_sort(l, reinterpret_cast<hipStream_t>(stream)));
}

int64_t mxq_expert_sort_workspace(int64_t count, int64_t n_experts) {
  if (count <= 0 || count > kMaxDim || n_experts < 1 || n_experts > kMaxExperts) return 0;
  return sort_workspace(count, n_experts);
}

mxq_status mxq_dispatch(const void* x, mxq_dtype dt, int64_t tokens, int64_t width, int64_t ldx,
                        const int32_t* positions, int64_t top_k, int64_t rows, mxq_rows fmt, void* out, void* scales,
                        void* stream) {
  if (!is_dtype(dt) || fmt < MXQ_ROWS_COPY || fmt > MXQ_ROWS_FP8) return MXQ_EINVAL;
  if (mxq_status s = check_rows(tokens, top_k, rows, width)) return s;
  if (tokens == 0 || rows == 0) return MXQ_OK;
  if (!x || !positions || !out || (fmt != MXQ_ROWS_COPY && !scales)) return MXQ_EINVAL;
  if (ldx < width || ldx > ((int64_t)1 << 40) / tokens) return MXQ_ESHAPE;
  if ((fmt == MXQ_ROWS_MXFP4 && width % 32) || (fmt == MXQ_ROWS_FP8 && width % 128)) return MXQ_ESHAPE;
  if (!aligned(positions, 4) || !aligned(out, 16) || (fmt == MXQ_ROWS_FP8 && !aligned(scales, 4))) return MXQ_EALIGN;
  if (fmt == MXQ_ROWS_COPY ? !aligned(x, size_of(dt)) : !aligned(x, 16) || ldx * size_of(dt) % 16) return MXQ_EALIGN;
  RowsLaunch l{};
  l.x = x;
  l.x_f32 = dt == MXQ_F32;
  l.ldx = ldx;
  l.tokens = tokens;
  l.width = width;
  l.rows = rows;
  l.positions = positions;
  l.top_k = (int)top_k;
  l.fmt = fmt;
  l.out = out;
  l.scales = scales;
  return from_hip(launch_dispatch(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_combine(const void* y, mxq_dtype y_dt, int64_t rows, int64_t width, const int32_t* positions,
                       const float* weights, int64_t tokens, int64_t top_k, const void* residual, void* out,
                       mxq_dtype out_dt, void* stream) {
  if (!is_dtype(y_dt) || !is_dtype(out_dt)) return MXQ_EINVAL;
  if (mxq_status s = check_rows(tokens, top_k, rows, width)) return s;
  if (tokens == 0) return MXQ_OK;
  if ((rows > 0 && !y) || !positions || !out) return MXQ_EINVAL;
  if (!aligned(y, 16) || !aligned(positions, 4) || !aligned(weights, 4) || !aligned(residual, 16) || !aligned(out, 16))
    return MXQ_EALIGN;
  RowsLaunch l{};
  l.x = y;
  l.x_f32 = y_dt == MXQ_F32;
  l.tokens = tokens;
  l.width = width;
  l.rows = rows;
  l.positions = positions;
  l.top_k = (int)top_k;
  l.weights = weights;
  l.res = residual;
  l.out = out;
  l.out_f32 = out_dt == MXQ_F32;
  return from_hip(launch_combine(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_combine_grad(const void* grad, mxq_dtype grad_dt, const void* y, mxq_dtype y_dt, int64_t rows,
                            int64_t width, const int32_t* positions, const float* weights, int64_t tokens,
                            int64_t top_k, void* dy, float* dw, void* stream) {
  if (!is_dtype(grad_dt) || !is_dtype(y_dt)) return MXQ_EINVAL;
  if (mxq_status s = check_rows(tokens, top_k, rows, width)) return s;
  if (tokens == 0) return MXQ_OK;
  if (!grad || !positions || (rows > 0 && (!dy || (dw && !y)))) return MXQ_EINVAL;
  if (rows == 0 && !dw) return MXQ_OK;
  if (!aligned(grad, 16) || !aligned(y, 16) || !aligned(positions, 4) || !aligned(weights, 4) || !aligned(dy, 16) ||
      !aligned(dw, 4))
    return MXQ_EALIGN;
  RowsLaunch l{};
  l.x = grad;
  l.x_f32 = grad_dt == MXQ_F32;
  l.tokens = tokens;
  l.width = width;
  l.rows = rows;
  l.positions = positions;
  l.top_k = (int)top_k;
  l.weights = weights;
  l.res = y;
  l.out = dy;
  l.out_f32 = y_dt == MXQ_F32;
  l.dw = dw;
  return from_hip(launch_combine_grad(l, reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_fp8_quantize(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q8,
                            float* scales, void* stream) {
  if (!is_dtype(dt) || rows < 0 || cols < 0) return MXQ_EINVAL;
  if (rows == 0) return MXQ_OK;
  if (!x || !q8 || !scales) return MXQ_EINVAL;
  if (cols == 0 || cols > kMaxDim / 2 || ldx < cols || ldx > ((int64_t)1 << 40) / rows) return MXQ_ESHAPE;
  if (!aligned(x, size_of(dt)) || !aligned(q8, 16) || !aligned(scales, 4)) return MXQ_EALIGN;
  return from_hip(launch_fp8_quantize(x, dt == MXQ_F32, rows, cols, ldx, q8, scales,
                                      reinterpret_cast<hipStream_t>(stream)));
}

mxq_status mxq_fp8_act_grad(const void* dy, mxq_dtype dt, const uint8_t* z8, const float* z_scales, int64_t rows,
                            int64_t n, mxq_act act, const int64_t* offsets, int64_t n_experts, void* dz, float* db,
                            void* h, void* workspace, void* stream) {
  if (!is_dtype(dt) || act < MXQ_ACT_NONE || act > MXQ_ACT_SWIGLU || rows < 0 || n < 0) return MXQ_EINVAL;
  if (offsets ? (n_experts < 1 || n_experts > kMaxExperts) : n_experts != 1) return MXQ_EINVAL;
  if (rows == 0 && !db) return MXQ_OK;
  if (rows > 0 && (!dy || !z8 || !z_scales || !dz || (db && !workspace))) return MXQ_EINVAL;
  if (n == 0 || n > kMaxDim || rows > kMaxDim || rows > ((int64_t)1 << 40) / n) return MXQ_ESHAPE;
  if (act == MXQ_ACT_SWIGLU && n % 2) return MXQ_ESHAPE;
  // the grids enumerate row blocks x column tiles (16 bytes of 64 lanes) and groups x column tiles
  const int64_t tile = 64 * 16 / size_of(dt);
  if (act_grad_blocks(rows, n_experts, act_grad_rows(rows, n)) * ((n + tile - 1) / tile) >= kMaxGrid / 64 ||
      n_experts * ((n + 63) / 64) >= kMaxGrid / 256)
    return MXQ_ESHAPE;
  if (!aligned(dy, 16) || !aligned(z8, 16) || !aligned(z_scales, 4) || !aligned(dz, 16) || !aligned(db, 16) ||
      !aligned(h, 16) || !aligned(workspace, 16) || !aligned(offsets, 8))
    return MXQ_EALIGN;
  ActGradLaunch l{};
  l.dy = dy;
  l.z = z8;
  l.z_scales = z_scales;
  l.f32 = dt == MXQ_F32;
  l.rows = rows;
  l.n = n;
  l.act = (int)act;
  l.offsets = offsets;
  l.groups = (int)n_experts;
  l.dz = dz;
  l.h = h;
  l.db = db;
  l.partials = static_cast<float*>(workspace);
  l.block_rows = act_grad_rows(rows, n);
  return from_hip(launch_fp8_act_grad(l, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
