/*
 * mxq_moe.h - C ABI of libmxq's operators around the experts' products (mxq_gemm.h): the
 * choice of experts, the rows of every expert, tokens sent to those rows and their results
 * brought back, each with its gradient, and values before an activation kept in 8 bits.
 * Pointers, streams, ownership, status codes and byte layouts are those of mxq.h.
 *
 * T tokens choose k experts each; assignment t k + j is token t's choice j. Its row among
 * the rows of all experts is positions[t, j]; a position outside [0, rows) (-1, as
 * mxq_expert_sort writes it) stands for an assignment without a row, which reads and
 * writes nothing. Two assignments must not have the same row.
 *
 * Limits: fewer than 2^31 assignments, rows and tokens, 2^40 elements of a matrix, 2^22
 * columns of a row that is sent or combined (beyond them MXQ_ESHAPE), 4096 experts, 64
 * choices of a token (MXQ_EINVAL). 0 tokens, or 0 rows to write, are no-ops.
 */
#ifndef MXQ_MOE_H_
#define MXQ_MOE_H_

#include "mxq_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mxq_route - the top_k largest logits of every token and their softmax weights.
 * logits   [tokens, n_experts] of dt, row stride ld >= n_experts.
 * experts  int32 [tokens, top_k]: in falling order of the logits, equal ones (and -0 and
 *          +0) in rising order of the expert; NaN counts as larger than +Inf. A logit of
 *          -Inf is never chosen: choices left over are -1.
 * weights  fp32 [tokens, top_k]: renorm == 0: softmax over all experts; renorm == 1:
 *          softmax over the chosen ones. 0 where the expert is -1. A NaN or +Inf among the
 *          logits that the softmax runs over makes the token's weights NaN.
 * 1 <= top_k <= n_experts, top_k <= 64, n_experts <= 4096; logits aligned to its type,
 * weights and experts to 4 bytes.
 */
mxq_status mxq_route(const void* logits, mxq_dtype dt, int64_t tokens, int64_t n_experts, int64_t ld,
                     int64_t top_k, int renorm, float* weights, int32_t* experts, void* stream);

/*
 * mxq_route_grad - the gradient of mxq_route. dw [tokens, top_k] is the gradient of the
 * weights; weights and experts are what mxq_route wrote, for the same logits and renorm.
 *   S = sum_j w_j dw_j
 *   dlogits[e] = sum over j with experts[j] == e of w_j dw_j, less S p_e (renorm == 0,
 *   p the softmax over all experts) or S times the weights of e (renorm == 1)
 * dlogits  [tokens, n_experts] of dt, dense (rounded once). Choices outside
 *          [0, n_experts) are left out, whatever their dw. mxq_route names an expert once for
 *          a token; the terms of one named more often are added up in no stated order.
 * logits   as in mxq_route; not read with renorm == 1 (may be NULL). ld is then ignored.
 */
mxq_status mxq_route_grad(const float* dw, const float* weights, const int32_t* experts, const void* logits,
                          mxq_dtype dt, int64_t tokens, int64_t n_experts, int64_t ld, int64_t top_k, int renorm,
                          void* dlogits, void* stream);

/*
 * mxq_expert_sort - the rows of every expert: `count` assignments sorted by expert, those
 * of one expert in their own order.
 * experts    int32 [count]; a value outside [0, n_experts) is an assignment without a row.
 * offsets    int64 [n_experts + 1]: rows of expert e are [offsets[e], offsets[e + 1]).
 * positions  int32 [count]: the row of every assignment, or -1.
 * order      int32 [count]: the assignment of every row; -1 from row offsets[n_experts] on.
 * workspace  mxq_expert_sort_workspace(count, n_experts) bytes on the device, 16-byte
 *            aligned; its contents do not matter. May be NULL where that is 0.
 * 0 <= count < 2^31, 1 <= n_experts <= 4096. count == 0 writes the offsets alone.
 */
mxq_status mxq_expert_sort(const int32_t* experts, int64_t count, int64_t n_experts, int64_t* offsets,
                           int32_t* positions, int32_t* order, void* workspace, void* stream);

/* Host helper: bytes of workspace that mxq_expert_sort needs. */
int64_t mxq_expert_sort_workspace(int64_t count, int64_t n_experts);

typedef enum { MXQ_ROWS_COPY = 0, MXQ_ROWS_MXFP4 = 1, MXQ_ROWS_FP8 = 2 } mxq_rows;

/*
 * mxq_dispatch - every token's row to the rows of its assignments:
 *   out[positions[t, j]] = x[t]
 * x        [tokens, width] of dt, row stride ldx >= width.
 * out      [rows, width]: MXQ_ROWS_COPY of dt, as x; MXQ_ROWS_MXFP4 codes uint8 [rows, width/2]
 *          and E8M0 scales uint8 [rows, width/32], the bits that mxq_quantize gives (nearest
 *          even); MXQ_ROWS_FP8 E4M3 uint8 [rows, width] and fp32 scales [rows, width/128], the
 *          bits that mxq_fp8_quantize gives. Rows of no assignment are left as they are.
 * scales   NULL for MXQ_ROWS_COPY.
 * width % 32 == 0 for MXFP4 and % 128 for FP8. Alignment: out 16 bytes, fp32 scales 4; x its
 * type for MXQ_ROWS_COPY, else 16 bytes with rows that start on 16 bytes.
 * Its gradient is mxq_combine without weights. 1 <= top_k <= 64.
 */
mxq_status mxq_dispatch(const void* x, mxq_dtype dt, int64_t tokens, int64_t width, int64_t ldx,
                        const int32_t* positions, int64_t top_k, int64_t rows, mxq_rows fmt, void* out,
                        void* scales, void* stream);

/*
 * mxq_combine - the rows of every token's assignments, weighted and added up:
 *   out[t] = residual[t] + sum_j weights[t, j] y[positions[t, j]]
 * y         [rows, width] of y_dt.
 * weights   fp32 [tokens, top_k], or NULL: all 1. Weights of assignments without a row do
 *           not matter (nor do rows of no assignment).
 * residual  [tokens, width] of out_dt, or NULL: zero. It may be out itself.
 * out       [tokens, width] of out_dt: sums in fp32 in the order of j, the residual last,
 *           rounded once.
 * y, residual and out 16-byte aligned. 1 <= top_k <= 64.
 */
mxq_status mxq_combine(const void* y, mxq_dtype y_dt, int64_t rows, int64_t width, const int32_t* positions,
                       const float* weights, int64_t tokens, int64_t top_k, const void* residual, void* out,
                       mxq_dtype out_dt, void* stream);

/*
 * mxq_combine_grad - the gradient of mxq_combine. grad [tokens, width] of grad_dt is the
 * gradient of its output (and of its residual).
 *   dy[positions[t, j]] = weights[t, j] grad[t]         of y_dt, rounded once
 *   dw[t, j] = sum over the columns of grad[t] y[positions[t, j]]    fp32; 0 without a row
 * y    [rows, width] of y_dt; may be NULL where dw is.
 * dy   [rows, width]; rows of no assignment are left as they are. It may be y itself.
 * dw   fp32 [tokens, top_k], or NULL. Its sums are taken in a fixed order.
 * grad, y and dy 16-byte aligned. 1 <= top_k <= 64.
 */
mxq_status mxq_combine_grad(const void* grad, mxq_dtype grad_dt, const void* y, mxq_dtype y_dt, int64_t rows,
                            int64_t width, const int32_t* positions, const float* weights, int64_t tokens,
                            int64_t top_k, void* dy, float* dw, void* stream);

/*
 * mxq_fp8_quantize - rows in E4M3 with a power-of-two scale for each 128 columns: the FP8
 * operand of the products, and the form in which z is kept for mxq_fp8_act_grad.
 * x       [rows, cols] of dt, row stride ldx >= cols.
 * q8      uint8 [rows, cols], the nearest E4M3 value of x / s (ties to even, sign kept).
 * scales  fp32 [rows, ceil(cols / 128)], the last one of a row for what is left of it:
 *         s = 2^i, i >= -126 the smallest with max|x| / s <= 448 (i = 0 where all are
 *         zero). A group that meets NaN or Inf gets scale NaN and codes 0x7F.
 * Alignment: x its type, q8 16 bytes, scales 4. Any cols >= 1.
 */
mxq_status mxq_fp8_quantize(const void* x, mxq_dtype dt, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q8,
                            float* scales, void* stream);

/*
 * mxq_fp8_act_grad - mxq_act_grad from z in FP8: with z the values that mxq_fp8_quantize's
 * z8 [rows, n] and z_scales [rows, ceil(n / 128)] stand for (a scale is read through its
 * exponent field; 255: NaN),
 *   dz = act'(z) dy                            [rows, n] of dt
 *   db[e] = sum of dz over the rows of expert e    fp32 [groups, n], or NULL
 *   h = act(z)                                 [rows, n], SWIGLU [rows, n/2], of dt, or NULL
 * dy, dt, offsets, n_experts, db, workspace (mxq_act_grad_workspace) and the order of sums
 * as in mxq_act_grad. dy, z8, dz, db and h 16-byte aligned, z_scales 4. h may be dy itself.
 */
mxq_status mxq_fp8_act_grad(const void* dy, mxq_dtype dt, const uint8_t* z8, const float* z_scales, int64_t rows,
                            int64_t n, mxq_act act, const int64_t* offsets, int64_t n_experts, void* dz, float* db,
                            void* h, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_MOE_H_ */
