/*
 * mxq_gemm.h - C ABI of libmxq's matrix products on the operands that mxq.h's entry
 * points write, and of the gradient of their epilogue. Pointers, streams, ownership,
 * status codes and the byte layouts of codes and scales are those of mxq.h.
 *
 * Operands. Every product contracts the last index of both operands:
 * C[i, j] = sum_t A[i, t] B[j, t]. A row of k elements is held as
 *   MXQ_OPERAND_MXFP4   codes uint8 [rows, k/2], scales uint8 E8M0 [rows, k/32]; k % 32 == 0
 *   MXQ_OPERAND_FP8     E4M3 uint8 [rows, k], scales fp32 [rows, k/128], read through
 *                       their exponent field (2^(field - 127); 255: NaN); k % 128 == 0
 * dense and row-major: what mxq_quantize, mxq_rht_quantize, mxq_fp8_to_mxfp4 and
 * mxq_mxfp4_to_fp8 write. With the column-wise outputs the three products of a linear
 * layer y = x W^T are the same call: Fprop (x rows, W rows), Dgrad (dy rows, W's
 * column-wise output) and Wgrad (dy's and x's column-wise outputs).
 * The NVFP4 formats are not operands (the matrix cores scale blocks of 32, not 16).
 *
 * Precision. Products of two MXFP4 operands are formed exactly and summed in fp32 by
 * the scaled matrix instructions. The matrix cores add FP8 products in groups of eight,
 * in which what lies 2^-14 and more below the largest is lost (measured), and the groups
 * in fp32: the error does not grow with k, is 1.4e-5 of the result's norm on normal
 * data, about 1e-4 of the sum of the magnitudes where they spread widely, and 7 x 2^-13
 * of it (8.5e-4) at worst. Products with an FP8 operand take them only where the result
 * is rounded to bf16 (2e-3); with fp32 results, and for few rows, both operands are
 * widened to bf16 - exact for every E2M1 and E4M3 value times its scale whose magnitude
 * is at least 2^-126 and below 2^128, below which it may be lost and beyond which it is
 * infinite - and multiplied there, again exactly with sums in fp32.
 * NaN scales give NaN in the rows (columns) of the result that they belong to.
 */
#ifndef MXQ_GEMM_H_
#define MXQ_GEMM_H_

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MXQ_OPERAND_MXFP4 = 0, MXQ_OPERAND_FP8 = 1 } mxq_operand;

/*
 * Activations, on fp32 values:
 *   MXQ_ACT_RELU    max(z, 0)                 MXQ_ACT_SILU  z sigmoid(z)
 *   MXQ_ACT_GELU    z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
 *   MXQ_ACT_SWIGLU  silu(z[2j]) z[2j + 1]: gate and up are interleaved (row 2j of the
 *                   weight is gate j, row 2j + 1 is up j), n is even and the result
 *                   has n/2 columns
 */
typedef enum {
  MXQ_ACT_NONE = 0,
  MXQ_ACT_RELU = 1,
  MXQ_ACT_GELU = 2,
  MXQ_ACT_SILU = 3,
  MXQ_ACT_SWIGLU = 4
} mxq_act;

/*
 * mxq_gemm - z = A B^T + bias, d = act(z) + residual.
 * a, a_scales  operand [m, k];  b, b_scales  operand [n, k]. b_fmt may be FP8 only where
 *              a_fmt is (else MXQ_EUNSUPPORTED).
 * bias         [n] of bias_dt, or NULL.
 * residual     [m, dn] of d_dt, or NULL; dn = n/2 for MXQ_ACT_SWIGLU, else n. It may be
 *              d itself: the call then adds to d.
 * d            [m, dn] of d_dt (bf16 or fp32; rounded once, to nearest even).
 * z            [m, n] of d_dt, or NULL: z as mxq_act_grad takes it. It must not
 *              overlap d or residual.
 * Alignment: codes 16 bytes, fp32 scales and fp32 bias 4, bf16 bias 2, residual, d and
 * z 16; E8M0 scales may start at any byte (on a multiple of 4 they are read faster). m >= 0 (0: nothing is done), 1 <= n < 2^31, m < 2^31, 1 <= k <= 2^22.
 */
mxq_status mxq_gemm(const uint8_t* a, const void* a_scales, mxq_operand a_fmt, const uint8_t* b,
                    const void* b_scales, mxq_operand b_fmt, int64_t m, int64_t n, int64_t k,
                    const void* bias, mxq_dtype bias_dt, mxq_act act, const void* residual, void* d,
                    mxq_dtype d_dt, void* z, void* stream);

/*
 * mxq_grouped_gemm - mxq_gemm for tokens grouped by expert: row r of A, of expert e
 * (offsets[e] <= r < offsets[e + 1]), is multiplied by B[e] and gets bias[e].
 * a [rows, k], b [n_experts, n, k], bias [n_experts, n], residual, d and z as above.
 * offsets: device int64 [n_experts + 1], offsets[0] = 0, nondecreasing,
 * offsets[n_experts] = rows; experts may be empty and need no padding. They are read
 * on the device; values outside [0, rows] are clamped, so malformed offsets give
 * unspecified output but no access outside the buffers. 1 <= n_experts <= 4096.
 */
mxq_status mxq_grouped_gemm(const uint8_t* a, const void* a_scales, mxq_operand a_fmt, const uint8_t* b,
                            const void* b_scales, mxq_operand b_fmt, int64_t rows, int64_t n, int64_t k,
                            const int64_t* offsets, int64_t n_experts, const void* bias,
                            mxq_dtype bias_dt, mxq_act act, const void* residual, void* d,
                            mxq_dtype d_dt, void* z, void* stream);

/*
 * mxq_grouped_wgrad - the weight gradient of every expert over its own tokens,
 *   d[e][i][j] = add[e][i][j] + sum over the tokens t of expert e of Y[t][i] X[t][j],
 * both operands as mxq_fp4_row_to_fp8_col writes them: E4M3 columns y [n, ld_y] and
 * x [k, ld_x], fp32 power-of-two scales y_scales [n, ld_ys] and x_scales [k, ld_xs],
 * one per 128-token group of an expert. Of a column, tokens from rows (rounded up to 16)
 * on and scales from (rows + 127 n_experts) / 128 on are not read: both operands may be
 * slices of wider tensors.
 * add, d: [n_experts, n, k] of d_dt; add may be NULL (zero) or d itself. An expert
 * without tokens gives add, or zeros; so does rows == 0.
 * offsets as in mxq_grouped_gemm. rows <= ld_y, ld_x <= 2^23, multiples of 16;
 * (rows + 127 n_experts) / 128 <= ld_ys, ld_xs < 2^22. y, x, add, d 16-byte aligned, scales 4,
 * offsets 8. n, k < 2^31.
 */
mxq_status mxq_grouped_wgrad(const uint8_t* y, const float* y_scales, int64_t ld_y, int64_t ld_ys,
                             const uint8_t* x, const float* x_scales, int64_t ld_x, int64_t ld_xs,
                             int64_t rows, int64_t n, int64_t k, const int64_t* offsets,
                             int64_t n_experts, const void* add, void* d, mxq_dtype d_dt, void* stream);

/*
 * mxq_act_grad - the gradient of the epilogue. dy [rows, dn] is the gradient of
 * d = act(z) (+ residual, whose gradient is dy itself), z [rows, n] what mxq_gemm kept:
 *   dz = act'(z) dy            [rows, n] of dt (SWIGLU: of both halves of each pair)
 *   db[e] = sum of the fp32 values of dz over the rows of expert e, fp32 [groups, n]
 * dt: the type of dy, z and dz. offsets == NULL: one group of all rows (n_experts is
 * then 1); otherwise as in mxq_grouped_gemm. db may be NULL. A group without rows has
 * db = 0; so has rows == 0. The sums are taken in a fixed order: equal inputs give
 * equal bits.
 * workspace: mxq_act_grad_workspace(rows, n, n_experts) bytes on the device, 16-byte
 * aligned, needed when db is given and that is not 0; its contents do not matter.
 * dz may be z (the gradient is then written over it). dy, z, dz, db 16-byte aligned.
 */
mxq_status mxq_act_grad(const void* dy, const void* z, mxq_dtype dt, int64_t rows, int64_t n, mxq_act act,
                        const int64_t* offsets, int64_t n_experts, void* dz, float* db, void* workspace,
                        void* stream);

/* Host helper: bytes of workspace that mxq_act_grad needs for a bias gradient. */
int64_t mxq_act_grad_workspace(int64_t rows, int64_t n, int64_t n_experts);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_GEMM_H_ */
