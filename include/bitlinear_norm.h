/*
 * bitlinear_norm.h -- the step between two layers: the residual's addition,
 * the sub-layer norm and 8-bit codes of its output, in one launch.
 *
 * A layer's output joins the residual stream, and the next layer's norm reads
 * the sum ("BitNet b1.58 2B4T Technical Report", section 2, names the
 * sub-layer norm; its formula is the reading stated for
 * bitlinear_subln_quant_act in bitlinear.h).  Conventions, status codes and
 * bitlinear_last_error() are those of bitlinear.h.
 *
 * Per token, with x widened to binary32 and rounding to nearest even:
 *   total    = the binary32 sum x + residual, rounded to the residual's type,
 *              or x where there is no residual;
 *   r, x_hat = as bitlinear_subln_quant_act defines them for the row `total`
 *              (exact sum of squares, r in binary32, x_hat = RN32(RN32(total * g) * r)).
 * Whatever a row holds, the other rows' results do not depend on it.
 */
#ifndef BITLINEAR_NORM_H
#define BITLINEAR_NORM_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The sum and step A1's int8 codes of its norm: the same bits as the addition
 * followed by bitlinear_subln_quant_act.
 *
 *   x         [T, K] of dtype x_dtype (BL_F32 or BL_BF16), 16-byte aligned.
 *   residual  [T, K] of dtype r_dtype (BL_F32 or BL_BF16), 16-byte aligned, or NULL
 *             for the norm of x alone (r_dtype is then not looked at).
 *   gain      [K] float32, 16-byte aligned.
 *   eps_n     the norm's epsilon, finite and > 0.
 *   T, K      1 <= T <= 2^24, 16 <= K <= BITLINEAR_MAX_K, K % 16 == 0.
 *   total     [T, K] output of dtype r_dtype, 16-byte aligned; NULL exactly where
 *             residual is.  It may be the residual itself, or x where their
 *             dtypes are the same; no other output may overlap an input.
 *   xq        [T, K] int8 output, 16-byte aligned.
 *   scale     [T] float32 output: max |x_hat| (takes the place of absmax).
 *   rowsum    [T] int32 output sum_k xq[t,k], or NULL.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_ARG
 * (eps_n, or total without a residual), BL_ERR_HIP. */
bl_status bitlinear_add_subln_quant_act(const void* x, int x_dtype, const void* residual,
                                        int r_dtype, const float* gain, float eps_n, int64_t T,
                                        int64_t K, void* total, int8_t* xq, float* scale,
                                        int32_t* rowsum, void* stream);

/* The sum and the e4m3 codes of its norm, one scale per group of 128 along K:
 * bitlinear_quant_act_f8 (bitlinear_f8.h) of x_hat.
 *
 *   x .. total  as bitlinear_add_subln_quant_act.
 *   xq        [T, K] e4m3 output, 16-byte aligned.
 *   scales    [ceil(K / 128), T] float32 output: scales[g * T + t].
 * A row whose mean square is no binary32 number (a NaN or infinity in `total`, or a
 * square sum beyond binary32's range) gets NaN for every code.
 * Errors: as bitlinear_add_subln_quant_act. */
bl_status bitlinear_add_subln_quant_act_f8(const void* x, int x_dtype, const void* residual,
                                           int r_dtype, const float* gain, float eps_n, int64_t T,
                                           int64_t K, void* total, uint8_t* xq, float* scales,
                                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_NORM_H */
