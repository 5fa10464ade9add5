/*
 * bitlinear_f8.h -- linear layers in 8-bit floating point with a scale for
 * each block of 128, for the matrices of a ternary model that take neither
 * ternary nor 4-bit weights (its vocabulary projection, its first and last
 * layers).
 *
 * The pages keep such matrices in higher precision ("BitNet b1.58 2B4T
 * Technical Report", section 2) and give no 8-bit format; the one below is
 * this library's.  Conventions, status codes and bitlinear_last_error() are
 * those of bitlinear.h.
 *
 * Codes are e4m3 bytes (sign, 4 exponent bits of bias 7, 3 significand bits,
 * no infinities, largest value 448).  A group of values v with m = max |v| is
 * held as, every operation binary32 with one rounding to nearest even:
 *   m'    = max(m, 2^-100),
 *   code  = e4m3(v * (448 / m')),     never above 448 in magnitude,
 *   scale = m' / 448,
 * and a code c stands for c * scale.
 *
 * Tokens: one group per 128 consecutive k of a row (the last may be shorter),
 * codes [T, K], scales group-major: [ceil(K / 128), T], scales[g * T + t], so
 * that neighbouring tokens' scales of one group are neighbours in memory.
 * Matrices: one group per block of 128 rows x 128 columns (the last ones may
 * be smaller), codes [N, K] row-major, scales [ceil(N / 128), ceil(K / 128)].
 *
 * A value that is NaN or infinite gets a NaN code (0x7f or 0xff), and the other
 * codes and the scale of its group may then be any.  All outputs of a token, or of a matrix
 * row, with a NaN code are NaN.  Groups, tokens and rows without one do not depend on it.
 */
#ifndef BITLINEAR_F8_H
#define BITLINEAR_F8_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantises tokens.
 *
 *   x        [T, K] of dtype x_dtype (BL_F32 or BL_BF16), 16-byte aligned.
 *   T, K     1 <= T <= 2^24, 16 <= K <= BITLINEAR_MAX_K, K % 16 == 0.
 *   xq       [T, K] e4m3 output, 16-byte aligned.
 *   scales   [ceil(K / 128), T] float32 output.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_HIP. */
bl_status bitlinear_quant_act_f8(const void* x, int x_dtype, int64_t T, int64_t K, uint8_t* xq,
                                 float* scales, void* stream);

/* Quantises one matrix.
 *
 *   w        [N, K] float32, 16-byte aligned.
 *   N, K     1 <= N <= 2^26, 16 <= K <= BITLINEAR_MAX_K, K % 16 == 0, N * K <= 2^38.
 *   codes    [N, K] e4m3 output, 16-byte aligned.
 *   scales   [ceil(N / 128), ceil(K / 128)] float32 output.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bitlinear_pack_weights_f8(const float* w, int64_t N, int64_t K, uint8_t* codes,
                                    float* scales, void* stream);

/* The values that a matrix stands for, RN32(code * scale).
 *
 *   codes, scales, N, K   as bitlinear_pack_weights_f8.
 *   w        [N, K] float32 output, 16-byte aligned.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bitlinear_unpack_weights_f8(const uint8_t* codes, const float* scales, int64_t N,
                                      int64_t K, float* w, void* stream);

/* Or'ed to y_dtype BL_BF16: sums may be cut, see bitlinear_forward_f8. */
#define BL_CUT_SUMS 0x100

/* y[t, n] = sum over blocks g of (x_scales[g, t] * w_scales[n / 128, g])
 *           * sum_{k in g} xq[t, k] * w[n, k].
 * Products and sums in binary32, for either type of output and any number of
 * tokens.  Sums go in an order that depends on the shape and the device's number of
 * CUs alone: the same inputs give the same bits on every call.
 *
 * With BL_CUT_SUMS (BL_BF16 | BL_CUT_SUMS as y_dtype) the caller allows matrix
 * instructions of twice the rate that keep fewer bits: of eight products of
 * neighbouring k (8 i .. 8 i + 7) all bits below 2^-13 of the largest one's power of
 * two are cut off, so a sum is within 7 * 2^-13 of its products' magnitudes (4e-5
 * to 5e-5 of the result in the norm, for activations without outlying features)
 * before it is rounded to bfloat16.  Few tokens may be summed in binary32 all the same.
 *
 *   w, w_scales   as bitlinear_pack_weights_f8 writes them.
 *   xq, x_scales  as bitlinear_quant_act_f8 writes them; both code arrays 16-byte aligned.
 *   T, N, K  1 <= T <= 2^24, T * N <= 2^36, N and K as bitlinear_pack_weights_f8.
 *   y_dtype  BL_F32, or BL_BF16 (the binary32 result rounded to nearest even), the latter
 *            with or without BL_CUT_SUMS.
 *   y        [T, N] output, aligned to its element.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_HIP. */
bl_status bitlinear_forward_f8(const uint8_t* w, const float* w_scales, const uint8_t* xq,
                               const float* x_scales, int64_t T, int64_t N, int64_t K, void* y,
                               int y_dtype, void* stream);

/* bitlinear_quant_act_f8 of x, then bitlinear_forward_f8: the same results.
 *
 *   x, x_dtype   as bitlinear_quant_act_f8.
 *   w, w_scales, T, N, K, y, y_dtype   as bitlinear_forward_f8.
 *   xq, x_scales   the tokens' codes and scales (written), as bitlinear_quant_act_f8.
 * Errors: as the two calls, before either is made. */
bl_status bitlinear_linear_f8(const void* x, int x_dtype, const uint8_t* w, const float* w_scales,
                              int64_t T, int64_t N, int64_t K, uint8_t* xq, float* x_scales,
                              void* y, int y_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_F8_H */
