/*
 * bitlinear_w4.h -- linear layers with 4-bit weights and one scale per group
 * of a row (W4A8), for the matrices of a ternary model that do not take
 * ternary weights, such as its vocabulary projection.
 *
 * The pages only compare with 4-bit post-training quantisation ("BitNet b1.58
 * 2B4T Technical Report", section 4.2) and give no format; the one below is
 * this library's.  The activations are step A1's int8 tokens, so the same
 * bitlinear_quant_act or bitlinear_subln_quant_act output feeds ternary and
 * 4-bit matrices alike.  Conventions, status codes and bitlinear_last_error()
 * are those of bitlinear.h.
 *
 * Values.  Row n is cut into groups of G weights along K; a weight of group g
 * stands for (t - z[n,g]) * s[n,g] with t and z whole numbers in [-8, 7] and s
 * a bfloat16 scale (binary32's range, so no scale of a finite matrix leaves
 * it; its 8 significant bits are rounded once, before the codes are chosen).
 * Without zero points z is 0.
 *
 * Packed layout.  Row n occupies 64 * ceil(K / 128) bytes at byte offset
 * n * 64 * ceil(K / 128), one run of 64 bytes per block of 128 weights.  In a
 * block, byte i (0..3) of little-endian word j (0..3) of 16-byte chunk q
 * (0..3) holds, as two's complement nibbles, the t of
 *   k = 32j + 8q + i      in its low four bits,
 *   k = 32j + 8q + 4 + i  in its high four bits,
 * so word j of the four chunks is one group of 32 and a masked word is four
 * consecutive k as int8 multiples of 16.  Nibbles past K are 0.
 */
#ifndef BITLINEAR_W4_H
#define BITLINEAR_W4_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a packed row: 64 * ceil(K / 128). */
int64_t bitlinear_w4_row_bytes(int64_t K);

/* Quantises and packs one weight matrix.  Per group of G weights w, every
 * operation binary32 with one rounding unless said otherwise:
 *   without zero points:  s = bf16(max |w| / 7), z = 0,
 *                         t = clamp(rne(w / s), -8, 7);
 *   with zero points:     lo = min(w, 0), hi = max(w, 0), s = bf16((hi - lo) / 15),
 *                         z = clamp(rne(-lo / s), 0, 15) - 8,
 *                         t = clamp(rne(w / s) + z, -8, 7).
 * A group whose s is 0 (all zero, or too small for bfloat16) gets t = z = 0.
 * hi - lo has to be finite.
 *
 *   w        [N, K] float32 weights, row-major, 16-byte aligned.
 *   G        32, 64 or 128.
 *   N, K     1 <= N <= 2^26, G <= K <= BITLINEAR_MAX_K, K % G == 0, N * K <= 2^38.
 *   packed   [N, bitlinear_w4_row_bytes(K)] uint8 output, 16-byte aligned.
 *   scales   [N, K / G] bfloat16 output (uint16 bit patterns), 2-byte aligned.
 *   zeros    [N, K / G] int8 output z, or NULL for no zero points.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_ARG (G), BL_ERR_HIP. */
bl_status bitlinear_pack_weights_w4(const float* w, int64_t N, int64_t K, int64_t G,
                                    uint8_t* packed, uint16_t* scales, int8_t* zeros,
                                    void* stream);

/* The values that a packed matrix stands for: w[n,k] = (t - z) * s, exact in binary32.
 *
 *   packed, scales, zeros, N, K, G   as bitlinear_pack_weights_w4 (zeros NULL: z = 0).
 *   w        [N, K] float32 output, 16-byte aligned.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_ARG (G), BL_ERR_HIP. */
bl_status bitlinear_unpack_weights_w4(const uint8_t* packed, const uint16_t* scales,
                                      const int8_t* zeros, int64_t N, int64_t K, int64_t G,
                                      float* w, void* stream);

/* y[t, n] = (sum over groups g of s[n,g] * sum_{k in g} (t[n,k] - z[n,g]) * xq[t,k])
 *           * max(absmax[t], eps) / 127.
 * Each group's sum is exact in int32; the sum over groups is in binary32, in
 * an order that depends on the shape alone, so the same inputs give the same
 * bits on every call.
 *
 *   packed, scales, zeros, N, K, G   as bitlinear_pack_weights_w4 (zeros NULL: z = 0).
 *   xq       [T, K] int8 from bitlinear_quant_act, 16-byte aligned.
 *   absmax   [T] float32 from bitlinear_quant_act.
 *   T        1 <= T <= 2^24, T * N <= 2^36.
 *   y        [T, N] float32 output, 4-byte aligned.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_ARG (G), BL_ERR_HIP. */
bl_status bitlinear_forward_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                               const int8_t* xq, const float* absmax, int64_t T, int64_t N,
                               int64_t K, int64_t G, float* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_W4_H */
