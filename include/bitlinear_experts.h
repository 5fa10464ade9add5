/*
 * bitlinear_experts.h -- routed experts: BitLinear layers of which every token
 * takes k out of E, and the router that says which.
 *
 * "BitNet解读" (future work) names 1-bit mixtures of experts as the method's
 * next step and gives no details; each expert is read here as a BitLinear of
 * its own (its own ternary matrix and gamma), so every product below has the
 * numerics of bitlinear_linear_grouped and bitlinear_gated_relu2 on the rows
 * that its expert was given.  Conventions, numerical contract, status codes
 * and bitlinear_last_error() are those of bitlinear.h.
 *
 * Slots.  The T * k (token, rank) pairs, pair index t * k + j, are put in
 * order of their experts, pairs of one expert in order of their index; a
 * pair's place is its slot.  Expert e has the slots offsets[e] ..
 * offsets[e + 1] - 1.  A token whose row of logits has fewer than k usable
 * entries (all of a padded row may be masked) leaves pairs without an
 * expert; they have no slot, and the last T * k - offsets[E] slots are empty.
 * No call reads an empty slot's row for a result or writes to it.
 */
#ifndef BITLINEAR_EXPERTS_H
#define BITLINEAR_EXPERTS_H

#include "bitlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BITLINEAR_MAX_EXPERTS 1024
#define BITLINEAR_MAX_TOP_K 32

/* What a token's weights add up to (argument `share`). */
typedef enum {
  BL_SHARE_CHOSEN = 0, /* softmax over the token's chosen logits: they add up to 1 */
  BL_SHARE_ALL = 1     /* softmax over all its usable logits: the chosen ones' part of 1 */
} bl_share;

/* Rows of a tensor (arguments `x_rows` and `y_rows`). */
typedef enum {
  BL_ROWS_TOKENS = 0, /* one row per token: [T, .] */
  BL_ROWS_SLOTS = 1   /* one row per slot: [T * k, .] */
} bl_rows;

/* Where a batch of tokens goes: a HOST struct of device pointers, as
 * bitlinear_route_experts fills the arrays.  The kernels keep every access in
 * bounds whatever the arrays hold (offsets are taken as lying in [0, T * k]
 * and not decreasing, other entries are clamped); with contents that the
 * router would not write the results mean nothing. */
typedef struct bl_routing {
  int64_t T, k, E;         /* 1 <= T <= 2^24, 1 <= k <= 32, k <= E <= 1024, T * k < 2^30 */
  const int32_t* offsets;  /* [E + 1] first slot of each expert, then the slots in use */
  const int32_t* pairs;    /* [T * k] pair index of each slot, -1 in the empty ones */
  const int32_t* slots;    /* [T, k] slot of each pair, -1 without an expert (BL_ROWS_TOKENS outputs) */
  const float* weights;    /* [T, k] weight of each pair (BL_ROWS_TOKENS outputs) */
} bl_routing;

/* Bytes of device workspace that bitlinear_route_experts needs (0 for up to
 * 64 tokens; `workspace` may then be NULL). */
size_t bitlinear_route_workspace_bytes(int64_t T, int64_t E);

/* The router: each token's k largest logits, their softmax weights, and the
 * slots of all pairs.  Equal logits go to the lower expert first (-0 equals
 * +0); -inf (a mask) and NaN are never taken.  With l_max the token's largest
 * logit, u(l) = 1 where l = l_max and exp(l - l_max) elsewhere,
 *   weights[t, j] = u(l of rank j) / sum of u over the chosen (or all) logits,
 * in binary32.  Ranks beyond the usable logits get expert -1 and weight 0.
 * The same inputs give the same bits on every call.
 *
 *   logits   [T, E] scores of dtype BL_F32 (4-byte aligned) or BL_BF16 (2-byte).
 *   T, E, k  as in bl_routing.
 *   share    BL_SHARE_CHOSEN or BL_SHARE_ALL.
 *   ids      [T, k] int32 output: experts by falling logit.
 *   weights  [T, k] float32 output.
 *   offsets, pairs, slots   int32 outputs as in bl_routing.
 *   workspace  device scratch, 4-byte aligned, of at least
 *            bitlinear_route_workspace_bytes(T, E) bytes; overwritten.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_ARG
 * (share), BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bitlinear_route_experts(const void* logits, int dtype, int64_t T, int64_t E, int64_t k,
                                  int share, int32_t* ids, float* weights, int32_t* offsets,
                                  int32_t* pairs, int32_t* slots, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* The routed tokens' gate and up projections with the squared-ReLU gate:
 * row p of h is what bitlinear_gated_relu2 gives for the token of slot p with
 * the matrices of its expert.  Each token is quantised once (step A1), however
 * many experts it has.
 *
 *   routing     offsets and pairs (slots and weights are not read).
 *   x           [T, K] activations of dtype x_dtype (BL_F32 or BL_BF16), 16-byte aligned.
 *   packed_gu   [E, 2N, K/4]: each expert's rows as bitlinear_interleave_rows
 *               writes them (2i gate, 2i + 1 up), 16-byte aligned.
 *   gamma_gate, gamma_up   [E] float32 each, one per expert.
 *   N, K        1 <= N <= 2^25, 16 <= K <= BITLINEAR_MAX_K, K % 16 == 0, 2 E N K <= 2^38,
 *               T * k * 2N <= 2^36.  Fast up to T * K < 2^31 and 2N * K < 2^35; larger
 *               products run some three times longer per row.
 *   h           [T * k, N] bfloat16 output (uint16 bit patterns), by slot; rows of
 *               empty slots are left as they were.
 *   xq          [T, K] int8 activations (written), 16-byte aligned.
 *   absmax      [T] token absmax (written), 4-byte aligned.  In both, rows of tokens
 *               without an expert may be left as they were.
 *   acc         [T * k, 2N] exact int32 sums by slot, interleaved as the rows, or NULL.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_HIP. */
bl_status bitlinear_gated_relu2_experts(const bl_routing* routing, const void* x, int x_dtype,
                                        const uint8_t* packed_gu, const float* gamma_gate,
                                        const float* gamma_up, int64_t N, int64_t K, uint16_t* h,
                                        int8_t* xq, float* absmax, int32_t* acc, void* stream);

/* Bytes of device workspace that bitlinear_linear_experts needs with
 * BL_ROWS_TOKENS outputs (with BL_ROWS_SLOTS outputs: none). */
size_t bitlinear_experts_workspace_bytes(int64_t T, int64_t k, int64_t N);

/* Steps A1-A3 of one BitLinear per expert: the row of every slot in use times
 * the matrix of its expert (for instance the down projections).
 *   y_slot[p, n] = (sum_k t_e[n,k] * xq[row(p),k]) * gamma[e] * max(absmax[row(p)], eps) / 127,
 * row(p) = p (x_rows = BL_ROWS_SLOTS) or the slot's token (BL_ROWS_TOKENS).
 *   y_rows = BL_ROWS_SLOTS:  y = y_slot, [T * k, N]; rows of empty slots are left
 *                            as they were.
 *   y_rows = BL_ROWS_TOKENS: y[t, n] = sum over j of weights[t, j] * y_slot[slots[t, j], n],
 *                            [T, N], added in order of j in binary32, pairs
 *                            without a slot left out (a token without any gets 0).
 *
 *   routing    offsets and pairs; slots and weights too with BL_ROWS_TOKENS outputs.
 *   x          activations of dtype x_dtype (BL_F32 or BL_BF16), 16-byte aligned.
 *   packed     [E, N, K/4] from bitlinear_pack_weights, 16-byte aligned.
 *   gamma      [E] float32.
 *   N, K       1 <= N <= 2^26, 16 <= K <= BITLINEAR_MAX_K, K % 16 == 0, E N K <= 2^38,
 *              T * k * N <= 2^36.  Fast up to (rows of x) * K < 2^31 and N * K < 2^35;
 *              larger products run some three times longer per row (split the batch).
 *   y          float32 output, 4-byte aligned.
 *   xq         int8 activations (written), as many rows as x, 16-byte aligned.
 *   absmax     row absmax (written), one per row of x, 4-byte aligned.  In both, rows of
 *              empty slots or of tokens without an expert may be left as they were.
 *   acc        [T * k, N] exact int32 sums by slot, or NULL (BL_ROWS_SLOTS outputs only).
 *   workspace  device scratch, 16-byte aligned, of at least
 *              bitlinear_experts_workspace_bytes(T, k, N) bytes with BL_ROWS_TOKENS
 *              outputs; overwritten.  NULL otherwise.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_DTYPE, BL_ERR_ARG
 * (x_rows, y_rows, acc with BL_ROWS_TOKENS outputs), BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bitlinear_linear_experts(const bl_routing* routing, const void* x, int x_dtype,
                                   int x_rows, const uint8_t* packed, const float* gamma,
                                   int64_t N, int64_t K, float* y, int y_rows, int8_t* xq,
                                   float* absmax, int32_t* acc, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_EXPERTS_H */
