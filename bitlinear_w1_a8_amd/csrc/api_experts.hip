// C ABI of the routed-expert and 4-bit operators (declared in
// include/bitlinear_experts.h and include/bitlinear_w4.h): argument checks on
// the host, then kernel launches on the caller's stream.
#include "api_util.h"
#include "experts.h"

using bl::aligned;
using bl::check_k;
using bl::fail;
using bl::kMaxN;
using bl::kMaxNK;
using bl::kMaxT;
using bl::kMaxTN;
using bl::launched;

namespace {

constexpr int64_t kMaxPairs = int64_t(1) << 30;   // slot numbers are int32

bl_status check_counts(const char* fn, int64_t t, int64_t k, int64_t e) {
  if (t < 1 || t > kMaxT) return fail(BL_ERR_SHAPE, "%s: T=%lld out of range", fn, (long long)t);
  if (e < 1 || e > BITLINEAR_MAX_EXPERTS)
    return fail(BL_ERR_SHAPE, "%s: E=%lld must be in [1, %d]", fn, (long long)e,
                BITLINEAR_MAX_EXPERTS);
  if (k < 1 || k > BITLINEAR_MAX_TOP_K || k > e || t * k >= kMaxPairs)
    return fail(BL_ERR_SHAPE, "%s: k=%lld must be in [1, min(E, %d)] with T*k below 2^30", fn,
                (long long)k, BITLINEAR_MAX_TOP_K);
  return BL_OK;
}

bl_status check_group(const char* fn, int64_t n, int64_t k, int64_t g) {
  if (g != 32 && g != 64 && g != 128)
    return fail(BL_ERR_ARG, "%s: G=%lld must be 32, 64 or 128", fn, (long long)g);
  if (k < g || k > BITLINEAR_MAX_K || k % g != 0)
    return fail(BL_ERR_SHAPE, "%s: K=%lld must be a multiple of G=%lld up to %d", fn, (long long)k,
                (long long)g, BITLINEAR_MAX_K);
  if (n < 1 || n > kMaxN || n * k > kMaxNK)
    return fail(BL_ERR_SHAPE, "%s: N=%lld out of range", fn, (long long)n);
  return BL_OK;
}

}  // namespace

extern "C" {

size_t bitlinear_route_workspace_bytes(int64_t T, int64_t E) {
  return T < 1 || T > kMaxT || E < 1 || E > BITLINEAR_MAX_EXPERTS ? 0
                                                                  : bl::route_workspace_bytes(T, E);
}

bl_status bitlinear_route_experts(const void* logits, int dtype, int64_t T, int64_t E, int64_t k,
                                  int share, int32_t* ids, float* weights, int32_t* offsets,
                                  int32_t* pairs, int32_t* slots, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const char* fn = "bitlinear_route_experts";
  if (!logits || !ids || !weights || !offsets || !pairs || !slots)
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (dtype != BL_F32 && dtype != BL_BF16) return fail(BL_ERR_DTYPE, "%s: unknown dtype %d", fn, dtype);
  if (bl_status rc = check_counts(fn, T, k, E)) return rc;
  if (share != BL_SHARE_CHOSEN && share != BL_SHARE_ALL)
    return fail(BL_ERR_ARG, "%s: unknown share %d (BL_SHARE_CHOSEN or BL_SHARE_ALL)", fn, share);
  const size_t need = bl::route_workspace_bytes(T, E);
  if (need && !workspace) return fail(BL_ERR_NULL, "%s: NULL workspace", fn);
  if (!aligned(logits, dtype == BL_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(pairs, 4) || !aligned(slots, 4) || !aligned(workspace, 4))
    return fail(BL_ERR_ALIGN, "%s: logits need their dtype's, the others 4-byte alignment", fn);
  if (workspace_bytes < need)
    return fail(BL_ERR_WORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes, need);
  return launched(fn, bl::launch_route(logits, dtype == BL_BF16, T, E, k, share, ids, weights,
                                       offsets, pairs, slots, static_cast<int32_t*>(workspace),
                                       static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_gated_relu2_experts(const bl_routing* routing, const void* x, int x_dtype,
                                        const uint8_t* packed_gu, const float* gamma_gate,
                                        const float* gamma_up, int64_t N, int64_t K, uint16_t* h,
                                        int8_t* xq, float* absmax, int32_t* acc, void* stream) {
  const char* fn = "bitlinear_gated_relu2_experts";
  if (!routing || !x || !packed_gu || !gamma_gate || !gamma_up || !h || !xq || !absmax)
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  const bl_routing& r = *routing;
  if (!r.offsets || !r.pairs) return fail(BL_ERR_NULL, "%s: NULL offsets or pairs", fn);
  if (x_dtype != BL_F32 && x_dtype != BL_BF16)
    return fail(BL_ERR_DTYPE, "%s: unknown x_dtype %d", fn, x_dtype);
  if (bl_status rc = check_counts(fn, r.T, r.k, r.E)) return rc;
  if (bl_status rc = check_k(fn, K)) return rc;
  if (N < 1 || N > kMaxN / 2 || 2 * N * K > kMaxNK / r.E || r.T * r.k > kMaxTN / (2 * N))
    return fail(BL_ERR_SHAPE, "%s: N=%lld out of range", fn, (long long)N);
  if (!aligned(x, 16) || !aligned(packed_gu, 16) || !aligned(xq, 16) || !aligned(gamma_gate, 4) ||
      !aligned(gamma_up, 4) || !aligned(absmax, 4) || !aligned(h, 2) || !aligned(acc, 4) ||
      !aligned(r.offsets, 4) || !aligned(r.pairs, 4))
    return fail(BL_ERR_ALIGN, "%s: x, packed_gu and xq need 16-byte, h 2-byte, the others "
                "4-byte alignment", fn);
  return launched(fn, bl::launch_gated_experts(r, x, x_dtype == BL_BF16, packed_gu, gamma_gate,
                                               gamma_up, 2 * N, K, h, xq, absmax, acc,
                                               static_cast<hipStream_t>(stream)));
}

size_t bitlinear_experts_workspace_bytes(int64_t T, int64_t k, int64_t N) {
  if (T < 1 || T > kMaxT || k < 1 || k > BITLINEAR_MAX_TOP_K || N < 1 || T * k > kMaxTN / N) return 0;
  return (size_t)T * (size_t)k * (size_t)N * sizeof(float);
}

bl_status bitlinear_linear_experts(const bl_routing* routing, const void* x, int x_dtype,
                                   int x_rows, const uint8_t* packed, const float* gamma,
                                   int64_t N, int64_t K, float* y, int y_rows, int8_t* xq,
                                   float* absmax, int32_t* acc, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const char* fn = "bitlinear_linear_experts";
  if (!routing || !x || !packed || !gamma || !y || !xq || !absmax)
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  const bl_routing& r = *routing;
  if (x_rows != BL_ROWS_TOKENS && x_rows != BL_ROWS_SLOTS)
    return fail(BL_ERR_ARG, "%s: unknown x_rows %d", fn, x_rows);
  if (y_rows != BL_ROWS_TOKENS && y_rows != BL_ROWS_SLOTS)
    return fail(BL_ERR_ARG, "%s: unknown y_rows %d", fn, y_rows);
  const bool combine = y_rows == BL_ROWS_TOKENS;
  if (!r.offsets || !r.pairs || (combine && (!r.slots || !r.weights)))
    return fail(BL_ERR_NULL, "%s: NULL offsets, pairs, slots or weights", fn);
  if (combine && acc)
    return fail(BL_ERR_ARG, "%s: acc is per slot (BL_ROWS_SLOTS outputs only)", fn);
  if (x_dtype != BL_F32 && x_dtype != BL_BF16)
    return fail(BL_ERR_DTYPE, "%s: unknown x_dtype %d", fn, x_dtype);
  if (bl_status rc = check_counts(fn, r.T, r.k, r.E)) return rc;
  if (bl_status rc = check_k(fn, K)) return rc;
  if (N < 1 || N > kMaxN || N * K > kMaxNK / r.E || r.T * r.k > kMaxTN / N)
    return fail(BL_ERR_SHAPE, "%s: N=%lld out of range", fn, (long long)N);
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(xq, 16) || !aligned(gamma, 4) ||
      !aligned(y, 4) || !aligned(absmax, 4) || !aligned(acc, 4) || !aligned(workspace, 16) ||
      !aligned(r.offsets, 4) || !aligned(r.pairs, 4) ||
      (combine && (!aligned(r.slots, 4) || !aligned(r.weights, 4))))
    return fail(BL_ERR_ALIGN, "%s: x, packed, xq and workspace need 16-byte, the others "
                "4-byte alignment", fn);
  if (combine) {
    if (!workspace) return fail(BL_ERR_NULL, "%s: NULL workspace", fn);
    const size_t need = bitlinear_experts_workspace_bytes(r.T, r.k, N);
    if (workspace_bytes < need)
      return fail(BL_ERR_WORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes, need);
  }
  return launched(fn, bl::launch_linear_experts(r, x, x_dtype == BL_BF16, x_rows, packed, gamma, N,
                                                K, y, y_rows, xq, absmax, acc,
                                                static_cast<float*>(workspace),
                                                static_cast<hipStream_t>(stream)));
}

size_t bitlinear_experts_ffn_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t F, int64_t K,
                                             int64_t N) {
  if (T < 1 || T > kMaxT || E < 1 || E > BITLINEAR_MAX_EXPERTS || k < 1 || k > BITLINEAR_MAX_TOP_K ||
      F < 1 || F > BITLINEAR_MAX_K || K < 1 || K > BITLINEAR_MAX_K || N < 1 || N > kMaxN ||
      T * k > kMaxTN / N || T * k > kMaxTN / (2 * F))
    return 0;
  return bl::layer_workspace_bytes(T, E, k, F, K, N);
}

bl_status bitlinear_experts_ffn(const void* logits, int logits_dtype, int64_t T, int64_t E,
                                int64_t k, int share, const void* x, int x_dtype,
                                const float* absmax, const uint8_t* packed_gu,
                                const float* gamma_gate, const float* gamma_up, int64_t F,
                                int64_t K, const uint8_t* packed_down, const float* gamma_down,
                                int64_t N, float* y, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const char* fn = "bitlinear_experts_ffn";
  // sizes first: the workspace query answers 0 for those out of range, so that there may be none
  if (bl_status rc = check_counts(fn, T, k, E)) return rc;
  if (bl_status rc = check_k(fn, K)) return rc;
  if (F < 16 || F > BITLINEAR_MAX_K || F % 16 != 0 || 2 * F * K > kMaxNK / E ||
      T * k > kMaxTN / (2 * F))
    return fail(BL_ERR_SHAPE, "%s: F=%lld must be a multiple of 16 in [16, %d], with E*2F*K up to 2^38 "
                "and T*k*2F up to 2^36", fn, (long long)F, BITLINEAR_MAX_K);
  if (N < 1 || N > kMaxN || N * F > kMaxNK / E || T * k > kMaxTN / N)
    return fail(BL_ERR_SHAPE, "%s: N=%lld out of range", fn, (long long)N);
  if (!logits || !x || !packed_gu || !gamma_gate || !gamma_up || !packed_down || !gamma_down || !y ||
      !workspace || (x_dtype == BL_CODES && !absmax))
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (logits_dtype != BL_F32 && logits_dtype != BL_BF16)
    return fail(BL_ERR_DTYPE, "%s: unknown logits_dtype %d", fn, logits_dtype);
  if (x_dtype != BL_F32 && x_dtype != BL_BF16 && x_dtype != BL_CODES)
    return fail(BL_ERR_DTYPE, "%s: unknown x_dtype %d", fn, x_dtype);
  if (x_dtype != BL_CODES && absmax)
    return fail(BL_ERR_ARG, "%s: absmax belongs to int8 codes (BL_CODES)", fn);
  if (share != BL_SHARE_CHOSEN && share != BL_SHARE_ALL)
    return fail(BL_ERR_ARG, "%s: unknown share %d (BL_SHARE_CHOSEN or BL_SHARE_ALL)", fn, share);
  if (!aligned(x, 16) || !aligned(packed_gu, 16) || !aligned(packed_down, 16) ||
      !aligned(workspace, 16) || !aligned(logits, logits_dtype == BL_F32 ? 4 : 2) ||
      !aligned(absmax, 4) || !aligned(gamma_gate, 4) || !aligned(gamma_up, 4) ||
      !aligned(gamma_down, 4) || !aligned(y, 4))
    return fail(BL_ERR_ALIGN, "%s: x, the packed matrices and workspace need 16-byte, logits their "
                "dtype's, the others 4-byte alignment", fn);
  const size_t need = bl::layer_workspace_bytes(T, E, k, F, K, N);
  if (workspace_bytes < need)
    return fail(BL_ERR_WORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, workspace_bytes, need);
  return launched(fn, bl::launch_layer({logits, x, absmax, packed_gu, packed_down, gamma_gate,
                                        gamma_up, gamma_down, T, E, k, F, K, N, y, workspace,
                                        logits_dtype == BL_BF16, share, x_dtype},
                                       static_cast<hipStream_t>(stream)));
}

int64_t bitlinear_w4_row_bytes(int64_t K) { return K < 1 ? 0 : bl::w4_row_bytes(K); }

bl_status bitlinear_pack_weights_w4(const float* w, int64_t N, int64_t K, int64_t G,
                                    uint8_t* packed, uint16_t* scales, int8_t* zeros,
                                    void* stream) {
  const char* fn = "bitlinear_pack_weights_w4";
  if (!w || !packed || !scales) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_group(fn, N, K, G)) return rc;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 2))
    return fail(BL_ERR_ALIGN, "%s: w and packed need 16-byte, scales 2-byte alignment", fn);
  return launched(fn, bl::launch_pack_w4(w, N, K, (int)G, packed, scales, zeros,
                                         static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_unpack_weights_w4(const uint8_t* packed, const uint16_t* scales,
                                      const int8_t* zeros, int64_t N, int64_t K, int64_t G,
                                      float* w, void* stream) {
  const char* fn = "bitlinear_unpack_weights_w4";
  if (!w || !packed || !scales) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_group(fn, N, K, G)) return rc;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 2))
    return fail(BL_ERR_ALIGN, "%s: w and packed need 16-byte, scales 2-byte alignment", fn);
  return launched(fn, bl::launch_unpack_w4(packed, scales, zeros, N, K, (int)G, w,
                                           static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_forward_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                               const int8_t* xq, const float* absmax, int64_t T, int64_t N,
                               int64_t K, int64_t G, float* y, void* stream) {
  const char* fn = "bitlinear_forward_w4";
  if (!packed || !scales || !xq || !absmax || !y)
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_group(fn, N, K, G)) return rc;
  if (T < 1 || T > kMaxT || T > kMaxTN / N)
    return fail(BL_ERR_SHAPE, "%s: T=%lld out of range", fn, (long long)T);
  if (!aligned(packed, 16) || !aligned(scales, 2) || !aligned(xq, 16) || !aligned(absmax, 4) ||
      !aligned(y, 4))
    return fail(BL_ERR_ALIGN, "%s: packed and xq need 16-byte, scales 2-byte, the others 4-byte "
                "alignment", fn);
  return launched(fn, bl::launch_forward_w4(packed, scales, zeros, xq, absmax, T, N, K, (int)G, y,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
