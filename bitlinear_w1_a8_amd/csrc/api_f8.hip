// C ABI of the residual norms and of the 8-bit floating point products
// (declared in include/bitlinear_norm.h and include/bitlinear_f8.h): argument
// checks on the host, then kernel launches on the caller's stream.
#include <math.h>

#include "api_util.h"
#include "f8.h"

using bl::aligned;
using bl::check_k;
using bl::fail;
using bl::kMaxN;
using bl::kMaxNK;
using bl::kMaxT;
using bl::kMaxTN;
using bl::launched;

namespace {

bl_status check_dtype(const char* fn, const char* what, int dtype) {
  if (dtype != BL_F32 && dtype != BL_BF16)
    return fail(BL_ERR_DTYPE, "%s: unknown %s %d", fn, what, dtype);
  return BL_OK;
}

bl_status check_t(const char* fn, int64_t t) {
  if (t < 1 || t > kMaxT) return fail(BL_ERR_SHAPE, "%s: T=%lld out of range", fn, (long long)t);
  return BL_OK;
}

bl_status check_matrix(const char* fn, int64_t n, int64_t k) {
  if (bl_status rc = check_k(fn, k)) return rc;
  if (n < 1 || n > kMaxN || n * k > kMaxNK)
    return fail(BL_ERR_SHAPE, "%s: N=%lld out of range", fn, (long long)n);
  return BL_OK;
}

bl_status norm(const char* fn, const bl::NormCall& c, int x_dtype, int r_dtype, hipStream_t stream) {
  if (!c.x || !c.gain || !c.xq || !c.scale || (c.residual && !c.total))
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (!c.residual && c.total) return fail(BL_ERR_ARG, "%s: total without a residual", fn);
  if (bl_status rc = check_dtype(fn, "x_dtype", x_dtype)) return rc;
  if (c.residual)
    if (bl_status rc = check_dtype(fn, "r_dtype", r_dtype)) return rc;
  if (!(c.eps_n > 0.0f) || !isfinite(c.eps_n))
    return fail(BL_ERR_ARG, "%s: eps_n must be finite and > 0", fn);
  if (bl_status rc = check_t(fn, c.T)) return rc;
  if (bl_status rc = check_k(fn, c.K)) return rc;
  if (!aligned(c.x, 16) || !aligned(c.residual, 16) || !aligned(c.gain, 16) ||
      !aligned(c.total, 16) || !aligned(c.xq, 16) || !aligned(c.scale, 4) || !aligned(c.rowsum, 4))
    return fail(BL_ERR_ALIGN, "%s: x, residual, gain, total and xq need 16-byte, the others "
                "4-byte alignment", fn);
  return launched(fn, bl::launch_add_subln(c, stream));
}

bl_status check_product(const char* fn, const uint8_t* w, const float* w_scales, const uint8_t* xq,
                        const float* x_scales, int64_t t, int64_t n, int64_t k, const void* y,
                        int y_dtype) {
  if (!w || !w_scales || !xq || !x_scales || !y)
    return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (y_dtype != (BL_BF16 | BL_CUT_SUMS))
    if (bl_status rc = check_dtype(fn, "y_dtype", y_dtype)) return rc;
  if (bl_status rc = check_matrix(fn, n, k)) return rc;
  if (t < 1 || t > kMaxT || t > kMaxTN / n)
    return fail(BL_ERR_SHAPE, "%s: T=%lld out of range", fn, (long long)t);
  if (!aligned(w, 16) || !aligned(xq, 16) || !aligned(w_scales, 4) || !aligned(x_scales, 4) ||
      !aligned(y, y_dtype == BL_F32 ? 4 : 2))
    return fail(BL_ERR_ALIGN, "%s: w and xq need 16-byte, the scales 4-byte alignment, y its "
                "element's", fn);
  return BL_OK;
}

}  // namespace

extern "C" {

bl_status bitlinear_add_subln_quant_act(const void* x, int x_dtype, const void* residual,
                                        int r_dtype, const float* gain, float eps_n, int64_t T,
                                        int64_t K, void* total, int8_t* xq, float* scale,
                                        int32_t* rowsum, void* stream) {
  const bl::NormCall c{x, residual, gain, eps_n, T, K, total, xq, scale, rowsum,
                       x_dtype == BL_BF16, r_dtype == BL_BF16, false};
  return norm("bitlinear_add_subln_quant_act", c, x_dtype, r_dtype, static_cast<hipStream_t>(stream));
}

bl_status bitlinear_add_subln_quant_act_f8(const void* x, int x_dtype, const void* residual,
                                           int r_dtype, const float* gain, float eps_n, int64_t T,
                                           int64_t K, void* total, uint8_t* xq, float* scales,
                                           void* stream) {
  const bl::NormCall c{x, residual, gain, eps_n, T, K, total, xq, scales, nullptr,
                       x_dtype == BL_BF16, r_dtype == BL_BF16, true};
  return norm("bitlinear_add_subln_quant_act_f8", c, x_dtype, r_dtype,
              static_cast<hipStream_t>(stream));
}

bl_status bitlinear_quant_act_f8(const void* x, int x_dtype, int64_t T, int64_t K, uint8_t* xq,
                                 float* scales, void* stream) {
  const char* fn = "bitlinear_quant_act_f8";
  if (!x || !xq || !scales) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_dtype(fn, "x_dtype", x_dtype)) return rc;
  if (bl_status rc = check_t(fn, T)) return rc;
  if (bl_status rc = check_k(fn, K)) return rc;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(scales, 4))
    return fail(BL_ERR_ALIGN, "%s: x and xq need 16-byte, scales 4-byte alignment", fn);
  return launched(fn, bl::launch_quant_f8(x, x_dtype == BL_BF16, T, K, xq, scales,
                                          static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_pack_weights_f8(const float* w, int64_t N, int64_t K, uint8_t* codes,
                                    float* scales, void* stream) {
  const char* fn = "bitlinear_pack_weights_f8";
  if (!w || !codes || !scales) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_matrix(fn, N, K)) return rc;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(BL_ERR_ALIGN, "%s: w and codes need 16-byte, scales 4-byte alignment", fn);
  return launched(fn, bl::launch_pack_f8(w, N, K, codes, scales, static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_unpack_weights_f8(const uint8_t* codes, const float* scales, int64_t N,
                                      int64_t K, float* w, void* stream) {
  const char* fn = "bitlinear_unpack_weights_f8";
  if (!w || !codes || !scales) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_matrix(fn, N, K)) return rc;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(BL_ERR_ALIGN, "%s: w and codes need 16-byte, scales 4-byte alignment", fn);
  return launched(fn, bl::launch_unpack_f8(codes, scales, N, K, w, static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_forward_f8(const uint8_t* w, const float* w_scales, const uint8_t* xq,
                               const float* x_scales, int64_t T, int64_t N, int64_t K, void* y,
                               int y_dtype, void* stream) {
  const char* fn = "bitlinear_forward_f8";
  if (bl_status rc = check_product(fn, w, w_scales, xq, x_scales, T, N, K, y, y_dtype)) return rc;
  return launched(fn, bl::launch_forward_f8(w, w_scales, xq, x_scales, T, N, K, y, y_dtype,
                                            static_cast<hipStream_t>(stream)));
}

bl_status bitlinear_linear_f8(const void* x, int x_dtype, const uint8_t* w, const float* w_scales,
                              int64_t T, int64_t N, int64_t K, uint8_t* xq, float* x_scales,
                              void* y, int y_dtype, void* stream) {
  const char* fn = "bitlinear_linear_f8";
  if (!x) return fail(BL_ERR_NULL, "%s: NULL pointer argument", fn);
  if (bl_status rc = check_dtype(fn, "x_dtype", x_dtype)) return rc;
  if (bl_status rc = check_product(fn, w, w_scales, xq, x_scales, T, N, K, y, y_dtype)) return rc;
  if (!aligned(x, 16)) return fail(BL_ERR_ALIGN, "%s: x needs 16-byte alignment", fn);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = bl::launch_quant_f8(x, x_dtype == BL_BF16, T, K, xq, x_scales, s);
  if (e == hipSuccess)
    e = bl::launch_forward_f8(w, w_scales, xq, x_scales, T, N, K, y, y_dtype, s);
  return launched(fn, e);
}

}  // extern "C"
