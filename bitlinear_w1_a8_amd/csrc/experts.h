// Internal declarations of the routed-expert and 4-bit operators.
#pragma once

#include "bitlinear_experts.h"
#include "bitlinear_w4.h"
#include "bl_internal.h"

namespace bl {

// ---------------------------------------------------------------- router (route.hip)

constexpr int kRouteTokens = 64;   // tokens of a block: one bit each in an expert's mask

size_t route_workspace_bytes(int64_t t, int64_t e);
hipError_t launch_route(const void* logits, int bf16, int64_t t, int64_t e, int64_t k, int share,
                        int32_t* ids, float* weights, int32_t* offsets, int32_t* pairs,
                        int32_t* slots, int32_t* workspace, hipStream_t stream);

// ---------------------------------------------------------------- experts (experts.hip)

hipError_t launch_gated_experts(const bl_routing& r, const void* x, int bf16, const uint8_t* packed,
                                const float* gamma_gate, const float* gamma_up, int64_t n,
                                int64_t k, uint16_t* h, int8_t* xq, float* absmax, int32_t* acc,
                                hipStream_t stream);   // n: rows of gate and up together
hipError_t launch_linear_experts(const bl_routing& r, const void* x, int bf16, int x_rows,
                                 const uint8_t* packed, const float* gamma, int64_t n, int64_t k,
                                 float* y, int y_rows, int8_t* xq, float* absmax, int32_t* acc,
                                 float* workspace, hipStream_t stream);

// ---------------------------------------------------------------- 4-bit weights (w4.hip)

inline int64_t w4_row_bytes(int64_t k) { return (k + 127) / 128 * 64; }
hipError_t launch_pack_w4(const float* w, int64_t n, int64_t k, int g, uint8_t* packed,
                          uint16_t* scales, int8_t* zeros, hipStream_t stream);
hipError_t launch_unpack_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                            int64_t n, int64_t k, int g, float* w, hipStream_t stream);
hipError_t launch_forward_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                             const int8_t* xq, const float* absmax, int64_t t, int64_t n,
                             int64_t k, int g, float* y, hipStream_t stream);

}  // namespace bl
