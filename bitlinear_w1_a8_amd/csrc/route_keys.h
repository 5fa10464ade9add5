// Device code shared by the router and the whole routed layer: logits as keys,
// and reductions over a token's lanes.
#pragma once

#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

// unsigned key of a logit, growing with its value; 0 for -inf and NaN
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -__builtin_inff())) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);     // -0 becomes +0
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((int)key < 0 ? key & 0x7fffffffu : ~key);
}

// OP over the LANES lanes of a token (16 or 64), the result in each.
template <int LANES, typename T, typename OP>
__device__ __forceinline__ T over_lanes(T v, OP op) {
  static_assert(sizeof(T) == 4 && (LANES == 16 || LANES == 64), "one DPP row, or four");
  auto with = [&](auto ctrl) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                              0xF, 0xF, false);
    v = op(v, __builtin_bit_cast(T, o));
  };
  with(std::integral_constant<int, 0xB1>{});    // quad_perm 1,0,3,2
  with(std::integral_constant<int, 0x4E>{});    // quad_perm 2,3,0,1
  with(std::integral_constant<int, 0x141>{});   // row_half_mirror
  with(std::integral_constant<int, 0x140>{});   // row_mirror
  if constexpr (LANES == 64) {
    auto row = [&](int l) {
      return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    };
    v = op(op(row(0), row(16)), op(row(32), row(48)));
  }
  return v;
}

}  // namespace
}  // namespace bl
