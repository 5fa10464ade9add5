// Internal declarations of the residual norms and of the 8-bit floating point
// products.
#pragma once

#include "bitlinear_f8.h"
#include "bitlinear_norm.h"
#include "bl_internal.h"

namespace bl {

constexpr int kF8Block = 128;              // values per scale, along K and along N
constexpr float kF8Top = 448.0f;           // largest e4m3
constexpr float kF8Floor = 0x1p-100f;      // floor of a group's absmax: 448 / m stays finite

inline int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

// One norm call; residual NULL: none.  xq int8 with scale [T] and rowsum, or
// (f8) e4m3 with scale [groups, T].
struct NormCall {
  const void* x;
  const void* residual;
  const float* gain;
  float eps_n;
  int64_t T, K;
  void* total;
  void* xq;
  float* scale;
  int32_t* rowsum;
  bool x_bf16, r_bf16, f8;
};
hipError_t launch_add_subln(const NormCall& c, hipStream_t stream);

hipError_t launch_quant_f8(const void* x, int bf16, int64_t t, int64_t k, uint8_t* xq,
                           float* scales, hipStream_t stream);
hipError_t launch_pack_f8(const float* w, int64_t n, int64_t k, uint8_t* codes, float* scales,
                          hipStream_t stream);
hipError_t launch_unpack_f8(const uint8_t* codes, const float* scales, int64_t n, int64_t k,
                            float* w, hipStream_t stream);
hipError_t launch_forward_f8(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs,
                             int64_t t, int64_t n, int64_t k, void* y, int y_dtype,
                             hipStream_t stream);   // y_dtype with or without BL_CUT_SUMS

// ---------------------------------------------------------------- device helpers

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Two binary32 values as bfloat16 (nearest, ties to even), the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}

// Eight consecutive activations widened to binary32: one 16-byte load of
// bfloat16, or two of binary32.
template <bool BF16>
struct Vec8 {
  uint4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(row) +
                                                    at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          f[2 * j] = __uint_as_float(w[j] << 16);
          f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          f[4 * i + j] = __uint_as_float(w[j]);
        }
      }
    }
  }
};

// Largest |f| of eight as a bit pattern (patterns of magnitudes order like their values).
__device__ __forceinline__ int absmax8(const float (&f)[8]) {
  int m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, (int)(__float_as_uint(f[i]) & 0x7fffffffu));
  return m;
}

// Maximum over the 16 lanes of a DPP row, in each of them.
__device__ __forceinline__ int row_max16(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false));  // row_mirror
  return v;
}

// Four values times `inv` as e4m3 codes in one word: one binary32 product each,
// then nearest even.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return (uint32_t)w;
}

}  // namespace bl
