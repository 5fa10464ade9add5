// Device code shared by the kernels for a few routed rows: raw activations and
// step A1, and the contraction of 16 weight rows with rows in LDS.
#pragma once

#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

enum Mode { kInt8 = 0, kBf16 = 1, kF32 = 2 };

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* glb_ptr_t;

// Four raw activations (elements k .. k + 3 of a row) as loaded, and widened
// to binary32.
template <int MODE>
struct Raw4 {
  std::conditional_t<MODE == kBf16, uint2, uint4> v;
  __device__ __forceinline__ void load(const void* row, int k) {
    v = *reinterpret_cast<const decltype(v)*>(static_cast<const unsigned char*>(row) +
                                              (MODE == kBf16 ? 2 : 4) * k);
  }
  __device__ __forceinline__ void clear() { v = {}; }
  __device__ __forceinline__ void widen(float (&f)[4]) const {
    if constexpr (MODE == kBf16) {
      f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
      f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
      f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
      f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
  }
  __device__ __forceinline__ int max_bits() const {   // of magnitudes, which order as ints
    float f[4];
    widen(f);
    int m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, (int)(__float_as_uint(f[i]) & 0x7fffffffu));
    return m;
  }
};

// Step A1 of four activations, as the act-quant kernel: one binary32 product,
// half to even, clipped; the codes in one word.
template <int MODE>
__device__ __forceinline__ uint32_t quant4(const Raw4<MODE>& raw, float s) {
  float f[4];
  raw.widen(f);
  int q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = (int)fminf(fmaxf(rintf(f[i] * s), -kQb), kQb);
  const uint32_t lo = __builtin_amdgcn_perm((uint32_t)q[1], (uint32_t)q[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm((uint32_t)q[3], (uint32_t)q[2], 0x04000c0cu);
  return lo | hi;
}

// Codes of a packed word as an MFMA operand.
__device__ __forceinline__ v4i operand(uint32_t w) {
  return v4i{(int)codes_of(w, 0), (int)codes_of(w, 1), (int)codes_of(w, 2), (int)codes_of(w, 3)};
}

// 16 weight rows (lane (qg, r) takes 64 k, 16 bytes, of row r per chunk) against
// up to 16 int8 rows in LDS over all of K; w holds the row's first U chunks and
// is filled again as it empties.  x: the lane's row, at 64 qg.
template <int U, int Q>
__device__ __forceinline__ v4i few_contract(uint4 (&w)[U], const uint32_t* wrow,
                                            const unsigned char* x, int qg, int K16, int nchunks) {
  v4i acc = {0, 0, 0, 0};
  for (int c0 = 0; c0 < nchunks; c0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u >= nchunks) break;
      const uint4* xv = reinterpret_cast<const uint4*>(x + (c0 + u) * 256);
      const uint4 p = settle<Q>(w[u], 16 * (c0 + u) + 4 * qg, K16);
      const uint32_t word[4] = {p.x, p.y, p.z, p.w};
      // the buffer's next chunk at once
      if (c0 + U + u < nchunks) w[u] = load_quad<Q>(wrow, 16 * (c0 + U + u) + 4 * qg, K16);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint4 q = xv[v];
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            operand(word[v]), v4i{(int)q.x, (int)q.y, (int)q.z, (int)q.w}, acc, 0, 0, 0);
      }
    }
  }
  return acc;
}

}  // namespace
}  // namespace bl
