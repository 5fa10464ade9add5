// 4-bit weights with one bfloat16 scale per group of a row: packing, unpacking
// and the product with int8 tokens (W4A8).
//
// Product.  A masked nibble, left in the high half of its byte, is 16 t as an
// int8: (w << 4) & 0xF0F0F0F0 and w & 0xF0F0F0F0 turn a packed word into eight
// consecutive k of MFMA operand in three VALU operations, with no table and no
// offset to take off.  The int8 MFMA sums a group exactly; the sum is converted
// once per group and multiplied by the group's scale, 1/16 (a power of two)
// and the token's absmax / 127 follow in the epilogue.  Zero points need the
// group's sum of q as well, which one more MFMA against a matrix of ones
// gives, in the same lanes as the products.
//
// The tokens are the rows (A) and the weights the columns (B) of the 16 x 16
// result: every lane then works on one weight row, so it has one scale per
// group.
#include <algorithm>
#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

constexpr int kBlock = 128;      // weights per packed block (64 bytes)

__device__ __forceinline__ float bf16_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f_bf16(float f) {   // finite f >= 0, nearest even
  uint32_t b = __float_as_uint(f);
  b += 0x7FFFu + ((b >> 16) & 1u);
  return (uint16_t)(b >> 16);
}

// ------------------------------------------------------------------ packing

// Four neighbouring lanes hold one block of a row: lane q its 16-byte chunk,
// weights k = 32j + 8q + i.  A group of 32, 64 or 128 is one, two or four of
// the j over the four lanes.
template <int G, bool ZEROS>
__global__ __launch_bounds__(256) void k_pack_w4(const float* __restrict__ w, int64_t n, int K,
                                                 uint4* __restrict__ packed,
                                                 uint16_t* __restrict__ scales,
                                                 int8_t* __restrict__ zeros) {
  constexpr int GJ = G / 32, NG = 4 / GJ;           // words per group, groups per block
  const int blocks = (K + kBlock - 1) / kBlock, kg = K / G;
  const int64_t units = n * blocks * 4;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += step) {
    const int64_t b = u >> 2, row = b / blocks;
    const int q = (int)(u & 3), blk = (int)(b - row * blocks);
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = blk * kBlock + 32 * j + 8 * q;  // whole runs of 8 are in or out (K % 32 == 0)
      if (k < K) {
        const float4* src = reinterpret_cast<const float4*>(w + row * K + k);
        const float4 a = src[0], c = src[1];
        v[j][0] = a.x; v[j][1] = a.y; v[j][2] = a.z; v[j][3] = a.w;
        v[j][4] = c.x; v[j][5] = c.y; v[j][6] = c.z; v[j][7] = c.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      }
    }
    uint32_t word[4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float lo = 0.0f, hi = 0.0f;                   // of the weights and 0
#pragma unroll
      for (int j = g * GJ; j < (g + 1) * GJ; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo = fminf(lo, v[j][i]);
          hi = fmaxf(hi, v[j][i]);
        }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, d));
        hi = fmaxf(hi, __shfl_xor(hi, d));
      }
      const uint16_t sb = f_bf16(ZEROS ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
      const float s = bf16_f(sb);
      float z = 0.0f;
      if (ZEROS && s > 0.0f) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) - 8.0f;
      const int gi = blk * NG + g;
      if (q == 0 && gi < kg) {
        scales[row * kg + gi] = sb;
        if (ZEROS) zeros[row * kg + gi] = (int8_t)z;
      }
#pragma unroll
      for (int j = g * GJ; j < (g + 1) * GJ; ++j) {
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float t = s > 0.0f ? fminf(fmaxf(rintf(v[j][i] / s) + z, -8.0f), 7.0f) : 0.0f;
          if (blk * kBlock + 32 * j >= K) t = 0.0f;
          o |= ((uint32_t)(int)t & 15u) << (8 * (i & 3) + 4 * (i >> 2));
        }
        word[j] = o;
      }
    }
    packed[u] = make_uint4(word[0], word[1], word[2], word[3]);
  }
}

template <bool ZEROS>
__global__ __launch_bounds__(256) void k_unpack_w4(const uint4* __restrict__ packed,
                                                   const uint16_t* __restrict__ scales,
                                                   const int8_t* __restrict__ zeros, int64_t n,
                                                   int K, int G, float* __restrict__ w) {
  const int blocks = (K + kBlock - 1) / kBlock, kg = K / G;
  const int64_t units = n * blocks * 4;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += step) {
    const int64_t b = u >> 2, row = b / blocks;
    const int q = (int)(u & 3), blk = (int)(b - row * blocks);
    const uint4 p = packed[u];
    const uint32_t word[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = blk * kBlock + 32 * j + 8 * q;
      if (k >= K) continue;
      const int64_t gi = row * kg + k / G;
      const float s = bf16_f(scales[gi]);
      const int z = ZEROS ? zeros[gi] : 0;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int sh = 8 * (i & 3) + 4 * (i >> 2);
        const int t = (int)(word[j] << (28 - sh)) >> 28;
        f[i] = (float)(t - z) * s;
      }
      float4* dst = reinterpret_cast<float4*>(w + row * K + k);
      dst[0] = make_float4(f[0], f[1], f[2], f[3]);
      dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// ------------------------------------------------------------------ product

// Up to 16 tokens and 16 weight rows per block; the waves take the blocks of
// 128 k in turn and add their sums through LDS in order.
template <int G, bool ZEROS>
__global__ __launch_bounds__(256) void k_w4_rows(const uint4* __restrict__ packed,
                                                 const uint16_t* __restrict__ scales,
                                                 const int8_t* __restrict__ zeros,
                                                 const int8_t* __restrict__ xq,
                                                 const float* __restrict__ absmax, int T, int N,
                                                 int K, float* __restrict__ y) {
  constexpr int kWaves = 4;
  __shared__ float red[kWaves][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, r = lane & 15;
  const int blocks = (K + kBlock - 1) / kBlock, kg = K / G;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const int n = min(n0 + r, N - 1), t = min(t0 + r, T - 1);
  const uint4* wrow = packed + (int64_t)n * blocks * 4 + q;
  const int8_t* xrow = xq + (int64_t)t * K + 8 * q;
  const uint16_t* srow = scales + (int64_t)n * kg;
  const int8_t* zrow = ZEROS ? zeros + (int64_t)n * kg : nullptr;

  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = wave; b < blocks; b += kWaves) {
    const uint4 p = wrow[b * 4];
    const uint32_t word[4] = {p.x, p.y, p.z, p.w};
    uint2 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = b * kBlock + 32 * j;
      x[j] = k < K ? *reinterpret_cast<const uint2*>(xrow + k) : make_uint2(0, 0);
    }
    auto lo = [&](int j) { return (int)((word[j] << 4) & 0xF0F0F0F0u); };
    auto hi = [&](int j) { return (int)(word[j] & 0xF0F0F0F0u); };
    auto scaled = [&](const v4i& acc, const v4i& ones, int g) {
      const int gi = b * (kBlock / G) + g;
      if (gi >= kg) return;                           // past K: codes and tokens are 0
      const float s = bf16_f(srow[gi]);
      const int z = ZEROS ? 16 * zrow[gi] : 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int a = ZEROS ? acc[v] - z * ones[v] : acc[v];
        sum[v] = fmaf((float)a, s, sum[v]);
      }
    };
    if constexpr (G == 32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long a = (long)(((unsigned long)x[j].y << 32) | x[j].x);
        const long bb = (long)(((unsigned long)(uint32_t)hi(j) << 32) | (uint32_t)lo(j));
        v4i acc = {0, 0, 0, 0}, one = {0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, bb, acc, 0, 0, 0);
        if (ZEROS) one = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, 0x0101010101010101l, one, 0, 0, 0);
        scaled(acc, one, j);
      }
    } else {
      const v4i one8 = {0x01010101, 0x01010101, 0x01010101, 0x01010101};
      v4i acc = {0, 0, 0, 0}, one = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const v4i a = {(int)x[2 * i].x, (int)x[2 * i].y, (int)x[2 * i + 1].x, (int)x[2 * i + 1].y};
        const v4i bb = {lo(2 * i), hi(2 * i), lo(2 * i + 1), hi(2 * i + 1)};
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, bb, acc, 0, 0, 0);
        if (ZEROS) one = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, one8, one, 0, 0, 0);
        if (G == 64 || i == 1) {
          scaled(acc, one, G == 64 ? i : 0);
          acc = one = v4i{0, 0, 0, 0};
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][v][lane] = sum[v];
  __syncthreads();
  // lane 16 a + c of register v holds token 4a + v, weight row c
  const int tok = threadIdx.x >> 4, col = threadIdx.x & 15;
  if (t0 + tok >= T || n0 + col >= N) return;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += red[w][tok & 3][(tok >> 2) * 16 + col];
  const float m = fmaxf(absmax[t0 + tok], kEps) / kQb;
  y[(int64_t)(t0 + tok) * N + n0 + col] = s * (m * 0.0625f);
}

unsigned stream_grid(int64_t units) {
  return (unsigned)std::min<int64_t>((units + 255) / 256, 16 * (int64_t)device_cus());
}

template <typename F>
hipError_t by_group(int g, bool zeros, F&& f) {
  auto z = [&](auto gc) {
    if (zeros) f(gc, std::true_type{});
    else f(gc, std::false_type{});
  };
  if (g == 32) z(std::integral_constant<int, 32>{});
  else if (g == 64) z(std::integral_constant<int, 64>{});
  else z(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pack_w4(const float* w, int64_t n, int64_t k, int g, uint8_t* packed,
                          uint16_t* scales, int8_t* zeros, hipStream_t stream) {
  const unsigned grid = stream_grid(n * ((k + kBlock - 1) / kBlock) * 4);
  return by_group(g, zeros != nullptr, [&](auto gc, auto zc) {
    k_pack_w4<decltype(gc)::value, decltype(zc)::value><<<grid, 256, 0, stream>>>(
        w, n, (int)k, reinterpret_cast<uint4*>(packed), scales, zeros);
  });
}

hipError_t launch_unpack_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                            int64_t n, int64_t k, int g, float* w, hipStream_t stream) {
  const unsigned grid = stream_grid(n * ((k + kBlock - 1) / kBlock) * 4);
  const auto* p = reinterpret_cast<const uint4*>(packed);
  if (zeros) k_unpack_w4<true><<<grid, 256, 0, stream>>>(p, scales, zeros, n, (int)k, g, w);
  else k_unpack_w4<false><<<grid, 256, 0, stream>>>(p, scales, zeros, n, (int)k, g, w);
  return hipGetLastError();
}

hipError_t launch_forward_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                             const int8_t* xq, const float* absmax, int64_t t, int64_t n,
                             int64_t k, int g, float* y, hipStream_t stream) {
  // grid.y holds at most 65535 blocks: more tokens go in several launches
  for (int64_t t0 = 0; t0 < t; t0 += 65535 * 16) {
    const int64_t nt = std::min<int64_t>(t - t0, 65535 * 16);
    const dim3 grid((unsigned)((n + 15) / 16), (unsigned)((nt + 15) / 16));
    const hipError_t e = by_group(g, zeros != nullptr, [&](auto gc, auto zc) {
      k_w4_rows<decltype(gc)::value, decltype(zc)::value><<<grid, 256, 0, stream>>>(
          reinterpret_cast<const uint4*>(packed), scales, zeros, xq + t0 * k, absmax + t0, (int)nt,
          (int)n, (int)k, y + t0 * n);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bl
