// Products of e4m3 tokens with e4m3 matrices, one scale per block of 128, and
// the quantisation of matrices.
//
// A block of 128 along K is summed from a zero accumulator; its binary32 sums
// are then multiplied by the token's scale times the block's and added in
// binary32.  The operands' order along K does not matter as long as both use
// the same one, so a lane takes whole 16-byte pieces of its row.
//
// Two kinds of matrix instruction.  The e4m3 ones (v_mfma_f32_32x32x64_f8f6f4, 2048
// multiply-adds per cycle and SIMD counted as flops) add the products of eight
// neighbouring k with what lies 2^14 and more below the largest of the eight cut
// off, measured on 16x16x128, 16x16x32, 32x32x64 and 32x32x16 alike: a sum is off by up
// to 7 * 2^-13 of its magnitudes' sum (seen: 2^-12.7; 4e-5 to 5e-5 in the norm), more
// than a binary32 result may be and a fortieth of what its rounding to bfloat16
// costs.  The f16 ones at half the rate hold every e4m3 exactly and add in binary32
// (8e-8 in the norm).  So binary32 outputs, and batches that the stream of
// weights bounds, take the f16 ones; bfloat16 outputs of many tokens the e4m3 ones.
#include <algorithm>
#include <type_traits>

#include "f8.h"

namespace bl {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* glb_ptr_t;

// 32 x 32 x 64 product of e4m3 operands (no hardware scales: those are powers of two).
__device__ __forceinline__ v16f mfma32(const v8i& a, const v8i& b, const v16f& c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// The eight e4m3 codes of two words as binary16, exact.
__device__ __forceinline__ v8h halves8(uint32_t lo, uint32_t hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ v8i operand8(const uint4& a, const uint4& b) {
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Four outputs n .. n + 3 of a token; n + i < N is checked where the last are cut off.
template <bool BF16>
__device__ __forceinline__ void store4(void* y, int64_t at, int n, int N, const float (&v)[4]) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(y) + at + n;
    const uint32_t a = bf16_pair(v[0], v[1]), b = bf16_pair(v[2], v[3]);
    if ((N & 3) == 0 && n < N) {
      *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
    } else {
      if (n < N) p[0] = (uint16_t)a;
      if (n + 1 < N) p[1] = (uint16_t)(a >> 16);
      if (n + 2 < N) p[2] = (uint16_t)b;
      if (n + 3 < N) p[3] = (uint16_t)(b >> 16);
    }
  } else {
    float* p = static_cast<float*>(y) + at + n;
    if ((N & 3) == 0 && n < N) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) p[i] = v[i];
    }
  }
}

// ------------------------------------------------------------------ few tokens

// Up to 16 TT tokens against 16 RT rows per block; the block's waves take the
// blocks of K in turn and their sums meet in LDS, added in order of the waves.
// Every load goes straight to registers, U blocks of K ahead.
constexpr int kFewWaves = 4;

template <int TT, int RT, int U, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_f8_few(const uint8_t* __restrict__ w,
                                                           const float* __restrict__ ws,
                                                           const uint8_t* __restrict__ xq,
                                                           const float* __restrict__ xs, int T,
                                                           int N, int K, void* __restrict__ y) {
  __shared__ float red[kFewWaves][RT * TT][4][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb_all = (K + kF8Block - 1) / kF8Block;
  const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * TT;
  const float* wsr = ws + (int64_t)(n0 / kF8Block) * kb_all;
  const uint8_t* wrow[RT];
  const uint8_t* xrow[TT];
  int tok[TT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = w + (int64_t)min(n0 + 16 * i + r, N - 1) * K;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    tok[j] = min(t0 + 16 * j + r, T - 1);
    xrow[j] = xq + (int64_t)tok[j] * K;
  }
  struct Buf {
    uint4 a[RT][2], b[TT][2];
    float s[TT], ws;
  };
  auto load = [&](Buf& f, int kb) {
    kb = min(kb, kb_all - 1);
    const int k0 = min(kb * kF8Block + 32 * g, K - 16), k1 = min(kb * kF8Block + 32 * g + 16, K - 16);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      f.a[i][0] = *reinterpret_cast<const uint4*>(wrow[i] + k0);
      f.a[i][1] = *reinterpret_cast<const uint4*>(wrow[i] + k1);
    }
    f.ws = wsr[kb];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      f.b[j][0] = *reinterpret_cast<const uint4*>(xrow[j] + k0);
      f.b[j][1] = *reinterpret_cast<const uint4*>(xrow[j] + k1);
      f.s[j] = xs[(int64_t)kb * T + tok[j]];
    }
  };
  v4f acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  Buf buf[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load(buf[u], wave + u * kFewWaves);
  for (int k0 = wave; k0 < kb_all; k0 += U * kFewWaves) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * kFewWaves;
      if (kb >= kb_all) break;
      Buf f = buf[u];
      if (kb + U * kFewWaves < kb_all) load(buf[u], kb + U * kFewWaves);
      if ((kb + 1) * kF8Block > K) {           // tokens are zero past K
        const int k = kb * kF8Block + 32 * g;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          if (k >= K) f.b[j][0] = make_uint4(0, 0, 0, 0);
          if (k + 16 >= K) f.b[j][1] = make_uint4(0, 0, 0, 0);
        }
      }
      v4f p[RT][TT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) p[i][j] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {            // 32 k: eight per lane
        auto part = [&](const uint4 (&v)[2]) {
          return q & 1 ? halves8(v[q >> 1].z, v[q >> 1].w) : halves8(v[q >> 1].x, v[q >> 1].y);
        };
        v8h a[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) a[i] = part(f.a[i]);
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const v8h b = part(f.b[j]);
#pragma unroll
          for (int i = 0; i < RT; ++i)
            p[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i], b, p[i][j], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const float s = f.s[j] * f.ws;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[i][j][v], s, acc[i][j][v]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][i * TT + j][v][lane] = acc[i][j][v];
  lds_sync();
  // lane (g, r): rows 4 g .. 4 g + 3 of token r of a tile
  for (int q = wave; q < RT * TT; q += kFewWaves) {
    const int t = t0 + 16 * (q % TT) + r;
    float s[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      s[v] = red[0][q][v][lane];
#pragma unroll
      for (int p = 1; p < kFewWaves; ++p) s[v] += red[p][q][v][lane];
    }
    if (t < T) store4<BF16>(y, (int64_t)t * N, n0 + 16 * (q / TT) + 4 * g, N, s);
  }
}

// ------------------------------------------------------------------ many tokens

// 16 zero bytes, read in place of what lies past K.
__device__ __align__(16) uint8_t kZeros[16];

// 128 rows x 128 tokens per block, four waves of 64 x 64, one block of K per
// step through two LDS buffers filled directly from memory.  In a buffer, row r
// has its eight 16-byte pieces at 128 r, piece c at place c ^ (r & 7), so that
// eight lanes reading one piece of eight rows reach all banks.
// NATIVE: e4m3 instructions; else each wave widens its operands to f16.
template <bool BF16, bool NATIVE>
__global__ __launch_bounds__(256) void k_f8_tile(const uint8_t* __restrict__ w,
                                                 const float* __restrict__ ws,
                                                 const uint8_t* __restrict__ xq,
                                                 const float* __restrict__ xs, int T, int N, int K,
                                                 int t_tiles, int tiles, void* __restrict__ y) {
  __shared__ __align__(16) uint8_t lds[2][2][128 * 128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb_all = (K + kF8Block - 1) / kF8Block;
  // block b runs on XCD b % 8: each gets a run of neighbouring tiles
  const int per = (tiles + 7) / 8;
  const int item = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (blockIdx.x / 8 >= per || item >= tiles) return;
  const int n0 = item / t_tiles * 128, t0 = item % t_tiles * 128;
  const float* wsr = ws + (int64_t)(n0 / kF8Block) * kb_all;

  // rows of this wave's loads: 8 per instruction, four instructions per operand
  const int lr = lane >> 3, piece = (lane & 7) ^ lr;
  const uint8_t* src[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = wave * 32 + i * 8 + lr;
    src[0][i] = w + (int64_t)min(n0 + row, N - 1) * K;
    src[1][i] = xq + (int64_t)min(t0 + row, T - 1) * K;
  }
  auto fetch = [&](int b, int kb) {
    const int k = kb * kF8Block + 16 * piece;
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = k < K ? src[o][i] + k : kZeros;
        __builtin_amdgcn_global_load_lds((glb_ptr_t)p, (lds_ptr_t)(&lds[b][o][(wave * 32 + i * 8) * 128]),
                                         16, 0, 0);
      }
  };
  const int h = lane >> 5, c = lane & 31;
  const int wr = (wave >> 1) * 64, wt = (wave & 1) * 64;
  const int tok[2] = {min(t0 + wt + c, T - 1), min(t0 + wt + 32 + c, T - 1)};
  v16f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  fetch(0, 0);
  for (int kb = 0; kb < kb_all; ++kb) {
    const int b = kb & 1;
    float s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j] = xs[(int64_t)kb * T + tok[j]] * wsr[kb];
    wait_vmem<0>();
    lds_sync();                                     // buffer b is whole, the other one is free
    if (kb + 1 < kb_all) fetch(b ^ 1, kb + 1);
    uint4 fa[2][4], fb[2][4];
    auto frag = [&](const uint8_t* base, int row, uint4 (&f)[4]) {
      const uint8_t* p = base + row * 128;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f[q] = *reinterpret_cast<const uint4*>(p + 16 * ((2 * q + h) ^ (row & 7)));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      frag(lds[b][0], wr + 32 * i + c, fa[i]);
      frag(lds[b][1], wt + 32 * i + c, fb[i]);
    }
    if constexpr (NATIVE) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v16f p = {};
          p = mfma32(operand8(fa[i][0], fa[i][1]), operand8(fb[j][0], fb[j][1]), p);
          p = mfma32(operand8(fa[i][2], fa[i][3]), operand8(fb[j][2], fb[j][3]), p);
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(p[v], s[j], acc[i][j][v]);
        }
    } else {
      v16f p[2][2] = {};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        auto part = [&](const uint4 (&v)[4]) {
          return q & 1 ? halves8(v[q >> 1].z, v[q >> 1].w) : halves8(v[q >> 1].x, v[q >> 1].y);
        };
        const v8h a[2] = {part(fa[0]), part(fa[1])}, bb[2] = {part(fb[0]), part(fb[1])};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            p[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], bb[j], p[i][j], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(p[i][j][v], s[j], acc[i][j][v]);
    }
  }
  // lane (h, c): token c, rows 8 q + 4 h + v of a 32 x 32 tile
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = t0 + wt + 32 * j + c;
      if (t >= T) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        store4<BF16>(y, (int64_t)t * N, n0 + wr + 32 * i + 8 * q + 4 * h, N, v);
      }
    }
}

// ------------------------------------------------------------------ matrices

// One block of 128 x 128 per workgroup, in registers between the maximum and
// the codes: 32 lanes have a row's 512 bytes.
__global__ __launch_bounds__(256) void k_pack_f8(const float* __restrict__ w, int64_t N, int K,
                                                 int kb_all, int64_t units,
                                                 uint8_t* __restrict__ codes,
                                                 float* __restrict__ scales) {
  __shared__ int most[4];
  const int tid = threadIdx.x;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t nb = u / kb_all;
    const int kb = (int)(u - nb * kb_all), k = kb * kF8Block + 4 * (tid & 31);
    const int64_t n0 = nb * kF8Block + (tid >> 5);
    float4 v[16];
    int m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t n = n0 + 8 * i;
      v[i] = make_float4(0, 0, 0, 0);
      if (n < N && k < K) v[i] = *reinterpret_cast<const float4*>(w + n * K + k);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      m = max(m, max((int)(__float_as_uint(v[i].x) & 0x7fffffffu), (int)(__float_as_uint(v[i].y) & 0x7fffffffu)));
      m = max(m, max((int)(__float_as_uint(v[i].z) & 0x7fffffffu), (int)(__float_as_uint(v[i].w) & 0x7fffffffu)));
    }
    m = wave_max_nonneg(m);
    __syncthreads();                                 // the last round's maxima have been read
    if ((tid & 63) == 0) most[tid >> 6] = m;
    __syncthreads();
    m = max(max(most[0], most[1]), max(most[2], most[3]));
    const float top = fmaxf(__int_as_float(m), kF8Floor), inv = kF8Top / top;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t n = n0 + 8 * i;
      if (n < N && k < K)
        *reinterpret_cast<uint32_t*>(codes + n * K + k) = f8_codes4(v[i].x, v[i].y, v[i].z, v[i].w, inv);
    }
    if (tid == 0) scales[u] = top / kF8Top;
  }
}

__global__ __launch_bounds__(256) void k_unpack_f8(const uint32_t* __restrict__ codes,
                                                   const float* __restrict__ scales, int64_t units,
                                                   int K, int kb_all, float4* __restrict__ w) {
  const int k4 = K >> 2;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t n = u / k4;
    const int k = 4 * (int)(u - n * k4);
    const float s = scales[n / kF8Block * kb_all + k / kF8Block];
    const int c = (int)codes[u];
    const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
    w[u] = make_float4(lo[0] * s, lo[1] * s, hi[0] * s, hi[1] * s);
  }
}

template <bool BF16>
hipError_t forward(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs, int64_t t,
                   int64_t n, int64_t k, void* y, hipStream_t stream) {
  if (t <= 64) {
    const dim3 grid((unsigned)((n + 31) / 32), 1);
    auto* f = t <= 16 ? k_f8_few<1, 2, 4, BF16> : t <= 32 ? k_f8_few<2, 2, 2, BF16> : k_f8_few<4, 2, 2, BF16>;
    f<<<grid, 64 * kFewWaves, 0, stream>>>(w, ws, xq, xs, (int)t, (int)n, (int)k, y);
    return hipGetLastError();
  }
  // T * N <= 2^36: at most 2^23 tiles, 2^31 threads
  const int t_tiles = (int)((t + 127) / 128), tiles = (int)((n + 127) / 128 * t_tiles);
  k_f8_tile<BF16, BF16><<<(unsigned)((tiles + 7) / 8 * 8), 256, 0, stream>>>(
      w, ws, xq, xs, (int)t, (int)n, (int)k, t_tiles, tiles, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_forward_f8(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs,
                             int64_t t, int64_t n, int64_t k, void* y, int bf16,
                             hipStream_t stream) {
  return bf16 ? forward<true>(w, ws, xq, xs, t, n, k, y, stream)
              : forward<false>(w, ws, xq, xs, t, n, k, y, stream);
}

hipError_t launch_pack_f8(const float* w, int64_t n, int64_t k, uint8_t* codes, float* scales,
                          hipStream_t stream) {
  const int kb = (int)f8_blocks(k);
  const int64_t units = f8_blocks(n) * kb;
  k_pack_f8<<<(unsigned)std::min<int64_t>(units, 1 << 20), 256, 0, stream>>>(w, n, (int)k, kb, units,
                                                                            codes, scales);
  return hipGetLastError();
}

hipError_t launch_unpack_f8(const uint8_t* codes, const float* scales, int64_t n, int64_t k,
                            float* w, hipStream_t stream) {
  const int64_t units = n * (k / 4);
  k_unpack_f8<<<(unsigned)std::min<int64_t>((units + 255) / 256, 1 << 16), 256, 0, stream>>>(
      reinterpret_cast<const uint32_t*>(codes), scales, units, (int)k, (int)f8_blocks(k),
      reinterpret_cast<float4*>(w));
  return hipGetLastError();
}

}  // namespace bl
