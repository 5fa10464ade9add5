// 4-bit weights with one bfloat16 scale per group of a row: packing, unpacking
// and the product with int8 tokens (W4A8).
//
// Product.  A masked nibble, left in the high half of its byte, is 16 t as an
// int8: (w << 4) & 0xF0F0F0F0 and w & 0xF0F0F0F0 turn a packed word into eight
// consecutive k of MFMA operand in three VALU operations, with no table and no
// offset to take off.  The int8 MFMA sums a group exactly; the sum is converted
// once per group and multiplied by the group's scale; 1/16 (a power of two)
// and the token's absmax / 127 follow in the epilogue.  Zero points come off
// the codes, five more operations per word, as t - z still fits an int8.
//
// The tokens are the rows (A) and the weights the columns (B) of the 16 x 16
// result: every lane then works on one weight row, so it has one scale per
// group.
#include <algorithm>
#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float bf16_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f_bf16(float f) {   // finite f >= 0, nearest even
  uint32_t b = __float_as_uint(f);
  b += 0x7FFFu + ((b >> 16) & 1u);
  return (uint16_t)(b >> 16);
}

// ------------------------------------------------------------------ packing

// Four neighbouring lanes hold one block of a row: lane q its 16-byte chunk,
// weights k = 32j + 8q + i.  A group of 32, 64 or 128 is one, two or four of
// the j over the four lanes.  Bound by reading the weights (8192 x 28672: 0.94
// GB in 246-260 us, 4.1-4.3 TB/s in and out together, a copy's 4.75).
template <int G, bool ZEROS, typename INDEX>
__global__ __launch_bounds__(256) void k_pack_w4(const float* __restrict__ w, INDEX units, int K,
                                                 uint4* __restrict__ packed,
                                                 uint16_t* __restrict__ scales,
                                                 int8_t* __restrict__ zeros) {
  constexpr int GJ = G / 32, NG = 4 / GJ;           // words per group, groups per block
  const INDEX blocks = (INDEX)((K + kBlock - 1) / kBlock);
  const int kg = K / G;
  for (INDEX u = (INDEX)blockIdx.x * 256 + threadIdx.x; u < units; u += (INDEX)gridDim.x * 256) {
    const INDEX b = u >> 2;
    const int64_t row = b / blocks;
    const int q = (int)(u & 3), blk = (int)(b - (INDEX)row * blocks);
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

// Eight neighbouring lanes hold one block of a row, lane (q, p) the low (p = 0)
// or high nibbles of chunk q: per word j they write 128 consecutive bytes.
// Bound by these writes (8192 x 28672: 235-238 us, 4.5 TB/s in and out together).
// INDEX: a 32-bit unsigned type where it numbers all lanes.
template <bool ZEROS, typename INDEX>
__global__ __launch_bounds__(256) void k_unpack_w4(const uint4* __restrict__ packed,
                                                   const uint16_t* __restrict__ scales,
                                                   const int8_t* __restrict__ zeros, INDEX units,
                                                   int K, int G, float* __restrict__ w) {
  const INDEX blocks = (INDEX)((K + kBlock - 1) / kBlock);
  const int kg = K / G;
  for (INDEX u = (INDEX)blockIdx.x * 256 + threadIdx.x; u < units; u += (INDEX)gridDim.x * 256) {
    const INDEX b = u >> 3, row = b / blocks;
    const int p = (int)(u & 1), q = (int)(u >> 1 & 3), blk = (int)(b - row * blocks);
    const uint4 v = packed[(int64_t)(u >> 1)];
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = blk * kBlock + 32 * j + 8 * q + 4 * p;
      if (k >= K) continue;
      const int64_t gi = (int64_t)row * kg + k / G;
      const float s = bf16_f(scales[gi]);
      const int z = ZEROS ? zeros[gi] : 0;
      const uint32_t c = p ? word[j] : word[j] << 4;
      auto value = [&](int i) { return (float)(((int)(c << (24 - 8 * i)) >> 28) - z) * s; };
      *reinterpret_cast<float4*>(w + (int64_t)row * K + k) =
          make_float4(value(0), value(1), value(2), value(3));
    }
  }
}

// ------------------------------------------------------------------ product

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* glb_ptr_t;

// Eight codes of a packed word, times 16, as two int8 operand words.
__device__ __forceinline__ int low16(uint32_t w) { return (int)((w << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ int high16(uint32_t w) { return (int)(w & 0xF0F0F0F0u); }

// Eight codes less their group's zero point, as two int8 operand words: with
// zz = z + 8 in every byte, bytes 0x80 + (t + 8) - (z + 8), none of which
// borrows from the next, then the sign bit turned over (t - z lies in [-15, 15]).
__device__ __forceinline__ int low_z(uint32_t w, uint32_t zz) {
  return (int)((((w & 0x0F0F0F0Fu) ^ 0x88888888u) - zz) ^ 0x80808080u);
}
__device__ __forceinline__ int high_z(uint32_t w, uint32_t zz) { return low_z(w >> 4, zz); }

// CNT consecutive scales (or zero points) of a row.  Rows have any alignment:
// inside a row they are loaded in as few pieces as there are words, which the
// hardware takes at any address; a run that may reach past the row's end
// (TAIL) goes element by element, those past the end as 0.
template <typename E, int CNT>
struct Run {
  static constexpr int kWords = (CNT * (int)sizeof(E) + 3) / 4;
  uint32_t w[kWords];
  template <bool TAIL>
  __device__ __forceinline__ void load(const E* __restrict__ row, int at, int end) {
    if constexpr (!TAIL) {
      __builtin_memcpy(w, row + at, CNT * sizeof(E));
    } else {
      using U = std::make_unsigned_t<E>;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < CNT; ++i) {
        const uint32_t e = (U)row[min(at + i, end - 1)];
        constexpr int kPer = 4 / (int)sizeof(E);
        w[i / kPer] |= (at + i < end ? e : 0u) << (8 * (int)sizeof(E) * (i % kPer));
      }
    }
  }
  __device__ __forceinline__ float scale(int i) const {    // E = uint16_t
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t zero_bytes(int i) const {   // E = int8_t: z + 8, four times
    const uint32_t z = __builtin_amdgcn_perm(w[i >> 2], w[i >> 2], 0x01010101u * (uint32_t)(i & 3));
    return (z ^ 0x08080808u) & 0x0F0F0F0Fu;
  }
};

// A few tokens (decode), as many as LDS holds whole (16 of rows up to 9472, one
// of the longest): the weights stream once.  A team of `team` waves has 16 weight rows and splits their
// blocks into runs; a wave holds two buffers of U blocks (1 KiB each), one on
// its way while it works on the other, and goes on to its next rows without a
// pause where it is a team of its own.  Bound by the weight stream (2560 ->
// 128256, one token: 170 MB in 33.8 us, 5.0 TB/s; a pure read stream reaches
// 6.3); with few rows by latency (6912 -> 2560, 7 tokens, groups of 32: 10.5 MB in
// 10.8 us on 160 of 256 CUs).
// NV: result registers in use (1: one token, 4: up to 16).
template <int G, bool ZEROS, int NV, int U>
__global__ __launch_bounds__(512) void k_w4_few(const uint4* __restrict__ packed,
                                                const uint16_t* __restrict__ scales,
                                                const int8_t* __restrict__ zeros,
                                                const int8_t* __restrict__ xq,
                                                const float* __restrict__ absmax, int T, int N,
                                                int K, int team, float* __restrict__ y) {
  constexpr int NG = kBlock / G;                    // groups per block
  extern __shared__ __align__(16) unsigned char xs[];   // [T][token_stride(K)]
  __shared__ float red[8][NV][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int blocks = (K + kBlock - 1) / kBlock, kg = K / G, stride = (int)token_stride(K);
  const int tiles = (N + 15) / 16, teams = 8 / team;
  const int part = wave % team;
  const int per = (blocks + team - 1) / team;       // blocks of a wave's run
  const int b0 = part * per, b1 = min(b0 + per, blocks);
  const int runs = (max(b1 - b0, 0) + U - 1) / U;   // its groups of U, per tile

  // tokens: straight into LDS, 16 bytes per lane, zeros past K
  for (int t = wave; t < T; t += 8) {
    const int8_t* src = xq + (int64_t)t * K;
    for (int k0 = 0; k0 < blocks * kBlock; k0 += 1024) {
      const int k = k0 + 16 * lane;
      if (k < K)
        __builtin_amdgcn_global_load_lds((glb_ptr_t)(src + k), (lds_ptr_t)(xs + t * stride + k0), 16,
                                         0, 0);
      else if (k < blocks * kBlock)
        *reinterpret_cast<uint4*>(xs + t * stride + k) = make_uint4(0, 0, 0, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  struct Buf {
    Run<uint16_t, U * NG> s;
    Run<int8_t, U * NG> z;
    uint4 w[U];
  };
  // First block that group `g` of the run loads: its own, or for the row's last
  // blocks U before the end, so that a load group lies inside the row.
  auto first_of = [&](int g) { return max(min(b0 + g * U, blocks - U), 0); };
  // group `g` of the tile's: rows past N read row N - 1
  auto load = [&](Buf& b, int tile, int g) {
    const int n = min(tile * 16 + r, N - 1), c = first_of(g);
    const uint16_t* srow = scales + (int64_t)n * kg;
    const int8_t* zrow = ZEROS ? zeros + (int64_t)n * kg : nullptr;
    if ((c + U) * NG <= kg) {
      b.s.template load<false>(srow, c * NG, kg);
      if constexpr (ZEROS) b.z.template load<false>(zrow, c * NG, kg);
    } else {
      b.s.template load<true>(srow, c * NG, kg);
      if constexpr (ZEROS) b.z.template load<true>(zrow, c * NG, kg);
    }
    const uint4* row = packed + (int64_t)n * blocks * 4 + q;
#pragma unroll
    for (int u = 0; u < U; ++u) b.w[u] = row[4 * min(c + u, blocks - 1)];
  };
  float sum[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) sum[v] = 0.0f;
  const unsigned char* xrow = xs + min(r, T - 1) * stride + 8 * q;
  auto work = [&](const Buf& b, int g) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = first_of(g) + u, lo = b0 + g * U;
      if ((uint32_t)(c - lo) >= (uint32_t)(b1 - lo)) continue;   // another group's (wave-uniform)
      uint2 x[4];                                   // the lane's 8 k of each group of 32
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = *reinterpret_cast<const uint2*>(xrow + c * kBlock + 32 * j);
      const uint32_t w[4] = {b.w[u].x, b.w[u].y, b.w[u].z, b.w[u].w};
      auto add = [&](const v4i& acc, int i) {
        const float s = b.s.scale(u * NG + i);
#pragma unroll
        for (int v = 0; v < NV; ++v) sum[v] = fmaf((float)acc[v], s, sum[v]);
      };
      // operand words of group of 32 number j
      auto low = [&](int j) {
        if constexpr (ZEROS) return low_z(w[j], b.z.zero_bytes(u * NG + j * 32 / G));
        else return low16(w[j]);
      };
      auto high = [&](int j) {
        if constexpr (ZEROS) return high_z(w[j], b.z.zero_bytes(u * NG + j * 32 / G));
        else return high16(w[j]);
      };
      const v4i none = {0, 0, 0, 0};
      if constexpr (G == 32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const long a = (long)(((unsigned long)x[j].y << 32) | x[j].x);
          const long w8 = (long)(((unsigned long)(uint32_t)high(j) << 32) | (uint32_t)low(j));
          add(__builtin_amdgcn_mfma_i32_16x16x32_i8(a, w8, none, 0, 0, 0), j);
        }
      } else {
        v4i acc = none;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              v4i{(int)x[2 * i].x, (int)x[2 * i].y, (int)x[2 * i + 1].x, (int)x[2 * i + 1].y},
              v4i{low(2 * i), high(2 * i), low(2 * i + 1), high(2 * i + 1)}, acc, 0, 0, 0);
          if (G == 64 || i == 1) {
            add(acc, G == 64 ? i : 0);
            acc = none;
          }
        }
      }
    }
  };
  // lane 16 a + c of register v: token 4a + v, weight row c
  auto store = [&](int tile) {
    const int n = tile * 16 + r;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int t = 4 * q + v;
      if (n < N && t < T && (NV > 1 || q == 0))
        y[(int64_t)t * N + n] = sum[v] * (fmaxf(absmax[t], kEps) / kQb * (ZEROS ? 1.0f : 0.0625f));
      sum[v] = 0.0f;
    }
  };

  const int step = (int)gridDim.x * teams, first = (int)blockIdx.x * teams + wave / team;
  Buf buf[2];
  const bool busy = runs > 0 && first < tiles;
  if (busy) load(buf[0], first, 0);
  __builtin_amdgcn_sched_barrier(0);
  if (busy) wait_vmem<U>();                         // this wave's tokens are in LDS
  else wait_vmem<0>();
  lds_sync();
  if (team == 1) {
    // one run of groups over all of the wave's tiles, two buffers in turn
    int tile = first, g = 0, ntile = first, ng = 0;   // group in work; group on its way
    auto next = [&](Buf& b) {
      if (++ng == runs) {
        ng = 0;
        ntile += step;
      }
      if (ntile < tiles) load(b, ntile, ng);
    };
    auto turn = [&](Buf& now, Buf& then) {
      next(then);
      work(now, g);
      if (++g == runs) {
        store(tile);
        g = 0;
        tile += step;
      }
    };
    while (tile < tiles) {
      turn(buf[0], buf[1]);
      if (tile >= tiles) break;
      turn(buf[1], buf[0]);
    }
  } else {
    // every team of the block as often, for the barriers
    for (int base = (int)blockIdx.x * teams; base < tiles; base += step) {
      const int tile = base + wave / team;
      if (tile < tiles) {
        for (int g = 0; g < runs; g += 2) {
          if (g + 1 < runs) load(buf[1], tile, g + 1);
          work(buf[0], g);
          if (g + 2 < runs) load(buf[0], tile, g + 2);
          if (g + 1 < runs) work(buf[1], g + 1);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) red[wave][v][lane] = sum[v];
      }
      if (runs > 0 && tile + step < tiles) load(buf[0], tile + step, 0);
      lds_sync();
      if (part == 0 && tile < tiles) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          for (int w = 1; w < team; ++w) sum[v] += red[wave + w][v][lane];
        store(tile);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) sum[v] = 0.0f;
      if (base + step < tiles) lds_sync();          // red is free again
    }
  }
}

// Many tokens: int8 tokens through LDS (global -> LDS directly, three stages,
// one barrier per 128 k), weights straight into registers, WMF row fragments
// of 32 x 32 per wave on v_mfma_i32_32x32x32_i8.  Lane (m, h) takes chunks 2h
// and 2h + 1 of weight row m: word j of the two is 16 consecutive k of the
// block's group of 32 number j.
//
// A group's sums are converted and scaled in registers, two VALU operations of
// four cycles per register and group, against 32 cycles of MFMA per 32 k and
// fragment: for groups of 32 and 64 that is the largest part, not the matrix
// cores, but it does not fill the time either (2560 -> 6912, 2048 tokens, groups
// of 64, 70 us: VALU issue 98 of 160 thousand cycles, MFMA 35; the four waves of a
// block meet at a barrier every 128 k).  Groups of 32 / 64 / 128: 96 / 77 / 60 us
// back to back, with zero points 106 / 89 / 72.  Zero points come off the codes (t - z fits an int8;
// five more operations per word, which all row fragments share) and not off the
// sums (two operations per register).
//
// WK > 1 (few tiles): WK groups of waves split K, each with its own stages,
// and add their sums through LDS in order.
template <int WN, int WK, int WMF, int G, bool ZEROS, bool TAIL>
__global__ __launch_bounds__(WN * WK * 64, WMF == 2 ? 3 : 1) void k_w4_tile(const uint4* __restrict__ packed,
                                                          const uint16_t* __restrict__ scales,
                                                          const int8_t* __restrict__ zeros,
                                                          const int8_t* __restrict__ xq,
                                                          const float* __restrict__ absmax, int T,
                                                          int N, int K, float* __restrict__ y) {
  constexpr int NG = kBlock / G;
  constexpr int BM = 32 * WMF, BN = 32 * WN, kThreads = WN * WK * 64;
  constexpr int kATot = BM / 8, kAChunks = (kATot + WN - 1) / WN;   // 1 KiB pieces of a stage
  constexpr int kStage = BM * kBlock;
  __shared__ __align__(16) unsigned char A0[WK * kStage], A1[WK * kStage], A2[WK * kStage];
  __shared__ float scale[BM];
  __shared__ float red[WK > 1 ? (WK - 1) * WN : 1][WK > 1 ? WMF * 16 : 1][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wk = wave / WN;
  auto stage_of = [&](auto st) -> unsigned char* {
    constexpr int S = decltype(st)::value;
    if constexpr (S == 0) return A0 + wk * kStage;
    else if constexpr (S == 1) return A1 + wk * kStage;
    else return A2 + wk * kStage;
  };
  const int h = lane >> 5, m = lane & 31;
  const int blocks = (K + kBlock - 1) / kBlock, kg = K / G;
  const int per = (blocks + WK - 1) / WK;           // blocks of 128 k per group of waves
  const int b0 = min(wk * per, blocks - 1), nb = min(per, blocks - wk * per);   // nb < 1: none

  // tiles in equal runs to the XCDs, four row blocks at a time, down the rows first
  const int64_t ntn = (N + BN - 1) / BN, ntm = (T + BM - 1) / BM, tiles = ntn * ntm;
  const int64_t per_xcd = (tiles + 7) / 8;
  const int64_t tile = (blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
  if (blockIdx.x / 8 >= per_xcd || tile >= tiles) return;
  const int64_t gid = tile / (4 * ntn), first_m = gid * 4, r_in = tile - gid * 4 * ntn;
  const int64_t gsize = ntm - first_m < 4 ? ntm - first_m : 4;
  const int m0 = (int)(first_m + r_in % gsize) * BM, n0 = (int)(r_in / gsize) * BN;

  // without zero points the codes are 16 t
  for (int i = tid; i < BM; i += kThreads)
    scale[i] = m0 + i < T ? fmaxf(absmax[m0 + i], kEps) / kQb * (ZEROS ? 1.0f : 0.0625f) : 0.0f;

  // activations: 1 KiB = 8 rows x 128 bytes; row r's 16-byte slot p holds slot
  // p ^ ((r >> 1) & 7), which spreads an operand read over the banks.  Slots
  // past K meet codes of 0 and scales of 0: they take the row's last bytes
  const int8_t* asrc[kAChunks];
  int aslot[kAChunks];
#pragma unroll
  for (int i = 0; i < kAChunks; ++i) {
    const int c = min(wn * kAChunks + i, kATot - 1), row = 8 * c + (lane >> 3);
    asrc[i] = xq + (int64_t)min(m0 + row, T - 1) * K;
    aslot[i] = 16 * ((lane & 7) ^ ((row >> 1) & 7));
  }
  const int64_t n = min(n0 + wn * 32 + m, N - 1);
  const uint4* wsrc = packed + n * blocks * 4 + 2 * h;
  const uint16_t* ssrc = scales + n * kg;
  const int8_t* zsrc = ZEROS ? zeros + n * kg : nullptr;
  struct Frag {
    uint4 w0, w1;
    Run<uint16_t, NG> s;
    Run<int8_t, NG> z;
  };
  Frag frag[3];
  auto issue = [&](int i, auto st) {                // block i of this group's, the last one again past it
    constexpr int S = decltype(st)::value;
    const int b = b0 + max(min(i, nb - 1), 0);
#pragma unroll
    for (int u = 0; u < kAChunks; ++u)
      __builtin_amdgcn_global_load_lds(
          (glb_ptr_t)(asrc[u] + min(b * kBlock + aslot[u], K - 16)),
          (lds_ptr_t)(stage_of(st) + min(wn * kAChunks + u, kATot - 1) * 1024), 16, 0, 0);
    frag[S].s.template load<TAIL>(ssrc, b * NG, kg);
    if constexpr (ZEROS) frag[S].z.template load<TAIL>(zsrc, b * NG, kg);
    frag[S].w0 = wsrc[4 * b];
    frag[S].w1 = wsrc[4 * b + 1];
  };
  constexpr int kLoads = kAChunks + 3 + ZEROS;      // at least: a wave's loads per step

  v16f sum[WMF];
#pragma unroll
  for (int i = 0; i < WMF; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) sum[i][v] = 0.0f;

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  __builtin_amdgcn_s_waitcnt(0);
  issue(0, I0{});
  __builtin_amdgcn_sched_barrier(0);
  issue(1, I1{});
  __builtin_amdgcn_sched_barrier(0);
  wait_vmem<kLoads>();                              // block 0 (the second one stays in flight)
  lds_sync();

  const int swz = (m >> 1) & 7;
  // One block of 128 k on stage S.  REFILL: stage S + 2 takes block b + 2, and
  // the step ends when all but the loads of that refill have come back; the
  // last steps load nothing more and wait for all there is.  (With no branch
  // in the loop and the refill fenced off, a counted wait leaves exactly the
  // refill in flight.)
  auto step = [&](auto st, int b, auto refill) {
    constexpr int S = decltype(st)::value;
    constexpr bool REFILL = decltype(refill)::value;
    if constexpr (REFILL) {
      issue(b + 2, std::integral_constant<int, (S + 2) % 3>{});
      __builtin_amdgcn_sched_barrier(0);
    }
    const unsigned char* At = stage_of(st) + m * kBlock;
    // operand words of the block's four groups of 32
    v4i w[4];
    const uint32_t u[8] = {frag[S].w0.x, frag[S].w0.y, frag[S].w0.z, frag[S].w0.w,
                           frag[S].w1.x, frag[S].w1.y, frag[S].w1.z, frag[S].w1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!ZEROS) {
        w[j] = v4i{low16(u[j]), high16(u[j]), low16(u[4 + j]), high16(u[4 + j])};
      } else {
        const uint32_t zz = frag[S].z.zero_bytes(j / (G / 32));
        w[j] = v4i{low_z(u[j], zz), high_z(u[j], zz), low_z(u[4 + j], zz), high_z(u[4 + j], zz)};
      }
    }
    v16i zero;
#pragma unroll
    for (int v = 0; v < 16; ++v) zero[v] = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      v16i acc[WMF];
#pragma unroll
      for (int jj = 0; jj < G / 32; ++jj) {
        const int j = g * (G / 32) + jj;
#pragma unroll
        for (int i = 0; i < WMF; ++i) {
          const uint4 t = *reinterpret_cast<const uint4*>(At + i * 32 * kBlock + 16 * ((2 * j + h) ^ swz));
          acc[i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
              v4i{(int)t.x, (int)t.y, (int)t.z, (int)t.w}, w[j], jj ? acc[i] : zero, 0, 0, 0);
        }
      }
      // waves whose run has ended add nothing
      const float s = WK == 1 || b < nb ? frag[S].s.scale(g) : 0.0f;
#pragma unroll
      for (int i = 0; i < WMF; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) sum[i][v] = fmaf((float)acc[i][v], s, sum[i][v]);
    }
    wait_vmem<REFILL ? kLoads : 0>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  int b = 0;
  for (; b + 3 <= per; b += 3) {
    step(I0{}, b, std::true_type{});
    step(I1{}, b + 1, std::true_type{});
    step(I2{}, b + 2, std::true_type{});
  }
  wait_vmem<0>();   // the last two stages (no load may land in LDS after the block has ended)
  lds_sync();
  if (b < per) step(I0{}, b, std::false_type{});
  if (b + 1 < per) step(I1{}, b + 1, std::false_type{});

  if constexpr (WK > 1) {
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < WMF; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) red[wave - WN][i * 16 + v][lane] = sum[i][v];
    }
    lds_sync();
    if (wk > 0) return;
#pragma unroll
    for (int i = 0; i < WMF; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        for (int k = 0; k < WK - 1; ++k) sum[i][v] += red[k * WN + wn][i * 16 + v][lane];
  }
  // the lane's first output; the others' offsets from it are the same in every
  // lane (scalar), and whole tiles need no bounds
  const int col = n0 + wn * 32 + m, row0 = 4 * h;
  float* const out = y + ((int64_t)(m0 + row0) * N + col);
  auto finish = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int i = 0; i < WMF; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int at = i * 32 + (v >> 2) * 8 + (v & 3);
        if (WHOLE || (m0 + row0 + at < T && col < N)) out[(int64_t)at * N] = sum[i][v] * scale[row0 + at];
      }
  };
  if (m0 + BM <= T && n0 + BN <= N) finish(std::true_type{});
  else finish(std::false_type{});
}

unsigned stream_grid(int64_t units) {
  return (unsigned)std::min<int64_t>((units + 255) / 256, 16 * (int64_t)device_cus());
}

// f(G, ZEROS), which launches and returns the launch's status.
template <typename F>
hipError_t by_group(int g, bool zeros, F&& f) {
  auto z = [&](auto gc) -> hipError_t {
    return zeros ? f(gc, std::true_type{}) : f(gc, std::false_type{});
  };
  if (g == 32) return z(std::integral_constant<int, 32>{});
  if (g == 64) return z(std::integral_constant<int, 64>{});
  return z(std::integral_constant<int, 128>{});
}

}  // namespace

hipError_t launch_pack_w4(const float* w, int64_t n, int64_t k, int g, uint8_t* packed,
                          uint16_t* scales, int8_t* zeros, hipStream_t stream) {
  const int64_t units = n * ((k + kBlock - 1) / kBlock) * 4;
  const unsigned grid = stream_grid(units);
  const bool small = units + 256 * (int64_t)grid < (int64_t(1) << 32);   // u never wraps
  return by_group(g, zeros != nullptr, [&](auto gc, auto zc) {
    auto go = [&](auto ic) {
      using I = decltype(ic);
      k_pack_w4<decltype(gc)::value, decltype(zc)::value, I><<<grid, 256, 0, stream>>>(
          w, (I)units, (int)k, reinterpret_cast<uint4*>(packed), scales, zeros);
      return hipGetLastError();
    };
    return small ? go(uint32_t{}) : go(uint64_t{});
  });
}

hipError_t launch_unpack_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                            int64_t n, int64_t k, int g, float* w, hipStream_t stream) {
  const int64_t units = n * ((k + kBlock - 1) / kBlock) * 8;
  const unsigned grid = stream_grid(units);
  const auto* p = reinterpret_cast<const uint4*>(packed);
  auto go = [&](auto zc, auto ic) {
    using I = decltype(ic);
    k_unpack_w4<decltype(zc)::value, I><<<grid, 256, 0, stream>>>(p, scales, zeros, (I)units, (int)k,
                                                                  g, w);
  };
  const bool small = units + 256 * (int64_t)grid < (int64_t(1) << 32);   // u never wraps
  if (zeros) small ? go(std::true_type{}, uint32_t{}) : go(std::true_type{}, uint64_t{});
  else small ? go(std::false_type{}, uint32_t{}) : go(std::false_type{}, uint64_t{});
  return hipGetLastError();
}

hipError_t launch_forward_w4(const uint8_t* packed, const uint16_t* scales, const int8_t* zeros,
                             const int8_t* xq, const float* absmax, int64_t t, int64_t n,
                             int64_t k, int g, float* y, hipStream_t stream) {
  const auto* w = reinterpret_cast<const uint4*>(packed);
  const W4Plan plan = w4_plan(t, n, k, g, device_cus());
  if (plan.wn) {
    return by_group(g, zeros != nullptr, [&](auto gc, auto zc) {
      constexpr int G = decltype(gc)::value;
      constexpr bool Z = decltype(zc)::value;
      auto go = [&](auto wn, auto wk, auto wmf) {
        constexpr int WN = decltype(wn)::value, WK = decltype(wk)::value, WMF = decltype(wmf)::value;
        constexpr int BM = 32 * WMF, BN = 32 * WN;
        auto kern = k_w4_tile<WN, WK, WMF, G, Z, false>;
        if constexpr (G < kBlock)
          if (k % kBlock) kern = k_w4_tile<WN, WK, WMF, G, Z, true>;
        const int64_t tiles = ((t + BM - 1) / BM) * ((n + BN - 1) / BN);
        kern<<<(unsigned)((tiles + 7) / 8 * 8), 64 * WN * WK, 0, stream>>>(
            w, scales, zeros, xq, absmax, (int)t, (int)n, (int)k, y);
        return hipGetLastError();
      };
      using I1 = std::integral_constant<int, 1>;
      using I2 = std::integral_constant<int, 2>;
      using I4 = std::integral_constant<int, 4>;
      using I8 = std::integral_constant<int, 8>;
      if (plan.wn == 1) return go(I1{}, I8{}, I1{});
      if (plan.wn == 2) return go(I2{}, I4{}, I1{});
      if constexpr (G == kBlock)
        if (plan.wn == 8) return go(I8{}, I1{}, I4{});
      if (plan.wk == 2) return go(I4{}, I2{}, I1{});
      return plan.wmf == 2 ? go(I4{}, I1{}, I2{}) : go(I4{}, I1{}, I1{});
    });
  }
  const int64_t stride = token_stride(k), tiles = (n + 15) / 16;
  const int team = plan.team;
  for (int64_t t0 = 0; t0 < t; t0 += plan.tokens) {
    const int64_t nt = std::min(t - t0, plan.tokens);
    const size_t lds = (size_t)(nt * stride);
    // two blocks per CU where their LDS fits, going on from tile to tile
    // (2560 -> 128256, one token: 1 / 2 / 3 / 4 blocks 43 / 33 / 35 / 34 us)
    const int64_t per_cu = lds + 12288 <= (size_t)kMaxLds / 2 ? 2 : 1;
    const int64_t grid = std::min<int64_t>((tiles * team + 7) / 8, per_cu * device_cus());
    const hipError_t e = by_group(g, zeros != nullptr, [&](auto gc, auto zc) {
      constexpr int G = decltype(gc)::value;
      constexpr bool Z = decltype(zc)::value;
      auto go = [&](auto kern) {
        const hipError_t lds_ok = kern.allow_lds();
        if (lds_ok != hipSuccess) return lds_ok;
        kern.kernel<<<(unsigned)grid, 512, lds, stream>>>(w, scales, zeros, xq + t0 * k, absmax + t0,
                                                   (int)nt, (int)n, (int)k, team, y + t0 * n);
        return hipGetLastError();
      };
      return nt == 1 ? go(Kernel<k_w4_few<G, Z, 1, kAhead>>{})
                     : go(Kernel<k_w4_few<G, Z, 4, kAhead>>{});
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bl
