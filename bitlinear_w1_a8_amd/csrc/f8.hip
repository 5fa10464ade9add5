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
// neighbouring k (8 i .. 8 i + 7) with all bits below 2^-13 of the largest one's power of
// two (its factors' exponents added) cut off, towards zero; measured on 16x16x128,
// 16x16x32, 32x32x64 and 32x32x16 alike.  Each of the other seven loses less than 2^-13 of
// the largest, so a sum is off by up to 7 * 2^-13 of its magnitudes' sum (seen: 2^-12.7; 4e-5
// to 5e-5 in the norm for Gaussian data), which is more than sums in binary32 may be.  The f16 ones at half the
// rate hold every e4m3 exactly and add in binary32 (8e-8 in the norm).  So products take
// the f16 ones, and the e4m3 ones only where the caller has asked for cut sums.
#include <algorithm>
#include <type_traits>

#include "experts.h"
#include "f8.h"
#include "f8_plan.h"

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

// Four outputs n .. n + 3 of a token; n + i < N is checked where the last are cut
// off.  y is aligned to its element only, which a wide store does not mind here.
template <bool BF16>
__device__ __forceinline__ void store4(void* y, int64_t at, int n, int N, const float (&v)[4]) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(y) + at + n;
    const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    if (n + 3 < N) {
      __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (n + i < N) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(y) + at + n;
    if (n + 3 < N) {
      __builtin_memcpy(p, v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (n + i < N) p[i] = v[i];
    }
  }
}

// ------------------------------------------------------------------ few tokens

// Up to 16 TT tokens against 16 RT rows per block or, not FULL, fewer, so that more CUs
// have a block (13 tokens, 6912 -> 2560, 12 rows 8.3 -> 8.0 us; one token, 8192 -> 2000, 8
// rows 7.4 -> 6.4, 8192 -> 128, 4 rows 7.0 -> 5.5).  The block's waves take the blocks of K
// in turn and their sums meet in LDS, added in order of the waves.  Every load goes straight
// to registers, two blocks of K ahead of its use (four: 128256 rows 82 us, two: 56).  Bound
// by the stream of weights (one token, 2560 -> 128256: 328 MB in 55 us, 6.0 TB/s; a pure
// read stream reaches 6.2), with few rows by latency: two blocks of K ahead per wave (13
// tokens, 6912 -> 2560: 17.7 MB in 8.0 us, seven blocks of K per wave one after the other,
// 62% of the wave cycles waiting).
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 2;

template <int TT, int RT, bool FULL, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_f8_few(const uint8_t* __restrict__ w,
                                                           const float* __restrict__ ws,
                                                           const uint8_t* __restrict__ xq,
                                                           const float* __restrict__ xs, int T,
                                                           int N, int K, int rows_, int t_tiles,
                                                           void* __restrict__ y) {
  constexpr int WV = kFewWaves, U = kFewAhead;
  __shared__ float red[WV][RT * TT][4][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb_all = (K + kF8Block - 1) / kF8Block;
  const int rows = FULL ? 16 * RT : rows_;
  const int n0 = blockIdx.x / t_tiles * rows, t0 = blockIdx.x % t_tiles * 16 * TT;
  // one scale for the lane's outputs: four rows from a multiple of four on, or whole tiles
  const float* wsr = ws + (int64_t)(min(n0 + (FULL ? 0 : 4 * g), N - 1) / kF8Block) * kb_all;
  const uint8_t* wrow[RT];
  const uint8_t* xrow[TT];
  int tok[TT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wrow[i] = w + (int64_t)min(n0 + min(16 * i + r, rows - 1), N - 1) * K;
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
    const int k0 = min(kb * kF8Block + 16 * g, K - 16), k1 = min(kb * kF8Block + 64 + 16 * g, K - 16);
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
  for (int u = 0; u < U; ++u) load(buf[u], wave + u * WV);
  for (int k0 = wave; k0 < kb_all; k0 += U * WV) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * WV;
      if (kb >= kb_all) break;
      Buf f = buf[u];
      if (kb + U * WV < kb_all) load(buf[u], kb + U * WV);
      if ((kb + 1) * kF8Block > K) {           // tokens are zero past K
        const int k = kb * kF8Block + 16 * g;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          if (k >= K) f.b[j][0] = make_uint4(0, 0, 0, 0);
          if (k + 64 >= K) f.b[j][1] = make_uint4(0, 0, 0, 0);
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
  for (int q = wave; q < RT * TT; q += WV) {
    const int t = t0 + 16 * (q % TT) + r;
    float s[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      s[v] = red[0][q][v][lane];
#pragma unroll
      for (int p = 1; p < WV; ++p) s[v] += red[p][q][v][lane];
    }
    const int n = 16 * (q / TT) + 4 * g;
    if (t < T && n < rows) store4<BF16>(y, (int64_t)t * N, n0 + n, N, s);
  }
}

// ------------------------------------------------------------------ many tokens

// What the tiled kernels have in common.  A tile of BM rows and BT tokens comes one
// block of K at a time through LDS buffers filled directly from memory, by ROWS of the
// block's waves in equal parts.  In a buffer, row r has its eight 16-byte pieces at
// 128 r, piece c at place c ^ (r >> 1 & 7), so that sixteen lanes reading one piece
// of their rows reach all 64 banks (c ^ (r & 7): half of them; 256 x 128 tiles, 250 x 28672
// x 8192 92 -> 82 us).  The buffers of different steps are objects of their own, named at
// compile time: with one array indexed by the step the compiler waits for every load on
// its way before each LDS read (4096 x 8192 x 8192: 366 -> 296 us).
// TAIL: the last block of K is a partial one.
template <int BM, int BT, int WAVES, bool TAIL>
struct Loads {
  static constexpr int LM = BM / (8 * WAVES), LT = BT / (8 * WAVES), kCount = LM + LT;
  static_assert(LM % 2 == 0 && LT % 2 == 0, "a wave's first load of an operand is an even one");
  __amdgpu_buffer_rsrc_t wb, xb;
  int off[2], piece, wave, K;

  // The tile's rows that exist as buffers: what lies behind them is read as zeros.
  __device__ __forceinline__ Loads(const uint8_t* w, const uint8_t* xq, int n0, int t0, int T, int N,
                                   int K, int wave, int lane)
      : wave(wave), K(K) {
    constexpr int kRaw = 0x00027000;                // raw 32-bit buffer
    wb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(w) + (int64_t)n0 * K, 0,
                                           min(BM, N - n0) * K, kRaw);
    xb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(xq) + (int64_t)t0 * K, 0,
                                           min(BT, T - t0) * K, kRaw);
    // the piece that a lane brings: of even loads, and with bit 2 turned of odd ones
    const int lr = lane >> 3;
    piece = (lane & 7) ^ (lr >> 1);
    off[0] = lr * K + 16 * piece;
    off[1] = lr * K + 16 * (piece ^ 4);
  }
  // Load number i (8 rows) of block kb into the buffers a (rows) and b (tokens).  A piece
  // past K is the row's last one, whose token is zeroed when it is used.
  __device__ __forceinline__ void send(int i, int kb, uint8_t* a, uint8_t* b) const {
    const int row = i < LM ? (wave * LM + i) * 8 : (wave * LT + i - LM) * 8;
    int at = off[i & 1] + row * K + kb * kF8Block;
    if constexpr (TAIL) at -= max(kb * kF8Block + 16 * (piece ^ (4 * (i & 1))) - (K - 16), 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(i < LM ? wb : xb, (lds_ptr_t)((i < LM ? a : b) + row * kF8Block),
                                             16, at, 0, 0, 0);
  }
};

// One wave's scales of the blocks of K: its rows' and, per token, FT tokens' of a lane.
template <int FT>
struct Scales {
  const float *ws, *xs;
  int64_t T;
  uint32_t tok[FT], zero;
  float w, x[FT];
  __device__ __forceinline__ Scales(const float* ws_, const float* xs_, int n, int t, int T_, int N,
                                    int kb_all, int c)
      : ws(ws_ + (int64_t)min(n / kF8Block, (N - 1) / kF8Block) * kb_all), xs(xs_), T(T_), zero(0) {
#pragma unroll
    for (int j = 0; j < FT; ++j) tok[j] = 4u * (uint32_t)min(t + 32 * j + c, T_ - 1);   // bytes
    // a vector load of the rows' scale: a scalar one shares the LDS reads' counter, out of
    // order, and each of them would wait for all
    __asm__ volatile("" : "+v"(zero));
  }
  __device__ __forceinline__ void load(int kb) {
    auto at = [](const float* base, uint32_t bytes) {
      return *reinterpret_cast<const float*>(reinterpret_cast<const char*>(base) + bytes);
    };
    w = at(ws + kb, zero);
#pragma unroll
    for (int j = 0; j < FT; ++j) x[j] = at(xs + kb * T, tok[j]);
  }
};

__device__ __forceinline__ v8h halves_part(const uint4 (&v)[4], int q) {
  return q & 1 ? halves8(v[q >> 1].z, v[q >> 1].w) : halves8(v[q >> 1].x, v[q >> 1].y);
}

// Zeros in the pieces of a token past K; piece 2 q + h of a lane.
__device__ __forceinline__ void cut_tail(uint4 (&f)[4], int kb, int h, int K) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t keep = kb * kF8Block + 16 * (2 * q + h) < K ? ~0u : 0u;
    f[q].x &= keep; f[q].y &= keep; f[q].z &= keep; f[q].w &= keep;
  }
}

// Tile number of a workgroup: workgroup b runs on XCD b % 8, and each XCD gets a
// run of neighbouring tiles; false for those left over.
__device__ __forceinline__ bool tile_of(int tiles, int& item) {
  const int per = (tiles + 7) / 8, at = (int)(blockIdx.x / 8);
  item = (int)(blockIdx.x % 8) * per + at;
  return at < per && item < tiles;
}

// Lane (h, c) of a 32 x 32 tile has token c and rows 8 q + 4 h + v.
template <bool BF16>
__device__ __forceinline__ void store_tile(const v16f& a, void* y, int t, int n, int h, int T, int N) {
  if (t >= T) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float v[4] = {a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
    store4<BF16>(y, (int64_t)t * N, n + 8 * q + 4 * h, N, v);
  }
}

using S0 = std::integral_constant<int, 0>;
using S1 = std::integral_constant<int, 1>;
using S2 = std::integral_constant<int, 2>;

// WR x WT waves of 64 rows x 64 tokens each, GROUPS times: each group takes
// every GROUPS-th block of K through buffers of its own, and their sums meet at the end, in
// order.  A wave takes about a microsecond per block of K, most of it issue, so where there
// are few tiles the CU's other SIMDs take other blocks of K; LDS holds what is on its way.
// (6912 -> 2560, 256 tokens, binary32 outputs: 64 x 64 in two groups with three buffers 27.1 us,
// in four with two 24.6, in three with three 22.4; 128 x 64 in two with three 32.7; 128 x 128 in
// two with two 50.)
// NATIVE: e4m3 instructions (cut sums); else each wave widens its operands to f16.
template <bool BF16, bool NATIVE, bool TAIL, int WR, int WT, int GROUPS, int STAGES>
__global__ __launch_bounds__(64 * WR * WT * GROUPS) void k_f8_tile(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, const uint8_t* __restrict__ xq,
    const float* __restrict__ xs, int T, int N, int K, int t_tiles, int tiles,
    void* __restrict__ y) {
  constexpr int kWaves = WR * WT, BM = 64 * WR, BT = 64 * WT, kA = BM * kF8Block, kB = BT * kF8Block;
  __shared__ __align__(16) uint8_t a0[GROUPS * kA], b0[GROUPS * kB], a1[GROUPS * kA], b1[GROUPS * kB];
  __shared__ __align__(16) uint8_t a2[STAGES > 2 ? GROUPS * kA : 16], b2[STAGES > 2 ? GROUPS * kB : 16];
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = all % kWaves, group = all / kWaves;
  auto buf_a = [&](auto stage) -> uint8_t* {
    constexpr int S = decltype(stage)::value;
    if constexpr (S == 0) return a0 + group * kA;
    else if constexpr (S == 1) return a1 + group * kA;
    else return a2 + group * kA;
  };
  auto buf_b = [&](auto stage) -> uint8_t* {
    constexpr int S = decltype(stage)::value;
    if constexpr (S == 0) return b0 + group * kB;
    else if constexpr (S == 1) return b1 + group * kB;
    else return b2 + group * kB;
  };
  int item;
  if (!tile_of(tiles, item)) return;
  const int n0 = item / t_tiles * BM, t0 = item % t_tiles * BT;
  const int wr = (wave / WT) * 64, wt = (wave % WT) * 64;
  const int kb_all = (K + kF8Block - 1) / kF8Block, steps = (kb_all + GROUPS - 1) / GROUPS;
  auto block = [&](int i) { return min(i * GROUPS + group, kb_all - 1); };
  using L = Loads<BM, BT, kWaves, TAIL>;
  const L loads(w, xq, n0, t0, T, N, K, wave, lane);
  Scales<2> scales(ws, xs, n0 + wr, t0 + wt, T, N, kb_all, c);

  v16f acc[2][2] = {};
  scales.load(block(0));
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < L::kCount; ++i) loads.send(i, block(0), buf_a(S0{}), buf_b(S0{}));
  if constexpr (STAGES == 3) {
#pragma unroll
    for (int i = 0; i < L::kCount; ++i) loads.send(i, block(1), buf_a(S1{}), buf_b(S1{}));
  }
  auto step = [&](auto stage, int at) {
    constexpr int S = decltype(stage)::value;
    using R = std::integral_constant<int, (S + STAGES - 1) % STAGES>;
    __builtin_amdgcn_sched_barrier(0);
    // all but the loads of the step before, which came after its scales'
    wait_vmem<(STAGES - 2) * L::kCount>();
    lds_sync();                                     // this buffer is whole, R's is free
    __builtin_amdgcn_sched_barrier(0);
    float sc[2];
    const bool mine = at * GROUPS + group < kb_all; // a group's last step may be one too many
#pragma unroll
    for (int j = 0; j < 2; ++j) sc[j] = mine ? scales.x[j] * scales.w : 0.0f;
    scales.load(block(at + 1));                     // past the end: the last block once more
    __builtin_amdgcn_sched_barrier(0);
    // piece 2 q + h of a row sits at its first address with bits 5 and 6 turned by q
    int ra = (wr + c) * kF8Block + 16 * (h ^ (c >> 1 & 7)), rb = (wt + c) * kF8Block + 16 * (h ^ (c >> 1 & 7));
    __asm__ volatile("" : "+v"(ra), "+v"(rb));      // made anew: kept, they cost eight registers
    uint4 fa[2][4], fb[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        fa[i][q] = *reinterpret_cast<const uint4*>(buf_a(stage) + (ra ^ (32 * q)) + 32 * i * kF8Block);
        fb[i][q] = *reinterpret_cast<const uint4*>(buf_b(stage) + (rb ^ (32 * q)) + 32 * i * kF8Block);
      }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (TAIL) {
#pragma unroll
      for (int j = 0; j < 2; ++j) cut_tail(fb[j], block(at), h, K);
    }
    // the other buffer's loads go out between the tiles: a wave issues in order, and a full
    // memory queue would hold its LDS reads back
    auto refill = [&](int tile) {
#pragma unroll
      for (int i = 0; i < L::kCount; ++i)
        if (min(i / 2, 3) == tile) loads.send(i, block(at + STAGES - 1), buf_a(R{}), buf_b(R{}));
    };
    auto add = [&](int i, int j, const v16f& p) {
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(p[v], sc[j], acc[i][j][v]);
    };
    const v16f zero = {};
    if constexpr (NATIVE) {
      v16f p[2];                                    // a tile's sums are scaled while the next one's are formed
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) {
        const int i = tile / 2, j = tile % 2, now = tile & 1;
        p[now] = mfma32(operand8(fa[i][0], fa[i][1]), operand8(fb[j][0], fb[j][1]), zero);
        p[now] = mfma32(operand8(fa[i][2], fa[i][3]), operand8(fb[j][2], fb[j][3]), p[now]);
        refill(tile);
        if (tile > 0) add((tile - 1) / 2, (tile - 1) % 2, p[now ^ 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      add(1, 1, p[1]);
    } else {
      v8h hb[2][8];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 8; ++q) hb[j][q] = halves_part(fb[j], q);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v16f p[2];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const v8h f = halves_part(fa[i], q);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            p[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, hb[j][q], q ? p[j] : zero, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          refill(2 * i + j);
          add(i, j, p[j]);
        }
      }
    }
  };
  int at = 0;
  for (; at + STAGES <= steps; at += STAGES) {
    step(S0{}, at);
    step(S1{}, at + 1);
    if constexpr (STAGES == 3) step(S2{}, at + 2);
  }
  if (at < steps) step(S0{}, at);
  if constexpr (STAGES == 3)
    if (at + 1 < steps) step(S1{}, at + 1);
  wait_vmem<0>();                                   // loads past the end land before LDS is used anew
  if constexpr (GROUPS > 1) {
    constexpr int kSums = 2 * 16 * 64 * kWaves;     // half of a group's sums
    static_assert(GROUPS * kA >= (GROUPS - 1) * kSums * 4, "half of the groups' sums in one buffer");
    lds_sync();
    float* part[2] = {reinterpret_cast<float*>(a0), reinterpret_cast<float*>(a1)};
    const int me = wave * 64 + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (group) part[i][(group - 1) * kSums + (j * 16 + v) * 64 * kWaves + me] = acc[i][j][v];
    lds_sync();
    if (group) return;
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g)            // in order of the groups
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] += part[i][g * kSums + (j * 16 + v) * 64 * kWaves + me];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      store_tile<BF16>(acc[i][j], y, t0 + wt + 32 * j + c, n0 + wr + 32 * i, h, T, N);
}

// 256 x 256 tiles with the e4m3 instructions (cut sums, bfloat16 outputs): 2 x 4 waves of 128 x 64 in two groups of
// four, one wave of each on a SIMD, in turn.  While one group runs its matrix
// instructions (phase M) the other scales its last sums, reads its next operands from
// LDS and sends for the next block of K (phase L); a barrier ends each phase.  A wave
// issues a vector instruction every eight cycles at best, so the sixteen multiply-adds
// that scale a tile take as long as the tile's two matrix instructions: in the same
// phase they would add up.  (2048 x 6912 x 2560: all eight waves in step 49-51 us, this
// 41 in a row.)
//
// Four pairs of phases per block of K, one row of tiles each.  Group 1 is one phase
// behind: in step kb group 0 has the phases 8 kb .. 8 kb + 7, L first, group 1 the same
// plus 1.  The last L of group 1 is phase 8 kb + 7, so after that phase's barrier block
// kb's buffer is free, and step kb + 1 sends for block kb + 2 into it.  Block kb + 1 is read
// from phase 8 (kb + 1) on: each wave waits for its own part of it in its last L of
// step kb, which group 1 ends with the phase before that.
template <bool TAIL>
__global__ __launch_bounds__(512) void k_f8_turns(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, const uint8_t* __restrict__ xq,
    const float* __restrict__ xs, int T, int N, int K, int t_tiles, int tiles,
    void* __restrict__ y) {
  constexpr int BM = 256, BT = 256;
  __shared__ __align__(16) uint8_t a0[BM * kF8Block], b0[BT * kF8Block], a1[BM * kF8Block], b1[BT * kF8Block];
  auto buf_a = [&](auto stage) -> uint8_t* { return decltype(stage)::value ? a1 : a0; };
  auto buf_b = [&](auto stage) -> uint8_t* { return decltype(stage)::value ? b1 : b0; };
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = wave >> 2;
  int item;
  if (!tile_of(tiles, item)) return;
  const int n0 = item / t_tiles * BM, t0 = item % t_tiles * BT;
  const int wr = (wave >> 2) * 128, wt = (wave & 3) * 64;
  const int kb_all = (K + kF8Block - 1) / kF8Block;
  using L = Loads<BM, BT, 8, TAIL>;
  const L loads(w, xq, n0, t0, T, N, K, wave, lane);
  Scales<2> scales(ws, xs, n0 + wr, t0 + wt, T, N, kb_all, c);

  v16f acc[4][2] = {}, p[2] = {};                   // p: sums not yet scaled
  float sc[2] = {};
  scales.load(0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < L::kCount; ++i) loads.send(i, 0, buf_a(S0{}), buf_b(S0{}));
  wait_vmem<0>();
  lds_sync();
  if (group) lds_sync();                            // one phase behind
  __builtin_amdgcn_sched_barrier(0);

  auto pending = [&](int i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(p[j][v], sc[j], acc[i][j][v]);
  };
  auto step = [&](auto stage, int kb) {
    using R = std::integral_constant<int, 1 - decltype(stage)::value>;
    const int next = min(kb + 1, kb_all - 1);       // past the end the last block once more, not read
    uint4 fb[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // ---- phase L
      // piece 2 q + h of a row sits at its first address with bits 5 and 6 turned by q
      int ra = (wr + 32 * i + c) * kF8Block + 16 * (h ^ (c >> 1 & 7));
      int rb = (wt + c) * kF8Block + 16 * (h ^ (c >> 1 & 7));
      __asm__ volatile("" : "+v"(ra), "+v"(rb));    // made anew: kept, they would not fit
      uint4 fa[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        fa[q] = *reinterpret_cast<const uint4*>(buf_a(stage) + (ra ^ (32 * q)));
        if (i == 0)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            fb[j][q] = *reinterpret_cast<const uint4*>(buf_b(stage) + (rb ^ (32 * q)) + 32 * j * kF8Block);
      }
      __builtin_amdgcn_sched_barrier(0);
      pending((i + 3) % 4);
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) sc[j] = scales.x[j] * scales.w;
        scales.load(next);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (TAIL) {
        if (i == 0)
#pragma unroll
          for (int j = 0; j < 2; ++j) cut_tail(fb[j], kb, h, K);
      }
      if (i == 3) wait_vmem<0>();
      lds_sync();
      __builtin_amdgcn_sched_barrier(0);
      // ---- phase M
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v16f zero = {};
        p[j] = mfma32(operand8(fa[0], fa[1]), operand8(fb[j][0], fb[j][1]), zero);
        p[j] = mfma32(operand8(fa[2], fa[3]), operand8(fb[j][2], fb[j][3]), p[j]);
        if (i < 2)
#pragma unroll
          for (int l = 0; l < 2; ++l) loads.send(4 * i + 2 * j + l, next, buf_a(R{}), buf_b(R{}));
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      lds_sync();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(L::kCount == 8, "two loads with each tile of the first two rows");
  int kb = 0;
  for (; kb + 2 <= kb_all; kb += 2) {
    step(S0{}, kb);
    step(S1{}, kb + 1);
  }
  if (kb < kb_all) step(S0{}, kb);
  if (!group) lds_sync();
  pending(3);
  wait_vmem<0>();                                   // loads past the end land before the block ends
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      store_tile<true>(acc[i][j], y, t0 + wt + 32 * j + c, n0 + wr + 32 * i, h, T, N);
}

// ------------------------------------------------------------------ matrices

// One block of 128 x 128 per workgroup, in registers between the maximum and
// the codes: 32 lanes have a row's 512 bytes.  Bound by memory (28672 x 8192, 940 MB read
// and 235 written in 205 us, 5.7 TB/s; 576 x 2512 3.8, its launch).
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

// Four codes per thread; bound by memory (28672 x 8192 206 us, 5.7 TB/s).
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

// T * N <= 2^36: about 2^24 tiles of 64 x 64 at most, of 192 threads, fewer than 2^32.
template <int BM, int BT, typename F>
hipError_t launch_tiles(F whole, F tail, int threads, const uint8_t* w, const float* ws, const uint8_t* xq,
                        const float* xs, int64_t t, int64_t n, int64_t k, void* y, hipStream_t stream) {
  const int t_tiles = (int)((t + BT - 1) / BT), tiles = (int)((n + BM - 1) / BM * t_tiles);
  (k % kF8Block ? tail : whole)<<<(unsigned)((tiles + 7) / 8 * 8), threads, 0, stream>>>(
      w, ws, xq, xs, (int)t, (int)n, (int)k, t_tiles, tiles, y);
  return hipGetLastError();
}

template <bool BF16, bool CUT, int WR, int WT, int GROUPS, int STAGES>
hipError_t launch_tile(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs, int64_t t,
                       int64_t n, int64_t k, void* y, hipStream_t stream) {
  return launch_tiles<64 * WR, 64 * WT>(k_f8_tile<BF16, CUT, false, WR, WT, GROUPS, STAGES>,
                                        k_f8_tile<BF16, CUT, true, WR, WT, GROUPS, STAGES>,
                                        64 * WR * WT * GROUPS, w, ws, xq, xs, t, n, k, y, stream);
}

template <bool BF16, bool CUT>
hipError_t forward(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs, int64_t t,
                   int64_t n, int64_t k, void* y, hipStream_t stream) {
  const F8Kernel kernel = f8_kernel(t, n, k, CUT, device_cus());
  switch (kernel) {
    case kF8Few1:
    case kF8Few2: {
      const int rows = kernel == kF8Few2 ? 32 : f8_few_rows(t, n, device_cus());
      const int t_tiles = (int)((t + 63) / 64);
      const unsigned grid = (unsigned)((n + rows - 1) / rows * t_tiles);
      auto few = [&](auto full) {
        constexpr bool F = decltype(full)::value;
        return t <= 16 ? k_f8_few<1, 1, F, BF16> : t <= 32 ? k_f8_few<2, 1, F, BF16> : k_f8_few<4, 1, F, BF16>;
      };
      auto* f = rows == 32 ? k_f8_few<2, 2, true, BF16>
              : rows == 16 ? few(std::true_type{})
                           : few(std::false_type{});
      f<<<grid, 64 * kFewWaves, 0, stream>>>(w, ws, xq, xs, (int)t, (int)n, (int)k, rows, t_tiles, y);
      return hipGetLastError();
    }
    case kF8Turns:
      return launch_tiles<256, 256>(k_f8_turns<false>, k_f8_turns<true>, 512, w, ws, xq, xs, t, n, k, y, stream);
    case kF8Wide: return launch_tile<BF16, CUT, 4, 2, 1, 3>(w, ws, xq, xs, t, n, k, y, stream);
    case kF8Square: return launch_tile<BF16, CUT, 2, 2, 2, 2>(w, ws, xq, xs, t, n, k, y, stream);
    case kF8Tall: return launch_tile<BF16, CUT, 2, 1, 2, 3>(w, ws, xq, xs, t, n, k, y, stream);
    default: return launch_tile<BF16, CUT, 1, 1, 3, 3>(w, ws, xq, xs, t, n, k, y, stream);
  }
}

}  // namespace

hipError_t launch_forward_f8(const uint8_t* w, const float* ws, const uint8_t* xq, const float* xs,
                             int64_t t, int64_t n, int64_t k, void* y, int y_dtype,
                             hipStream_t stream) {
  return y_dtype == BL_F32    ? forward<false, false>(w, ws, xq, xs, t, n, k, y, stream)
         : y_dtype == BL_BF16 ? forward<true, false>(w, ws, xq, xs, t, n, k, y, stream)
                              : forward<true, true>(w, ws, xq, xs, t, n, k, y, stream);
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
