// Products of routed tokens with their experts' ternary matrices (steps A2 +
// A3 per expert), ragged: expert e has the slots offsets[e] .. offsets[e + 1],
// known on the device only.  The grid covers the most row blocks that any
// split of P slots over E experts can make (each expert adds at most one
// partly filled one), every block finds its expert and rows from the offsets,
// and the blocks left over end at once.
#include <algorithm>
#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

// Batches whose step A1 is repeated by every block instead of launched on its
// own.  Gated, 64 experts of 2560 -> 2 x 1024, 8 per token, on one card: T = 1
// 7.5 against 9.3 us, T = 2 10.0 / 11.3, T = 4 13.1 / 13.5, T = 6 17.3 / 15.7.
constexpr int kFewTokens = 4;
// Weighted sums in one launch (k_experts_token), whose blocks stream a token's
// experts whoever else uses them: up to 32 pairs, or one per expert (64 experts of 1024 ->
// 2560, 8 per token: T = 1 5.7 against 11.8 us, T = 8 13.6 / 16.3, T = 12
// 18.5 / 16.8; 16 experts of 2048 -> 2560, 4 per token: T = 8 13.0 / 15.7, T = 12
// 17.5 / 15.9).
bool token_wins(int64_t p, int64_t e) { return p <= 32 || p <= e; }
// Slots per expert, were all alike, up to which the experts' rows go to
// k_experts_few rather than to the tiled kernel: fewer where that one's tiles
// fill the device (gated, 64 experts of 2560 -> 2 x 1024: 4 / 6 / 8 slots 22.7 /
// 23.8 / 26.0 against 24.2 / 24.4 / 25.6 us; 1024 -> 2560: 17.9 / 19.2 at 6 / 8
// slots against 17.7 / 18.4) than where they do not (8 experts of 2560 -> 2 x
// 1728: 12 / 24 slots 13.5 / 18.3 against 16.0 / 16.9; 16 experts: 8 / 12 slots
// 16.8 / 20.3 against 17.5 / 19.1, of 1728 -> 2560 13.0 / 14.1 against 14.9 / 15.1).
bool few_wins(int64_t p, int64_t e, int64_t n) {
  const bool fill = std::min(p, e) * ((n + 127) / 128) > 2 * device_cus();
  return p <= (fill ? 6 : 12) * e;
}

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

// LDS row stride of int8 activations: whole chunks of 256 k, zero past K, and
// 16 bytes that spread the rows of one operand read over the banks.
__host__ __device__ constexpr int few_stride(int k) { return ((k + 255) & ~255) + 16; }

// A few rows per expert (decode batches): up to R <= 16 slots of one expert,
// their int8 rows whole in LDS, against 16 weight rows per wave over all of K
// on v_mfma_i32_16x16x64_i8, which contracts the codes t + 1; each row's sum of
// q comes off at the end.  No wave waits for another after the rows are staged
// and none adds to another's sums, so a wave is one run of loads: its first U
// chunks (256 k of 16 rows, 1 KiB) are in flight while the rows are staged.
// Gated, 33 tokens, 6 of 64 experts each, 2560 -> 2 x 1000, weights from memory: the
// 45 experts hit, 58 MB, in 18.5 us (3.1 TB/s; 15.2 where part of the weights is
// still in the cache behind the L2s): the waves wait, VALU issue is 17 thousand
// of some 44 thousand cycles.  One token, 8 experts, 2560 -> 2 x 1024: 8.7 us, of
// which the launch and three dependent loads are more than half.
// MODE kBf16, kF32: step A1 happens in the staging (every block of an expert
// repeats it: for batches of a few tokens, whose own launch would cost more),
// and the first block of an expert writes the codes and absmax of the tokens
// whose first rank it has.
template <int MODE, bool GATED, int U, int Q>
__global__ __launch_bounds__(512) void k_experts_few(const Slots slots,
                                                     const uint32_t* __restrict__ packed,
                                                     const float* __restrict__ gamma,
                                                     const float* __restrict__ gamma2,
                                                     const void* __restrict__ x,
                                                     const float* __restrict__ absmax, int N, int K,
                                                     int R, int first, float* __restrict__ y,
                                                     uint16_t* __restrict__ h,
                                                     int32_t* __restrict__ acc_out,
                                                     int8_t* __restrict__ xq_out,
                                                     float* __restrict__ absmax_out) {
  extern __shared__ __align__(16) unsigned char xs[];   // [R][few_stride(K)], then raw [R][K]
  __shared__ int qsum[16], amax[16];
  int expert, p0, p1;
  if (!find_rows(slots, first + (int)blockIdx.y, R, expert, p0, p1)) return;
  const int nrow = p1 - p0;
  const int tid = threadIdx.x, lane = tid & 63, nthreads = blockDim.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), nwaves = nthreads >> 6;
  const int qg = lane >> 4, r = lane & 15;
  const int K16 = K >> 4, nchunks = (K + 255) >> 8, stride = few_stride(K);
  const int n0 = (blockIdx.x * nwaves + wave) * 16;

  // The rows first, straight into LDS, then the weights: loads come back in
  // order, so the rows can be worked on while the weights are in flight.
  constexpr int kBytes = MODE == kInt8 ? 1 : MODE == kBf16 ? 2 : 4;
  const int my_row = slot_row(slots, p0 + min(r, nrow - 1));   // of slot r, in every wave
  const int row_bytes = K * kBytes;
  unsigned char* land = MODE == kInt8 ? xs : xs + R * stride;     // int8 rows, or raw ones
  const int land_stride = MODE == kInt8 ? stride : row_bytes;
  for (int i = wave; i < nrow; i += nwaves) {
    const unsigned char* src = static_cast<const unsigned char*>(x) +
                               (int64_t)__builtin_amdgcn_readlane(my_row, i) * row_bytes;
    for (int b = 0; b < row_bytes; b += 1024)
      if (b + 16 * lane < row_bytes)
        __builtin_amdgcn_global_load_lds((glb_ptr_t)(src + b + 16 * lane),
                                         (lds_ptr_t)(land + i * land_stride + b), 16, 0, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  // weights: lane (qg, r) takes 64 k (16 bytes) of row r per chunk; rows past N
  // are computed, never stored
  const int n = min(n0 + r, N - 1);
  const uint32_t* wrow = packed + ((int64_t)expert * N + n) * K16;
  uint4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = load_quad<Q>(wrow, 16 * min(u, nchunks - 1) + 4 * qg, K16);
  __builtin_amdgcn_sched_barrier(0);
  if (tid < 16) qsum[tid] = amax[tid] = 0;
  wait_vmem<U>();                                   // this wave's rows are in LDS
  lds_sync();
  if constexpr (MODE == kInt8) {
    for (int i = wave; i < nrow; i += nwaves) {
      uint4* row = reinterpret_cast<uint4*>(xs + i * stride);
      int s = 0;
      for (int v = lane; v < K16; v += 64) {
        const uint4 q = row[v];
        s = __builtin_amdgcn_sdot4((int)q.x, 0x01010101, s, false);
        s = __builtin_amdgcn_sdot4((int)q.y, 0x01010101, s, false);
        s = __builtin_amdgcn_sdot4((int)q.z, 0x01010101, s, false);
        s = __builtin_amdgcn_sdot4((int)q.w, 0x01010101, s, false);
      }
      if (K16 + lane < 16 * nchunks) row[K16 + lane] = make_uint4(0, 0, 0, 0);   // fewer than 16
      s = wave_sum_i(s);
      if (lane == 0) qsum[i] = s;
    }
  } else {
    for (int i = 0; i < nrow; ++i) {
      int m = 0;
      for (int k = 4 * tid; k < K; k += 4 * nthreads) {
        Raw4<MODE> f;
        f.load(land + i * land_stride, k);
        m = max(m, f.max_bits());
      }
      m = wave_max_nonneg(m);
      if (lane == 0) atomicMax(&amax[i], m);
    }
    lds_sync();
    for (int i = 0; i < nrow; ++i) {
      const float a = __int_as_float(amax[i]), s = kQb / fmaxf(a, kEps);
      const int row = __builtin_amdgcn_readlane(my_row, i);
      // the block that writes a token's codes: its first rank's, or, with one
      // row per slot, the slot's
      const bool out = blockIdx.x == 0 && (slots.k == 0 || slots.pairs[p0 + i] == row * slots.k);
      int sum = 0;
      for (int k = 4 * tid; k < nchunks * 256; k += 4 * nthreads) {
        Raw4<MODE> f;
        f.clear();
        if (k < K) f.load(land + i * land_stride, k);
        const uint32_t q = quant4(f, s);
        sum = __builtin_amdgcn_sdot4((int)q, 0x01010101, sum, false);
        *reinterpret_cast<uint32_t*>(xs + i * stride + k) = q;
        if (out && k < K) *reinterpret_cast<uint32_t*>(xq_out + (int64_t)row * K + k) = q;
      }
      sum = wave_sum_i(sum);
      if (lane == 0) atomicAdd(&qsum[i], sum);
      if (out && tid == 0) absmax_out[row] = a;
    }
  }
  lds_sync();

  const unsigned char* xrow = xs + (r < nrow ? r : 0) * stride + 64 * qg;
  v4i acc = {0, 0, 0, 0};
  for (int c0 = 0; c0 < nchunks; c0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u >= nchunks) break;
      const uint4* xv = reinterpret_cast<const uint4*>(xrow + (c0 + u) * 256);
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

  // lane (qg, r) holds rows 4 qg .. 4 qg + 3 of slot r
  if (r >= nrow) return;
  const int64_t p = p0 + r;
  const int nn = n0 + 4 * qg;
  const float a = MODE == kInt8 ? absmax[my_row] : __int_as_float(amax[r]);   // lane r's row
  const int qs = qsum[r];
  if (acc_out) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (nn + v < N) acc_out[p * N + nn + v] = acc[v] - qs;
  }
  if constexpr (GATED) {
    const double gg = gamma_m(gamma[expert], a), gu = gamma_m(gamma2[expert], a);
#pragma unroll
    for (int v = 0; v < 4; v += 2)
      if (nn + v < N)
        h[p * (N >> 1) + ((nn + v) >> 1)] = gated_relu2_bf16(acc[v] - qs, acc[v + 1] - qs, gg, gu);
  } else {
    const float sc = out_scale(gamma[expert], a);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (nn + v < N) y[p * N + nn + v] = (float)(acc[v] - qs) * sc;
  }
}

// The weighted sum for a few tokens, in one launch: a block has one token and
// 16 outputs, each of its k slots a team of `team` waves that split K.  A team
// quantises its slot's row (step A1; every block of the token repeats it) and
// contracts it with the slot's expert; the teams' exact sums meet in LDS, and
// the rescale and the sum over the ranks follow in order.  k * team <= 16.
// Bound by its trips to memory one after another: slot, offsets, row and weights
// (8 of 64 experts of 1024 -> 2560, 5.2 MB of weights: 6.6 us from memory, 5.7
// from the cache).
template <int MODE, int U, int Q>
__global__ __launch_bounds__(1024) void k_experts_token(const Slots slots,
                                                        const int32_t* __restrict__ slot_of,
                                                        const float* __restrict__ weights, int topk,
                                                        int team, const uint32_t* __restrict__ packed,
                                                        const float* __restrict__ gamma,
                                                        const void* __restrict__ x, int N, int K,
                                                        float* __restrict__ y,
                                                        int8_t* __restrict__ xq_out,
                                                        float* __restrict__ absmax_out) {
  extern __shared__ __align__(16) unsigned char xs[];   // [topk][few_stride(K)]
  __shared__ int amax[16], tile[16][16];
  __shared__ float scale[16], share[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qg = lane >> 4, r = lane & 15;
  const int t = blockIdx.y, j = wave / team, part = wave - j * team;
  const int K16 = K >> 4, nchunks = (K + 255) >> 8, stride = few_stride(K);
  const int per = (nchunks + team - 1) / team, c0 = part * per, c1 = min(c0 + per, nchunks);
  const int n0 = blockIdx.x * 16;
  if (tid < 256) (&tile[0][0])[tid] = 0;
  if (tid < 16) amax[tid] = 0;

  const int slot = min(slot_of[(int64_t)t * topk + j], slots.P - 1);   // below 0: no expert
  int expert = 0;                    // experts whose slots end at or before this one
  for (int base = 0; base < slots.E; base += 64) {
    const int e = base + lane;
    expert += __builtin_popcountll(__ballot(e < slots.E && slots.offsets[e + 1] <= slot));
  }
  expert = min(expert, slots.E - 1);
  const int row = slots.k ? t : max(slot, 0);
  constexpr int kBytes = MODE == kBf16 ? 2 : 4;
  const void* xrow = static_cast<const unsigned char*>(x) + (int64_t)row * K * kBytes;
  const uint32_t* wrow = packed + ((int64_t)expert * N + min(n0 + r, N - 1)) * K16;
  const bool live = slot >= 0 && c0 < c1;               // wave-uniform
  // the row before the weights, as above; its first U chunks stay in registers
  Raw4<MODE> xr[U];
  uint4 w[U];
  if (live) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(c0 + u, c1 - 1) * 256 + 4 * lane;
      xr[u].load(xrow, min(k, K - 4));
      if (k >= K) xr[u].clear();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      w[u] = load_quad<Q>(wrow, 16 * min(c0 + u, c1 - 1) + 4 * qg, K16);
  }
  const float g = gamma[expert];
  lds_sync();
  if (live) {
    int m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) m = max(m, xr[u].max_bits());
    for (int c = c0 + U; c < c1; ++c) {
      const int k = c * 256 + 4 * lane;
      if (k < K) {
        Raw4<MODE> f;
        f.load(xrow, k);
        m = max(m, f.max_bits());
      }
    }
    m = wave_max_nonneg(m);
    if (lane == 0) atomicMax(&amax[j], m);
  }
  lds_sync();
  const float a = __int_as_float(amax[j]);
  if (part == 0 && lane == 0) {
    scale[j] = out_scale(g, a);
    share[j] = slot >= 0 ? weights[(int64_t)t * topk + j] : 0.0f;
  }
  if (live) {
    const float s = kQb / fmaxf(a, kEps);
    const bool out = blockIdx.x == 0 && (slots.k == 0 || j == 0);
    int sum = 0;
    auto put = [&](const Raw4<MODE>& f, int k) {
      const uint32_t q = quant4(f, s);
      sum = __builtin_amdgcn_sdot4((int)q, 0x01010101, sum, false);
      *reinterpret_cast<uint32_t*>(xs + j * stride + k) = q;
      if (out && k < K) *reinterpret_cast<uint32_t*>(xq_out + (int64_t)row * K + k) = q;
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < c1) put(xr[u], (c0 + u) * 256 + 4 * lane);
    for (int c = c0 + U; c < c1; ++c) {
      const int k = c * 256 + 4 * lane;
      Raw4<MODE> f;
      f.clear();
      if (k < K) f.load(xrow, k);
      put(f, k);
    }
    if (out && part == 0 && lane == 0) absmax_out[row] = a;
    sum = wave_sum_i(sum);
    wave_lds_sync();                                  // this wave's own chunks: no block barrier
    // every column of the second operand is the one row: each holds the sums
    v4i acc = {0, 0, 0, 0};
    const unsigned char* xq = xs + j * stride + 64 * qg;
    for (int b0 = c0; b0 < c1; b0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b0 + u >= c1) break;
        const uint4* xv = reinterpret_cast<const uint4*>(xq + (b0 + u) * 256);
        const uint4 p = settle<Q>(w[u], 16 * (b0 + u) + 4 * qg, K16);
        const uint32_t word[4] = {p.x, p.y, p.z, p.w};
        if (b0 + U + u < c1) w[u] = load_quad<Q>(wrow, 16 * (b0 + U + u) + 4 * qg, K16);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint4 b = xv[v];
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              operand(word[v]), v4i{(int)b.x, (int)b.y, (int)b.z, (int)b.w}, acc, 0, 0, 0);
        }
      }
    }
    if (r == 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v) atomicAdd(&tile[j][4 * qg + v], acc[v] - sum);
    }
  }
  lds_sync();
  if (tid < 16 && n0 + tid < N) {
    float s = 0.0f;
    for (int i = 0; i < topk; ++i)
      if (slot_of[(int64_t)t * topk + i] >= 0) s = fmaf(share[i], (float)tile[i][tid] * scale[i], s);
    y[(int64_t)t * N + n0 + tid] = s;
  }
}

// y[t] = sum over j of weights[t, j] * rows[slots[t, j]], in order of j.  Bound
// by reading the slots' rows, which the product has just written (2048 tokens
// of 8 x 2560: 168 MB in, 21 out in 27 us, 7 TB/s, so mostly from the cache
// behind the L2s).
__global__ __launch_bounds__(256) void k_experts_combine(const float* __restrict__ rows,
                                                         const int32_t* __restrict__ slots,
                                                         const float* __restrict__ weights, int k,
                                                         int P, int N, int col_blocks,
                                                         int64_t units, float* __restrict__ y) {
  const bool vec = (N & 3) == 0;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {   // (token, 1024 columns)
  const int t = (int)(u / col_blocks), cb = (int)(u - (int64_t)t * col_blocks);
  const int n0 = cb * 1024 + 4 * threadIdx.x;
  if (n0 >= N) continue;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) {
    const int slot = slots[(int64_t)t * k + j];
    if (slot < 0) continue;
    const float w = weights[(int64_t)t * k + j];
    const float* row = rows + (int64_t)min(slot, P - 1) * N + n0;
    if (vec) {
      const float4 v = *reinterpret_cast<const float4*>(row);
      s[0] = fmaf(w, v.x, s[0]); s[1] = fmaf(w, v.y, s[1]);
      s[2] = fmaf(w, v.z, s[2]); s[3] = fmaf(w, v.w, s[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + i < N) s[i] = fmaf(w, row[i], s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < N) y[(int64_t)t * N + n0 + i] = s[i];
  }
}

// Step A1 of any number of rows.  A launch has fewer than 2^32 threads and a
// row takes up to 1024 of them, so 2^21 rows go at a time.
hipError_t quant_rows(const void* x, int bf16, int64_t rows, int64_t k, int8_t* xq, float* absmax,
                      hipStream_t stream) {
  constexpr int64_t kMost = int64_t(1) << 21;
  hipError_t e = hipSuccess;
  for (int64_t r = 0; e == hipSuccess && r < rows; r += kMost)
    e = launch_quant(static_cast<const unsigned char*>(x) + r * k * (bf16 ? 2 : 4), bf16,
                     std::min(rows - r, kMost), k, xq + r * k, absmax + r, nullptr, stream);
  return e;
}

// LDS of k_experts_few for R rows: the int8 rows, and the raw ones that they
// are made from.
size_t few_lds(int64_t k, int rows, int mode) {
  return (size_t)rows * (few_stride((int)k) + (mode == kInt8 ? 0 : mode == kBf16 ? 2 * k : 4 * k));
}
bool few_fits(int64_t k, int rows, int mode) {
  return few_lds(k, rows, mode) <= (size_t)kMaxLds;
}

template <int MODE, bool GATED>
hipError_t launch_few(const Slots& s, const uint8_t* packed, const float* gamma,
                      const float* gamma2, const void* x, const float* absmax, int64_t n,
                      int64_t k, int rows, float* y, uint16_t* h, int32_t* acc, int8_t* xq_out,
                      float* absmax_out, hipStream_t stream) {
  const auto* w = reinterpret_cast<const uint32_t*>(packed);
  // 128 weight rows per block where that leaves blocks enough (gated, 64
  // experts of 2560 -> 2 x 1024, 8 slots each: 27.6 -> 24.3 us), else 64
  const int waves = ((n + 127) / 128) * std::min(s.P, s.E) >= 512 ? 8 : 4;
  const int64_t blocks = row_blocks(s.P, s.E, rows), bn = 16 * waves;
  const size_t lds = few_lds(k, rows, MODE);
  auto go = [&](auto kern) {
    hipError_t e = kern.allow_lds();
    for (int64_t b = 0; e == hipSuccess && b < blocks; b += 65535) {   // grid.y: at most 65535
      const dim3 grid((unsigned)((n + bn - 1) / bn), (unsigned)std::min<int64_t>(blocks - b, 65535));
      kern.kernel<<<grid, 64 * waves, lds, stream>>>(s, w, gamma, gamma2, x, absmax, (int)n, (int)k, rows,
                                              (int)b, y, h, acc, xq_out, absmax_out);
      e = hipGetLastError();
    }
    return e;
  };
  if (k < 64) return go(Kernel<k_experts_few<MODE, GATED, 2, kWords>>{});
  auto by_depth = [&](auto quads) {
    constexpr int Q = decltype(quads)::value;
    switch (few_depth(k)) {
      case 2: return go(Kernel<k_experts_few<MODE, GATED, 2, Q>>{});
      case 4: return go(Kernel<k_experts_few<MODE, GATED, 4, Q>>{});
      case 6: return go(Kernel<k_experts_few<MODE, GATED, 6, Q>>{});
      case 8: return go(Kernel<k_experts_few<MODE, GATED, 8, Q>>{});
      default: return go(Kernel<k_experts_few<MODE, GATED, 10, Q>>{});
    }
  };
  return k % 64 ? by_depth(std::integral_constant<int, kShort>{})
                : by_depth(std::integral_constant<int, kWhole>{});
}

template <int MODE>
hipError_t launch_token(const Slots& s, const bl_routing& r, const uint8_t* packed,
                        const float* gamma, const void* x, int64_t n, int64_t k, float* y,
                        int8_t* xq, float* absmax, hipStream_t stream) {
  const int nchunks = (int)((k + 255) / 256);
  const int topk = (int)r.k, team = std::max(1, std::min(16 / topk, (nchunks + 3) / 4));
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)r.T);
  const size_t lds = (size_t)topk * few_stride((int)k);
  auto go = [&](auto kern) {
    hipError_t e = kern.allow_lds();
    if (e != hipSuccess) return e;
    kern.kernel<<<grid, 64 * topk * team, lds, stream>>>(s, r.slots, r.weights, topk, team,
                                                  reinterpret_cast<const uint32_t*>(packed), gamma,
                                                  x, (int)n, (int)k, y, xq, absmax);
    return hipGetLastError();
  };
  if (k < 64) return go(Kernel<k_experts_token<MODE, 4, kWords>>{});
  return k % 64 ? go(Kernel<k_experts_token<MODE, 4, kShort>>{})
                : go(Kernel<k_experts_token<MODE, 4, kWhole>>{});
}

// Steps A2 + A3 of int8 rows by the kernel for their number and length.
template <bool GATED>
hipError_t launch_products(const Slots& s, int64_t x_rows, const uint8_t* packed,
                           const float* gamma, const float* gamma2, const int8_t* xq,
                           const float* absmax, int64_t n, int64_t k, float* y, uint16_t* h,
                           int32_t* acc, hipStream_t stream) {
  // the tiled kernel's 32-bit offsets, and blocks of 256 threads in a grid: past
  // them the rows go to the decode kernel, 16 at a time with the weights again
  // (64 experts of 8192 -> 2560, 8 per token, by slot: 32752 tokens 6.4 ms, 32768,
  // where rows * K reaches 2^31, 17.7)
  const bool tiled = k >= 64 && x_rows * k < (int64_t(1) << 31) &&
                     n * (k / 16) < (int64_t(1) << 31) &&
                     (n + 127) / 128 * row_blocks(s.P, s.E, 32) < (int64_t(1) << 24) - 8;
  if (tiled && !few_wins(s.P, s.E, n))
    return launch_gemm_experts(s, packed, gamma, gamma2, xq, absmax, n, k, y, h, acc, stream);
  int rows = 16;                       // as many as LDS holds; one of the longest fits
  while (!few_fits(k, rows, kInt8)) rows /= 2;
  return launch_few<kInt8, GATED>(s, packed, gamma, gamma2, xq, absmax, n, k, rows, y, h, acc,
                                  nullptr, nullptr, stream);
}

}  // namespace

hipError_t launch_gated_experts(const bl_routing& r, const void* x, int bf16, const uint8_t* packed,
                                const float* gamma_gate, const float* gamma_up, int64_t n,
                                int64_t k, uint16_t* h, int8_t* xq, float* absmax, int32_t* acc,
                                hipStream_t stream) {
  const Slots s{r.offsets, r.pairs, (int)r.E, (int)(r.T * r.k), (int)r.k};
  if (r.T <= kFewTokens && few_fits(k, kFewTokens, bf16 ? kBf16 : kF32)) {
    auto* f = bf16 ? launch_few<kBf16, true> : launch_few<kF32, true>;
    return f(s, packed, gamma_gate, gamma_up, x, nullptr, n, k, kFewTokens, nullptr, h, acc, xq,
             absmax, stream);
  }
  hipError_t e = quant_rows(x, bf16, r.T, k, xq, absmax, stream);
  if (e != hipSuccess) return e;
  return launch_products<true>(s, r.T, packed, gamma_gate, gamma_up, xq, absmax, n, k, nullptr, h,
                               acc, stream);
}

hipError_t launch_linear_experts(const bl_routing& r, const void* x, int bf16, int x_rows,
                                 const uint8_t* packed, const float* gamma, int64_t n, int64_t k,
                                 float* y, int y_rows, int8_t* xq, float* absmax, int32_t* acc,
                                 float* workspace, hipStream_t stream) {
  const bool combine = y_rows == BL_ROWS_TOKENS;
  const int64_t p = r.T * r.k, rows = x_rows == BL_ROWS_TOKENS ? r.T : p;
  const Slots s{r.offsets, r.pairs, (int)r.E, (int)p, x_rows == BL_ROWS_TOKENS ? (int)r.k : 0};
  // the last: blocks of up to 1024 threads, fewer than 2^32 of them in a row of the grid
  if (combine && r.k <= 16 && token_wins(p, r.E) && few_fits(k, (int)r.k, kInt8) && n < (1 << 25)) {
    auto* f = bf16 ? launch_token<kBf16> : launch_token<kF32>;
    return f(s, r, packed, gamma, x, n, k, y, xq, absmax, stream);
  }
  float* out = combine ? workspace : y;
  hipError_t e;
  if (r.T <= kFewTokens && few_fits(k, kFewTokens, bf16 ? kBf16 : kF32)) {
    auto* f = bf16 ? launch_few<kBf16, false> : launch_few<kF32, false>;
    e = f(s, packed, gamma, nullptr, x, nullptr, n, k, kFewTokens, out, nullptr, acc, xq, absmax,
          stream);
  } else {
    e = quant_rows(x, bf16, rows, k, xq, absmax, stream);
    if (e != hipSuccess) return e;
    e = launch_products<false>(s, rows, packed, gamma, nullptr, xq, absmax, n, k, out, nullptr,
                               acc, stream);
  }
  if (e != hipSuccess || !combine) return e;
  const int col_blocks = (int)((n + 1023) / 1024);
  const int64_t units = r.T * col_blocks;
  k_experts_combine<<<(unsigned)std::min<int64_t>(units, 1 << 20), 256, 0, stream>>>(
      out, r.slots, r.weights, (int)r.k, (int)p, (int)n, col_blocks, units, y);
  return hipGetLastError();
}

}  // namespace bl
