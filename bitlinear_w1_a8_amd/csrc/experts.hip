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

// The routing as the kernels take it.
struct Slots {
  const int32_t* offsets;
  const int32_t* pairs;
  int E, P;
  int k;                  // pairs / k is the row of x; 0: x has one row per slot
};

__device__ __forceinline__ int slot_row(const Slots& s, int p) {
  if (s.k == 0) return p;
  const int pair = min(max(s.pairs[p], 0), s.P - 1);
  return (int)((uint32_t)pair / (uint32_t)s.k);
}

// Block `c` of `rows` slots each, counted over the experts in order: its
// expert and slots p0 .. p1 - 1 (all in [0, P)), or false when there are
// fewer.  Called by whole waves, with the same result in each.
__device__ __forceinline__ bool find_rows(const Slots& s, int c, int rows, int& expert, int& p0,
                                          int& p1) {
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int base = 0; base < s.E; base += 64) {
    const int e = base + lane;
    int lo = 0, hi = 0;
    if (e < s.E) {
      lo = min(max(s.offsets[e], 0), s.P);
      hi = min(max(s.offsets[e + 1], lo), s.P);
    }
    const int n = (hi - lo + rows - 1) / rows;
    int sum = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    const int total = __builtin_amdgcn_readlane(sum, 63);
    if (c < seen + total) {
      const int at = __builtin_ctzll(__ballot(seen + sum > c));
      const int first = __builtin_amdgcn_readlane(seen + sum - n, at);
      lo = __builtin_amdgcn_readlane(lo, at);
      hi = __builtin_amdgcn_readlane(hi, at);
      expert = base + at;
      p0 = lo + (c - first) * rows;
      p1 = min(p0 + rows, hi);
      return true;
    }
    seen += total;
  }
  return false;
}

// Row blocks of `rows` slots that P slots over E experts can make at most.
int64_t row_blocks(int64_t p, int64_t e, int64_t rows) {
  return std::min(p, p / rows + std::min(p, e));
}

// Few rows per expert (decode): up to 16 slots of one expert against 16 RT of
// its rows per block; the waves split K and add their sums through LDS.  As
// in the decode kernels of a single matrix, v_mfma_i32_16x16x64_i8 contracts
// the codes t + 1 and each wave takes the sum of q over its own k off again.
template <int VEC, int RT, int U, bool GATED>
__global__ __launch_bounds__(256) void k_experts_rows(const Slots slots,
                                                      const uint32_t* __restrict__ packed,
                                                      const float* __restrict__ gamma,
                                                      const float* __restrict__ gamma2,
                                                      const int8_t* __restrict__ xq,
                                                      const float* __restrict__ absmax, int N,
                                                      int K, int first, float* __restrict__ y,
                                                      uint16_t* __restrict__ h,
                                                      int32_t* __restrict__ acc_out) {
  constexpr int kWaves = 4, kRows = 16 * RT;
  __shared__ int red[kWaves][RT * 4][64];
  int expert, p0, p1;
  if (!find_rows(slots, first + (int)blockIdx.y, 16, expert, p0, p1)) return;
  const int nrow = p1 - p0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int qg = lane >> 4, r = lane & 15;
  const int K16 = K >> 4;
  const int nchunks = (K16 + 4 * VEC - 1) / (4 * VEC);
  const int n0 = blockIdx.x * kRows;

  const uint32_t* wrow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int n = min(n0 + 16 * rt + r, N - 1);     // rows past N are computed, never stored
    wrow[rt] = packed + ((int64_t)expert * N + n) * K16;
  }
  const bool valid = r < nrow;
  const int8_t* xrow = xq + (int64_t)slot_row(slots, valid ? p0 + r : p0) * K;

  v4i acc[RT];
  int qs = 0;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] = v4i{0, 0, 0, 0};
  for (int c0 = wave * U; c0 < nchunks; c0 += kWaves * U) {
    uint32_t wv[U][RT][VEC], xv[U][4 * VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int wi = (c0 + u) * 4 * VEC + qg * VEC;
      const bool kvalid = wi < K16;                 // VEC divides K16 when VEC > 1
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if constexpr (VEC == 4) {
          const uint4 w4 =
              kvalid ? *reinterpret_cast<const uint4*>(wrow[rt] + wi) : make_uint4(0, 0, 0, 0);
          wv[u][rt][0] = w4.x; wv[u][rt][1] = w4.y; wv[u][rt][2] = w4.z; wv[u][rt][3] = w4.w;
        } else {
          wv[u][rt][0] = kvalid ? wrow[rt][wi] : 0u;
        }
      }
      const uint4* src = reinterpret_cast<const uint4*>(xrow + (int64_t)wi * 16);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const uint4 x4 = kvalid && valid ? src[v] : make_uint4(0, 0, 0, 0);
        xv[u][4 * v + 0] = x4.x; xv[u][4 * v + 1] = x4.y;
        xv[u][4 * v + 2] = x4.z; xv[u][4 * v + 3] = x4.w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int d = 0; d < 4 * VEC; ++d)
        qs = __builtin_amdgcn_sdot4((int)xv[u][d], 0x01010101, qs, false);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const v4i b = {(int)xv[u][4 * v + 0], (int)xv[u][4 * v + 1], (int)xv[u][4 * v + 2],
                       (int)xv[u][4 * v + 3]};
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint32_t w = wv[u][rt][v];
          const v4i a = {(int)codes_of(w, 0), (int)codes_of(w, 1), (int)codes_of(w, 2),
                         (int)codes_of(w, 3)};
          acc[rt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc[rt], 0, 0, 0);
        }
      }
    }
  }
  qs += __shfl_xor(qs, 16);
  qs += __shfl_xor(qs, 32);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wave][rt * 4 + v][lane] = acc[rt][v] - qs;
  __syncthreads();

  const float g = gamma[expert];
  auto sum_of = [&](int nl, int tl) {
    const int i = nl & 15, slot = (nl >> 4) * 4 + (i & 3), ln = (i >> 2) * 16 + tl;
    int s = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += red[w][slot][ln];
    return s;
  };
  if constexpr (GATED) {
    // rows 2i (gate) and 2i + 1 (up) make output n0 / 2 + i
    const float g2 = gamma2[expert];
    for (int idx = threadIdx.x; idx < kRows / 2 * nrow; idx += 256) {
      const int pl = idx % (kRows / 2), tl = idx / (kRows / 2);
      const int n = n0 + 2 * pl;
      if (n >= N) continue;
      const int sg = sum_of(2 * pl, tl), su = sum_of(2 * pl + 1, tl);
      const int64_t p = p0 + tl;
      if (acc_out) {
        acc_out[p * N + n] = sg;
        acc_out[p * N + n + 1] = su;
      }
      const float a = absmax[slot_row(slots, p0 + tl)];
      h[p * (N >> 1) + (n >> 1)] = gated_relu2_bf16(sg, su, gamma_m(g, a), gamma_m(g2, a));
    }
  } else {
    for (int idx = threadIdx.x; idx < kRows * nrow; idx += 256) {
      const int nl = idx % kRows, tl = idx / kRows;
      const int n = n0 + nl;
      if (n >= N) continue;
      const int s = sum_of(nl, tl);
      const int64_t o = (int64_t)(p0 + tl) * N + n;
      if (acc_out) acc_out[o] = s;
      y[o] = (float)s * out_scale(g, absmax[slot_row(slots, p0 + tl)]);
    }
  }
}

// y[t] = sum over j of weights[t, j] * rows[slots[t, j]], in order of j.
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

template <bool GATED>
hipError_t launch_rows(const Slots& s, const uint8_t* packed, const float* gamma,
                       const float* gamma2, const int8_t* xq, const float* absmax, int64_t n,
                       int64_t k, float* y, uint16_t* h, int32_t* acc, hipStream_t stream) {
  const auto* w = reinterpret_cast<const uint32_t*>(packed);
  const int64_t blocks = row_blocks(s.P, s.E, 16);
  for (int64_t b = 0; b < blocks; b += 65535) {     // grid.y holds at most 65535 blocks
    const dim3 grid((unsigned)((n + 15) / 16), (unsigned)std::min<int64_t>(blocks - b, 65535));
    if (k % 64 == 0)
      k_experts_rows<4, 1, 2, GATED><<<grid, 256, 0, stream>>>(s, w, gamma, gamma2, xq, absmax,
                                                               (int)n, (int)k, (int)b, y, h, acc);
    else
      k_experts_rows<1, 1, 4, GATED><<<grid, 256, 0, stream>>>(s, w, gamma, gamma2, xq, absmax,
                                                               (int)n, (int)k, (int)b, y, h, acc);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gated_experts(const bl_routing& r, const void* x, int bf16, const uint8_t* packed,
                                const float* gamma_gate, const float* gamma_up, int64_t n,
                                int64_t k, uint16_t* h, int8_t* xq, float* absmax, int32_t* acc,
                                hipStream_t stream) {
  const Slots s{r.offsets, r.pairs, (int)r.E, (int)(r.T * r.k), (int)r.k};
  hipError_t e = launch_quant(x, bf16, r.T, k, xq, absmax, nullptr, stream);
  if (e != hipSuccess) return e;
  return launch_rows<true>(s, packed, gamma_gate, gamma_up, xq, absmax, n, k, nullptr, h, acc,
                           stream);
}

hipError_t launch_linear_experts(const bl_routing& r, const void* x, int bf16, int x_rows,
                                 const uint8_t* packed, const float* gamma, int64_t n, int64_t k,
                                 float* y, int y_rows, int8_t* xq, float* absmax, int32_t* acc,
                                 float* workspace, hipStream_t stream) {
  const bool combine = y_rows == BL_ROWS_TOKENS;
  const int64_t p = r.T * r.k;
  const Slots s{r.offsets, r.pairs, (int)r.E, (int)p, x_rows == BL_ROWS_TOKENS ? (int)r.k : 0};
  hipError_t e = launch_quant(x, bf16, x_rows == BL_ROWS_TOKENS ? r.T : p, k, xq, absmax, nullptr,
                              stream);
  if (e != hipSuccess) return e;
  float* rows = combine ? workspace : y;
  e = launch_rows<false>(s, packed, gamma, nullptr, xq, absmax, n, k, rows, nullptr, acc, stream);
  if (e != hipSuccess || !combine) return e;
  const int col_blocks = (int)((n + 1023) / 1024);
  const int64_t units = r.T * col_blocks;
  k_experts_combine<<<(unsigned)std::min<int64_t>(units, 1 << 20), 256, 0, stream>>>(
      rows, r.slots, r.weights, (int)r.k, (int)p, (int)n, col_blocks, units, y);
  return hipGetLastError();
}

}  // namespace bl
