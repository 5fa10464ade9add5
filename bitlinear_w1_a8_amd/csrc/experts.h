// Internal declarations of the routed-expert and 4-bit operators.
#pragma once

#include <atomic>

#include "bitlinear_experts.h"
#include "bitlinear_w4.h"
#include "bl_internal.h"
#include "experts_plan.h"
#include "w4_plan.h"

namespace bl {

// A kernel that may ask for more dynamic LDS than the 64 KiB that a launch
// gets without saying so; said once per kernel and device (saying it again,
// as two threads may, does no harm).
template <auto KERNEL>
struct Kernel {
  static constexpr auto kernel = KERNEL;
  hipError_t allow_lds() const {
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (set.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL),
                            hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
    if (e == hipSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

// ---------------------------------------------------------------- router (route.hip)

constexpr int kOneBlock = 64;      // tokens that one block routes alone: a bit each in an expert's mask
constexpr int kRouteTokens = 32;   // tokens of a block where there are more

size_t route_workspace_bytes(int64_t t, int64_t e);
hipError_t launch_route(const void* logits, int bf16, int64_t t, int64_t e, int64_t k, int share,
                        int32_t* ids, float* weights, int32_t* offsets, int32_t* pairs,
                        int32_t* slots, int32_t* workspace, hipStream_t stream);

// ---------------------------------------------------------------- ragged rows

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
// fewer, or when the counts of overlapping experts pass 32 bits.  Called by
// whole waves, with the same result in each.
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
      const unsigned long long reach = __ballot(seen + sum > c);
      const int at = reach ? __builtin_ctzll(reach) : 0;
      const int first = __builtin_amdgcn_readlane(seen + sum - n, at);
      lo = __builtin_amdgcn_readlane(lo, at);
      hi = __builtin_amdgcn_readlane(hi, at);
      expert = base + at;
      p0 = lo + (c - first) * rows;
      p1 = min(p0 + rows, hi);
      return reach != 0 && expert < s.E && p0 >= lo && p0 < hi;
    }
    seen += total;
  }
  return false;
}

// Row blocks of `rows` slots that P slots over E experts can make at most.
inline int64_t row_blocks(int64_t p, int64_t e, int64_t rows) {
  const int64_t most = p / rows + (p < e ? p : e);
  return most < p ? most : p;
}

// Row blocks of `rows` slots that the experts make together (whole waves).
__device__ __forceinline__ int count_row_blocks(const Slots& s, int rows) {
  int n = 0;
  for (int e = threadIdx.x & 63; e < s.E; e += 64) {
    const int lo = min(max(s.offsets[e], 0), s.P), hi = min(max(s.offsets[e + 1], lo), s.P);
    n += (hi - lo + rows - 1) / rows;
  }
  return wave_sum_i(n);
}

// Words `at` .. `at` + 3 of a packed row of `words`, for products with
// activations that are zero past K: words past the row's end may be any.
//   kWhole  K % 64 == 0: a 16-byte load (quads past the end repeat the last).
//   kShort  rows lie on 4-byte boundaries, where 16-byte loads may, and a quad
//           that reaches past the row's end is loaded from its last four words;
//           settle() moves it down, at use, so that the load is not waited for
//           earlier.  (Gated, 33 tokens, 64 experts of 2576 -> 2 x 1000: single
//           words 46.5 us, moved at once 27.7, at use 25.3.)
//   kWords  K < 64, fewer than four words: one by one.
enum Quads { kWhole = 0, kShort = 1, kWords = 2 };
template <int Q>
__device__ __forceinline__ uint4 load_quad(const uint32_t* row, int at, int words) {
  if constexpr (Q == kWhole) {
    return *reinterpret_cast<const uint4*>(row + min(at, words - 4));
  } else if constexpr (Q == kShort) {
    uint32_t w[4];
    __builtin_memcpy(w, row + min(at, words - 4), 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(row[min(at, words - 1)], row[min(at + 1, words - 1)],
                      row[min(at + 2, words - 1)], row[min(at + 3, words - 1)]);
  }
}
template <int Q>
__device__ __forceinline__ uint4 settle(uint4 w, int at, int words) {
  if constexpr (Q == kShort) {
    const int by = at - min(at, words - 4);
    if (by & 1) { w.x = w.y; w.y = w.z; w.z = w.w; }
    if (by & 2) { w.x = w.z; w.y = w.w; }
  }
  return w;
}

// ---------------------------------------------------------------- experts (experts.hip, gemm.hip)

// The tiled MFMA kernel over each expert's rows: y (or, gated, h) by slot.
// K >= 64, rows of x times K below 2^31, N * K / 16 below 2^31.
hipError_t launch_gemm_experts(const Slots& s, const uint8_t* packed, const float* gamma,
                               const float* gamma2, const int8_t* xq, const float* absmax,
                               int64_t n, int64_t k, float* y, uint16_t* h, int32_t* acc,
                               hipStream_t stream);

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
