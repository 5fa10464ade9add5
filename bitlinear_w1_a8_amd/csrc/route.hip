// The router of the expert layers: each token's k largest logits, their
// softmax weights, and the slots of all (token, rank) pairs in expert order.
//
// Selection.  A wave owns a token and holds its E logits in registers, VPL
// consecutive ones per lane, as keys whose unsigned order is that of the
// values (0 for a masked one).  A rank is one wave maximum of the lanes' best
// keys and a ballot; lanes hold consecutive experts, so the first lane of the
// ballot has the lowest expert among equals.
//
// Slots.  A block takes 64 tokens, whose choice of expert e is one 64-bit
// mask: a pair's place among its expert's pairs of the block is the number of
// mask bits below its token.  The masks are integers set by or, so nothing
// depends on an order of execution.  Up to 64 tokens one block does
// everything; more take a second kernel that turns the blocks' counts into
// starts (one wave per expert) and a third that writes the slots.
#include <type_traits>

#include "experts.h"

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxE = BITLINEAR_MAX_EXPERTS;
static_assert(kMaxE <= kThreads, "one thread per expert");

// unsigned key of a logit, growing with its value; 0 for -inf and NaN
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -__builtin_inff())) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);     // -0 becomes +0
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((int)key < 0 ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ uint32_t wave_max_u(uint32_t u) {
  auto mx = [](uint32_t a, int b) { return a > (uint32_t)b ? a : (uint32_t)b; };
  u = mx(u, __builtin_amdgcn_update_dpp(0, (int)u, 0xB1, 0xF, 0xF, false));
  u = mx(u, __builtin_amdgcn_update_dpp(0, (int)u, 0x4E, 0xF, 0xF, false));
  u = mx(u, __builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xF, 0xF, false));
  u = mx(u, __builtin_amdgcn_update_dpp(0, (int)u, 0x140, 0xF, 0xF, false));
  const uint32_t a = mx(__builtin_amdgcn_readlane((int)u, 0), __builtin_amdgcn_readlane((int)u, 16));
  const uint32_t b = mx(__builtin_amdgcn_readlane((int)u, 32), __builtin_amdgcn_readlane((int)u, 48));
  return a > b ? a : b;
}

// Exclusive sum over the block's threads of one count per thread, and the
// total; part: kWaves ints of LDS.
__device__ __forceinline__ int block_scan(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) part[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int p = part[w];
    if (w < wave) before += p;
    all += p;
  }
  total = all;
  return before + s - v;
}

// Top k of one block's tokens; marks each choice in the masks.
template <int VPL, bool BF16>
__device__ __forceinline__ void choose(const void* __restrict__ logits, int64_t t0, int nt, int E,
                                       int k, int share, int32_t* __restrict__ ids,
                                       float* __restrict__ weights, unsigned long long* mask) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i < nt; i += kWaves) {
    const int64_t t = t0 + i;
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane * VPL + v;
      key[v] = 0;
      if (e < E) {
        float f;
        if constexpr (BF16)
          f = __uint_as_float((uint32_t) static_cast<const uint16_t*>(logits)[t * E + e] << 16);
        else
          f = static_cast<const float*>(logits)[t * E + e];
        key[v] = key_of(f);
      }
    }
    uint32_t best = 0, top = 0;
    int at = 0;
    float total = 0.0f, mine = 0.0f;     // lane j keeps rank j
    int my_id = -1;
    auto refresh = [&]() {
      best = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (key[v] > best) { best = key[v]; at = v; }
    };
    refresh();
    if (share == BL_SHARE_ALL) {
      top = wave_max_u(best);
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (key[v]) s += key[v] == top ? 1.0f : expf(value_of(key[v]) - value_of(top));
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
      total = s;
    }
    for (int j = 0; j < k; ++j) {
      const uint32_t m = wave_max_u(best);
      if (m == 0) break;                                  // nothing usable left
      if (j == 0) top = m;
      const int src = __builtin_ctzll(__ballot(best == m));
      const int e = __builtin_amdgcn_readlane(lane * VPL + at, src);
      const float u = m == top ? 1.0f : expf(value_of(m) - value_of(top));
      if (share == BL_SHARE_CHOSEN) total += u;
      if (lane == j) {
        my_id = e;
        mine = u;
      }
      if (lane == src) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (v == at) key[v] = 0;
        refresh();
      }
    }
    if (lane < k) {
      ids[t * k + lane] = my_id;
      weights[t * k + lane] = my_id < 0 ? 0.0f : mine / total;
      if (my_id >= 0) atomicOr(&mask[my_id], 1ull << i);
    }
  }
}

__device__ __forceinline__ int below(unsigned long long m, int i) {
  return __builtin_popcountll(m & ((1ull << i) - 1));
}

// Slots of a block's pairs: `start[e]` is the first slot of the block's pairs
// of expert e.
__device__ __forceinline__ void place(int64_t t0, int nt, int k, const int32_t* __restrict__ ids,
                                      const unsigned long long* mask, const int* start,
                                      int32_t* __restrict__ pairs, int32_t* __restrict__ slots) {
  for (int i = threadIdx.x; i < nt * k; i += kThreads) {
    const int64_t pair = t0 * k + i;
    const int e = ids[pair];
    int slot = -1;
    if (e >= 0) {
      slot = start[e] + below(mask[e], i / k);
      pairs[slot] = (int32_t)pair;
    }
    slots[pair] = slot;
  }
}

// Up to 64 tokens: everything in one block.
template <int VPL, bool BF16>
__global__ __launch_bounds__(kThreads) void k_route_one(const void* __restrict__ logits, int T,
                                                        int E, int k, int share,
                                                        int32_t* __restrict__ ids,
                                                        float* __restrict__ weights,
                                                        int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ pairs,
                                                        int32_t* __restrict__ slots) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ int start[kMaxE], part[kWaves];
  const int e = threadIdx.x;
  mask[e] = 0;
  __syncthreads();
  choose<VPL, BF16>(logits, 0, T, E, k, share, ids, weights, mask);
  __syncthreads();
  int used;
  const int first = block_scan(__builtin_popcountll(mask[e]), part, used);
  start[e] = first;
  if (e < E) offsets[e] = first;
  if (e == 0) offsets[E] = used;
  for (int p = used + threadIdx.x; p < T * k; p += kThreads) pairs[p] = -1;
  __syncthreads();                 // the ids written above by this block are read back below
  place(0, T, k, ids, mask, start, pairs, slots);
}

// More tokens, first kernel: choices, and each block's count per expert.
// workspace: counts [E][blocks], then totals [E].
template <int VPL, bool BF16>
__global__ __launch_bounds__(kThreads) void k_route_choose(const void* __restrict__ logits, int T,
                                                           int E, int k, int share,
                                                           int32_t* __restrict__ ids,
                                                           float* __restrict__ weights,
                                                           int32_t* __restrict__ counts) {
  __shared__ unsigned long long mask[kMaxE];
  const int e = threadIdx.x;
  mask[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kRouteTokens;
  choose<VPL, BF16>(logits, t0, min(kRouteTokens, T - t0), E, k, share, ids, weights, mask);
  __syncthreads();
  if (e < E) counts[(int64_t)e * gridDim.x + blockIdx.x] = __builtin_popcountll(mask[e]);
}

// Second kernel, one wave per expert: counts -> pairs of the expert in earlier blocks.
__global__ __launch_bounds__(64) void k_route_starts(int32_t* __restrict__ counts, int blocks,
                                                     int32_t* __restrict__ totals) {
  const int lane = threadIdx.x;
  int32_t* c = counts + (int64_t)blockIdx.x * blocks;
  int before = 0;
  for (int b = 0; b < blocks; b += 64) {
    const int v = b + lane < blocks ? c[b + lane] : 0;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    if (b + lane < blocks) c[b + lane] = before + s - v;
    before += __builtin_amdgcn_readlane(s, 63);
  }
  if (lane == 0) totals[blockIdx.x] = before;
}

// Third kernel: offsets (block 0) and every pair's slot.
__global__ __launch_bounds__(kThreads) void k_route_place(const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ totals, int T,
                                                          int E, int k,
                                                          const int32_t* __restrict__ ids,
                                                          int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ pairs,
                                                          int32_t* __restrict__ slots) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ int start[kMaxE], part[kWaves];
  const int e = threadIdx.x, blocks = gridDim.x;
  mask[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kRouteTokens, nt = min(kRouteTokens, T - t0);
  for (int i = threadIdx.x; i < nt * k; i += kThreads) {
    const int id = ids[(int64_t)t0 * k + i];
    if (id >= 0) atomicOr(&mask[id], 1ull << (i / k));
  }
  int used;
  const int first = block_scan(e < E ? totals[e] : 0, part, used);   // also orders the masks
  start[e] = e < E ? first + counts[(int64_t)e * blocks + blockIdx.x] : 0;
  if (blockIdx.x == 0) {
    if (e < E) offsets[e] = first;
    if (e == 0) offsets[E] = used;
  }
  for (int64_t p = used + (int64_t)blockIdx.x * kThreads + e; p < (int64_t)T * k;
       p += (int64_t)blocks * kThreads)
    pairs[p] = -1;
  __syncthreads();
  place(t0, nt, k, ids, mask, start, pairs, slots);
}

}  // namespace

size_t route_workspace_bytes(int64_t t, int64_t e) {
  const int64_t blocks = (t + kRouteTokens - 1) / kRouteTokens;
  return blocks <= 1 ? 0 : (size_t)((blocks + 1) * e) * sizeof(int32_t);
}

hipError_t launch_route(const void* logits, int bf16, int64_t t, int64_t e, int64_t k, int share,
                        int32_t* ids, float* weights, int32_t* offsets, int32_t* pairs,
                        int32_t* slots, int32_t* workspace, hipStream_t stream) {
  const int blocks = (int)((t + kRouteTokens - 1) / kRouteTokens);
  auto go = [&](auto vpl, auto bf) {
    constexpr int V = decltype(vpl)::value;
    constexpr bool B = decltype(bf)::value;
    if (blocks == 1)
      k_route_one<V, B><<<1, kThreads, 0, stream>>>(logits, (int)t, (int)e, (int)k, share, ids,
                                                    weights, offsets, pairs, slots);
    else
      k_route_choose<V, B><<<blocks, kThreads, 0, stream>>>(logits, (int)t, (int)e, (int)k, share,
                                                            ids, weights, workspace);
  };
  auto by_width = [&](auto bf) {
    if (e <= 64) go(std::integral_constant<int, 1>{}, bf);
    else if (e <= 128) go(std::integral_constant<int, 2>{}, bf);
    else if (e <= 256) go(std::integral_constant<int, 4>{}, bf);
    else go(std::integral_constant<int, 16>{}, bf);
  };
  if (bf16) by_width(std::true_type{});
  else by_width(std::false_type{});
  if (blocks > 1) {
    int32_t* totals = workspace + (int64_t)blocks * e;
    k_route_starts<<<(unsigned)e, 64, 0, stream>>>(workspace, blocks, totals);
    k_route_place<<<blocks, kThreads, 0, stream>>>(workspace, totals, (int)t, (int)e, (int)k, ids,
                                                   offsets, pairs, slots);
  }
  return hipGetLastError();
}

}  // namespace bl
