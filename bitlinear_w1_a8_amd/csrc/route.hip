// The router of the expert layers: each token's k largest logits, their
// softmax weights, and the slots of all (token, rank) pairs in expert order.
//
// Selection.  LANES lanes (a row of 16, or a whole wave for many experts or
// ranks) own a token and hold its E logits in registers, VPL consecutive ones
// per lane, as keys whose unsigned order is that of the values (0 for a masked
// one).  A rank is a maximum over them and the lowest expert that has it, both
// by DPP; the weights' exponentials follow once the ranks are known, lane j's
// for rank j.  With a row per token a wave's instructions serve four tokens
// (8192 tokens, 128 experts, k = 8, the whole router: a wave per token with an
// exponential in every rank 23.5 us, this 12.6; 64 tokens 17.1 -> 9.5).  Bound by
// latency: of that choice's 6.6 us VALU issue is 6.2 thousand cycles (2.6 us); a
// wave lives 12 thousand, two thirds of them waiting for its logits (two bytes
// a load) and along the DPP chains of the ranks, with two waves per SIMD to
// cover it.
//
// Slots.  A block takes up to 64 tokens, whose choices of expert e are one
// 64-bit mask: a pair's place among its expert's pairs of the block is the number of
// mask bits below its token.  The masks are integers set by or, so nothing
// depends on an order of execution.  Up to 64 tokens one block does
// everything; more are chosen 32 per block (64 leave half the CUs idle at 8192
// tokens: 15.2 -> 14.0 us), a last kernel writes the slots, and where the counts are
// many one in between turns them into starts (one wave per expert, four counts a
// lane: 14.0 -> 12.6).
#include <type_traits>

#include "route_keys.h"

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kChooseThreads = 16 * kRouteTokens;   // a row of lanes per token
constexpr int kMaxE = BITLINEAR_MAX_EXPERTS;
static_assert(kMaxE <= kThreads, "one thread per expert");

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

// Top k of one block's tokens; marks each choice in the masks.  k <= LANES.
template <int THREADS, int LANES, int VPL, bool BF16>
__device__ __forceinline__ void choose(const void* __restrict__ logits, int64_t t0, int nt, int E,
                                       int k, int share, int32_t* __restrict__ ids,
                                       float* __restrict__ weights, unsigned long long* mask) {
  constexpr int kTeams = THREADS / LANES;
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  auto lower = [](int a, int b) { return a < b ? a : b; };
  auto sum = [](float a, float b) { return a + b; };
  // whole waves go round; tokens past the end repeat the last one, not stored
  for (int base = 0; base < nt; base += kTeams) {
    if (base + team / (64 / LANES) * (64 / LANES) >= nt) break;    // wave-uniform
    const int i = base + team;
    const int64_t t = t0 + min(i, nt - 1);
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int64_t o = t * E + min(lane * VPL + v, E - 1);
      float f;
      if constexpr (BF16)
        f = __uint_as_float((uint32_t) static_cast<const uint16_t*>(logits)[o] << 16);
      else
        f = static_cast<const float*>(logits)[o];
      key[v] = lane * VPL + v < E ? key_of(f) : 0;
    }
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) best = larger(best, key[v]);
    const uint32_t top = over_lanes<LANES>(best, larger);
    const float top_value = value_of(top);
    float all = 0.0f;
    if (share == BL_SHARE_ALL) {
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (key[v]) all += key[v] == top ? 1.0f : expf(value_of(key[v]) - top_value);
    }
    uint32_t mine = 0;                   // lane j keeps rank j
    int my_id = -1;
    for (int j = 0; j < k; ++j) {
      best = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) best = larger(best, key[v]);
      const uint32_t m = over_lanes<LANES>(best, larger);
      int e = kMaxE;
#pragma unroll
      for (int v = VPL - 1; v >= 0; --v) e = key[v] == m ? lane * VPL + v : e;
      e = over_lanes<LANES>(e, lower);
#pragma unroll
      for (int v = 0; v < VPL; ++v) key[v] = lane * VPL + v == e ? 0 : key[v];
      if (lane == j) {
        mine = m;
        my_id = m ? e : -1;              // 0: nothing usable left
      }
    }
    float u = 0.0f;
    if (mine) u = mine == top ? 1.0f : expf(value_of(mine) - top_value);
    const float total = over_lanes<LANES>(share == BL_SHARE_ALL ? all : u, sum);
    if (i < nt && lane < k) {
      const int64_t o = t * k + lane;
      ids[o] = my_id;
      weights[o] = my_id < 0 ? 0.0f : u / total;
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
template <int LANES, int VPL, bool BF16>
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
  choose<kThreads, LANES, VPL, BF16>(logits, 0, T, E, k, share, ids, weights, mask);
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
template <int LANES, int VPL, bool BF16>
__global__ __launch_bounds__(kChooseThreads) void k_route_choose(const void* __restrict__ logits,
                                                                 int T, int E, int k, int share,
                                                                 int32_t* __restrict__ ids,
                                                                 float* __restrict__ weights,
                                                                 int32_t* __restrict__ counts) {
  __shared__ unsigned long long mask[kMaxE];
  for (int e = threadIdx.x; e < E; e += kChooseThreads) mask[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kRouteTokens;
  choose<kChooseThreads, LANES, VPL, BF16>(logits, t0, min(kRouteTokens, T - t0), E, k, share, ids,
                                           weights, mask);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kChooseThreads)
    counts[(int64_t)e * gridDim.x + blockIdx.x] = __builtin_popcountll(mask[e]);
}

// Second kernel, one wave per expert: counts -> pairs of the expert in earlier blocks.
__global__ __launch_bounds__(64) void k_route_starts(int32_t* __restrict__ counts, int blocks,
                                                     int32_t* __restrict__ totals) {
  const int lane = threadIdx.x;
  int32_t* c = counts + (int64_t)blockIdx.x * blocks;
  int before = 0;
  for (int b0 = 0; b0 < blocks; b0 += 256) {
    const int b = b0 + 4 * lane;
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = b + i < blocks ? c[b + i] : 0;
    const int own = v[0] + v[1] + v[2] + v[3];
    int s = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    int at = before + s - own;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b + i < blocks) c[b + i] = at;
      at += v[i];
    }
    before += __builtin_amdgcn_readlane(s, 63);
  }
  if (lane == 0) totals[blockIdx.x] = before;
}

// Last kernel: offsets (block 0) and every pair's slot.
// SUM: counts[] holds the blocks' counts as the first kernel left them, and
// every block adds up the earlier blocks' and all blocks' for itself (few
// enough, see launch_route); else k_route_starts has done so.
template <bool SUM>
__global__ __launch_bounds__(kThreads) void k_route_place(const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ totals, int T,
                                                          int E, int k,
                                                          const int32_t* __restrict__ ids,
                                                          int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ pairs,
                                                          int32_t* __restrict__ slots) {
  __shared__ unsigned long long mask[kMaxE];
  __shared__ int start[kMaxE], part[kWaves], whole[SUM ? kMaxE : 1];
  const int e = threadIdx.x, blocks = gridDim.x;
  mask[e] = 0;
  start[e] = 0;
  if (SUM) whole[e] = 0;
  __syncthreads();
  if constexpr (SUM) {
    // teams of 16 threads per expert
    for (int x = e / 16; x < E; x += kThreads / 16) {
      int before = 0, all = 0;
      for (int b = e % 16; b < blocks; b += 16) {
        const int c = counts[(int64_t)x * blocks + b];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      auto sum = [](int a, int b) { return a + b; };
      before = over_lanes<16>(before, sum);
      all = over_lanes<16>(all, sum);
      if (e % 16 == 0) {
        start[x] = before;
        whole[x] = all;
      }
    }
  }
  const int t0 = blockIdx.x * kRouteTokens, nt = min(kRouteTokens, T - t0);
  for (int i = threadIdx.x; i < nt * k; i += kThreads) {
    const int id = ids[(int64_t)t0 * k + i];
    if (id >= 0) atomicOr(&mask[id], 1ull << (i / k));
  }
  __syncthreads();
  int used;
  const int first = block_scan(e < E ? (SUM ? whole[e] : totals[e]) : 0, part, used);
  if (e < E) start[e] = first + (SUM ? start[e] : counts[(int64_t)e * blocks + blockIdx.x]);
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

// Every block of the last kernel adds up the counts itself, 64 experts by 16
// blocks a round, where that takes few rounds; else a kernel in between does
// (8 rounds, 4096 tokens x 64 experts 9.5 against 10.1 us, 2048 x 128 11.1 / 11.7;
// 16 rounds, 8192 x 64 11.3 / 10.4, 4096 x 128 12.8 / 12.0; 1 round, 256 x 128
// 10.1 / 11.5).
bool sum_wins(int64_t blocks, int64_t e) { return (blocks + 15) / 16 * ((e + 63) / 64) <= 8; }

size_t route_workspace_bytes(int64_t t, int64_t e) {
  const int64_t blocks = (t + kRouteTokens - 1) / kRouteTokens;
  return t <= kOneBlock ? 0 : (size_t)((blocks + 1) * e) * sizeof(int32_t);
}

hipError_t launch_route(const void* logits, int bf16, int64_t t, int64_t e, int64_t k, int share,
                        int32_t* ids, float* weights, int32_t* offsets, int32_t* pairs,
                        int32_t* slots, int32_t* workspace, hipStream_t stream) {
  const int blocks = (int)((t + kRouteTokens - 1) / kRouteTokens);
  auto go = [&](auto lanes, auto vpl, auto bf) {
    constexpr int L = decltype(lanes)::value, V = decltype(vpl)::value;
    constexpr bool B = decltype(bf)::value;
    if (t <= kOneBlock)
      k_route_one<L, V, B><<<1, kThreads, 0, stream>>>(logits, (int)t, (int)e, (int)k, share, ids,
                                                       weights, offsets, pairs, slots);
    else
      k_route_choose<L, V, B><<<blocks, kChooseThreads, 0, stream>>>(
          logits, (int)t, (int)e, (int)k, share, ids, weights, workspace);
  };
  auto by_width = [&](auto bf) {
    using Row = std::integral_constant<int, 16>;
    using Wave = std::integral_constant<int, 64>;
    if (k <= 16 && e <= 64) go(Row{}, std::integral_constant<int, 4>{}, bf);
    else if (k <= 16 && e <= 128) go(Row{}, std::integral_constant<int, 8>{}, bf);
    else if (k <= 16 && e <= 256) go(Row{}, std::integral_constant<int, 16>{}, bf);
    else go(Wave{}, std::integral_constant<int, 16>{}, bf);
  };
  if (bf16) by_width(std::true_type{});
  else by_width(std::false_type{});
  if (t > kOneBlock) {
    int32_t* totals = workspace + (int64_t)blocks * e;
    if (sum_wins(blocks, e)) {
      k_route_place<true><<<blocks, kThreads, 0, stream>>>(workspace, nullptr, (int)t, (int)e, (int)k,
                                                           ids, offsets, pairs, slots);
    } else {
      k_route_starts<<<(unsigned)e, 64, 0, stream>>>(workspace, blocks, totals);
      k_route_place<false><<<blocks, kThreads, 0, stream>>>(workspace, totals, (int)t, (int)e,
                                                            (int)k, ids, offsets, pairs, slots);
    }
  }
  return hipGetLastError();
}

}  // namespace bl
