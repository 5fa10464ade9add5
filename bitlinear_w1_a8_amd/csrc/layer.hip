// A whole routed layer for a few tokens in two launches: the router with the
// gate and up projections, then the down projections with the weighted sum.
// The same operations in the same precision as the router, the gated and the
// linear calls one after the other, so the same bits.
//
// No launch of its own for the router, nor slots.  A block of the first kernel
// belongs to one expert, and whether a token takes that expert needs no
// selection: its rank is the number of the token's logits before it (larger,
// or equal at a lower place), one comparison per logit.  Its rows go
// to place token * k + rank, which the second kernel finds by itself.  One more
// block chooses and weighs each token's experts for the second kernel while
// the others stream weights.
#include <algorithm>
#include <type_traits>

#include "experts_rows.h"
#include "layer_plan.h"
#include "route_keys.h"

namespace bl {
namespace {

struct Router {
  const void* logits;
  int T, E, k, share, bf16;
  int32_t* ids;                    // [T, k]
  float* weights;                  // [T, k]
};

__device__ __forceinline__ uint32_t logit_key(const Router& r, int64_t at) {
  return key_of(r.bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(r.logits)[at] << 16)
                       : static_cast<const float*>(r.logits)[at]);
}

// The router's choice (route.hip), a DPP row per token: ranks by falling logit, and
// weights with the same sums in the same order.
__device__ __forceinline__ void choose_rows(const Router& r) {
  const int lane = threadIdx.x & 15, t = threadIdx.x >> 4;
  if ((int)(threadIdx.x >> 6) * 4 >= r.T) return;               // whole waves
  const int64_t row = (int64_t)min(t, r.T - 1) * r.E;
  const int per = r.E <= 64 ? 4 : r.E <= 128 ? 8 : 16;          // consecutive logits per lane
  auto larger = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  auto lower = [](int a, int b) { return a < b ? a : b; };
  auto sum = [](float a, float b) { return a + b; };
  uint32_t key[16];
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int e = lane * per + v;
    key[v] = v < per && e < r.E ? logit_key(r, row + e) : 0;
  }
  uint32_t best = 0;
#pragma unroll
  for (int v = 0; v < 16; ++v) best = larger(best, key[v]);
  const uint32_t top = over_lanes<16>(best, larger);
  const float top_value = value_of(top);
  float all = 0.0f;
  if (r.share == BL_SHARE_ALL) {
#pragma unroll
    for (int v = 0; v < 16; ++v)
      if (key[v]) all += key[v] == top ? 1.0f : expf(value_of(key[v]) - top_value);
  }
  uint32_t mine = 0;
  int my_id = -1;
  for (int j = 0; j < r.k; ++j) {
    best = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) best = larger(best, key[v]);
    const uint32_t m = over_lanes<16>(best, larger);
    int e = kLayerExperts;
#pragma unroll
    for (int v = 15; v >= 0; --v) e = v < per && key[v] == m ? lane * per + v : e;
    e = over_lanes<16>(e, lower);
#pragma unroll
    for (int v = 0; v < 16; ++v) key[v] = lane * per + v == e && v < per ? 0 : key[v];
    if (lane == j) {
      mine = m;
      my_id = m ? e : -1;
    }
  }
  float u = 0.0f;
  if (mine) u = mine == top ? 1.0f : expf(value_of(mine) - top_value);
  const float total = over_lanes<16>(r.share == BL_SHARE_ALL ? all : u, sum);
  if (t < r.T && lane < r.k) {
    r.ids[t * r.k + lane] = my_id;
    r.weights[t * r.k + lane] = my_id < 0 ? 0.0f : u / total;
  }
}

// Keys of a token's logits, 64 v + lane in key[v].
struct Keys {
  uint32_t key[kLayerExperts / 64];
  __device__ __forceinline__ Keys(const Router& r, int t) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int v = 0; v < kLayerExperts / 64; ++v) {
      const int e = v * 64 + lane;
      key[v] = e < r.E ? logit_key(r, (int64_t)t * r.E + e) : 0;
    }
  }
  __device__ __forceinline__ uint32_t of(int e) const {
    uint32_t k = 0;
#pragma unroll
    for (int v = 0; v < kLayerExperts / 64; ++v)
      if (e >> 6 == v) k = __builtin_amdgcn_readlane(key[v], e & 63);
    return k;
  }
};

// The expert of a token's rank j, -1 if fewer logits are usable, by a block of four
// waves: each counts for every key what comes before it among 16 of every 64 keys.
__device__ __forceinline__ int expert_of_rank(const Keys& a, int E, int j, int wave,
                                              int (*part)[kLayerExperts]) {
  constexpr int V = kLayerExperts / 64;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * 64 >= E) break;
    int before = 0;
#pragma unroll
    for (int w = 0; w < V; ++w) {
      if (w * 64 >= E) break;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int l = wave * 16 + i;
        const uint32_t other = __builtin_amdgcn_readlane(a.key[w], l);
        // equal keys: the lower expert first (key 0, unusable, is not asked for)
        before += other > a.key[v] - (w < v || (w == v && l < lane) ? 1u : 0u);
      }
    }
    part[wave][v * 64 + lane] = before;
  }
  lds_sync();
  int expert = -1;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * 64 >= E) break;
    const int e = v * 64 + lane, before = part[0][e] + part[1][e] + part[2][e] + part[3][e];
    const uint64_t here = __ballot(a.key[v] && before == j);
    if (here) expert = v * 64 + __builtin_ctzll(here);
  }
  return expert;
}

// Gate and up projections (as k_experts_few): block (row tile, 1 + expert) or, PAIRS,
// (row tile, 1 + token * k + rank), and the block (0, 0) that chooses.  Most blocks of an
// expert have nothing to do while few tokens meet many experts; a block of a pair
// first finds its expert, and ends if an earlier token takes the same one.
// N rows of gate and up together; h by token * k + rank.
// Bound by latency: the start of its blocks, the logits, then the tokens and the
// weights (one token, 8 of 64 experts of 2560 -> 2 x 1024, 10.5 MB in 8.6 us; 16 tokens, 40 of
// 64 taken, 53 MB in 18 us, where a third of the cycles issue vector instructions).
template <int MODE, bool PAIRS, int U, int Q>
__global__ __launch_bounds__(512) void k_layer_gate(const Router rt,
                                                    const uint32_t* __restrict__ packed,
                                                    const float* __restrict__ gamma_gate,
                                                    const float* __restrict__ gamma_up,
                                                    const void* __restrict__ x,
                                                    const float* __restrict__ absmax, int N, int K,
                                                    uint16_t* __restrict__ h) {
  extern __shared__ __align__(16) unsigned char xs[];   // [T][few_stride(K)], then raw [T][K]
  __shared__ int rank[kLayerTokens], qsum[kLayerTokens], amax[kLayerTokens];
  if (blockIdx.y == 0) {
    if (blockIdx.x == 0) choose_rows(rt);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, nthreads = blockDim.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), nwaves = nthreads >> 6;
  const int qg = lane >> 4, r = lane & 15;

  // ranks of the block's expert: -1 where a token does not take it
  if (tid < kLayerTokens) {
    rank[tid] = -1;
    qsum[tid] = amax[tid] = 0;
  }
  int expert = blockIdx.y - 1;
  auto keep = [&](int t, uint32_t own, int before) {
    before = wave_sum_i(before);
    if (lane == 0 && own && before < rt.k) rank[t] = before;
  };
  if constexpr (PAIRS) {
    __shared__ int part[4][kLayerExperts];
    const int t0 = expert / rt.k, j = expert - t0 * rt.k;
    const Keys a(rt, t0), b(rt, min(wave, rt.T - 1));
    expert = expert_of_rank(a, rt.E, j, wave, part);
    if (expert < 0) return;
    for (int t = wave; t < rt.T; t += 4) {
      const uint32_t own = b.of(expert);
      int before = 0;
#pragma unroll
      for (int v = 0; v < kLayerExperts / 64; ++v)
        before += b.key[v] > own || (b.key[v] == own && v * 64 + lane < expert);
      keep(t, own, before);
    }
  } else {
    lds_sync();
    for (int t = wave; t < rt.T; t += nwaves) {
      const int64_t row = (int64_t)t * rt.E;
      const uint32_t own = logit_key(rt, row + expert);
      int before = 0;
      for (int e = lane; e < rt.E; e += 64) {
        const uint32_t key = logit_key(rt, row + e);
        before += key > own || (key == own && e < expert);
      }
      keep(t, own, before);
    }
  }
  lds_sync();
  const int my_rank = rank[r];
  const uint32_t members = (uint32_t)__ballot(lane < 16 && my_rank >= 0);
  const int nrow = __builtin_popcount(members);
  if (nrow == 0) return;
  // lane r's token: the r-th member (the first in place of those that are missing)
  int token = __builtin_ctz(members);
  if (PAIRS && token != (int)(blockIdx.y - 1) / rt.k) return;   // an earlier token's block does it
  {
    uint32_t m = members;
    for (int i = 0; i < 16; ++i) {
      if (m && i == r) token = __builtin_ctz(m);
      m &= m - 1;
    }
  }
  const int place = token * rt.k + rank[token];
  float a = 0.0f;
  if constexpr (MODE == kInt8) a = absmax[token];
  const float g_gate = gamma_gate[expert], g_up = gamma_up[expert];

  const int K16 = K >> 4, nchunks = (K + 255) >> 8, stride = few_stride(K);
  const int n0 = (blockIdx.x * nwaves + wave) * 16;
  constexpr int kBytes = MODE == kInt8 ? 1 : MODE == kBf16 ? 2 : 4;
  const int row_bytes = K * kBytes;
  unsigned char* land = MODE == kInt8 ? xs : xs + rt.T * stride;
  const int land_stride = MODE == kInt8 ? stride : row_bytes;
  for (int i = wave; i < nrow; i += nwaves) {
    const unsigned char* src = static_cast<const unsigned char*>(x) +
                               (int64_t)__builtin_amdgcn_readlane(token, i) * row_bytes;
    for (int b = 0; b < row_bytes; b += 1024)
      if (b + 16 * lane < row_bytes)
        __builtin_amdgcn_global_load_lds((glb_ptr_t)(src + b + 16 * lane),
                                         (lds_ptr_t)(land + i * land_stride + b), 16, 0, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  const int n = min(n0 + r, N - 1);
  const uint32_t* wrow = packed + ((int64_t)expert * N + n) * K16;
  uint4 w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = load_quad<Q>(wrow, 16 * min(u, nchunks - 1) + 4 * qg, K16);
  __builtin_amdgcn_sched_barrier(0);
  wait_vmem<U>();
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
      if (K16 + lane < 16 * nchunks) row[K16 + lane] = make_uint4(0, 0, 0, 0);
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
      const float s = kQb / fmaxf(__int_as_float(amax[i]), kEps);
      int sum = 0;
      for (int k = 4 * tid; k < nchunks * 256; k += 4 * nthreads) {
        Raw4<MODE> f;
        f.clear();
        if (k < K) f.load(land + i * land_stride, k);
        const uint32_t q = quant4(f, s);
        sum = __builtin_amdgcn_sdot4((int)q, 0x01010101, sum, false);
        *reinterpret_cast<uint32_t*>(xs + i * stride + k) = q;
      }
      sum = wave_sum_i(sum);
      if (lane == 0) atomicAdd(&qsum[i], sum);
    }
  }
  lds_sync();

  const v4i acc = few_contract<U, Q>(w, wrow, xs + (r < nrow ? r : 0) * stride + 64 * qg, qg, K16, nchunks);

  // lane (qg, r) holds rows 4 qg .. 4 qg + 3 of member r
  if (r >= nrow) return;
  const int nn = n0 + 4 * qg, qs = qsum[r];
  if constexpr (MODE != kInt8) a = __int_as_float(amax[r]);
  const double gg = gamma_m(g_gate, a), gu = gamma_m(g_up, a);
#pragma unroll
  for (int v = 0; v < 4; v += 2)
    if (nn + v < N)
      h[(int64_t)place * (N >> 1) + ((nn + v) >> 1)] =
          gated_relu2_bf16(acc[v] - qs, acc[v + 1] - qs, gg, gu);
}

// Down projections and the weighted sum (as k_experts_token): a block has one
// token and 16 RT outputs, each of its k rows of h a team of `team` waves that
// split K; the rows do not wait for the experts' numbers, the weights do.
// (One token, 8 experts of 1024 -> 2560, 5.3 MB in 5.1 us: the latency of the number, the
// weights and three barriers.  16 tokens 17 us: an expert's weights are read, from the
// caches after the first time, and unpacked once per token, and each block quantises its
// token's rows: vector instructions issue in over half of the cycles.)
template <int RT, int U, int Q>
__global__ __launch_bounds__(1024) void k_layer_down(const int32_t* __restrict__ ids,
                                                     const float* __restrict__ weights, int topk,
                                                     int E, int team,
                                                     const uint32_t* __restrict__ packed,
                                                     const float* __restrict__ gamma,
                                                     const uint16_t* __restrict__ h, int N, int K,
                                                     float* __restrict__ y) {
  extern __shared__ __align__(16) unsigned char xs[];   // [topk][few_stride(K)]
  __shared__ int amax[kLayerTopK], tile[kLayerTopK][16 * RT];
  __shared__ float scale[kLayerTopK], share[kLayerTopK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int qg = lane >> 4, r = lane & 15;
  const int t = blockIdx.y, n0 = blockIdx.x * 16 * RT;
  const int j = wave / team, part = wave - j * team;
  const int K16 = K >> 4, nchunks = (K + 255) >> 8, stride = few_stride(K);
  const int per = (nchunks + team - 1) / team, c0 = part * per, c1 = min(c0 + per, nchunks);
  for (int i = tid; i < kLayerTopK * 16 * RT; i += blockDim.x) (&tile[0][0])[i] = 0;
  if (tid < kLayerTopK) amax[tid] = 0;

  const int pair = t * topk + j;
  const void* xrow = h + (int64_t)pair * K;
  const int id = ids[pair];
  Raw4<kBf16> xr[U];
  uint4 w[RT][U];
  const bool live = id >= 0 && c0 < c1;                 // wave-uniform
  const int expert = min(max(id, 0), E - 1);
  const uint32_t* wrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    wrow[i] = packed + ((int64_t)expert * N + min(n0 + 16 * i + r, N - 1)) * K16;
  if (live) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(c0 + u, c1 - 1) * 256 + 4 * lane;
      xr[u].load(xrow, min(k, K - 4));
      if (k >= K) xr[u].clear();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u)
        w[i][u] = load_quad<Q>(wrow[i], 16 * min(c0 + u, c1 - 1) + 4 * qg, K16);
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
        Raw4<kBf16> f;
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
    share[j] = id >= 0 ? weights[pair] : 0.0f;
  }
  if (live) {
    const float s = kQb / fmaxf(a, kEps);
    int sum = 0;
    auto put = [&](const Raw4<kBf16>& f, int k) {
      const uint32_t q = quant4(f, s);
      sum = __builtin_amdgcn_sdot4((int)q, 0x01010101, sum, false);
      *reinterpret_cast<uint32_t*>(xs + j * stride + k) = q;
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < c1) put(xr[u], (c0 + u) * 256 + 4 * lane);
    for (int c = c0 + U; c < c1; ++c) {
      const int k = c * 256 + 4 * lane;
      Raw4<kBf16> f;
      f.clear();
      if (k < K) f.load(xrow, k);
      put(f, k);
    }
    sum = wave_sum_i(sum);
    wave_lds_sync();                                    // this wave's own chunks: no block barrier
    v4i acc[RT] = {};
    const unsigned char* xq = xs + j * stride + 64 * qg;
    for (int b0 = c0; b0 < c1; b0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b0 + u >= c1) break;
        const uint4* xv = reinterpret_cast<const uint4*>(xq + (b0 + u) * 256);
        uint4 b[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) b[v] = xv[v];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint4 p = settle<Q>(w[i][u], 16 * (b0 + u) + 4 * qg, K16);
          const uint32_t word[4] = {p.x, p.y, p.z, p.w};
          if (b0 + U + u < c1) w[i][u] = load_quad<Q>(wrow[i], 16 * (b0 + U + u) + 4 * qg, K16);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                operand(word[v]), v4i{(int)b[v].x, (int)b[v].y, (int)b[v].z, (int)b[v].w}, acc[i], 0, 0, 0);
        }
      }
    }
    if (r == 0) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) atomicAdd(&tile[j][16 * i + 4 * qg + v], acc[i][v] - sum);
    }
  }
  lds_sync();
  if (tid < 16 * RT && n0 + tid < N) {
    float s = 0.0f;
    for (int i = 0; i < topk; ++i)
      if (ids[t * topk + i] >= 0) s = fmaf(share[i], (float)tile[i][tid] * scale[i], s);
    y[(int64_t)t * N + n0 + tid] = s;
  }
}

// ------------------------------------------------------------------ host

// Where the workspace holds what, in bytes; every part on a 256-byte border.
struct Layout {
  int64_t ids, weights, h, xq, absmax, offsets, pairs, slots, route, hq, habs, rows, end;
  Layout(int64_t t, int64_t e, int64_t k, int64_t f, int64_t kk, int64_t n) {
    const int64_t p = t * k;
    int64_t at = 0;
    auto part = [&](int64_t bytes) {
      const int64_t was = at;
      at += (bytes + 255) / 256 * 256;
      return was;
    };
    ids = part(4 * p);
    weights = part(4 * p);
    h = part(2 * p * f);
    xq = part(t * kk);
    absmax = part(4 * t);
    offsets = part(4 * (e + 1));
    pairs = part(4 * p);
    slots = part(4 * p);
    route = part((int64_t)route_workspace_bytes(t, e));
    hq = part(p * f);
    habs = part(4 * p);
    rows = part(4 * p * n);
    end = at;
  }
};

template <int MODE, bool PAIRS>
hipError_t launch_gate(const LayerCall& c, const LayerPlan& p, const Router& rt, const void* x,
                       const float* absmax, uint16_t* h, hipStream_t stream) {
  const int64_t n = 2 * c.F;
  const int bn = 16 * p.gate_waves;
  const dim3 grid((unsigned)((n + bn - 1) / bn), (unsigned)((PAIRS ? c.T * c.k : c.E) + 1));
  const size_t lds = (size_t)layer_rows_lds(c.K, c.T, MODE == kInt8 ? 0 : MODE == kBf16 ? 2 : 4);
  auto go = [&](auto kern) {
    hipError_t e = kern.allow_lds();
    if (e != hipSuccess) return e;
    kern.kernel<<<grid, 64 * p.gate_waves, lds, stream>>>(
        rt, reinterpret_cast<const uint32_t*>(c.gu), c.gamma_gate, c.gamma_up, x, absmax, (int)n,
        (int)c.K, h);
    return hipGetLastError();
  };
  if (c.K < 64) return go(Kernel<k_layer_gate<MODE, PAIRS, 2, kWords>>{});
  auto by_depth = [&](auto quads) {
    constexpr int Q = decltype(quads)::value;
    switch (few_depth(c.K)) {
      case 2: return go(Kernel<k_layer_gate<MODE, PAIRS, 2, Q>>{});
      case 4: return go(Kernel<k_layer_gate<MODE, PAIRS, 4, Q>>{});
      case 6: return go(Kernel<k_layer_gate<MODE, PAIRS, 6, Q>>{});
      case 8: return go(Kernel<k_layer_gate<MODE, PAIRS, 8, Q>>{});
      default: return go(Kernel<k_layer_gate<MODE, PAIRS, 10, Q>>{});
    }
  };
  return c.K % 64 ? by_depth(std::integral_constant<int, kShort>{})
                  : by_depth(std::integral_constant<int, kWhole>{});
}

template <int MODE>
hipError_t launch_gate(const LayerCall& c, const LayerPlan& p, const Router& rt, const void* x,
                       const float* absmax, uint16_t* h, hipStream_t stream) {
  return p.pairs ? launch_gate<MODE, true>(c, p, rt, x, absmax, h, stream)
                 : launch_gate<MODE, false>(c, p, rt, x, absmax, h, stream);
}

template <int RT>
hipError_t launch_down(const LayerCall& c, const LayerPlan& p, const Router& rt, const uint16_t* h,
                       hipStream_t stream) {
  const int topk = (int)c.k;
  const dim3 grid((unsigned)((c.N + 16 * RT - 1) / (16 * RT)), (unsigned)c.T);
  const size_t lds = (size_t)layer_rows_lds(c.F, topk, 0);
  auto go = [&](auto kern) {
    hipError_t e = kern.allow_lds();
    if (e != hipSuccess) return e;
    kern.kernel<<<grid, 64 * topk * p.team, lds, stream>>>(rt.ids, rt.weights, topk, (int)c.E, p.team,
                                                           reinterpret_cast<const uint32_t*>(c.down),
                                                           c.gamma_down, h, (int)c.N, (int)c.F, c.y);
    return hipGetLastError();
  };
  if (c.F < 64) return go(Kernel<k_layer_down<RT, 4, kWords>>{});
  return c.F % 64 ? go(Kernel<k_layer_down<RT, 4, kShort>>{}) : go(Kernel<k_layer_down<RT, 4, kWhole>>{});
}

}  // namespace

size_t layer_workspace_bytes(int64_t t, int64_t e, int64_t k, int64_t f, int64_t kk, int64_t n) {
  return (size_t)Layout(t, e, k, f, kk, n).end;
}

hipError_t launch_layer(const LayerCall& c, hipStream_t stream) {
  const Layout l(c.T, c.E, c.k, c.F, c.K, c.N);
  unsigned char* ws = static_cast<unsigned char*>(c.workspace);
  auto i32 = [&](int64_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  auto f32 = [&](int64_t at) { return reinterpret_cast<float*>(ws + at); };
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + l.h);
  int8_t* xq = reinterpret_cast<int8_t*>(ws + l.xq);
  hipError_t e;
  const int raw = c.x_dtype == BL_CODES ? 0 : c.x_dtype == BL_BF16 ? 2 : 4;
  const LayerPlan p = layer_plan(c.T, c.E, c.k, c.F, c.K, c.N, raw, device_cus());
  if (p.two) {
    const Router rt{c.logits, (int)c.T, (int)c.E, (int)c.k, c.share, c.logits_bf16, i32(l.ids), f32(l.weights)};
    if (p.own_quant) {
      e = launch_quant(c.x, raw == 2, c.T, c.K, xq, f32(l.absmax), nullptr, stream);
      if (e == hipSuccess) e = launch_gate<kInt8>(c, p, rt, xq, f32(l.absmax), h, stream);
    } else {
      e = raw == 0   ? launch_gate<kInt8>(c, p, rt, c.x, c.absmax, h, stream)
          : raw == 2 ? launch_gate<kBf16>(c, p, rt, c.x, nullptr, h, stream)
                     : launch_gate<kF32>(c, p, rt, c.x, nullptr, h, stream);
    }
    if (e != hipSuccess) return e;
    return p.down_tiles == 2 ? launch_down<2>(c, p, rt, h, stream) : launch_down<1>(c, p, rt, h, stream);
  }
  // the three calls, one after the other
  const bl_routing r{c.T, c.k, c.E, i32(l.offsets), i32(l.pairs), i32(l.slots), f32(l.weights)};
  e = launch_route(c.logits, c.logits_bf16, c.T, c.E, c.k, c.share, i32(l.ids), f32(l.weights),
                   i32(l.offsets), i32(l.pairs), i32(l.slots), i32(l.route), stream);
  if (e != hipSuccess) return e;
  if (c.x_dtype == BL_CODES)
    e = launch_gated_codes(r, static_cast<const int8_t*>(c.x), c.absmax, c.gu, c.gamma_gate,
                           c.gamma_up, 2 * c.F, c.K, h, stream);
  else
    e = launch_gated_experts(r, c.x, c.x_dtype == BL_BF16, c.gu, c.gamma_gate, c.gamma_up, 2 * c.F,
                             c.K, h, xq, f32(l.absmax), nullptr, stream);
  if (e != hipSuccess) return e;
  return launch_linear_experts(r, h, 1, BL_ROWS_SLOTS, c.down, c.gamma_down, c.N, c.F, c.y,
                               BL_ROWS_TOKENS, reinterpret_cast<int8_t*>(ws + l.hq), f32(l.habs),
                               nullptr, f32(l.rows), stream);
}

}  // namespace bl
