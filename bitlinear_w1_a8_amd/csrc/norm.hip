// The step between two layers: total = x + residual, the sub-layer norm of the
// sum, and its 8-bit codes (int8 with one scale per token, or e4m3 with one per
// 128), in one pass over memory.
//
// A block has one token and keeps the row in registers as u = total * g, eight
// consecutive elements per vector, two vectors per thread (what a longer row
// has beyond them is computed again from `total`, which each thread has itself
// written; one, two and four vectors are alike: 4096 x 2560 21.4 / 21.7 / 21.8 us, 1000
// x 28672 59.4 / 56.8 / 60.6, one token of 8192 4.0 / 3.6 / 4.3).  One exchange between the waves gives the sum of squares and
// the largest |u|; rounding is monotonic, so max |x_hat| = RN32(max |u| * r)
// and no second exchange is needed (a group of 128 is one DPP row of 16 lanes).
//
// The sum of squares.  ms = RN32(RN64(S / K)) is defined by the exact sum S.
// Squares of binary32 values are exact in binary64; each thread adds its own
// there, and the sums are added across the block: at most 160 additions on any
// path (8 per vector, up to 16 vectors; 6 in a wave; 16 waves), each off by
// 2^-53 of a sum of non-negative terms, so S lies within 2^-45 of the result.
// Where both ends of the interval of +- 2^-44 (which covers the rounding of the
// product with 1 / K and of the ends themselves) round to the same binary32,
// that is ms; all steps from S to ms are monotonic.  Else, about one row in
// 2^19 (of short bfloat16 rows, whose sums have few bits, more: one in 1700 of 144), the
// row is summed again exactly, in buckets by exponent (such a row of 144 5.9 us, any other
// 3.9).
//
// Bound by memory (binary32 x, bfloat16 residual, int8 codes, 9 bytes an element:
// 4096 x 2560 21.5 us, 4.4 TB/s; 1000 x 28672 56.8 us, 4.5; a large copy reaches 4.7), for
// few tokens by the latency of a launch, a load, the exchange and a store
// (one token of 2560 3.2 us).
#include <algorithm>
#include <type_traits>

#include "f8.h"

namespace bl {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kLimbs = 18;         // 576 bits: sums below 2^17 * 2^256 in units of 2^-298

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return v + __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
// Sum over the wave's lanes, uniform.
__device__ __forceinline__ double wave_sum_f64(double v) {
  v = add_dpp<0xB1>(v);
  v = add_dpp<0x4E>(v);
  v = add_dpp<0x141>(v);
  v = add_dpp<0x140>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

enum Residual { kNone = 0, kResF32 = 1, kResBf16 = 2 };

struct Args {
  const void* x;
  const void* residual;
  const float* gain;
  void* total;
  uint8_t* xq;
  float* scale;
  int32_t* rowsum;
  double inv_k;
  float eps_n;
  int K;
  int64_t T, row0;                 // all tokens; the first of this launch
};

constexpr int kVectors = 2;             // vectors per thread

template <bool XBF16, int RES, bool F8>
__global__ __launch_bounds__(1024) void k_add_subln(const Args a) {
  __shared__ double red_s[kMaxWaves];
  __shared__ int red_m[kMaxWaves], red_q[kMaxWaves];
  __shared__ unsigned long long hist[2][256];        // rare rows
  __shared__ unsigned long long word[kLimbs];
  __shared__ uint32_t limb[kLimbs];
  __shared__ double exact;
  const int K = a.K, nvec = K >> 3;
  const int64_t row = a.row0 + blockIdx.x;
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), nwaves = nthr >> 6;
  constexpr bool RBF16 = RES == kResBf16;
  const unsigned char* xr = static_cast<const unsigned char*>(a.x) + row * K * (XBF16 ? 2 : 4);
  const unsigned char* rr = static_cast<const unsigned char*>(a.residual) + row * K * (RBF16 ? 2 : 4);
  unsigned char* tr = static_cast<unsigned char*>(a.total) + row * K * (RBF16 ? 2 : 4);

  // total of eight elements, written
  auto join = [&](const Vec8<XBF16>& x, const Vec8<RBF16>& r, int at, float (&f)[8]) {
    x.widen(f);
    if constexpr (RES != kNone) {
      float g[8];
      r.widen(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
      uint4* out = reinterpret_cast<uint4*>(tr + (int64_t)at * (RBF16 ? 2 : 4));
      if constexpr (RBF16) {
        Vec8<true> t;
        t.v[0] = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                            bf16_pair(f[6], f[7]));
        out[0] = t.v[0];
        t.widen(f);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          out[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                              __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
      }
    }
  };
  // the same total again, as this thread has written it (or x itself)
  auto again = [&](int at, float (&f)[8]) {
    if constexpr (RES == kNone) {
      Vec8<XBF16> v;
      v.load(xr, at);
      v.widen(f);
    } else {
      Vec8<RBF16> v;
      v.load(tr, at);
      v.widen(f);
    }
  };
  auto times_gain = [&](int at, float (&f)[8]) {
    const float4 g0 = *reinterpret_cast<const float4*>(a.gain + at);
    const float4 g1 = *reinterpret_cast<const float4*>(a.gain + at + 4);
    f[0] *= g0.x; f[1] *= g0.y; f[2] *= g0.z; f[3] *= g0.w;
    f[4] *= g1.x; f[5] *= g1.y; f[6] *= g1.z; f[7] *= g1.w;
  };

  float u[kVectors][8];
  double sq = 0.0;
  int most = 0;
  {
    Vec8<XBF16> x[kVectors];
    Vec8<RBF16> r[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int v = tid + i * nthr;
      if (v < nvec) {
        x[i].load(xr, 8 * v);
        if constexpr (RES != kNone) r[i].load(rr, 8 * v);
      }
    }
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int v = tid + i * nthr;
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = 0.0f;
      if (v < nvec) {
        join(x[i], r[i], 8 * v, u[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double d = (double)u[i][e];
          sq = fma(d, d, sq);
        }
        times_gain(8 * v, u[i]);
        most = max(most, absmax8(u[i]));
      }
    }
  }
  for (int v = tid + kVectors * nthr; v < nvec; v += nthr) {
    Vec8<XBF16> x;
    Vec8<RBF16> r;
    float f[8];
    x.load(xr, 8 * v);
    if constexpr (RES != kNone) r.load(rr, 8 * v);
    join(x, r, 8 * v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = (double)f[e];
      sq = fma(d, d, sq);
    }
    times_gain(8 * v, f);
    most = max(most, absmax8(f));
  }

  sq = wave_sum_f64(sq);
  if constexpr (!F8) most = wave_max_nonneg(most);
  if (lane == 0) {
    red_s[wave] = sq;
    red_m[wave] = most;
  }
  lds_sync();
  double s = 0.0;
  int bm = 0;
  for (int w = 0; w < nwaves; ++w) {
    s += red_s[w];
    bm = max(bm, red_m[w]);
  }
  const double mean = s * a.inv_k;
  float ms = (float)(mean * (1.0 - 0x1p-44));
  if (ms != (float)(mean * (1.0 + 0x1p-44))) {       // the same in every thread
    for (int j = tid; j < 512; j += nthr) (&hist[0][0])[j] = 0ull;
    if (tid < kLimbs) word[tid] = 0ull;
    lds_sync();
    for (int v = tid; v < nvec; v += nthr) {
      float f[8];
      again(8 * v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(f[e]) & 0x7fffffffu;
        uint32_t m = b & 0x7fffffu;
        int ex = (int)(b >> 23);
        if (ex) m |= 0x800000u; else ex = 1;
        if (m) {                                     // m^2 in halves of 24 bits, at 2^(2 ex - 300)
          const unsigned long long q = (unsigned long long)m * m;
          atomicAdd(&hist[0][ex], q >> 24);
          atomicAdd(&hist[1][ex], q & 0xffffffull);
        }
      }
    }
    lds_sync();
    for (int j = tid; j < 512; j += nthr) {          // 32 bits at a time, carried afterwards
      const int ex = j & 255;
      const unsigned long long v = (&hist[0][0])[j];
      if (!v || ex == 255) continue;                 // (not finite: no defined result)
      const int at = 2 * ex + (j < 256 ? 22 : -2), l0 = at >> 5, o = at & 31;
      const unsigned long long lo = v << o;
      const uint32_t part[3] = {(uint32_t)lo, (uint32_t)(lo >> 32), o ? (uint32_t)(v >> (64 - o)) : 0u};
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (part[i]) atomicAdd(&word[l0 + i], (unsigned long long)part[i]);
    }
    lds_sync();
    if (tid == 0) {
      unsigned long long carry = 0;
      for (int i = 0; i < kLimbs; ++i) {
        carry += word[i];
        limb[i] = (uint32_t)carry;
        carry >>= 32;
      }
      exact = limbs_to_f64(limb, -298);
    }
    lds_sync();
    ms = (float)(exact / (double)K);
  }
  const float root = sqrtf(ms + a.eps_n);            // binary32, each rounded once
  float r = 1.0f / root;
  // a mean square that is no binary32 number gives no norm, which e4m3 codes can say
  if constexpr (F8)
    if (!(s < (double)__builtin_inff() && ms < __builtin_inff())) r = __builtin_nanf("");

  uint8_t* qr = a.xq + row * K;
  if constexpr (F8) {
    auto put = [&](int v, float (&f)[8]) {           // called by whole DPP rows
      const int gm = row_max16(v < nvec ? absmax8(f) : 0);
      const float m = fmaxf(__int_as_float(gm) * r, kF8Floor);
      const float inv = kF8Top / m;
      if (v < nvec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= r;
        *reinterpret_cast<uint2*>(qr + 8 * v) = make_uint2(f8_codes4(f[0], f[1], f[2], f[3], inv),
                                                           f8_codes4(f[4], f[5], f[6], f[7], inv));
        if ((v & 15) == 0) a.scale[(int64_t)(v >> 4) * a.T + row] = m / kF8Top;
      }
    };
#pragma unroll
    for (int i = 0; i < kVectors; ++i) put(tid + i * nthr, u[i]);
    for (int v0 = kVectors * nthr; v0 < nvec; v0 += nthr) {   // whole waves go round
      const int v = v0 + tid;
      float f[8] = {};
      if (v < nvec) {
        again(8 * v, f);
        times_gain(8 * v, f);
      }
      put(v, f);
    }
  } else {
    const float m = __int_as_float(bm) * r, sc = kQb / fmaxf(m, kEps);
    int sum = 0;
    auto put = [&](int v, float (&f)[8]) {
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = (int)fminf(fmaxf(rintf((f[4 * h + e] * r) * sc), -kQb), kQb);
          o |= (uint32_t)(q & 0xff) << (8 * e);
        }
        sum = __builtin_amdgcn_sdot4((int)o, 0x01010101, sum, false);
        w[h] = o;
      }
      *reinterpret_cast<uint2*>(qr + 8 * v) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
      if (tid + i * nthr < nvec) put(tid + i * nthr, u[i]);
    for (int v = tid + kVectors * nthr; v < nvec; v += nthr) {
      float f[8];
      again(8 * v, f);
      times_gain(8 * v, f);
      put(v, f);
    }
    if (a.rowsum) {
      sum = wave_sum_i(sum);
      if (lane == 0) red_q[wave] = sum;
      lds_sync();
      if (tid == 0) {
        int t = 0;
        for (int w = 0; w < nwaves; ++w) t += red_q[w];
        a.rowsum[row] = t;
      }
    }
    if (tid == 0) a.scale[row] = m;
  }
}

template <bool XBF16, int RES, bool F8>
hipError_t launch(const Args& base, int64_t t, hipStream_t stream) {
  const int64_t nvec = base.K / 8;
  // a launch has fewer than 2^32 threads, and a row takes up to 1024 of them
  constexpr int64_t kMost = int64_t(1) << 21;
  const int64_t thr = std::min<int64_t>(1024, ((nvec + kVectors - 1) / kVectors + 63) / 64 * 64);
  hipError_t e = hipSuccess;
  for (int64_t r = 0; e == hipSuccess && r < t; r += kMost) {
    Args a = base;
    a.row0 = r;
    const dim3 grid((unsigned)std::min(t - r, kMost)), block((unsigned)thr);
    k_add_subln<XBF16, RES, F8><<<grid, block, 0, stream>>>(a);
    e = hipGetLastError();
  }
  return e;
}

// e4m3 codes of tokens: 16 lanes per group of 128, one pass.  Bound by memory (4096
// tokens of 8192, bfloat16 22.3 us, 4.5 TB/s; binary32 31.3, 5.4), for few tokens by its
// launch (13 of 6912 2.4 us).
template <bool BF16>
__global__ __launch_bounds__(256) void k_quant_f8(const void* __restrict__ x, int64_t T, int K,
                                                  int groups, int64_t units,
                                                  uint8_t* __restrict__ xq,
                                                  float* __restrict__ scales) {
  const int l = threadIdx.x & 15;
  for (int64_t u = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); u < units;
       u += (int64_t)gridDim.x * 16) {
    const int64_t t = u / groups;
    const int g = (int)(u - t * groups), k = g * kF8Block + 8 * l;
    float f[8] = {};
    if (k < K) {
      Vec8<BF16> v;
      v.load(x, t * K + k);
      v.widen(f);
    }
    const float m = fmaxf(__int_as_float(row_max16(absmax8(f))), kF8Floor), inv = kF8Top / m;
    if (k < K)
      *reinterpret_cast<uint2*>(xq + t * K + k) = make_uint2(
          f8_codes4(f[0], f[1], f[2], f[3], inv), f8_codes4(f[4], f[5], f[6], f[7], inv));
    if (l == 0) scales[g * T + t] = m / kF8Top;
  }
}

}  // namespace

hipError_t launch_add_subln(const NormCall& c, hipStream_t stream) {
  const Args a{c.x, c.residual, c.gain, c.total, static_cast<uint8_t*>(c.xq), c.scale, c.rowsum,
               1.0 / (double)c.K, c.eps_n, (int)c.K, c.T, 0};
  const int res = !c.residual ? kNone : c.r_bf16 ? kResBf16 : kResF32;
  auto with = [&](auto xb, auto f8) {
    constexpr bool X = decltype(xb)::value, F = decltype(f8)::value;
    return res == kNone ? launch<X, kNone, F>(a, c.T, stream)
         : res == kResF32 ? launch<X, kResF32, F>(a, c.T, stream)
                          : launch<X, kResBf16, F>(a, c.T, stream);
  };
  using Y = std::true_type;
  using N = std::false_type;
  return c.x_bf16 ? (c.f8 ? with(Y{}, Y{}) : with(Y{}, N{})) : (c.f8 ? with(N{}, Y{}) : with(N{}, N{}));
}

hipError_t launch_quant_f8(const void* x, int bf16, int64_t t, int64_t k, uint8_t* xq,
                           float* scales, hipStream_t stream) {
  const int groups = (int)f8_blocks(k);
  const int64_t units = t * groups;
  const unsigned grid = (unsigned)std::min<int64_t>((units + 15) / 16, 1 << 20);
  if (bf16) k_quant_f8<true><<<grid, 256, 0, stream>>>(x, t, (int)k, groups, units, xq, scales);
  else k_quant_f8<false><<<grid, 256, 0, stream>>>(x, t, (int)k, groups, units, xq, scales);
  return hipGetLastError();
}

}  // namespace bl
