// How a whole routed layer runs, by sizes and the tokens' type: plain C++, so that
// it can be asked without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "experts_plan.h"
#include "w4_plan.h"

namespace bl {

constexpr int kLayerTokens = 16;   // most tokens of the two launches: the columns of an MFMA
constexpr int kRawTokens = 6;      // most whose step A1 every block repeats
constexpr int kPairTokens = 4;     // most whose blocks belong to (token, rank) pairs
constexpr int kLayerTopK = 16;     // most experts per token: one DPP row
constexpr int kLayerExperts = 256; // most experts: 16 logits per lane of a row

struct LayerPlan {
  bool two;          // the two launches of layer.hip; else the three calls' kernels, and nothing below
  bool own_quant;    // step A1 of raw tokens in a launch of its own before
  bool pairs;        // gate blocks per (token, rank), not per expert
  int gate_waves;    // of 16 weight rows each
  int down_tiles;    // 16 outputs each per block
  int team;          // waves that split a row of h
};

// LDS of int8 rows of k, with their raw values of `raw` bytes each (0: none).
inline int64_t layer_rows_lds(int64_t k, int64_t rows, int raw) { return rows * (few_stride((int)k) + raw * k); }

// raw: bytes per value of tokens that are not quantised yet (2 or 4), or 0.
inline LayerPlan layer_plan(int64_t t, int64_t e, int64_t k, int64_t f, int64_t kk, int64_t n, int raw,
                            int cus) {
  LayerPlan p{};
  // the last: blocks of up to 1024 threads, fewer than 2^32 of them in a row of the grid
  p.two = t <= kLayerTokens && k <= kLayerTopK && e <= kLayerExperts &&
          layer_rows_lds(kk, t, 0) <= kMaxLds && layer_rows_lds(f, k, 0) <= kMaxLds && n < (1 << 25);
  if (!p.two) return p;
  // Step A1 in every block, or in a launch of its own before.  Its own / in the blocks,
  // bfloat16, 8 of 64 experts of 2560 -> 1024 -> 2560: one token 16.2 / 13.9 us, four 22.4 /
  // 20.8, six 27.3 / 26.6, eight 29.5 / 30.4, sixteen 39.1 / 47.0; 2 of 16 of 4096, six 36.4 / 32.3,
  // eight 41.8 / 43.1.  Rows of binary32 take LDS from other blocks: three tokens of 2560
  // (38 KB) 20.1 / 19.3, four (51 KB) 22.5 / 25.6, of 4096 three (61 KB) 26.3 / 28.1.
  p.own_quant = raw && !(t <= kRawTokens && layer_rows_lds(kk, t, raw) <= (raw == 2 ? kMaxLds : 48 * 1024));
  // Blocks of (token, rank) pairs for at most four tokens, whose waves rank a token each,
  // where they spare a thousand blocks of experts that no token takes (about 2 us; to find
  // the expert takes 1.5).  Of 2560 -> 2 x 1024, 32 blocks an expert, per expert / per pair: one
  // token, 8 of 64 experts 10.4 / 8.7 us, of 128 10.7 / 8.4, of 256 13.1 / 11.3; four tokens,
  // 8 of 64 13.8 / 12.0; but one token, 8 of 16 7.6 / 8.2, 4 of 32 7.3 / 7.7.
  p.pairs = t <= kPairTokens && (e - t * k) * ((2 * f + 63) / 64) >= 1024;
  // 128 weight rows per block where that leaves blocks enough, else 64, as k_experts_few
  // (16 tokens, 8 of 64 experts: 22.8 -> 18.1 us; one token 11.0 / 7.8)
  p.gate_waves = !p.pairs && (2 * f + 127) / 128 * std::min(t * k, e) >= 512 ? 8 : 4;
  // 32 outputs per block where blocks of 16 would be more than four per CU, which
  // run at once (16 tokens, 8 of 64 experts, 1024 -> 2560: 18.1 -> 17.1 us; 3 tokens 6.4 / 6.6,
  // one 5.1 / 6.6; 64 outputs 19.5).  Blocks of one run of outputs side by side on an XCD,
  // for its L2, gained nothing (19.7).
  p.down_tiles = (n + 15) / 16 * t > 4 * cus ? 2 : 1;
  p.team = (int)std::max<int64_t>(1, std::min<int64_t>(16 / k, ((f + 255) / 256 + 3) / 4));
  return p;
}

}  // namespace bl
