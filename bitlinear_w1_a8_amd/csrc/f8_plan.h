// Which kernel an e4m3 product takes, by sizes and sums: plain C++, so that
// it can be asked without a device.
#pragma once

#include <stdint.h>

namespace bl {

enum F8Kernel {
  kF8Few1,     // k_f8_few, up to 16 rows per block
  kF8Few2,     // k_f8_few, 32 rows per block (17 to 32 tokens)
  kF8Small,    // k_f8_tile, 64 x 64, three groups of waves that share K
  kF8Tall,     // k_f8_tile, 128 x 64, two groups
  kF8Square,   // k_f8_tile, 128 x 128, two groups
  kF8Wide,     // k_f8_tile, 256 x 128
  kF8Turns,    // k_f8_turns, 256 x 256 (cut sums only)
};

// Up to 16 tokens the streaming kernel, beyond them the least of these estimates, in
// microseconds.  A kernel of tiles takes rounds of one tile per CU, each of them a
// time per block of 128 k and one for its start and end; the streaming kernel grows
// with rows and lots of 64 tokens per CU, and a launch of it has fewer than 2^32 threads
// (tiles always have, as T * N <= 2^36).  Fitted to graph replays of every kernel at 138
// sizes (8 to 2048 tokens) with weights from memory; what the rule takes was 0.8%
// behind the fastest on average, 15% at most.  Some of them, streaming / 64 x 64 / 128 x
// 64 / 128 x 128 / 256 x 128 / 256 x 256:
//   full sums, binary32 outputs
//    32 tokens, 2560 -> 6912      8.1 / 11.4 / 15.0 / 20.3 / 32.4
//    96 tokens, 6912 -> 2560     36.2 / 22.0 / 32.6 / 48.3 / 82.5
//   128 tokens, 5136 -> 13942    60.8 / 41.9 / 33.4 / 48.5 / 72.0
//   256 tokens, 8192 -> 28672     353 / 181 / 159 / 143 / 125
//   512 tokens, 28672 -> 8192     624 / 322 / 269 / 236 / 324
//  2048 tokens, 2560 -> 6912      256 / 162 / 118 / 106 / 85.6
//   cut sums, bfloat16 outputs
//    64 tokens, 8192 -> 28672     106 / 58.6 / 58.0 / 69.5 / 78.0 / 109
//   256 tokens, 2560 -> 6912     37.7 / 17.5 / 12.8 / 17.8 / 24.6 / 36.4
//   512 tokens, 8192 -> 8192      198 / 74.5 / 53.8 / 42.7 / 61.4 / 81.5
//  2048 tokens, 6912 -> 2560      345 / 97.9 / 73.7 / 70.9 / 53.6 / 88.5
//  2048 tokens, 2560 -> 6912      245 / 132 / 89.5 / 75.3 / 55.7 / 46.9
// The streaming kernel with 32 rows per block from 17 tokens on, where that leaves half the
// CUs a block (32 tokens, 2560 -> 6912 9.9 -> 8.1, 8192 -> 28672 80.9 -> 72.9; 13 tokens, 6912
// -> 2560 8.3 -> 11.7).
inline F8Kernel f8_kernel(int64_t t, int64_t n, int64_t k, bool cut, int cus) {
  if (t <= 16) return kF8Few1;
  const int64_t lots = (t + 63) / 64;
  const double blocks = (double)((k + 127) / 128);
  const double rows = (double)lots * (double)n * 1e-4 * (256.0 / cus);   // (fitted on 256 CUs)
  F8Kernel best = t <= 32 && (n + 31) / 32 >= cus / 2 ? kF8Few2 : kF8Few1;
  double least = t <= 32 ? 2.3 + 1.7 * rows + blocks * (0.14 + 0.22 * rows)
                         : 2.8 + 3.6 * rows + blocks * (0.235 + 0.3 * rows);
  if ((n + 15) / 16 * lots >= int64_t(1) << 23) least = 1e300;           // of 512 threads each
  struct Tile {
    F8Kernel kernel;
    int rows, tokens;
    double block[2], round[2];                      // full, cut sums
  };
  static constexpr Tile kTiles[] = {
      {kF8Small, 64, 64, {0.36, 0.29}, {4.2, 3.4}},    {kF8Tall, 128, 64, {0.59, 0.43}, {4.7, 3.5}},
      {kF8Square, 128, 128, {0.96, 0.69}, {6.2, 3.9}}, {kF8Wide, 256, 128, {1.55, 0.98}, {10, 6.3}},
      {kF8Turns, 256, 256, {0, 1.5}, {0, 8.7}}};
  for (const Tile& c : kTiles) {
    if (c.kernel == kF8Turns && !cut) continue;
    const int64_t tiles = ((n + c.rows - 1) / c.rows) * ((t + c.tokens - 1) / c.tokens);
    const double time = (double)((tiles + cus - 1) / cus) * (blocks * c.block[cut] + c.round[cut]);
    if (time < least) {
      least = time;
      best = c.kernel;
    }
  }
  return best;
}

// Rows per block of kF8Few1, a multiple of four: as few as make no more blocks than CUs.
inline int f8_few_rows(int64_t t, int64_t n, int cus) {
  for (int rows = 4; rows < 16; rows += 4)
    if ((n + rows - 1) / rows * ((t + 63) / 64) <= cus) return rows;
  return 16;
}

}  // namespace bl
