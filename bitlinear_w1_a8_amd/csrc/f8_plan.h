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
// sizes with weights from memory.  Measured again with these kernels (11 matrices, 17 to 2048
// tokens), what the rule takes was 0.3% (binary32 outputs), 0.4% (bfloat16) and 1.7% (cut
// sums) behind the fastest on average, and 8%, 14% and 25% (17 tokens, 28672 -> 8192) at
// most.  Some of them, streaming / 64 x 64 / 128 x 64 / 128 x 128 / 256 x 128 / 256 x 256:
//   full sums, binary32 outputs
//    32 tokens, 2560 -> 6912      8.2 / 11.2 / 14.9 / 20.2 / 32.3
//    96 tokens, 6912 -> 2560     36.4 / 22.0 / 32.4 / 48.1 / 82.4
//   128 tokens, 5136 -> 13942    81.3 / 41.7 / 33.1 / 48.2 / 71.5
//   256 tokens, 8192 -> 28672     563 / 186 / 167 / 146 / 127
//   512 tokens, 28672 -> 8192    1035 / 329 / 276 / 244 / 325
//  2048 tokens, 2560 -> 6912      408 / 163 / 121 / 110 / 90.2
//   full sums, bfloat16 outputs
//   256 tokens, 2560 -> 6912     53.0 / 21.7 / 15.8 / 21.8 / 34.7
//   512 tokens, 8192 -> 8192      319 / 101 / 80.2 / 64.6 / 95.4
//  2048 tokens, 2560 -> 6912      397 / 148 / 108 / 96.2 / 79.5
//   cut sums, bfloat16 outputs
//    64 tokens, 8192 -> 28672     146 / 56.3 / 55.4 / 68.3 / 72.0 / 106
//   256 tokens, 2560 -> 6912     53.1 / 17.6 / 12.4 / 17.4 / 24.1 / 36.3
//   512 tokens, 8192 -> 8192      319 / 76.4 / 55.1 / 43.4 / 61.2 / 81.3
//  2048 tokens, 6912 -> 2560      346 / 96.2 / 73.5 / 71.1 / 54.3 / 74.7
//  2048 tokens, 2560 -> 6912      396 / 135 / 91.6 / 76.6 / 56.9 / 46.5
// The streaming kernel with 32 rows per block from 17 tokens on, where that leaves half the
// CUs a block (32 tokens, 2560 -> 6912 10.1 -> 8.2; 17 tokens, 28672 -> 8192 65.5 -> 54.2).
// The border of 16 tokens is right for few rows and for up to 8 tokens, and costs large matrices
// up to a seventh at 16 (16 rows / 32 rows per block / best tiles, binary32 outputs):
//    16 tokens, 6912 -> 2560      8.8 / 14.5 / 21.3      2560 -> 6912      7.5 / 7.4 / 11.0
//    16 tokens, 28672 -> 8192    59.0 / 53.8 / 81.7      8192 -> 28672    58.3 / 63.7 / 51.3
//    16 tokens, 2560 -> 128256   81.0 / 96.4 / 76.2
//     8 tokens, 28672 -> 8192    49.8 / 49.4 / 80.4      8192 -> 28672    48.2 / 59.4 / 50.7
// so that 17 tokens take less time than 16 there (54.2, 51.2 and 75.4).
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
