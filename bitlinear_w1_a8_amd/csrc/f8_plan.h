// Which kernel an e4m3 product takes, by sizes and output type: plain C++, so that
// it can be asked without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

enum F8Kernel {
  kF8Few1,     // k_f8_few, 16 rows per block
  kF8Few2,     // k_f8_few, 32 rows per block
  kF8Split,    // k_f8_tile, 128 x 128, two groups of waves that share K
  kF8Wide,     // k_f8_tile, 256 x 128
  kF8Turns,    // k_f8_turns, 256 x 256 (bfloat16 outputs only)
};

// Up to 32 tokens the streaming kernel, beyond them the least of these estimates
// of the time per block of 128 k, in microseconds, from cases on 256 CUs with weights
// from memory: a kernel of tiles takes its time per round of one tile per CU,
// the streaming kernel grows with rows and tokens.  Streaming / 128 x 128 / 256 x 128 /
// 256 x 256, binary32 and bfloat16 outputs:
//    96 tokens, 2560 -> 2560    11.0 / 22.5 / 36.0       10.5 / 15.9 / 22.5 / 28.9 us
//    96 tokens, 2560 -> 6912    18.4 / 22.8 / 36.6       18.0 / 16.2 / 23.1 / 29.3
//   256 tokens, 2560 -> 6912    38.1 / 24.3 / 39.3       36.9 / 17.5 / 24.4 / 36.4
//   250 tokens, 8192 -> 28672    347 / 145 / 127          344 / 111 / 82 / 127
//   256 tokens, 28672 -> 8192    317 / 221 / 322          316 / 183 / 216 / 382
//  1024 tokens, 2560 -> 6912     129 / 56.0 / 44.5        125 / 39.7 / 28.4 / 42.6
//  2048 tokens, 6912 -> 2560     216 / 109 / 87.9         213 / 77.7 / 56.5 / 102
//  2048 tokens, 2560 -> 6912     248 / 108 / 87.9         242 / 79.0 / 57.8 / 51.8
//  4096 tokens, 2560 -> 6912     493 / 203 / 175          480 / 155 / 112 / 102
// 16 rows per block where blocks of 32 would leave half the CUs idle, and up to 16
// tokens always (13 tokens, 6912 -> 2560 8.3 against 11.7 us; 4 tokens, 8192 -> 28672
// 43.1 / 48.7; 32 tokens 12.4 / 16.2 and 80.8 / 72.2; 64 tokens, 2560 -> 6912 16.5 / 11.0).
inline F8Kernel f8_kernel(int64_t t, int64_t n, bool bf16, int cus) {
  const F8Kernel few = t <= 16 || (n + 31) / 32 < cus / 2 ? kF8Few1 : kF8Few2;
  if (t <= 32) return few;
  auto rounds = [&](int64_t rows, int64_t tokens) {
    const int64_t tiles = ((n + rows - 1) / rows) * ((t + tokens - 1) / tokens);
    return (double)((tiles + cus - 1) / cus);
  };
  const double cost[] = {(double)((t + 63) / 64) * (double)n * 7e-5 * (bf16 ? 1.3 : 1.0),
                         rounds(128, 128) * (bf16 ? 0.85 : 1.2), rounds(256, 128) * (bf16 ? 1.2 : 1.95),
                         rounds(256, 256) * 1.8};
  const F8Kernel kernel[] = {few, kF8Split, kF8Wide, kF8Turns};
  return kernel[std::min_element(cost, cost + (bf16 ? 4 : 3)) - cost];
}

}  // namespace bl
