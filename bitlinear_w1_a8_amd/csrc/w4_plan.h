// Which kernel a 4-bit product takes: plain C++, so that the choice can be
// asked without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

constexpr int kMaxLds = 150 * 1024;   // dynamic LDS of a block (a CU has 160 KiB, the static part included)

constexpr int kBlock = 128;           // weights per packed block (64 bytes)

// Blocks of 128 k that a wave of k_w4_few loads at a time, into each of two
// buffers (2560 -> 128256, one token: 2 / 4 / 5 / 8 blocks 34.7 / 34.5 / 35.0
// / 40.0 us; 8192 -> 28672: 34.6 / 28.9 / 34.4 / 31.4).
constexpr int kAhead = 4;

// LDS row stride of a token of k_w4_few: whole blocks of 128 k, and 16 bytes
// that spread the rows of one operand read over the banks.
constexpr int64_t token_stride(int64_t k) { return (k + kBlock - 1) / kBlock * kBlock + 16; }

struct W4Plan {
  // k_w4_tile<wn, wk, wmf>, or with wn = 0 k_w4_few
  int wn, wk, wmf;
  // k_w4_few: waves that split K, and tokens per pass over the matrix
  int team;
  int64_t tokens;
};

// T tokens, N rows of K weights in groups of G, on `cus` compute units.
inline W4Plan w4_plan(int64_t t, int64_t n, int64_t k, int g, int64_t cus) {
  auto tiles = [&](int64_t rows, int64_t cols) {
    return ((t + rows - 1) / rows) * ((n + cols - 1) / cols);
  };
  // k_w4_few keeps whole tokens in LDS: as many at a time as it holds, and a
  // pass over the matrix for each lot.  k_w4_tile reads the matrix once, so it
  // has the batches that would take three passes or more, and those of two but
  // for matrices so small that their tiles leave CUs idle and K is cut over
  // eight waves.  us, k_w4_few / k_w4_tile:
  //   one pass    2560 -> 128256, 16 tokens 41.8 / 62.3; 8192 -> 12288, 16 21.1 / 22.9;
  //               14336 -> 8192, 8 20.6 / 22.3; 28672 -> 8192, 5 33.3 / 39.5; 14336 ->
  //               16384, 10 35.7 / 39.4; 131072 -> 1024, 1 58.7 / 144.9
  //   two         28672 -> 8192, 6 55.4 / 38.9; 14336 -> 8192, 12 35.2 / 22.6; 10240 ->
  //               128256, 16 294 / 240; small ones: 28672 -> 4064, 10 36.3 / 36.9;
  //               28672 -> 2560, 10 37.1 / 38.9; 28672 -> 1024, 10 31.7 / 35.9; 14336 ->
  //               2560, 16 24.9 / 24.7, groups of 32 27.0 / 23.0; 131072 -> 1024, 2 105 / 146
  //   three, four 28672 -> 8192, 11 79.8 / 40.4, 16 104.7 / 42.5; 28672 -> 2560, 12 52.4 /
  //               39.5; 28672 -> 1024, 11 42.6 / 36.1; 131072 -> 1024, 3 150.5 / 146.1
  const int64_t most = std::min<int64_t>(16, kMaxLds / token_stride(k));
  const int64_t passes = (t + most - 1) / most, tiles16 = (n + 15) / 16;
  if (t <= 16 && (passes == 1 || (passes == 2 && tiles16 < cus))) {
    // K split over a team of waves while a wave has more than one load group and
    // twice the team still leaves one block per CU, two for one token (several
    // tokens are staged by every block: 2560 -> 6912, 7 tokens, groups of 32, teams
    // of 4 / 8 10.1 / 13.5 us).  Up to the border itself: 28672 -> 8192, where a team of
    // 4 makes one block per CU, 5 tokens, teams of 2 / 4 / 8 55.0 / 34.5 / 35.9 us, and
    // just beyond it, 28672 -> 8320, 55.3 / 56.2 / 47.5; 2560 -> 16384, 8 tokens, 1 / 2 / 4
    // 12.7 / 9.9 / 9.8; one token, 28672 -> 8192, 4 / 8 33.9 / 27.3, 2560 -> 16384, 2 / 4
    // 8.9 / 8.5.
    const int64_t per_cu = t == 1 ? 2 : 1, blocks = (k + kBlock - 1) / kBlock;
    int team = 1;
    while (team < 8 && 2 * tiles16 * team <= 8 * per_cu * cus && blocks > kAhead * team) team *= 2;
    return {0, 0, 0, team, most};
  }
  // the smallest tiles, with K split most, that do not outnumber the CUs; then
  // larger ones while each CU still gets one or more
  if (tiles(32, 32) <= cus) return {1, 8, 1, 0, 0};
  if (tiles(32, 64) <= cus) return {2, 4, 1, 0, 0};
  if (tiles(32, 128) <= cus) return {4, 2, 1, 0, 0};
  if (g == 128 && 8 * tiles(128, 256) >= 5 * cus) return {8, 1, 4, 0, 0};
  if (4 * tiles(64, 128) >= 5 * cus) return {4, 1, 2, 0, 0};
  return {4, 1, 1, 0, 0};
}

}  // namespace bl
