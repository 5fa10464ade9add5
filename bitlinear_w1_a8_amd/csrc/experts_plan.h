// Choices of the routed-expert kernels by size: plain C++, so that they can be
// asked without a device.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bl {

// Chunks of 256 k that a wave of k_experts_few has on their way: as many as the
// row has (in pairs, which keeps the kernels few), up to ten.  Loads past the
// row's end would fetch its last chunk again, and fewer than the row has come
// later.  Gated, 64 experts of K -> 2 x 1024, 33 tokens of 6, weights from memory,
// 2 / 4 / 6 / 8 / 10 / 12 / 16 chunks:
//   K =  512  10.4 / 11.2 / 12.3 / 13.5 / 14.9 / 16.2 / 19.9 us
//       1024  13.0 / 12.9 / 13.5 / 14.6 / 16.1 / 17.2 / 21.9
//       1280  15.2 / 14.6 / 14.4 / 14.7 / 15.2 / 15.8 / 18.5
//       1536  16.2 / 16.1 / 15.5 / 16.2 / 17.4 / 18.7 / 24.5
//       2048  19.1 / 19.5 / 18.7 / 18.6 / 19.0 / 20.0 / 25.2
//       2560  22.4 / 22.1 / 21.7 / 20.9 / 21.0 / 21.7 / 25.1
//       4096  35.3 / 34.4 / 33.6 / 32.4 / 29.7 / 29.8 / 30.5
//       6912  64.9 / 55.9 / 50.5 / 48.8 / 47.6 / 48.4 / 48.1
// 4 tokens of 8: 1280 9.9 / 9.5 / 9.5 / 9.7 / 10.0, 1536 10.7 / 10.3 / 10.3 / 10.7 / 11.4,
// 2048 12.0 / 11.8 / 11.6 / 12.1 / 12.6, 4096 19.1 / 18.3 / 17.7 / 17.7 / 17.7, 6912
// 40.0 / 33.6 / 30.4 / 29.4 / 28.7.
inline int few_depth(int64_t k) {
  const int64_t chunks = (k + 255) / 256;
  return (int)std::min<int64_t>((chunks + 1) / 2 * 2, 10);
}

// LDS row stride of int8 activations: whole chunks of 256 k, zero past K, and
// 16 bytes that spread the rows of one operand read over the banks.
constexpr int few_stride(int k) { return ((k + 255) & ~255) + 16; }

}  // namespace bl
