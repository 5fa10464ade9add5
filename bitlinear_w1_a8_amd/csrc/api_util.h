// Shared by the translation units that implement the C ABI: limits, argument
// checks and the thread's error message.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitlinear.h"

namespace bl {

constexpr int64_t kMaxT = int64_t(1) << 24;
constexpr int64_t kMaxN = int64_t(1) << 26;
constexpr int64_t kMaxNK = int64_t(1) << 38;  // keeps every gamma bucket below 2^62
constexpr int64_t kMaxTN = int64_t(1) << 36;  // y up to 256 GiB

// Records the message that bitlinear_last_error() returns and gives back `code`.
bl_status fail(bl_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// The status of a launch: BL_OK (which clears the message) or BL_ERR_HIP.
bl_status launched(const char* fn, hipError_t e);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bl_status check_k(const char* fn, int64_t k) {
  if (k < 16 || k > BITLINEAR_MAX_K || k % 16 != 0)
    return fail(BL_ERR_SHAPE, "%s: K=%lld must be a multiple of 16 in [16, %d]", fn,
                (long long)k, BITLINEAR_MAX_K);
  return BL_OK;
}

}  // namespace bl
