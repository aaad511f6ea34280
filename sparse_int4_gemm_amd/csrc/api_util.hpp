// What the C-ABI front ends (slim_api.cpp, attention_api.cpp) share: the
// per-thread error text, the pointer and device checks and the size limits.
// Not installed; not part of the ABI.
#pragma once

#include "slim.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace slim {

// Sets this thread's error text (slim_last_error) and returns `s`.
slim_status fail(slim_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns SLIM_OK (a call with nothing to do).
slim_status done();
// SLIM_OK if the current device is gfx950.
slim_status check_device();
// Status of a launch: clears the error text on success.
slim_status launched(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Largest sizes any call accepts: every product of two of them fits int64
// (the kernels' grid and offset math, and the size queries, stay exact).
constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 40;    // elements between batched problems

}  // namespace slim
