// Device helpers shared by the cache and attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.hpp"

namespace slim {

constexpr int kMaxLen = 1 << 30;      // lengths read from device memory are clamped to [0, kMaxLen]

__device__ __forceinline__ int seq_len(const PagedKV& kv, int b) {
    const int n = kv.lens[b];
    return n < 0 ? 0 : (n > kMaxLen ? kMaxLen : n);
}

// The sequence whose new tokens hold row t, by one wave: 64 sequences are
// looked at per step (a load and a ballot), so a batch of up to 64 costs one
// memory latency.  Returns -1 if t belongs to none.  Every lane gets the
// same answer, within [-1, seqs) whatever `starts` holds.
__device__ __forceinline__ int find_seq(const PagedKV& kv, int t) {
    if (!kv.starts) return t < kv.seqs ? t : -1;
    const int lane = threadIdx.x & 63;
    int lo = 0, n = kv.seqs;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lane * step;
        const uint64_t m = __ballot(at < n && kv.starts[lo + (at < n ? at : 0)] <= t);
        if (m == 0) return -1;
        const int c = 63 - __builtin_clzll(m);
        lo += c * step;
        n = n - c * step < step ? n - c * step : step;
    }
    return kv.starts[lo] <= t && t < kv.starts[lo + 1] ? lo : -1;
}

}  // namespace slim
