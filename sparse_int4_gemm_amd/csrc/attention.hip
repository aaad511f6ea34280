// Joins the partial results of rows whose keys were split over workgroups:
//
//   m = max_s m_s,  l = sum_s l_s 2^(m_s - m),  O = sum_s O_s 2^(m_s - m) / l.
//
// A workgroup joins S elements of one row: S / 4 threads hold four elements
// each, its groups of S / 4 threads take every (256 / (S / 4))-th split and add up through
// LDS in an order that does not depend on when the splits were written.  Bound
// by latency: few rows are cut into slices of 32 elements (32 rows of 256 splits
// of head size 128: 25 us whole, 8 us cut), many stay whole (1952 rows of 16 splits: 6 us
// whole, 22 us cut: four rounds of workgroups).
// A separate launch: joining in the workgroup that arrives last needs an
// agent-scope release in every workgroup, which cost more than the launch
// (131071 keys, 8 key heads: 294 us against 128 us).
#include "attention_device.hpp"

namespace slim {
namespace {

constexpr int kThreads = 256;

template <class T, int D, int S>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs a, int splits) {
    constexpr int kGroups = kThreads / (S / 4);              // S = 96: 10 groups of 24 threads, 16 idle
    __shared__ __align__(16) float part[kGroups][S];
    __shared__ float part_sum[kGroups];
    __shared__ float red[kThreads / 64];
    const int64_t row = blockIdx.x;
    const int token = (int)(blockIdx.x / (uint32_t)a.q_heads);
    // Rows of no sequence have no partial results, and their outputs are not this call's.
    if (a.kv.starts && (token < a.kv.starts[0] || token >= a.kv.starts[a.kv.seqs])) return;
    const Partials parts(a, D, splits);
    const float* ml = parts.ml + 2 * row * splits;
    if (ml[1] == kWhole) return;
    const int group = threadIdx.x / (S / 4), c = threadIdx.x % (S / 4) * 4, d = blockIdx.y * S + c;
    float top = -INFINITY;
    for (int s = threadIdx.x; s < splits; s += kThreads) top = fmaxf(top, ml[2 * s]);
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float ms = top == -INFINITY ? 0.0f : top;
    f4 acc = f4{0, 0, 0, 0};
    float sum = 0.0f;
#pragma unroll 4
    for (int s = group < kGroups ? group : splits; s < splits; s += kGroups) {
        const float f = exp2_fast(ml[2 * s] - ms), l = ml[2 * s + 1];
        const f4 x = *reinterpret_cast<const f4*>(parts.o + (row * splits + s) * D + d);
        sum += l * f;
        if (l != 0.0f) acc += x * f;               // a split without keys stored nothing
    }
    if (group < kGroups) {
        *reinterpret_cast<f4*>(&part[group][c]) = acc;
        if (c == 0) part_sum[group] = sum;
    }
    __syncthreads();
    if (group == 0) {
        acc = f4{0, 0, 0, 0};
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            acc += *reinterpret_cast<const f4*>(&part[i][c]);
            sum += part_sum[i];
        }
        store_row4<T>(a, token, (int)blockIdx.x - token * a.q_heads, D, d, acc, top, sum);
    }
}

template <class T, int D>
void launch(const AttnArgs& a, int splits, hipStream_t stream) {
    const int64_t rows = (int64_t)a.tokens * a.q_heads;
    if (rows * (D / 32) <= 1024)
        hipLaunchKernelGGL((attention_join_kernel<T, D, 32>), dim3((unsigned)rows, D / 32), dim3(kThreads), 0, stream, a,
                           splits);
    else
        hipLaunchKernelGGL((attention_join_kernel<T, D, D>), dim3((unsigned)rows), dim3(kThreads), 0, stream, a, splits);
}

template <class T>
void launch_dim(const AttnArgs& a, int splits, hipStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch<T, 64>(a, splits, stream);
        case 96: return launch<T, 96>(a, splits, stream);
        case 128: return launch<T, 128>(a, splits, stream);
        default: return launch<T, 256>(a, splits, stream);
    }
}

}  // namespace

hipError_t launch_attention_join(const AttnArgs& a, int splits, hipStream_t stream) {
    if (a.dtype == 0) launch_dim<Fp16>(a, splits, stream);
    else launch_dim<Bf16>(a, splits, stream);
    return hipGetLastError();
}

// Partials of a bounded number of (row, split) pairs, whatever the batch, so
// one workspace serves every batch of its heads.
size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    const size_t parts = (size_t)kAttnSplitRows * (size_t)(head_dim + 2) * sizeof(float);
    return (parts + 255) & ~size_t(255);
}

}  // namespace slim
