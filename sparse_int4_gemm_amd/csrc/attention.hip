// Joins the partial results of rows whose keys were split over workgroups:
//
//   m = max_s m_s,  l = sum_s l_s 2^(m_s - m),  O = sum_s O_s 2^(m_s - m) / l.
//
// One workgroup per output row; D/4 threads hold four elements each and the
// workgroup's thread groups take every (256 / (D/4))-th split, in an order that
// does not depend on when the splits arrived.  A separate launch: joining in
// the workgroup that arrives last needs an agent-scope release in every
// workgroup, which cost more than the launch (131071 keys, 8 key heads: 294 us
// against 128 us).
#include "attention_device.hpp"

namespace slim {
namespace {

constexpr int kThreads = 256;

template <class T, int D>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs a, int splits) {
    constexpr int kGroups = kThreads / (D / 4);              // D = 96: 10 groups of 24 threads, 16 idle
    __shared__ float part[kGroups][D];
    __shared__ float red[2][kThreads / 64];
    const int64_t row = blockIdx.x;
    const Partials parts(a, D, splits);
    const float* ml = parts.ml + 2 * row * splits;
    if (ml[1] == kWhole) return;
    float top = -INFINITY;
    for (int s = threadIdx.x; s < splits; s += kThreads) top = fmaxf(top, ml[2 * s]);
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float ms = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int s = threadIdx.x; s < splits; s += kThreads) sum += ml[2 * s + 1] * exp2_fast(ml[2 * s] - ms);
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = sum;
    const int group = threadIdx.x / (D / 4), d = (threadIdx.x - group * (D / 4)) * 4;
    if (group < kGroups) {
        f4 acc = f4{0, 0, 0, 0};
#pragma unroll 4
        for (int s = group; s < splits; s += kGroups)
            if (ml[2 * s + 1] != 0.0f)
                acc += *reinterpret_cast<const f4*>(parts.o + (row * splits + s) * D + d) * exp2_fast(ml[2 * s] - ms);
        *reinterpret_cast<f4*>(&part[group][d]) = acc;
    }
    __syncthreads();
    if (threadIdx.x < D / 4) {
        f4 acc = f4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kGroups; ++i) acc += *reinterpret_cast<const f4*>(&part[i][4 * threadIdx.x]);
        sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
        const int64_t token = row / a.q_heads;
        store_row4<T>(a, token, (int)(row - token * a.q_heads), D, 4 * threadIdx.x, acc, top, sum);
    }
}

template <class T>
void launch_dim(const AttnArgs& a, int splits, hipStream_t stream) {
    const dim3 grid((unsigned)(a.tokens * a.q_heads)), block(kThreads);
    switch (a.head_dim) {
        case 64: hipLaunchKernelGGL((attention_join_kernel<T, 64>), grid, block, 0, stream, a, splits); break;
        case 96: hipLaunchKernelGGL((attention_join_kernel<T, 96>), grid, block, 0, stream, a, splits); break;
        case 128: hipLaunchKernelGGL((attention_join_kernel<T, 128>), grid, block, 0, stream, a, splits); break;
        default: hipLaunchKernelGGL((attention_join_kernel<T, 256>), grid, block, 0, stream, a, splits); break;
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
    return kAttnReserved + ((parts + 255) & ~size_t(255));
}

}  // namespace slim
