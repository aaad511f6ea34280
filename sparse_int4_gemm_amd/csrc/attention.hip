// Attention over the paged cache, one wave per query row and head: the
// formulas as they stand, correct for every shape.
//
//   lane j scores key base + j:  s_j = scale * sum_d q_d k_jd
//   running maximum m and sum l over blocks of 64 keys,
//   lane owns the output elements d = lane + 64 i.
#include "attention_device.hpp"

namespace slim {
namespace {

__device__ __forceinline__ float to_float(uint16_t x, int dtype) {
    return dtype == 0 ? (float)__builtin_bit_cast(_Float16, x) : __builtin_bit_cast(float, (uint32_t)x << 16);
}
__device__ __forceinline__ uint16_t from_float(float x, int dtype) {
    return dtype == 0 ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint16_t, (__bf16)x);
}

__global__ __launch_bounds__(64) void attention_plain_kernel(AttnArgs a) {
    __shared__ float qs[256];
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int kvh = h / (a.q_heads / a.kv_heads), D = a.head_dim;
    const int b = find_seq(a.kv, t);
    if (b < 0) return;
    const int len = seq_len(a.kv, b);
    const int p = a.kv.starts ? len + t - a.kv.starts[b + 1] : len - 1;
    for (int d = lane; d < D; d += 64) qs[d] = to_float(a.q[t * a.sq + (int64_t)h * D + d], a.dtype);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    const int64_t capacity = (int64_t)a.kv.width << a.kv.page_shift;
    const int end = p + 1 < capacity ? p + 1 : (int)capacity;
    for (int base = 0; base < end; base += 64) {
        const int j = base + lane;
        bool seen = j < end && (a.window == 0 || j > p - a.window || j < a.sinks);
        int page = -1;
        if (seen) page = a.kv.table[(int64_t)b * a.kv.width + (j >> a.kv.page_shift)];
        seen = seen && page >= 0 && page < a.kv.pages;
        const int64_t row = seen ? ((((int64_t)page * a.kv_heads + kvh) << a.kv.page_shift) + (j & ((1 << a.kv.page_shift) - 1))) * D : 0;
        float s = -INFINITY;
        if (seen) {
            s = 0.0f;
            for (int d = 0; d < D; ++d) s = fmaf(qs[d], to_float(a.kv.k[row + d], a.dtype), s);
            s *= a.scale;
        }
        float top = s;
        for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.0f : mn;
        const float f = expf(m - ms), e = seen ? expf(s - ms) : 0.0f;
        m = mn;
        l = l * f;
        for (int i = 0; i < 4; ++i) o[i] *= f;
        for (int k = 0; k < 64; ++k) {
            if (!__shfl((int)seen, k)) continue;
            const float w = __shfl(e, k);
            const int64_t r = __shfl(row, k);
            l += w;
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < D) o[i] = fmaf(w, to_float(a.kv.v[r + lane + 64 * i], a.dtype), o[i]);
        }
    }
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < D)
            a.o[t * a.so + (int64_t)h * D + lane + 64 * i] = from_float(l == 0.0f ? 0.0f : o[i] / l, a.dtype);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

hipError_t launch_plain(const AttnArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(attention_plain_kernel, dim3((unsigned)a.tokens, (unsigned)a.q_heads), dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// Partials of the split form: at most kSplitTarget workgroups of at most 16
// rows, whatever the batch, so a workspace serves every batch of its heads.
size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    const int64_t share = q_heads / kv_heads;
    const size_t parts = (size_t)(kSplitTarget * (share < 16 ? share : 16)) * (size_t)(head_dim + 2) * sizeof(float);
    return kAttnCounters + ((parts + 255) & ~size_t(255));
}

hipError_t launch_attention_prefill(const AttnArgs& a, hipStream_t stream) { return launch_plain(a, stream); }

}  // namespace slim
