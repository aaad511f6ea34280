// slim_rope: rotary positions on rows of heads.
//
//   (a, b) -> (a cos - b sin, b cos + a sin) of every pair, angle = position * frequency.
//
// Bound by HBM (4 bytes an element, read and written once) for prompts, by
// launch and the chain position -> angle -> rows for single tokens.  A wave
// takes one token's rows, or a part of them, and forms the token's cosines and
// sines itself, in fp64, into its own part of LDS: a table of them would be
// read from HBM (8 bytes a pair) and end at some position.  The rows' loads
// are issued first and are in flight meanwhile.
//
// 4096 tokens of 32 heads of 128: 11.8 us, 5.7 TB/s, as a plain copy; one token 2.1 us.
#include "rope_device.hpp"

namespace slim {
namespace {

constexpr int kMaxHalf = 512;                 // head_dim is at most 1024

// N units a lane.  Waves of a token: `slices`.
template <class T, int C, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_kernel(RopeArgs a, int units, int slices) {
    extern __shared__ float2 rope_lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t task = (int64_t)blockIdx.x * kRopeWaves + wave;
    const int token = (int)(task / slices), slice = (int)(task - (int64_t)token * slices);
    if (token >= a.tokens) return;
    const int all = a.heads * units, first = slice * (64 * N) + lane;
    const uint16_t* x = a.x + token * a.sx;
    uint16_t* y = a.y + token * a.sy;
    float2* turns = rope_lds + wave * a.by.half;
    Vectors<C> v[N];
    Unit<C> u[N];
    int head[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = min(first + 64 * n, all - 1);
        head[n] = i / units;
        u[n] = unit_of<C>(a.by, a.head_dim, i - head[n] * units);
        load_unit<false>(v[n], u[n], x + head[n] * a.head_dim);
    }
    turns_to_lds(turns, a.by, a.positions[token]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (first + 64 * n >= all) continue;
        turn_unit<T>(v[n], u[n], a.by, turns);
        store_unit(v[n], u[n], y + head[n] * a.head_dim);
    }
}

// One unit a lane while the processor holds all waves at once, so that a token's
// chain is as short as can be, else four, so that fewer waves form its cosines
// (32 heads of 128, 512 tokens: 3.3 us with one, 4.3 with four; 2048, a round: 8.2 and 8.3; 4096: 13.3 and 11.8).
template <class T, int C>
hipError_t launch(const RopeArgs& a, hipStream_t stream) {
    const int units = units_of(a.by, a.head_dim, C), all = a.heads * units;
    const int n = rounds(a.tokens, all) > 1.0f ? 4 : 1, slices = (all + 64 * n - 1) / (64 * n);
    const int64_t tasks = (int64_t)a.tokens * slices;
    // A grid holds fewer than 2^32 threads; tokens past 2^25 waves go into further launches.
    const int64_t at_once = (int64_t(1) << 25) / slices;
    const size_t lds = (size_t)kRopeWaves * a.by.half * sizeof(float2);
    for (int64_t t = 0; t * slices < tasks; t += at_once) {
        RopeArgs b = a;
        b.x += t * a.sx;
        b.y += t * a.sy;
        b.positions += t;
        b.tokens = (int32_t)min(at_once, a.tokens - t);
        const dim3 grid((unsigned)(((int64_t)b.tokens * slices + kRopeWaves - 1) / kRopeWaves));
        if (n == 4) hipLaunchKernelGGL((rope_kernel<T, C, 4>), grid, dim3(64 * kRopeWaves), lds, stream, b, units, slices);
        else hipLaunchKernelGGL((rope_kernel<T, C, 1>), grid, dim3(64 * kRopeWaves), lds, stream, b, units, slices);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
    static_assert(kMaxHalf * kRopeWaves * sizeof(float2) <= 65536, "LDS without an attribute");
    const bool wide = rope_vector(a.by) == 8 && a.head_dim % 8 == 0;
    if (a.dtype == 0) return wide ? launch<Fp16, 8>(a, stream) : launch<Fp16, 4>(a, stream);
    return wide ? launch<Bf16, 8>(a, stream) : launch<Bf16, 4>(a, stream);
}

}  // namespace slim
