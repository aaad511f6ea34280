// Appending to the paged cache with the rotation of the keys (and of the
// step's queries) on the way, into pages of halves or of 4 bits, and reading
// rows of 4-bit pages back.
//
// A wave takes one token's rows of queries, keys and values, or a part of
// them: it finds the token's sequence and position (starts -> lens -> table), forms the
// position's cosines and sines in its own part of LDS, and turns, codes and
// writes what it loaded before.  Waves do not wait for each other, so a
// token cut over several only costs each of them the chain again.  Bound by HBM
// for prompts (halves: 4 bytes an element; 4 bits: 2.5), by launch and that chain for
// single tokens.
#include "kv_q4.hpp"
#include "rope_device.hpp"

namespace slim {
namespace {

constexpr int kMaxHalf = 128;                 // head_dim is at most 256
constexpr int kManyTokens = 512;              // from here on a lane takes several units

// Where a token's new row goes.
struct Target {
    int seq, pos, page, row;                  // page -1: nowhere
};

__device__ __forceinline__ Target target_of(const PagedKV& kv, int t) {
    Target x;
    x.page = -1;
    x.row = 0;
    x.pos = 0;
    x.seq = __builtin_amdgcn_readfirstlane(find_seq(kv, t));
    if (x.seq < 0) return x;
    x.pos = seq_len(kv, x.seq) - 1;
    if (kv.starts) x.pos += 1 + t - kv.starts[x.seq + 1];
    const int at = x.pos >> kv.page_shift;
    if (x.pos < 0 || at >= kv.width) return x;
    const int page = kv.table[(int64_t)x.seq * kv.width + at];
    if (page >= 0 && page < kv.pages) x.page = page;
    x.row = x.pos & ((1 << kv.page_shift) - 1);
    return x;
}

// The token and slice of this wave, tokens from token0 on; token >= tokens: none.
struct Task {
    int token, slice;
};
__device__ __forceinline__ Task task_of(int token0, int slices) {
    const uint32_t task = blockIdx.x * kRopeWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t token = task / (uint32_t)slices;
    return {token0 + (int)token, (int)(task - token * (uint32_t)slices)};
}

// Units (rope_device.hpp) of one token: those of the queries' heads, the
// keys' and the values'; of the values' units all stay as they are.
template <class T, int C, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_append_rope_kernel(AppendRopeArgs a, int token0, int units,
                                                                         int v_units, int slices) {
    __shared__ float2 lds[kRopeWaves][kMaxHalf];
    const Task task = task_of(token0, slices);
    const int t = task.token;
    if (t >= a.to.tokens) return;
    const int lane = threadIdx.x & 63, D = a.to.head_dim;
    float2* turns = lds[threadIdx.x >> 6];
    const int q_end = a.q_heads * units, k_end = q_end + a.to.kv_heads * units, all = k_end + a.to.kv_heads * v_units;
    const int first = task.slice * (64 * N) + lane;
    const Rotation none = {nullptr, 0, 0, 1.0};
    Vectors<C> v[N];
    Unit<C> u[N];
    int head[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = min(first + 64 * n, all - 1);
        const uint16_t* from;
        if (i < k_end) {
            const int j = i < q_end ? i : i - q_end;
            head[n] = j / units;
            u[n] = unit_of<C>(a.by, D, j - head[n] * units);
            from = i < q_end ? a.q + t * a.sq : a.to.k_new + t * a.to.sk;
        } else {
            head[n] = (i - k_end) / v_units;
            u[n] = unit_of<C>(none, D, i - k_end - head[n] * v_units);
            from = a.to.v_new + t * a.to.sv;
        }
        load_unit(v[n], u[n], from + head[n] * D);
    }
    const Target to = target_of(a.to.kv, t);
    if (to.seq < 0) return;
    turns_to_lds(turns, a.by, to.pos);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + 64 * n;
        if (i >= all) continue;
        turn_unit<T>(v[n], u[n], a.by, turns);
        if (i < q_end) {
            store_unit(v[n], u[n], a.q_out + t * a.sqo + head[n] * D);
        } else if (to.page >= 0) {
            uint16_t* pool = const_cast<uint16_t*>(i < k_end ? a.to.kv.k : a.to.kv.v);
            store_unit(v[n], u[n],
                       pool + ((((int64_t)to.page * a.to.kv_heads + head[n]) << a.to.kv.page_shift) + to.row) * D);
        }
    }
}

// One lane's eight elements of a key or value, and the eight they turn with.
struct Chunk {
    uint32_t own[4], other[2][2];
    int at;                                   // first element in its head
};

// First element of the four that elements at .. at + 3 turn with (halves layout).
__device__ __forceinline__ int partner(const Rotation& by, int at) {
    return at >= 2 * by.half ? at : at < by.half ? at + by.half : at - by.half;
}

// Elements of a chunk, turned in fp64 and rounded to fp32: what a code is
// chosen by must not depend on the order of fp32 operations.
template <class T>
__device__ __forceinline__ void turned_chunk(float (&y)[8], const Chunk& c, const Rotation& by, const double2* turns) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = T::low(c.own[j]);
        x[2 * j + 1] = T::high(c.own[j]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int at = c.at + 4 * q;
        if (at >= 2 * by.half) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[4 * q + j] = x[4 * q + j];
        } else if (by.interleaved) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const double2 r = turns[at / 2 + j];
                const double p = x[4 * q + 2 * j], s = x[4 * q + 2 * j + 1];
                y[4 * q + 2 * j] = (float)(p * r.x - s * r.y);
                y[4 * q + 2 * j + 1] = (float)(s * r.x + p * r.y);
            }
        } else {
            const bool low = at < by.half;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double2 r = turns[(low ? at : at - by.half) + j];
                const double own = x[4 * q + j];
                const double other = (j & 1) ? T::high(c.other[q][j >> 1]) : T::low(c.other[q][j >> 1]);
                y[4 * q + j] = (float)(own * r.x + other * (low ? -r.y : r.y));
            }
        }
    }
}

// The same into pages of 4 bits.  Keys and values go in chunks of eight
// elements a lane, four lanes a group of 32, so that a group's largest
// element is two exchanges away; a chunk's partners are loaded beside it (from the
// cache: the same row).
template <class T, int C, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_append_q4_kernel(AppendRopeArgs a, int token0, int units,
                                                                       int q_slices, int slices) {
    __shared__ double2 lds[kRopeWaves][kMaxHalf];
    const Task task = task_of(token0, slices);
    const int t = task.token;
    if (t >= a.to.tokens) return;
    const int lane = threadIdx.x & 63, D = a.to.head_dim;
    double2* turns = lds[threadIdx.x >> 6];
    if (task.slice < q_slices) {
        const int all = a.q_heads * units, first = task.slice * (64 * N) + lane;
        Vectors<C> v[N];
        Unit<C> u[N];
        int head[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = min(first + 64 * n, all - 1);
            head[n] = i / units;
            u[n] = unit_of<C>(a.by, D, i - head[n] * units);
            load_unit(v[n], u[n], a.q + t * a.sq + head[n] * D);
        }
        const Target to = target_of(a.to.kv, t);
        if (to.seq < 0) return;
        turns_to_lds(turns, a.by, to.pos);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (first + 64 * n >= all) continue;
            turn_unit<T>(v[n], u[n], a.by, turns);
            store_unit(v[n], u[n], a.q_out + t * a.sqo + head[n] * D);
        }
        return;
    }
    const int chunks = D / 8, half_all = a.to.kv_heads * chunks, all = 2 * half_all;       // of keys, then of values
    const int first = (task.slice - q_slices) * (64 * N) + lane;
    Chunk c[N];
    int head[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // (Lanes past the end repeat the last chunk's group in its order: `all` is a multiple of 4.)
        const int i = first + 64 * n < all ? first + 64 * n : all - 4 + (lane & 3);
        const bool key = i < half_all;
        const int j = key ? i : i - half_all;
        head[n] = j / chunks;
        c[n].at = (j - head[n] * chunks) * 8;
        const uint16_t* from = (key ? a.to.k_new + t * a.to.sk : a.to.v_new + t * a.to.sv) + head[n] * D;
        load_words<4>(c[n].own, from + c[n].at);
        if (key && !a.by.interleaved) {
#pragma unroll
            for (int q = 0; q < 2; ++q) load_words<2>(c[n].other[q], from + partner(a.by, c[n].at + 4 * q));
        }
    }
    const Target to = target_of(a.to.kv, t);
    if (to.page < 0) return;
    if ((task.slice - q_slices) * (64 * N) < half_all) turns_to_lds(turns, a.by, to.pos);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + 64 * n;
        const bool key = i < half_all;
        float x[8];
        if (key) {
            turned_chunk<T>(x, c[n], a.by, turns);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = T::low(c[n].own[j]);
                x[2 * j + 1] = T::high(c[n].own[j]);
            }
        }
        uint32_t e;
        const uint32_t codes = q4_encode<T>(x, e);
        if (i >= all) continue;
        const Q4Row at(to.page, a.to.kv_heads, a.to.kv.page_shift, D, head[n], to.row);
        unsigned char* pool = reinterpret_cast<unsigned char*>(const_cast<uint16_t*>(key ? a.to.kv.k : a.to.kv.v));
        *reinterpret_cast<uint32_t*>(pool + at.codes + c[n].at / 2) = codes;
        if ((lane & 3) == 0) pool[at.scales + (c[n].at / 32) * 16] = (unsigned char)e;
    }
}

// Rows of 4-bit pages as halves again.
template <class T, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_read_q4_kernel(AppendArgs a, int token0, int slices) {
    const Task task = task_of(token0, slices);
    const int t = task.token;
    if (t >= a.tokens) return;
    const int lane = threadIdx.x & 63, D = a.head_dim, chunks = D / 8, half_all = a.kv_heads * chunks;
    const Target to = target_of(a.kv, t);
    if (to.seq < 0) return;
    uint32_t codes[N], e[N];
    int head[N], at[N];
    const int first = task.slice * (64 * N) + lane;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = min(first + 64 * n, 2 * half_all - 1);
        const int j = i < half_all ? i : i - half_all;
        head[n] = j / chunks;
        at[n] = (j - head[n] * chunks) * 8;
        const unsigned char* pool = reinterpret_cast<const unsigned char*>(i < half_all ? a.kv.k : a.kv.v);
        const Q4Row row(max(to.page, 0), a.kv_heads, a.kv.page_shift, D, head[n], to.row);
        codes[n] = *reinterpret_cast<const uint32_t*>(pool + row.codes + at[n] / 2);
        e[n] = pool[row.scales + (at[n] / 32) * 16];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = first + 64 * n;
        if (i >= 2 * half_all) continue;
        uint16_t* y = const_cast<uint16_t*>(i < half_all ? a.k_new + t * a.sk : a.v_new + t * a.sv);
        const u4 x = q4_values<T>(codes[n], q4_scale(e[n]));
        *reinterpret_cast<u4*>(y + head[n] * D + at[n]) = to.page >= 0 ? x : u4{0, 0, 0, 0};
    }
}

// Calls launch(first token, grid) for as many tokens at a time as a grid's 2^32 threads hold.
template <class Launch>
hipError_t in_parts(int64_t tokens, int slices, Launch&& launch) {
    const int64_t at_once = (int64_t(1) << 25) / slices;
    for (int64_t t = 0; t < tokens; t += at_once) {
        const int64_t waves = min(at_once, tokens - t) * slices;
        launch((int)t, dim3((unsigned)((waves + kRopeWaves - 1) / kRopeWaves)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

const dim3 kBlock(64 * kRopeWaves);

template <class T, int C, int N>
hipError_t append_rope(const AppendRopeArgs& a, hipStream_t stream) {
    const Rotation none = {nullptr, 0, 0, 1.0};
    const int D = a.to.head_dim, units = units_of(a.by, D, C), v_units = units_of(none, D, C);
    const int all = (a.q_heads + a.to.kv_heads) * units + a.to.kv_heads * v_units;
    const int slices = (all + 64 * N - 1) / (64 * N);
    return in_parts(a.to.tokens, slices, [&](int t, dim3 grid) {
        hipLaunchKernelGGL((kv_append_rope_kernel<T, C, N>), grid, kBlock, 0, stream, a, t, units, v_units, slices);
    });
}

template <class T, int C, int N>
hipError_t append_q4(const AppendRopeArgs& a, hipStream_t stream) {
    const int D = a.to.head_dim, units = units_of(a.by, D, C);
    const int q_slices = (a.q_heads * units + 64 * N - 1) / (64 * N);
    const int slices = q_slices + (a.to.kv_heads * (D / 8) * 2 + 64 * N - 1) / (64 * N);
    return in_parts(a.to.tokens, slices, [&](int t, dim3 grid) {
        hipLaunchKernelGGL((kv_append_q4_kernel<T, C, N>), grid, kBlock, 0, stream, a, t, units, q_slices, slices);
    });
}

template <class T, int N>
hipError_t read_q4(const AppendArgs& a, hipStream_t stream) {
    const int slices = (a.kv_heads * (a.head_dim / 8) * 2 + 64 * N - 1) / (64 * N);
    return in_parts(a.tokens, slices, [&](int t, dim3 grid) {
        hipLaunchKernelGGL((kv_read_q4_kernel<T, N>), grid, kBlock, 0, stream, a, t, slices);
    });
}

// A token's rows are cut over as many waves as they fill with one unit a lane for
// few tokens (latency), four units a lane for many (loads in flight).
template <class T, int C>
hipError_t append_rope_n(const AppendRopeArgs& a, hipStream_t stream) {
    return a.to.tokens >= kManyTokens ? append_rope<T, C, 4>(a, stream) : append_rope<T, C, 1>(a, stream);
}
template <class T, int C>
hipError_t append_q4_n(const AppendRopeArgs& a, hipStream_t stream) {
    return a.to.tokens >= kManyTokens ? append_q4<T, C, 4>(a, stream) : append_q4<T, C, 1>(a, stream);
}
template <class T>
hipError_t read_q4_n(const AppendArgs& a, hipStream_t stream) {
    return a.tokens >= kManyTokens ? read_q4<T, 4>(a, stream) : read_q4<T, 1>(a, stream);
}

}  // namespace

hipError_t launch_kv_append_rope(const AppendRopeArgs& a, hipStream_t stream) {
    const bool wide = rope_vector(a.by) == 8;
    if (a.dtype == 0) return wide ? append_rope_n<Fp16, 8>(a, stream) : append_rope_n<Fp16, 4>(a, stream);
    return wide ? append_rope_n<Bf16, 8>(a, stream) : append_rope_n<Bf16, 4>(a, stream);
}

hipError_t launch_kv_append_q4(const AppendRopeArgs& a, hipStream_t stream) {
    const bool wide = rope_vector(a.by) == 8;
    if (a.dtype == 0) return wide ? append_q4_n<Fp16, 8>(a, stream) : append_q4_n<Fp16, 4>(a, stream);
    return wide ? append_q4_n<Bf16, 8>(a, stream) : append_q4_n<Bf16, 4>(a, stream);
}

hipError_t launch_kv_read_q4(const AppendArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? read_q4_n<Fp16>(a, stream) : read_q4_n<Bf16>(a, stream);
}

}  // namespace slim
