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
// single tokens.  Of 32 heads of 128, with their queries: 64 tokens 3.4 us into halves
// and 4.6 into 4 bits, 8192 tokens 79 us (5.1 TB/s) and 62 (4.9 TB/s).
#include "kv_q4.hpp"
#include "rope_device.hpp"

namespace slim {
namespace {

constexpr int kMaxHalf = 128;                 // head_dim is at most 256

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

// The token and slice of this wave, tokens from token0 on; token >= tokens (the call's, or its part's end): none.
// kRuns: an XCD (a workgroup's is its index mod 8) takes runs of 32 workgroups, where
// there are eight such runs left.  Pages of 4 bits need it, as 16 tokens share 16
// bytes of scales, and two a line of codes, that each XCD's L2 would read and write for
// itself (8763 tokens of 32 heads appended and read back: 126 MB written and 70 read
// without, 111 and 40 with, 106 -> 100 us; runs of 8: 102, of 128: 111; pages of halves, 8192 tokens: 78 and 80).
struct Task {
    int token, slice;
};
template <bool kRuns>
__device__ __forceinline__ Task task_of(int token0, int slices) {
    uint32_t block = blockIdx.x;
    if (kRuns && (block | 255) < gridDim.x) block = (block & ~255u) | (block & 7) * 32 | (block >> 3 & 31);
    const uint32_t task = block * kRopeWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t token = task / (uint32_t)slices;
    return {token0 + (int)token, (int)(task - token * (uint32_t)slices)};
}

// Units (rope_device.hpp) of one token: those of the queries' heads, the
// keys' and the values'; of the values' units all stay as they are.  The
// rows' loads are marked as read once, so that they leave the caches to what is written: 8763
// tokens of 32 heads on 8 alone 46.0 -> 43.4 us, behind the copies that
// make the rows 90 -> 79 together, with the attention after them 240 -> 238.
template <class T, int C, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_append_rope_kernel(AppendRopeArgs a, int token0, int units,
                                                                         int v_units, int slices) {
    __shared__ float2 lds[kRopeWaves][kMaxHalf];
    const Task task = task_of<false>(token0, slices);
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
        load_unit<true>(v[n], u[n], from + head[n] * D);
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

// Eight elements of a head, `own`, and those that they turn with, turned in fp64
// and rounded to fp32: what a code is chosen by must not depend on the order
// of fp32 operations.  first: the first element's place in its head; turns: of its fours.
template <class T>
__device__ __forceinline__ void turned_chunk(float (&y)[8], const uint32_t (&own)[4], const uint32_t (&other)[4], int first,
                                             const Rotation& by, const double2* turns) {
    const int step = by.half >> 2;                // from a pair to the next one in LDS (turn_place)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int at = first + 4 * q;
        float x[4], z[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[2 * j] = T::low(own[2 * q + j]);
            x[2 * j + 1] = T::high(own[2 * q + j]);
            z[2 * j] = T::low(other[2 * q + j]);
            z[2 * j + 1] = T::high(other[2 * q + j]);
        }
        if (at >= 2 * by.half) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[4 * q + j] = x[j];
        } else if (by.interleaved) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const double2 r = turns[turn_place(by, at / 2 + j)];
                const double p = x[2 * j], s = x[2 * j + 1];
                y[4 * q + 2 * j] = (float)(p * r.x - s * r.y);
                y[4 * q + 2 * j + 1] = (float)(s * r.x + p * r.y);
            }
        } else {
            const bool low = at < by.half;
            const double2* four = turns + ((low ? at : at - by.half) >> 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const double2 r = four[j * step];
                y[4 * q + j] = (float)((double)x[j] * r.x + (double)z[j] * (low ? -r.y : r.y));
            }
        }
    }
}

// The same into pages of 4 bits.  Keys and values go in chunks of eight
// elements a lane, whole heads side by side: four lanes are a group of 32, so that
// its largest element is two exchanges away, and the elements that a chunk
// turns with come from other lanes.  A token's work is a row of batches: of
// its queries (N / 2 units a lane), its keys, its values (N chunks a lane).  A wave
// takes `per` of them, the next one's loads in flight while it works on one,
// so that a prompt's tokens pay the chain and the cosines once or twice.
template <class T, int C, int D, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_append_q4_kernel(AppendRopeArgs a, int token0, Divisor units,
                                                                       int q_batches, int kv_batches, int per, int slices) {
    __shared__ double2 lds[kRopeWaves][kMaxHalf];
    const Task task = task_of<true>(token0, slices);
    const int t = task.token;
    if (t >= a.to.tokens) return;
    constexpr int kChunks = D / 8, kHeads = 64 / kChunks;           // of a head; heads of the wave's lanes
    const int lane = threadIdx.x & 63, q_all = a.q_heads * (int)units.d;
    const int my_head = min(lane / kChunks, kHeads - 1), at = lane % kChunks * 8;
    double2* turns = lds[threadIdx.x >> 6];
    const int first = task.slice * per, last = min(first + per, q_batches + 2 * kv_batches);

    struct Batch { uint32_t w[N][4]; };
    auto unit_at = [&](int i, int& head) {
        head = units.quotient((uint32_t)i);
        return unit_of<C>(a.by, D, i - head * (int)units.d);
    };
    auto load = [&](Batch& x, int b) {
        if (b < q_batches) {
            const uint16_t* q = a.q + t * a.sq;
#pragma unroll
            for (int n = 0; n < N / 2; ++n) {
                int head;
                const Unit<C> u = unit_at(min((b * (N / 2) + n) * 64 + lane, q_all - 1), head);
                Vectors<C> y;
                load_unit<true>(y, u, q + head * D);
#pragma unroll
                for (int j = 0; j < C / 2; ++j) {
                    x.w[2 * n][j] = y.a[0][j];
                    x.w[2 * n + 1][j] = y.a[1][j];
                }
            }
            return;
        }
        const bool key = b < q_batches + kv_batches;
        const uint16_t* row = key ? a.to.k_new + t * a.to.sk : a.to.v_new + t * a.to.sv;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int head = ((b - q_batches - (key ? 0 : kv_batches)) * N + n) * kHeads + my_head;
            // (Nobody reads these rows again.)
            const u4 own = __builtin_nontemporal_load(reinterpret_cast<const u4*>(row + (min(head, a.to.kv_heads - 1) * D + at)));
#pragma unroll
            for (int j = 0; j < 4; ++j) x.w[n][j] = own[j];
        }
    };
    Batch x, y;
    load(x, first);
    const Target to = target_of(a.to.kv, t);
    if (to.seq < 0) return;
    if (first < q_batches + kv_batches) turns_to_lds(turns, a.by, to.pos);

    // The lane that holds what this one's first four turn with, and whether its fours are the other way
    // round (halves that begin in the middle of a chunk; then of no other lane than the first four's).
    const bool crossed = (a.by.half & 7) != 0;
    auto lane_of = [&](int four) {
        const int f = at + 4 * four, p = f >= 2 * a.by.half ? f : f < a.by.half ? f + a.by.half : f - a.by.half;
        return 4 * (lane - at / 8 + p / 8);
    };
    const int from[2] = {lane_of(0), lane_of(1)};

    auto work = [&](const Batch& x, int b) {
        if (b < q_batches) {
#pragma unroll
            for (int n = 0; n < N / 2; ++n) {
                const int i = (b * (N / 2) + n) * 64 + lane;
                if (i >= q_all) continue;
                int head;
                const Unit<C> u = unit_at(i, head);
                Vectors<C> y;
#pragma unroll
                for (int j = 0; j < C / 2; ++j) {
                    y.a[0][j] = x.w[2 * n][j];
                    y.a[1][j] = x.w[2 * n + 1][j];
                }
                turn_unit<T>(y, u, a.by, turns);
                store_unit(y, u, a.q_out + t * a.sqo + head * D);
            }
            return;
        }
        if (to.page < 0) return;
        const bool key = b < q_batches + kv_batches;
        unsigned char* pool = reinterpret_cast<unsigned char*>(const_cast<uint16_t*>(key ? a.to.kv.k : a.to.kv.v));
        const Q4Row row(to.page, a.to.kv_heads, a.to.kv.page_shift, D, 0, to.row);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float z[8];
            if (key) {
                uint32_t other[4] = {0, 0, 0, 0};
                if (a.by.half && !a.by.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t word = crossed ? x.w[n][j ^ 2] : x.w[n][j];
                        other[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(from[j >> 1], (int)word);
                    }
                }
                turned_chunk<T>(z, x.w[n], other, at, a.by, turns);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[2 * j] = T::low(x.w[n][j]);
                    z[2 * j + 1] = T::high(x.w[n][j]);
                }
            }
            uint32_t e;
            const uint32_t codes = q4_encode<T>(z, e);
            const int head = ((b - q_batches - (key ? 0 : kv_batches)) * N + n) * kHeads + my_head;
            if (lane >= kHeads * kChunks || head >= a.to.kv_heads) continue;
            const uint32_t of_head = (uint32_t)head << a.to.kv.page_shift;        // rows before this head's
            *reinterpret_cast<uint32_t*>(pool + row.codes + (of_head * (D / 2) + at / 2)) = codes;
            if ((lane & 3) == 0) pool[row.scales + (of_head * (D / 32) + at / 32 * 16)] = (unsigned char)e;
        }
    };
    for (int b = first;;) {
        if (b + 1 < last) load(y, b + 1);
        work(x, b);
        if (++b >= last) break;
        if (b + 1 < last) load(x, b + 1);
        work(y, b);
        if (++b >= last) break;
    }
}

// Rows of 4-bit pages as halves again.  Bound by HBM: 8192 tokens of 32 heads of
// 128, 134 MB written and 36 read, 27 us (6.3 TB/s).  The stores pass the caches by: with
// those that fill them 8763 tokens took 39 us instead of 30 (and what reads the rows next comes from elsewhere: a copy of the
// cache, not the attention).  The appends' stores stay in the caches: past them
// the same 8763 tokens' append alone takes 42.5 us instead of 45.8, with the
// attention that follows 205.5 instead of 199.7.
template <class T, int N>
__global__ __launch_bounds__(64 * kRopeWaves) void kv_read_q4_kernel(AppendArgs a, int token0, int slices) {
    const Task task = task_of<true>(token0, slices);
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
        u4* at_y = reinterpret_cast<u4*>(y + head[n] * D + at[n]);
        const u4 z = to.page >= 0 ? x : u4{0, 0, 0, 0};
        if constexpr (N > 1) __builtin_nontemporal_store(z, at_y);
        else *at_y = z;
    }
}

// Calls launch(arguments, first token, grid) for as many tokens at a time as a grid's
// 2^32 threads hold; the arguments' `tokens` ends at the part's last one, so that what
// a part's last workgroup has over does nothing.
AppendArgs& of_tokens(AppendArgs& a) { return a; }
AppendArgs& of_tokens(AppendRopeArgs& a) { return a.to; }
template <class Args, class Launch>
hipError_t in_parts(Args a, int slices, Launch&& launch) {
    const int64_t at_once = (int64_t(1) << 25) / slices, tokens = of_tokens(a).tokens;
    for (int64_t t = 0; t < tokens; t += at_once) {
        const int64_t end = min(t + at_once, tokens);
        of_tokens(a).tokens = (int32_t)end;
        launch(a, (int)t, dim3((unsigned)(((end - t) * slices + kRopeWaves - 1) / kRopeWaves)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

const dim3 kBlock(64 * kRopeWaves);

template <class T, int C, int N>
hipError_t append_rope(const AppendRopeArgs& a, int units, int v_units, int all, hipStream_t stream) {
    const int slices = (all + 64 * N - 1) / (64 * N);
    return in_parts(a, slices, [&](const AppendRopeArgs& part, int t, dim3 grid) {
        hipLaunchKernelGGL((kv_append_rope_kernel<T, C, N>), grid, kBlock, 0, stream, part, t, units, v_units, slices);
    });
}

// Batches of a token, N as the kernel's.
template <int C, int D, int N>
struct Batches {
    int units, of_q, of_kv;
    explicit Batches(const AppendRopeArgs& a) {
        constexpr int kHeads = 64 / (D / 8) * N;                        // of a batch of keys or values
        units = units_of(a.by, D, C);
        of_q = (a.q_heads * units + 32 * N - 1) / (32 * N);
        of_kv = (a.to.kv_heads + kHeads - 1) / kHeads;
    }
    int all() const { return of_q + 2 * of_kv; }
};

// per: batches a wave takes.
template <class T, int C, int D, int N>
hipError_t append_q4(const AppendRopeArgs& a, int per, hipStream_t stream) {
    const Batches<C, D, N> n(a);
    const int slices = (n.all() + per - 1) / per;
    per = (n.all() + slices - 1) / slices;                              // as even as they come
    return in_parts(a, slices, [&](const AppendRopeArgs& part, int t, dim3 grid) {
        hipLaunchKernelGGL((kv_append_q4_kernel<T, C, D, N>), grid, kBlock, 0, stream, part, t, Divisor(n.units), n.of_q,
                           n.of_kv, per, slices);
    });
}

template <class T, int N>
hipError_t read_q4(const AppendArgs& a, int all, hipStream_t stream) {
    const int slices = (all + 64 * N - 1) / (64 * N);
    return in_parts(a, slices, [&](const AppendArgs& part, int t, dim3 grid) {
        hipLaunchKernelGGL((kv_read_q4_kernel<T, N>), grid, kBlock, 0, stream, part, t, slices);
    });
}

// How much a lane takes (32 heads of 128): one unit for few tokens, so that
// what a token needs is spread over as many waves as can be, more where
// the waves fill the processor anyway.  Halves: 256 tokens 4.6 us with one unit and 5.1
// with two, 512 7.8 and 7.2, 4096 43.5 and 43.3 (four: 44.8).  4 bits: 512 tokens (0.75 of a
// round of waves) 10.0 us with a batch of two and 11.0 with five of four, 1024
// 15.4 and 14.0, 4096 46.3 and 34.6.  Reading back: 256 tokens 4.0 us with one and
// 4.3 with eight, 512 5.5 and 4.5, 4096 24.1 and 16.6 (four: 18.9, sixteen: 16.9).
// (4 bits all without runs, see Task.)
template <class T, int C>
hipError_t append_rope_n(const AppendRopeArgs& a, hipStream_t stream) {
    const Rotation none = {nullptr, 0, 0, 1.0};
    const int D = a.to.head_dim, units = units_of(a.by, D, C), v_units = units_of(none, D, C);
    const int all = (a.q_heads + a.to.kv_heads) * units + a.to.kv_heads * v_units;
    return rounds(a.to.tokens, all) > 0.5f ? append_rope<T, C, 2>(a, units, v_units, all, stream)
                                           : append_rope<T, C, 1>(a, units, v_units, all, stream);
}
template <class T, int C, int D>
hipError_t append_q4_n(const AppendRopeArgs& a, hipStream_t stream) {
    return rounds(a.to.tokens, 64 * Batches<C, D, 2>(a).all()) > 1.0f ? append_q4<T, C, D, 4>(a, 5, stream)
                                                                      : append_q4<T, C, D, 2>(a, 1, stream);
}
template <class T, int C>
hipError_t append_q4_dim(const AppendRopeArgs& a, hipStream_t stream) {
    switch (a.to.head_dim) {
        case 64: return append_q4_n<T, C, 64>(a, stream);
        case 96: return append_q4_n<T, C, 96>(a, stream);
        case 128: return append_q4_n<T, C, 128>(a, stream);
        default: return append_q4_n<T, C, 256>(a, stream);
    }
}
template <class T>
hipError_t read_q4_n(const AppendArgs& a, hipStream_t stream) {
    const int all = a.kv_heads * (a.head_dim / 8) * 2;
    return rounds(a.tokens, all) > 0.5f ? read_q4<T, 8>(a, all, stream) : read_q4<T, 1>(a, all, stream);
}

}  // namespace

hipError_t launch_kv_append_rope(const AppendRopeArgs& a, hipStream_t stream) {
    const bool wide = rope_vector(a.by) == 8;
    if (a.dtype == 0) return wide ? append_rope_n<Fp16, 8>(a, stream) : append_rope_n<Fp16, 4>(a, stream);
    return wide ? append_rope_n<Bf16, 8>(a, stream) : append_rope_n<Bf16, 4>(a, stream);
}

// (Vectors of 4, for halves of a head that begin in the middle of a chunk, keep 20 bytes a lane in scratch
// memory: 8192 tokens of 32 heads on 8 of 96 take 44.0 us with rot_dim 24 and 37.3 with 32.)
hipError_t launch_kv_append_q4(const AppendRopeArgs& a, hipStream_t stream) {
    const bool wide = rope_vector(a.by) == 8;
    if (a.dtype == 0) return wide ? append_q4_dim<Fp16, 8>(a, stream) : append_q4_dim<Fp16, 4>(a, stream);
    return wide ? append_q4_dim<Bf16, 8>(a, stream) : append_q4_dim<Bf16, 4>(a, stream);
}

hipError_t launch_kv_read_q4(const AppendArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? read_q4_n<Fp16>(a, stream) : read_q4_n<Bf16>(a, stream);
}

}  // namespace slim
