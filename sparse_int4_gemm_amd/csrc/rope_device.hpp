// Rotary positions on the device: a wave turns rows of one token.
#pragma once

#include "attention_device.hpp"

namespace slim {

constexpr int kRopeWaves = 4;                 // waves of a workgroup; each has its own tokens, none waits for another

// Rounds of waves (32 on each of 256 CUs) that `units` of each token make with one a lane.
inline float rounds(int64_t tokens, int64_t units) { return (float)(tokens * ((units + 63) / 64)) / (256 * 32); }

// (cos, sin) * magnitude of pair i at position p.  The angle is taken in turns,
// in fp64: 1 / (2 pi) and two products, so off by at most 3 * 2^-53 of itself.
__device__ __forceinline__ double2 turn_of(const Rotation& by, int p, int i) {
    double t = (double)p * (by.freqs[i] * 0.15915494309189533577);       // 1 / (2 pi)
    t -= rint(t);
    double s, c;
    sincospi(2.0 * t, &s, &c);
    return make_double2(c * by.magnitude, s * by.magnitude);
}

// Where pair i lies in LDS: lanes work on fours of pairs, so those of the same
// place in their fours lie side by side (in the order of the pairs, sixteen
// lanes' would share a bank).
__device__ __forceinline__ int turn_place(const Rotation& by, int i) { return (i & 3) * (by.half >> 2) + (i >> 2); }

// All pairs of position p to the wave's own part of LDS.
template <class Turn>
__device__ __forceinline__ void turns_to_lds(Turn* to, const Rotation& by, int p) {
    for (int i = threadIdx.x & 63; i < by.half; i += 64) {
        const double2 t = turn_of(by, p, i);
        Turn& at = to[turn_place(by, i)];
        at.x = t.x;
        at.y = t.y;
    }
    // The wave's own LDS accesses are served in order; only the compiler must keep it.
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// A unit of work on one head: two vectors of C elements, C = 8 (or 4 where the
// halves of a head do not begin at whole vectors of 8), so that every pair
// lies in one unit.  Units below half / C turn C pairs, those behind them hold
// 2 C elements that stay as they are.
template <int C>
struct Unit {
    int at[2];                                // first element of both vectors
    int pair;                                 // first pair, or -1: not turned
    int last;                                 // vectors there are (an odd rest has one)
};

template <int C>
__device__ __forceinline__ Unit<C> unit_of(const Rotation& by, int head_dim, int u) {
    const int turned = by.half / C;
    Unit<C> x;
    x.last = 2;
    if (u < turned) {
        x.pair = u * C;
        x.at[0] = by.interleaved ? 2 * u * C : u * C;
        x.at[1] = by.interleaved ? x.at[0] + C : by.half + u * C;
    } else {
        x.pair = -1;
        x.at[0] = 2 * by.half + (u - turned) * 2 * C;
        x.at[1] = x.at[0] + C;
        if (x.at[1] >= head_dim) { x.last = 1; x.at[1] = x.at[0]; }
    }
    return x;
}

// Units of a head.
inline int units_of(const Rotation& by, int head_dim, int c) {
    return by.half / c + (head_dim - 2 * by.half + 2 * c - 1) / (2 * c);
}

template <int C>
struct Vectors {
    uint32_t a[2][C / 2];
};

// kOnce: rows that nobody reads again.
template <bool kOnce, int C>
__device__ __forceinline__ void load_unit(Vectors<C>& v, const Unit<C>& u, const uint16_t* head) {
    using Words = std::conditional_t<C == 8, u4, u2>;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Words* p = reinterpret_cast<const Words*>(head + u.at[i]);
        const Words x = kOnce ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
        for (int j = 0; j < C / 2; ++j) v.a[i][j] = x[j];
    }
}

template <int C>
__device__ __forceinline__ void store_unit(const Vectors<C>& v, const Unit<C>& u, uint16_t* head) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i >= u.last) continue;
        if constexpr (C == 8)
            *reinterpret_cast<u4*>(head + u.at[i]) = u4{v.a[i][0], v.a[i][1], v.a[i][2], v.a[i][3]};
        else
            *reinterpret_cast<u2*>(head + u.at[i]) = u2{v.a[i][0], v.a[i][1]};
    }
}

// Turns a unit's pairs in fp32; each result is rounded once, to the type.
template <class T, int C, class Turn>
__device__ __forceinline__ void turn_unit(Vectors<C>& v, const Unit<C>& u, const Rotation& by, const Turn* turns) {
    if (u.pair < 0) return;
    float x[2][C];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < C / 2; ++j) {
            x[i][2 * j] = T::low(v.a[i][j]);
            x[i][2 * j + 1] = T::high(v.a[i][j]);
        }
    float c[C], s[C];
    const Turn* fours = turns + (u.pair >> 2);
    const int step = by.half >> 2;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const Turn t = fours[(k & 3) * step + (k >> 2)];          // turn_place of pair + k
        c[k] = (float)t.x;
        s[k] = (float)t.y;
    }
    auto turn = [](float& a, float& b, float cos, float sin) {
        const float y = a * cos - b * sin;
        b = b * cos + a * sin;
        a = y;
    };
    if (by.interleaved) {
#pragma unroll
        for (int k = 0; k < C; ++k) turn(x[2 * k / C][2 * k % C], x[2 * k / C][2 * k % C + 1], c[k], s[k]);
    } else {
#pragma unroll
        for (int k = 0; k < C; ++k) turn(x[0][k], x[1][k], c[k], s[k]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < C / 2; ++j) v.a[i][j] = T::pack(x[i][2 * j], x[i][2 * j + 1]);
}

// The vector length that a rotation's halves allow.
inline int rope_vector(const Rotation& by) { return by.half % 8 ? 4 : 8; }

}  // namespace slim
