// What the attention kernels share: the half types' operations, which keys a
// query sees, the partial results of a split key axis, and the rule of the split.
#pragma once

#include "attention_util.hpp"
#include "mfma_util.hpp"

namespace slim {

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f16v __attribute__((ext_vector_type(16)));

// Operands travel as dwords of two halves; `pack` rounds to nearest even.
// kTop: log2 of the largest softmax weight that enters a product.  fp16 ends at
// 2^16 and, downwards, at 2^-24: with weights of 1 at most, those 2^-25 of the
// row's largest and below would be lost to the output, and not to the sum (a first key 25.5
// bits above 2^19 others: outputs 0.5% low), so they are taken as high as they
// go.  bf16 has the range of fp32.
struct Fp16 {
    static constexpr float kTop = 15.0f;
    static __device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f16v mfma32(u4 a, u4 b, f16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), h2));
    }
    static __device__ __forceinline__ float low(uint32_t x) { return (float)__builtin_bit_cast(h2, x)[0]; }
    static __device__ __forceinline__ float high(uint32_t x) { return (float)__builtin_bit_cast(h2, x)[1]; }
};
struct Bf16 {
    static constexpr float kTop = 0.0f;
    static __device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f16v mfma32(u4 a, u4 b, f16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x, y}), bf2));
    }
    static __device__ __forceinline__ float low(uint32_t x) { return __builtin_bit_cast(float, x << 16); }
    static __device__ __forceinline__ float high(uint32_t x) { return __builtin_bit_cast(float, x & 0xFFFF0000u); }
};

// 2^x by the hardware instruction (one ulp; results below 2^-126 are zero,
// which a weight relative to the row's maximum of 1 may lose).
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// N dwords from p; p is aligned to the largest power of two that divides N dwords.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&to)[N], const uint16_t* p) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u4 x = reinterpret_cast<const u4*>(w)[i];
            to[4 * i] = x[0]; to[4 * i + 1] = x[1]; to[4 * i + 2] = x[2]; to[4 * i + 3] = x[3];
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const u2 x = reinterpret_cast<const u2*>(w)[i];
            to[2 * i] = x[0]; to[2 * i + 1] = x[1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = w[i];
    }
}

// The keys that positions p0 .. p1 of one sequence see, as a run of tiles:
// those that hold sinks, then those from the first window's start on.
struct Span {
    int end;              // keys below min(p + 1, capacity of the table); 0 or less: nothing is seen
    int start;            // first key of the (first position's) window
    int sinks;

    __device__ __forceinline__ int sink_tiles(int t) const { return min((min(sinks, end) + t - 1) / t, start / t); }
    __device__ __forceinline__ int tiles(int t) const {
        return end <= 0 ? 0 : sink_tiles(t) + max(0, (end + t - 1) / t - start / t);
    }
    __device__ __forceinline__ int base(int i, int t) const {
        const int s = sink_tiles(t);
        return (i < s ? i : i - s + start / t) * t;
    }
    __device__ __forceinline__ bool seen(int j) const { return j < end && (j >= start || j < sinks); }
    __device__ __forceinline__ bool all_seen(int base, int t) const {
        return base + t <= end && (base >= start || base + t <= sinks);
    }
};

// Page of a sequence's key `key` (the same in all lanes), -1 if it has none
// (from `keys` on, or an entry out of range), through the scalar cache.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ int page_of(const AttnArgs& a, int b, int key, int keys) {
    key = __builtin_amdgcn_readfirstlane(key);
    if (key >= keys) return -1;
    const ScalarInts table = (ScalarInts)(uintptr_t)(a.kv.table + (int64_t)b * a.kv.width);
    const int page = table[key >> a.kv.page_shift];
    return page >= 0 && page < a.kv.pages ? page : -1;
}

// Of a single position p.
__device__ __forceinline__ Span key_span(const AttnArgs& a, int p) {
    // (32-bit: a 64-bit comparison goes to the vector unit, and what follows
    // from it with it.  The capacity is at most 2^30.)
    Span s;
    s.end = min(p + 1, a.kv.width << a.kv.page_shift);
    s.start = a.window ? max(0, p - a.window + 1) : 0;
    s.sinks = a.window ? a.sinks : 0;
    return s;
}

__device__ __forceinline__ float half_value(const AttnArgs& a, uint16_t x) {
    return a.dtype == 0 ? (float)__builtin_bit_cast(_Float16, x) : __builtin_bit_cast(float, (uint32_t)x << 16);
}

// One row over tiles [first, last) of `tiles` (KEYS keys each, at most 64) by
// the whole wave, straight from the formula: lane j scores key j of each tile, then owns
// the output elements lane + 64 i.  For rows that an infinity or NaN has
// reached in the matrix products, where it also meets weights of 0 and of
// either sign: here only keys that the row sees, and each with its weight.  A key
// at a time: some hundred times slower than the products.
template <int D, int KEYS>
__device__ void plain_row(const AttnArgs& a, const Span& tiles, int first, int last, const Span& row_span,
                          const int32_t* table, int kvh, const uint16_t* q, float (&o)[4], float& m, float& l) {
    const int lane = threadIdx.x & 63;
    const float scale = a.scale * 1.4426950408889634f;
    m = -INFINITY;
    l = 0.0f;
    for (int i = 0; i < 4; ++i) o[i] = 0.0f;
    for (int t = first; t < last; ++t) {
        const int j = tiles.base(t, KEYS) + lane;
        bool seen = lane < KEYS && row_span.seen(j);
        int page = -1;
        if (seen) page = table[j >> a.kv.page_shift];
        seen = seen && page >= 0 && page < a.kv.pages;
        const int64_t at = seen ? ((((int64_t)page * a.kv_heads + kvh) << a.kv.page_shift) +
                                   (j & ((1 << a.kv.page_shift) - 1))) * D : 0;
        float s = -INFINITY;
        if (seen) {
            s = 0.0f;
            for (int d = 0; d < D; ++d) s = fmaf(half_value(a, q[d]), half_value(a, a.kv.k[at + d]), s);
            s *= scale;
        }
        float top = s;
        for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2_fast(m - ms), w = seen ? exp2_fast(s - ms) : 0.0f;
        m = mn;
        l *= f;
        for (int i = 0; i < 4; ++i) o[i] *= f;
        for (uint64_t left = __ballot(seen); left; left &= left - 1) {
            const int k = __builtin_ctzll(left);
            const float wk = __shfl(w, k);
            const int64_t r = __shfl(at, k);
            l += wk;
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < D) o[i] = fmaf(wk, half_value(a, a.kv.v[r + lane + 64 * i]), o[i]);
        }
    }
}

// Writes four elements of an output row, and lse with the first of them.
// sum == 0: no key was seen, or none with a score above -inf.
template <class T>
__device__ __forceinline__ void store_row4(const AttnArgs& a, int64_t token, int head, int D, int d, f4 acc, float top,
                                           float sum) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (sum == 0.0f) acc = f4{0, 0, 0, 0};
    const u2 y = {T::pack(acc[0] * inv, acc[1] * inv), T::pack(acc[2] * inv, acc[3] * inv)};
    *reinterpret_cast<u2*>(a.o + token * a.so + (int64_t)head * D + d) = y;
    if (a.lse && d == 0)
        a.lse[token * a.q_heads + head] = sum == 0.0f ? -INFINITY : top * 0.6931471805599453f + logf(sum);
}

// Partial results of rows whose keys are split over workgroups: for each row
// (token * q_heads + head) and split the unscaled fp32 output, its maximum (in
// units of log2) and sum.  Every split of a sequence's row is marked, also one without
// keys (sum 0, no output stored), so attention_join_kernel needs no knowledge of
// how the row was cut; a row that needed no join is marked kWhole in its split 0.
constexpr float kWhole = -1.0f;

struct Partials {
    float* o;             // [rows][splits][D]
    float* ml;            // [rows][splits][2]
    int D, splits;
    __host__ __device__ Partials(const AttnArgs& a, int D_, int splits_) : D(D_), splits(splits_) {
        o = reinterpret_cast<float*>(a.ws);
        ml = o + (int64_t)a.tokens * a.q_heads * splits * D;
    }
    __device__ __forceinline__ void mark(int64_t row, int split, float top, float sum) const {
        float* at = ml + 2 * (row * splits + split);
        at[0] = top;
        at[1] = sum;
    }
    __device__ __forceinline__ void put4(int64_t row, int split, int d, f4 acc) const {
        *reinterpret_cast<f4*>(o + (row * splits + split) * D + d) = acc;
    }
};

// Writes what plain_row left in its wave's lanes: the output row, or where the
// keys are cut over workgroups its partial result.
template <class T, int D>
__device__ __forceinline__ void store_plain_row(const AttnArgs& a, const Partials& parts, bool cut, int64_t token, int head,
                                                int split, const float (&o)[4], float m, float l) {
    const int lane = threadIdx.x & 63;
    const int64_t row = token * a.q_heads + head;
    for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d >= D) continue;
        if (cut) parts.o[(row * parts.splits + split) * D + d] = o[i];
        else a.o[token * a.so + (int64_t)head * D + d] = (uint16_t)T::pack(l == 0.0f ? 0.0f : o[i] / l, 0.0f);
    }
    if (lane != 0) return;
    if (cut) parts.mark(row, split, m, l);
    else if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

}  // namespace slim
