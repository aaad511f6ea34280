// Pages of 4 bits a value: where a row's codes and scales lie, and the
// conversions (the format: include/slim.h).
#pragma once

#include "attention_device.hpp"

namespace slim {

// Bytes of one page of K or V.
__host__ __device__ __forceinline__ int64_t q4_page_bytes(int kv_heads, int page_shift, int head_dim) {
    return ((int64_t)kv_heads * head_dim << page_shift) * 17 / 32;
}

// Byte offsets in a pool of row r (0 .. page_size - 1) of head h in a page:
// its first code, and its scale of group 0; that of group g is 16 g further on.
struct Q4Row {
    int64_t codes, scales;
    __device__ __forceinline__ Q4Row(int64_t page, int kv_heads, int page_shift, int head_dim, int h, int r) {
        const int64_t base = page * q4_page_bytes(kv_heads, page_shift, head_dim);
        codes = base + ((int64_t)(h << page_shift) + r) * (head_dim / 2);
        scales = base + (((int64_t)kv_heads << page_shift) * (head_dim / 2)) +
                 ((int64_t)(h << page_shift) + (r & ~15)) * (head_dim / 32) + (r & 15);
    }
};

// A scale byte as the conversions take it: the exponent of an fp32.  255 makes NaN.
__device__ __forceinline__ float q4_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Byte i of four.  (The conversions read the exponent's eight bits and no
// others: checked for every code and exponent with other bits set, so one shift does.)
__device__ __forceinline__ float q4_scale_of(uint32_t bytes, int i) {
    return __builtin_bit_cast(float, i < 3 ? bytes << (23 - 8 * i) : bytes >> 1);
}

// The two values of byte I of `codes`, element 0 in the low half.
template <class T, int I>
__device__ __forceinline__ uint32_t q4_pair(uint32_t codes, float scale);
#define SLIM_Q4_PAIR(I)                                                                                              \
    template <>                                                                                                      \
    __device__ __forceinline__ uint32_t q4_pair<Fp16, I>(uint32_t codes, float scale) {                              \
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, I));              \
    }                                                                                                                \
    template <>                                                                                                      \
    __device__ __forceinline__ uint32_t q4_pair<Bf16, I>(uint32_t codes, float scale) {                              \
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));             \
    }
SLIM_Q4_PAIR(0)
SLIM_Q4_PAIR(1)
SLIM_Q4_PAIR(2)
SLIM_Q4_PAIR(3)
#undef SLIM_Q4_PAIR

// The eight values of a dword of codes.
template <class T>
__device__ __forceinline__ u4 q4_values(uint32_t codes, float scale) {
    return u4{q4_pair<T, 0>(codes, scale), q4_pair<T, 1>(codes, scale), q4_pair<T, 2>(codes, scale),
              q4_pair<T, 3>(codes, scale)};
}

// Largest and smallest e + 127 of a type.
template <class T> struct Q4Range;
template <> struct Q4Range<Fp16> { static constexpr int kLow = 127 - 23, kHigh = 127 + 13; };
template <> struct Q4Range<Bf16> { static constexpr int kLow = 127 - 125, kHigh = 127 + 125; };

// Codes of eight elements of a group whose 32 lie in four neighbouring lanes,
// and the group's e + 127 (the same in the four).
template <class T>
__device__ __forceinline__ uint32_t q4_encode(const float (&x)[8], uint32_t& e) {
    // As whole numbers, magnitudes have the order of their values, infinity and then NaN above all.
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __builtin_bit_cast(uint32_t, x[k]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    // m 2^E <= 7 * 2^e: e = E - 2 for m up to 1.75, E - 1 above (the addition carries into the exponent).
    const int fit = (int)((top + 0x1FFFFFu) >> 23) - 2;
    const bool finite = top < 0x7F800000u;
    e = finite ? (uint32_t)min(max(fit, Q4Range<T>::kLow), Q4Range<T>::kHigh) : 255u;
    const float scale = q4_scale(finite ? e : 127u);
    uint32_t codes = 0;
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[0], x[1], scale, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[2], x[3], scale, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[4], x[5], scale, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[6], x[7], scale, 3);
    return finite ? codes : 0u;
}

// Rows of codes as plain_row reads them.
template <int D>
struct Q4Rows {
    struct At { int64_t codes, scales; };
    static __device__ __forceinline__ At at(const AttnArgs& a, int page, int kvh, int r) {
        const Q4Row x(page, a.kv_heads, a.kv.page_shift, D, kvh, r);
        return {x.codes, x.scales};
    }
    static __device__ __forceinline__ At none() { return {0, 0}; }
    static __device__ __forceinline__ At of_lane(At at, int lane) { return {__shfl(at.codes, lane), __shfl(at.scales, lane)}; }
    static __device__ __forceinline__ float value(const AttnArgs&, const uint16_t* pool, At at, int d) {
        const unsigned char* p = reinterpret_cast<const unsigned char*>(pool);
        const uint32_t code = (uint32_t)p[at.codes + d / 2] >> (d & 1) * 4;
        return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, q4_scale(p[at.scales + d / 32 * 16]), 0)[0];
    }
};

}  // namespace slim
