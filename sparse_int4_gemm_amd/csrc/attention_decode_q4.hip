// slim_attention_decode_q4: attention of one new token per sequence, or of a
// few, over pages of 4 bits a value (attention_decode.hip has the mathematics;
// kv_q4.hpp the format).
//
//   s_j = scale q . k_j,  O = sum_j 2^(c s_j - m) v_j / l.
//
// Each wave streams tiles of 32 keys into registers, codes as they lie in the
// pages, a tile ahead of the one it computes on, and turns them into halves on
// the way into the matrix products: one instruction for every two values, with
// their scale (4.5 cycles a wave and pair, as a byte permute).
//  - Keys: lane (c, g) = (lane % 16, lane / 16) holds a quarter of key c's
//    elements, [D/4 g, D/4 (g + 1)), 16 bytes at head size 128, and eight of them
//    are its slots of one 16 x 16 x 32 product; queries lie the same way.
//  - Values: lane (c, g) holds D/16 elements of the four keys 4 g + i of each half
//    tile, whose weights it has already; two keys' elements are paired by a
//    byte permute as in attention_decode.hip.
//  - A half tile's scales are 16 bytes for each group of 32 elements: a byte a
//    lane for the keys, the four keys' dword for the values.
// A value's scale goes into its own conversion, so nothing is scaled after the
// products; weights enter them in two halves, as in attention_decode.hip.
//
// Bound by HBM in large batches: 64 sequences of 1 to 4096 tokens, 32 heads of
// 128, 105 us, 5.4 TB/s (a plain read of chunks of 4 KB in random order, as a page's head
// holds of them, reaches 5.75; in order 6.2).  One of 131071, 32 heads on 8: 30 us and the join's 5, 4.8 TB/s;
// 32 windows of 4100, 8 heads of 64, 18 to 20 us.  There a call's beginning and
// end are some 6 us.  Two tiles a wave are on their way; three (at head size 128
// more registers than there are) or four through LDS did not help (windows: 20.9
// and 20.9 us), and reading the codes alone, without any work on them, takes 87% of the time.
#include "kv_q4.hpp"

namespace slim {
namespace {

constexpr int kTile = 32;            // keys of one wave's step
constexpr float kLazy = 8.0f;        // a weight may pass 2^kUp by 2^kLazy before the maximum is raised

struct Place {
    int base, page[2];               // first key, pages of the 16-key halves (-1: none)
};

// Groups of 32 that a lane's elements of a key (D/4 from D/4 g on) lie in:
// the first, and where D/4 is no part of 32 (head sizes 96, 256) a second.
template <int D>
struct KeyGroups {
    static constexpr int kTwo = D == 96 || D == 256;
    static __device__ __forceinline__ uint32_t first(uint32_t g) { return D / 4 * g / 32; }
    static __device__ __forceinline__ uint32_t last(uint32_t g) { return (D / 4 * (g + 1) - 1) / 32; }
    // Whether chunk i of eight elements lies in the last.
    static __device__ __forceinline__ bool in_last(uint32_t g, uint32_t i) { return (D / 4 * g + 8 * i) / 32 != first(g); }
};
// The same of its elements of a value (D/16 from D/16 c on).
template <int D>
struct ValueGroups {
    static constexpr int kTwo = D == 96;
    static __device__ __forceinline__ uint32_t first(uint32_t c) { return D / 16 * c / 32; }
    static __device__ __forceinline__ uint32_t last(uint32_t c) { return (D / 16 * (c + 1) - 1) / 32; }
    static __device__ __forceinline__ bool in_last(uint32_t c, uint32_t e) { return (D / 16 * c + e) / 32 != first(c); }
};

// The registers of one tile.
template <int D>
struct Tile {
    static constexpr int kV = D == 256 ? 2 : 1;          // dwords that hold D/32 bytes
    uint32_t k[2][D / 32];
    uint32_t v[2][4][kV];
    uint32_t ks[2][2], vs[2][2];             // scales: a byte (first, last group); four keys' bytes
    Place at;
};

// (A uniform base and a lane's 32-bit offset for each load, so that the vector unit adds no addresses.)
template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& x, const AttnArgs& a, int kvh, const Place& at) {
    const uint32_t lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    x.at = at;
    const unsigned char *kp = reinterpret_cast<const unsigned char*>(a.kv.k), *vp = reinterpret_cast<const unsigned char*>(a.kv.v);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const Q4Row row(max(at.page[t], 0), a.kv_heads, a.kv.page_shift, D, kvh,
                        (at.base + 16 * t) & ((1 << a.kv.page_shift) - 1));
        const unsigned char *kc = kp + row.codes, *ks = kp + row.scales, *vc = vp + row.codes, *vs = vp + row.scales;
        const uint32_t k = c * (D / 2) + g * (D / 8);
        if constexpr (D == 96) {
#pragma unroll
            for (int i = 0; i < 3; ++i) x.k[t][i] = *reinterpret_cast<const uint32_t*>(kc + k + 4 * i);
        } else {
            load_words<D / 32>(x.k[t], reinterpret_cast<const uint16_t*>(kc + k));
        }
        x.ks[t][0] = ks[16 * KeyGroups<D>::first(g) + c];
        if constexpr (KeyGroups<D>::kTwo) x.ks[t][1] = ks[16 * KeyGroups<D>::last(g) + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned char* v = vc + (4 * g * (D / 2) + c * (D / 32)) + i * (D / 2);
            if constexpr (D == 64) x.v[t][i][0] = *reinterpret_cast<const uint16_t*>(v);
            // (Three bytes, and one that does not count: the next row's, or the scales' behind the last one.)
            else if constexpr (D == 96) __builtin_memcpy(&x.v[t][i][0], v, 4);
            else load_words<Tile<D>::kV>(x.v[t][i], reinterpret_cast<const uint16_t*>(v));
        }
        x.vs[t][0] = *reinterpret_cast<const uint32_t*>(vs + 16 * ValueGroups<D>::first(c) + 4 * g);
        if constexpr (ValueGroups<D>::kTwo)
            x.vs[t][1] = *reinterpret_cast<const uint32_t*>(vs + 16 * ValueGroups<D>::last(c) + 4 * g);
    }
}

// The largest of x over the four lanes of a column (lane % 16).
__device__ __forceinline__ float column_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, x), __builtin_bit_cast(int, x), false, false);
    const unsigned r0 = r[0], r1 = r[1];
    const float y = fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(int, y), __builtin_bit_cast(int, y), false, false);
    const unsigned s0 = s[0], s1 = s[1];
    return fmaxf(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}

// kWaves waves a workgroup, each with every kWaves-th tile.  A workgroup's up to
// 16 rows share a key head: its query heads of one new token, or with kMany (starts
// given) of several of a sequence.
template <class T, int D, int kWaves, bool kMany>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : 4) void attention_decode_q4_kernel(
    AttnArgs a, int splits, int chunk, int groups, int sort_most) {
    // (kMany: groups is not used, sort_most 0.)
    constexpr int VE = D / 16;
    __shared__ float o_join[kWaves][16][D + 4];
    __shared__ float m_join[kWaves][16], l_join[kWaves][16];
    __shared__ uint32_t bad_join[kWaves];        // a bit for each row that is not finite
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    // Row r of the block: head skip + r - past * share of the key head's, `past`
    // tokens behind row `token0`, by a product with the reciprocal (exact: attention_prefill.hip).
    int split, b, kvh, token0, skip, rows, p_first;
    const int share = a.q_heads / a.kv_heads;
    const float per_share = 1.0f / (float)share;
    auto past_of = [&](int r) { return kMany ? (int)(((float)(skip + r) + 0.5f) * per_share) : 0; };
    if constexpr (kMany) {
        const int slot = blockIdx.x / splits;
        split = blockIdx.x - slot * splits;
        kvh = blockIdx.y;
        Slot x;
        if (!find_slot(a, share, 4, slot, x)) return;
        b = x.b;
        const uint32_t r0 = (uint32_t)(x.tile * 16), past = r0 / (uint32_t)share;
        rows = (int)min((int64_t)16, (int64_t)x.count * share - r0);
        token0 = x.row_first + (int)past;
        skip = (int)(r0 - past * share);
        p_first = max(x.len - (x.to_row - x.row_first), -a.tokens) + (int)past;
    } else {
        int unit;                        // key head and group of 16 query heads
        if (sort_most) {
            // Longest sequences first, with all their heads (not split: see launch).
            const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x, rank = id / gridDim.y;
            unit = (int)(id - rank * gridDim.y);
            split = 0;
            b = __builtin_amdgcn_readfirstlane(longest_first(a.kv, (int)rank, sort_most));
        } else {
            split = blockIdx.x % splits;
            b = blockIdx.x / splits;
            unit = blockIdx.y;
        }
        kvh = unit / groups;
        token0 = b;
        skip = (unit - kvh * groups) * 16;
        rows = min(16, share - skip);
        p_first = seq_len(a.kv, b) - 1;
    }
    auto token_of = [&](int r) { return token0 + past_of(r); };
    auto head_of = [&](int r) { return kvh * share + skip + r - past_of(r) * share; };
    auto row_of = [&](int r) { return (int64_t)token_of(r) * a.q_heads + head_of(r); };

    // What the first row's position up to the last's see, what this lane's
    // sees, and what all of them see.
    const int p_last = p_first + __builtin_amdgcn_readfirstlane(past_of(rows - 1));
    Span span = key_span(a, p_last), mine = span, both = span;
    if constexpr (kMany) {
        const Span of_first = key_span(a, p_first);
        span.start = of_first.start;
        both.end = of_first.end;
        mine = key_span(a, c < rows ? p_first + past_of(c) : -1);
    }
    const int tiles = span.tiles(kTile);
    // At least `chunk` tiles a workgroup, more where the length passes what was planned for.
    const int per = max(chunk, (tiles + splits - 1) / splits);
    const int active = max(1, (tiles + per - 1) / per);
    const Partials parts(a, D, splits);
    if (split >= active) {
        if ((int)threadIdx.x < rows) parts.mark(row_of(threadIdx.x), split, -INFINITY, 0.0f);
        return;
    }
    const int first = split * per, last = min(tiles, first + per);

    // Slots of product i: elements D/4 g + 8 i + [0, 8).
    u4 qf[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        qf[i] = u4{0, 0, 0, 0};
        if (c < rows) qf[i] = *reinterpret_cast<const u4*>(a.q + token_of(c) * a.sq + (int64_t)head_of(c) * D + D / 4 * g + 8 * i);
    }
    // Scores are compared before they are scaled, so the scale's sign goes into the queries (exact).
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, keep = a.scale == 0.0f ? 0u : ~0u;
    const float scale = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.4426950408889634f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qf[i] = (qf[i] ^ flip) & keep;
    constexpr float kUp = T::kTop > kLazy ? T::kTop - kLazy : 0.0f;        // so that no weight passes 2^kTop
    float m = -INFINITY, l = 0.0f;
    f4 o[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) o[e] = f4{0, 0, 0, 0};

    auto step = [&](Tile<D>& x) {
        f4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = f4{0, 0, 0, 0};
            const float first_scale = q4_scale(x.ks[t][0]);
            float last_scale = first_scale;
            if constexpr (KeyGroups<D>::kTwo) last_scale = q4_scale(x.ks[t][1]);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                s[t] = T::mfma16(q4_values<T>(x.k[t][i], KeyGroups<D>::in_last(g, i) ? last_scale : first_scale), qf[i], s[t]);
        }
        // A tile whose every key is seen and owned needs no mask (the same answer in all lanes).
        if (!(both.all_seen(x.at.base, kTile) && x.at.page[0] >= 0 && x.at.page[1] >= 0)) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = x.at.base + 16 * t + 4 * g + i;
                    const bool any = x.at.page[t] >= 0 && span.seen(key);
                    if (!(kMany ? any && mine.seen(key) : any)) s[t][i] = -INFINITY;
                    if (!any) {
                        // What lies there must not reach 0 * v: codes of 0, and no scale that makes NaN of them.
                        // (What only other rows see may make a row NaN; it is computed again below.)
#pragma unroll
                        for (int e = 0; e < Tile<D>::kV; ++e) x.v[t][i][e] = 0;
                        x.vs[t][0] &= ~(0xFFu << 8 * i);
                        if constexpr (ValueGroups<D>::kTwo) x.vs[t][1] &= ~(0xFFu << 8 * i);
                    }
                }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = fmaf(column_max(top), scale, -kUp);
        if (__any(top > m + kLazy)) {
            const float mn = fmaxf(m, top), f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int e = 0; e < VE; ++e) o[e] *= f;
        }
        const float ms = m == -INFINITY ? 0.0f : m;          // nothing seen so far: all weights are 2^-inf = 0
        float w[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = exp2_fast(fmaf(s[j >> 2][j & 3], scale, -ms));
            sum += w[j];
        }
        l += sum;
        u4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = T::pack(w[2 * j], w[2 * j + 1]);
            lo[j] = T::pack(w[2 * j] - T::low(hi[j]), w[2 * j + 1] - T::high(hi[j]));
        }
        float vs[8], vs_last[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            vs[j] = q4_scale_of(x.vs[j >> 2][0], j & 3);
            if constexpr (ValueGroups<D>::kTwo) vs_last[j] = q4_scale_of(x.vs[j >> 2][1], j & 3);
        }
        // Elements e and e + 1 of a lane's: two keys' pairs, then their low and their high halves side by side.
        auto two = [&](auto byte, int word) {
            constexpr int e = 2 * decltype(byte)::value;
            u4 lows, highs;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t p[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int key = 2 * j + y;
                    float by = vs[key];
                    if constexpr (ValueGroups<D>::kTwo) by = ValueGroups<D>::in_last(c, e) ? vs_last[key] : by;
                    p[y] = q4_pair<T, e / 2>(x.v[key >> 2][key & 3][word], by);
                }
                lows[j] = __builtin_amdgcn_perm(p[1], p[0], 0x05040100u);
                highs[j] = __builtin_amdgcn_perm(p[1], p[0], 0x07060302u);
            }
            f4 &even = o[8 * word + e], &odd = o[8 * word + e + 1];
            even = T::mfma16(lows, lo, T::mfma16(lows, hi, even));
            odd = T::mfma16(highs, lo, T::mfma16(highs, hi, odd));
        };
#pragma unroll
        for (int word = 0; word < Tile<D>::kV; ++word) {
            two(std::integral_constant<int, 0>{}, word);
            two(std::integral_constant<int, 1>{}, word);
            if constexpr (VE > 4) two(std::integral_constant<int, 2>{}, word);
            if constexpr (VE > 6) two(std::integral_constant<int, 3>{}, word);
        }
    };

    // Two tiles in flight: the next one's loads are issued before the current
    // one is used, with the pages of the one after it.
    const int keys = max(0, span.end);
    auto place = [&](int i) {
        Place at;
        at.base = __builtin_amdgcn_readfirstlane(span.base(min(i, last - 1), kTile));
        at.page[0] = page_of(a, b, at.base, keys);
        at.page[1] = page_of(a, b, at.base + 16, keys);
        return at;
    };
    int i = first + wave;
    if (i < last) {
        Place next = place(i);
        Tile<D> x, y;
        load_tile<D>(x, a, kvh, next);
        next = place(i + kWaves);
        for (;;) {
            load_tile<D>(y, a, kvh, next);
            next = place(i + 2 * kWaves);
            step(x);
            i += kWaves;
            if (i >= last) break;
            load_tile<D>(x, a, kvh, next);
            next = place(i + 2 * kWaves);
            step(y);
            i += kWaves;
            if (i >= last) break;
        }
    }

    // Join the waves: a lane's o[e][r] is O^T of query c at d = (D/16)(4 g + r) + e.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        m_join[wave][c] = m;
        l_join[wave][c] = l;
    }
    if (c < rows) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < VE; ++e) o_join[wave][c][VE * (4 * g + r) + e] = o[e][r];
    }
    f4 probe = f4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < VE; ++e) probe += o[e] * 0.0f;
    const uint64_t odd = __ballot(c < rows && !(probe[0] + probe[1] + probe[2] + probe[3] == 0.0f));
    if (lane == 0) bad_join[wave] = (uint32_t)(odd | odd >> 16 | odd >> 32 | odd >> 48) & 0xFFFFu;
    __syncthreads();
    uint32_t bad = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) bad |= bad_join[w];
    bad = __builtin_amdgcn_readfirstlane(bad);
    for (int at = threadIdx.x; at < rows * (D / 4); at += 64 * kWaves) {
        const int r = at / (D / 4), d = (at - r * (D / 4)) * 4;
        if (bad >> r & 1) continue;
        float top = m_join[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_join[w][r]);
        const float ms = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        f4 acc = f4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = exp2_fast(m_join[w][r] - ms);
            sum += l_join[w][r] * f;
            acc += *reinterpret_cast<const f4*>(&o_join[w][r][d]) * f;
        }
        if (active == 1) {
            store_row4<T>(a, token_of(r), head_of(r), D, d, acc, top, sum);
            if (splits > 1 && d == 0) parts.mark(row_of(r), 0, top, kWhole);
        } else {
            parts.put4(row_of(r), split, d, acc);
            if (d == 0) parts.mark(row_of(r), split, top, sum);
        }
    }
    for (int r = wave; r < rows; r += kWaves) {
        if (!(bad >> r & 1)) continue;
        const int token = token_of(r), head = head_of(r);
        float x[4], top, sum;
        plain_row<D, kTile, Q4Rows<D>>(a, span, first, last, kMany ? key_span(a, p_first + past_of(r)) : span,
                                       a.kv.table + (int64_t)b * a.kv.width, kvh, a.q + token * a.sq + (int64_t)head * D, x,
                                       top, sum);
        store_plain_row<T, D>(a, parts, active > 1, token, head, split, x, top, sum);
        if (active == 1 && splits > 1 && lane == 0) parts.mark(row_of(r), 0, top, kWhole);
    }
}

// The plan.  Where there are enough key heads for all CUs, and for short
// lengths, one workgroup a key head.  It has 16 waves (8 at head size 256, whose
// registers hold no more) or 8 or 4, so that all workgroups run at once (ten
// sequences of 32 key heads and 2000 keys: 30.0 us with 16 waves, 25.3 with 8), and
// that a wave has some four tiles (500 keys of 32 key heads, four tiles for each of 4 waves or two of 8: one sequence
// 7.8 us with 4 and 7.4 with 8, nine 10.9 and 11.5).  More waves a workgroup and
// fewer workgroups of the same keys save the join: 32 sequences of 8 key heads in a
// window 19.5 us with 16 waves, 24.3 with 4 and the keys split.
// Otherwise the keys are split over workgroups, where that spares a SIMD
// kSplitFrom tiles (0.4 us each); that is what partial results and another
// launch cost: of 32 query heads on 8, 2000 keys of one sequence 13.6 us whole
// and 9.6 split, of four 13.8 and 11.4, of eight 14.3 and 15.0, of sixteen 14.7 and 16.5.
// The workgroups are then as small as gives at most kSplits of a key head (one sequence of 8000:
// 11.7 us with 62 of 4 waves, 10.6 with 31 of 8, 12.4 with 15 of 16; 131071: 39.1 with 64 of 8, 35.7 with 32 of 16)
// and two a CU (four of 8000: 17.1 with 1024 of 4 waves, 16.3 with 512 of 8).
// The plan knows the longest length only.  With a workgroup for every CU nothing is split, however uneven
// the lengths: one sequence of 131071 among 63 of 100, 32 heads on 8, takes 997 us, alone 34.
constexpr int kCus = 256, kSplitFrom = 10, kSplits = 32, kSortFrom = 512;

// Prompts (and chunks, and tokens to be verified) of up to kFewRows rows a key head on
// average, two blocks, go in blocks of 16 rows through this kernel, which reads the keys once for each block, longer
// ones through attention_prefill.hip with its blocks of 128 (2 tokens of 64 sequences
// of 2000, 32 heads on 8: 37 us here, 92 there; 4 of 32 of 4000, 32 heads:
// 114 and 195; 32 of 32 of 4000, 32 rows: 179 and 192; one of 24576, 32 heads on 8: 8 tokens, 32 rows, 23.7 and
// 27.6, 32 tokens, 128 rows, 40.4 and 41.2; 16 of 8 of 4096, 64 rows: 48.1 and 46.0).  The average
// decides for the whole batch: 61 tokens on 24576 beside 40 single ones of 1000, 32 heads on 8, take 196 us (apart 50 and 17), a prompt
// of 2048 beside 64 of them 81 (apart 55 and 19), beside 500 of them 194 (apart 55 and 111).
constexpr int kFewRows = 32;
// A sequence has at most kFewRows / 16 + 1 slots on average (find_slot), and there are at most 2^22
// sequences: their grid, of 4 waves a workgroup (plan_of: with more than 512 units), is one launch.
static_assert((kFewRows / 16 + 1) * (int64_t(1) << 22) * 64 * 4 < int64_t(1) << 32, "a grid holds fewer than 2^32 threads");

struct Plan {
    int64_t units;                   // key heads of blocks of rows, about
    int64_t most;                    // longest run of keys
    int tiles, waves, splits;
};

// Waves a CU holds, and a workgroup at most.
constexpr int most_waves(int head_dim) { return head_dim == 256 ? 8 : 16; }

Plan plan_of(const AttnArgs& a, int64_t units) {
    Plan x;
    const int kMost = most_waves(a.head_dim);
    x.units = units;
    x.most = a.max_len;
    if (a.window && (int64_t)a.window + a.sinks < x.most) x.most = (int64_t)a.window + a.sinks;
    x.tiles = (int)((x.most + kTile - 1) / kTile);
    x.splits = 1;
    const int64_t budget = kCus * kMost / units;             // waves of a unit that run at once
    if (x.tiles * (kCus - units) <= kSplitFrom * 4 * kCus) {
        const int few = units > kCus ? 4 : 2, wanted = (x.tiles + 3) / 4;
        x.waves = wanted <= few || budget < 8 ? 4 : wanted <= 8 || budget < 16 ? 8 : 16;
        x.waves = min(x.waves, kMost);
        return x;
    }
    const int64_t waves = min(budget, (int64_t)x.tiles), limit = kAttnSplitRows / ((int64_t)a.tokens * a.q_heads);
    for (x.waves = 4;; x.waves *= 2) {
        x.splits = (int)max((int64_t)1, min(waves / x.waves, limit));
        if (x.waves == kMost || (x.splits <= kSplits && units * x.splits <= 2 * kCus)) return x;
    }
}

template <class T, int D, int kWaves, bool kMany>
hipError_t launch_waves(const AttnArgs& a, const Plan& plan, hipStream_t stream) {
    const int share = a.q_heads / a.kv_heads, groups = (share + 15) / 16, splits = plan.splits;
    const int chunk = max(kWaves, (plan.tiles + splits - 1) / splits);
    // kMany: slots (find_slot).
    const int64_t blocks = kMany ? (int64_t)a.tokens * share / 16 + a.kv.seqs : a.tokens;
    const dim3 grid((unsigned)(blocks * splits), (unsigned)(kMany ? a.kv_heads : a.kv_heads * groups));
    // More than a round of workgroups: longest first (attention_decode.hip; 64 sequences of 1 to 4096
    // keys, 32 heads: 105 us, 142 in their order).
    const int sort_most = !kMany && kWaves == 4 && splits == 1 && plan.units > 2 * kCus && plan.most >= kSortFrom ? (int)plan.most : 0;
    hipLaunchKernelGGL((attention_decode_q4_kernel<T, D, kWaves, kMany>), grid, dim3(64 * kWaves), 0, stream, a, splits,
                       chunk, groups, sort_most);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || splits == 1 ? e : launch_attention_join(a, splits, stream);
}

template <class T, int D, bool kMany>
hipError_t launch(const AttnArgs& a, const Plan& plan, hipStream_t stream) {
    if (plan.waves == 4) return launch_waves<T, D, 4, kMany>(a, plan, stream);
    if constexpr (most_waves(D) == 16)
        if (plan.waves == 16) return launch_waves<T, D, 16, kMany>(a, plan, stream);
    return launch_waves<T, D, 8, kMany>(a, plan, stream);
}

template <class T, bool kMany>
hipError_t launch_dim(const AttnArgs& a, const Plan& plan, hipStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch<T, 64, kMany>(a, plan, stream);
        case 96: return launch<T, 96, kMany>(a, plan, stream);
        case 128: return launch<T, 128, kMany>(a, plan, stream);
        default: return launch<T, 256, kMany>(a, plan, stream);
    }
}

}  // namespace

hipError_t launch_attention_decode_q4(const AttnArgs& a, hipStream_t stream) {
    const Plan plan = plan_of(a, (int64_t)a.tokens * a.kv_heads * ((a.q_heads / a.kv_heads + 15) / 16));
    return a.dtype == 0 ? launch_dim<Fp16, false>(a, plan, stream) : launch_dim<Bf16, false>(a, plan, stream);
}

bool few_rows_q4(const AttnArgs& a) {
    return (int64_t)a.tokens * (a.q_heads / a.kv_heads) <= (int64_t)kFewRows * a.kv.seqs;
}

hipError_t launch_attention_few_q4(const AttnArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.tokens * (a.q_heads / a.kv_heads), blocks = (rows + 16 * a.kv.seqs - 1) / (16 * a.kv.seqs);
    const Plan plan = plan_of(a, a.kv.seqs * blocks * a.kv_heads);
    return a.dtype == 0 ? launch_dim<Fp16, true>(a, plan, stream) : launch_dim<Bf16, true>(a, plan, stream);
}

}  // namespace slim
