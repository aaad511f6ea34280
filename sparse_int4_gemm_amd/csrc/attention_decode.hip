// slim_attention_decode: attention of one new token per sequence.
//
//   s_j = scale q . k_j,  O = sum_j 2^(c s_j - m) v_j / l,  c = log2 e,
//   m a running maximum of c s_j - T::kTop, l the sum of the weights (all fp32).
//
// Bound by the keys and values read once from HBM (1 to 16 flops a byte), so
// the kernel is built around loads: each wave streams tiles of 32 keys
// straight into registers, one tile ahead of the one it computes on, and every
// load is as wide as the layout gives (16 bytes a lane at head size 128).
//  - One wave serves up to 16 query heads of a key head: the matrix
//    instruction's 16 columns; more take a workgroup for every 16, which reads
//    the keys again (64 sequences of 4096, 8 key heads: 183 us with 16 query heads
//    each, 295 with 20 or 32, 443 with 40).  Keys are its rows: S^T = K Q^T leaves a
//    lane with one query (column) and the 4 keys 16 t + 4 g + [0, 4) of each
//    16-key half t (g = lane / 16).
//  - O^T = V^T P^T then takes these weights as they lie: its 32 contraction
//    slots are bound to keys so that a lane's slots are the keys it
//    scored, and the lane loads exactly those 8 rows of V, head_dim/16
//    elements each.  Pairing two rows' 16-bit elements is one byte permute
//    per operand register: V is never transposed through LDS.
//  - Weights enter the product as two halves (high and low part of the fp32
//    value): the matrix unit idles anyway, and the result then keeps fp32
//    weights' accuracy.  An infinite value meets a low half of 0 or of the other
//    sign there: rows that are not finite at the end are computed again, each
//    weight whole (plain_row).
//  - A sequence's tiles are cut into chunks, one workgroup each; its 4 waves
//    take every fourth tile and join through LDS; the chunks of a row are joined
//    by attention_join_kernel.
//  - Page numbers come through the scalar cache a tile ahead: as vector loads
//    they would be waited for behind the keys in flight (131071 keys: 124 us
//    against 128).
// Measured (a stream of 4 GiB is read at 6.1 TB/s): 64 sequences
// of 4096 tokens, 32 heads of 128: 720 us, 6.0 TB/s; of 1 to 4096: 367 us, 5.9
// TB/s (longest first; the last long ones alone: 436); one of 131071, 8 key heads:
// 97 us, 5.5 TB/s; one of 33: 5.5 us, launch and the chain lens -> table -> keys -> join.
#include "attention_device.hpp"

namespace slim {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;            // keys of one wave's step

// Where a tile lies: its first key and the pages of its 16-key halves (-1: none).
struct Place {
    int base, page[2];
};

// The registers of one tile.
template <int D>
struct Tile {
    u4 k[2][D / 32];                 // K rows 16 t + lane % 16, elements 32 c + 8 g + [0, 8)
    uint32_t v[8][D / 32];           // V rows 16 t + 4 g + i, elements (D/16)(lane % 16) + [0, D/16)
    Place at;
};

template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& x, const AttnArgs& a, int kvh, const Place& at) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    x.at = at;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t row = (((int64_t)max(at.page[t], 0) * a.kv_heads + kvh) << a.kv.page_shift) +
                            ((at.base + 16 * t) & ((1 << a.kv.page_shift) - 1));
        const uint16_t* k = a.kv.k + row * D;
        const uint16_t* v = a.kv.v + row * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x.k[t][i] = *reinterpret_cast<const u4*>(k + c * D + 32 * i + 8 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words<D / 32>(x.v[4 * t + i], v + (4 * g + i) * D + (D / 16) * c);
    }
}

// The sequence in place `rank` when those of every 64 are taken longest first,
// in sixteen classes of length up to `most` (a class's in their own order): a
// load, and a ballot for each class down to the answer's.
__device__ __forceinline__ int longest_first(const PagedKV& kv, int rank, int most) {
    const int lane = threadIdx.x & 63, base = rank & ~63;
    const int len = seq_len(kv, min(base + lane, kv.seqs - 1));
    const int of = min((int)((float)len * (16.0f / (float)most)), 15);
    int left = rank & 63;
    uint64_t found = 0;
    for (int c = 15; c >= 0; --c) {
        found = __ballot(base + lane < kv.seqs && of == c);
        const int n = __builtin_popcountll(found);
        if (left < n) break;
        left -= n;
    }
    // The left-th of the class.
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(found >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)found, 0));
    const uint64_t at = __ballot((found >> lane & 1) && before == left);
    return base + (at == 0 ? 0 : __builtin_ctzll(at));
}

template <class T, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_decode_kernel(AttnArgs a, int splits, int chunk,
                                                                          int groups, int sort_most) {
    constexpr int VE = D / 16;
    __shared__ float o_join[kWaves][16][D + 4];
    __shared__ float m_join[kWaves][16], l_join[kWaves][16];
    __shared__ uint32_t bad_join[kWaves];        // a bit for each row that is not finite
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    int split, b, unit;                  // unit: key head and group of 16 query heads
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
    const int kvh = unit / groups, share = a.q_heads / a.kv_heads;
    const int h0 = kvh * share + (unit - kvh * groups) * 16;                   // this workgroup's query heads
    const int heads = min(16, (kvh + 1) * share - h0);

    const Span span = key_span(a, seq_len(a.kv, b) - 1);
    const int tiles = span.tiles(kTile);
    // At least `chunk` tiles a workgroup, more where the length passes what was planned for.
    const int per = max(chunk, (tiles + splits - 1) / splits);
    const int active = max(1, (tiles + per - 1) / per);
    const int64_t row0 = (int64_t)b * a.q_heads + h0;
    const Partials parts(a, D, splits);
    if (split >= active) {
        if ((int)threadIdx.x < heads) parts.mark(row0 + threadIdx.x, split, -INFINITY, 0.0f);
        return;
    }
    const int first = split * per, last = min(tiles, first + per);

    u4 qf[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        qf[i] = u4{0, 0, 0, 0};
        if (c < heads) qf[i] = *reinterpret_cast<const u4*>(a.q + b * a.sq + (int64_t)(h0 + c) * D + 32 * i + 8 * g);
    }
    const float scale = a.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.0f;
    f4 o[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) o[e] = f4{0, 0, 0, 0};

    auto step = [&](Tile<D>& x) {
        f4 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = f4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) s[t] = T::mfma16(x.k[t][i], qf[i], s[t]);
            s[t] *= scale;
        }
        // A tile whose every key is seen and owned needs no mask (the same answer in all lanes).
        if (!(span.all_seen(x.at.base, kTile) && x.at.page[0] >= 0 && x.at.page[1] >= 0)) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool seen = x.at.page[t] >= 0 && span.seen(x.at.base + 16 * t + 4 * g + i);
                    if (!seen) {
                        s[t][i] = -INFINITY;
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) x.v[4 * t + i][e] = 0;      // what lies there must not reach 0 * v
                    }
                }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top - T::kTop);            // the largest weight is 2^kTop
        const float ms = mn == -INFINITY ? 0.0f : mn;        // nothing seen so far: all weights are 2^-inf = 0
        const float f = exp2_fast(m - ms);
        m = mn;
        float w[8], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = exp2_fast(s[j >> 2][j & 3] - ms);
            sum += w[j];
        }
        l = l * f + sum;
        u4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi[j] = T::pack(w[2 * j], w[2 * j + 1]);
            lo[j] = T::pack(w[2 * j] - T::low(hi[j]), w[2 * j + 1] - T::high(hi[j]));
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            u4 vt;                                            // slots 2 j, 2 j + 1: two rows' element e
#pragma unroll
            for (int j = 0; j < 4; ++j)
                vt[j] = __builtin_amdgcn_perm(x.v[2 * j + 1][e >> 1], x.v[2 * j][e >> 1],
                                              (e & 1) ? 0x07060302u : 0x05040100u);
            o[e] = T::mfma16(vt, lo, T::mfma16(vt, hi, o[e] * f));
        }
    };

    // Two tiles in flight: the next one's loads are issued before the current
    // one is used, with the pages of the one after it.  At head size 256 two tiles (256
    // registers) do not fit; the CU's eight waves then keep eight 32 KB tiles
    // in flight between them.
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
        if constexpr (D > 128) {
            for (; i < last; i += kWaves) {
                Tile<D> x;
                load_tile<D>(x, a, kvh, next);
                next = place(i + kWaves);
                step(x);
            }
        } else {
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
    }

    // Join the waves: a lane's o[e][r] is O^T of query c at d = (D/16)(4 g + r) + e.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        m_join[wave][c] = m;
        l_join[wave][c] = l;
    }
    if (c < heads) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < VE; ++e) o_join[wave][c][VE * (4 * g + r) + e] = o[e][r];
    }
    f4 probe = f4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < VE; ++e) probe += o[e] * 0.0f;
    const uint64_t odd = __ballot(c < heads && !(probe[0] + probe[1] + probe[2] + probe[3] == 0.0f));
    if (lane == 0) bad_join[wave] = (uint32_t)(odd | odd >> 16 | odd >> 32 | odd >> 48) & 0xFFFFu;
    __syncthreads();
    static_assert(kWaves == 4, "the waves' rows below");
    const uint32_t bad = __builtin_amdgcn_readfirstlane(bad_join[0] | bad_join[1] | bad_join[2] | bad_join[3]);
    for (int at = threadIdx.x; at < heads * (D / 4); at += 64 * kWaves) {
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
            store_row4<T>(a, b, h0 + r, D, d, acc, top, sum);
            if (splits > 1 && d == 0) parts.mark(row0 + r, 0, top, kWhole);
        } else {
            parts.put4(row0 + r, split, d, acc);
            if (d == 0) parts.mark(row0 + r, split, top, sum);
        }
    }
    for (int r = wave; r < heads; r += kWaves) {
        if (!(bad >> r & 1)) continue;
        float x[4], top, sum;
        plain_row<D, kTile>(a, span, first, last, span, a.kv.table + (int64_t)b * a.kv.width, kvh,
                            a.q + b * a.sq + (int64_t)(h0 + r) * D, x, top, sum);
        store_plain_row<T, D>(a, parts, active > 1, b, h0 + r, split, x, top, sum);
        if (active == 1 && splits > 1 && lane == 0) parts.mark(row0 + r, 0, top, kWhole);
    }
}

// Splits: two workgroups a CU, each with at least kMinTiles tiles.  More of
// them cost more in partial results than they gain (131071 keys of 8 key heads: 512
// workgroups 100 us, 1024 103, 2048 111; 64 sequences of up to 900 at head size
// 256: 61 us unsplit, 87 in two), fewer tiles too (4 sequences of up to 8000, 8 key heads:
// 16 tiles 20.7 us, 8 tiles 24.1).  One number for the batch, from its size and
// longest length: a long sequence among enough short ones is not split (63 of
// 100 tokens and one of 131071, 8 key heads: 2582 us, the long one alone 98).
constexpr int kSplitTarget = 512, kMinTiles = 16, kSortFrom = 512;

template <class T, int D>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
    const int share = a.q_heads / a.kv_heads, groups = (share + 15) / 16;
    int64_t most = (int64_t)a.max_len;
    if (a.window && (int64_t)a.window + a.sinks < most) most = (int64_t)a.window + a.sinks;
    const int tiles = (int)((most + kTile - 1) / kTile);
    const int64_t units = (int64_t)a.tokens * a.kv_heads * groups;
    const int64_t want = min(kSplitTarget / units, (int64_t)((tiles + kMinTiles - 1) / kMinTiles));
    const int splits = (int)max((int64_t)1, min(want, kAttnSplitRows / ((int64_t)a.tokens * a.q_heads)));
    const int chunk = max(kWaves, (tiles + splits - 1) / splits);
    dim3 grid((unsigned)(a.tokens * splits), (unsigned)(a.kv_heads * groups));
    // More than one round of workgroups, so that none is split: the longest of
    // every 64 sequences first, or the last ones to begin end alone (64 sequences of 1 to
    // 4096, 32 key heads: 436 us in their order, 365 so; 128 of up to 8000, 8 key
    // heads 426 and 377; 64 of up to 900 at head size 256 207 and 170).  Not for
    // short ones, where finding a place costs more (512 of up to 100: 40.3 and
    // 45.6; 256 of up to 250 33.8 and 35.4, of up to 500 58.9 and 59.3).
    const int sort_most = units > kSplitTarget && most >= kSortFrom ? (int)most : 0;
    hipLaunchKernelGGL((attention_decode_kernel<T, D>), grid, dim3(64 * kWaves), 0, stream, a, splits, chunk, groups,
                       sort_most);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || splits == 1 ? e : launch_attention_join(a, splits, stream);
}

template <class T>
hipError_t launch_dim(const AttnArgs& a, hipStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch<T, 64>(a, stream);
        case 96: return launch<T, 96>(a, stream);
        case 128: return launch<T, 128>(a, stream);
        default: return launch<T, 256>(a, stream);
    }
}

}  // namespace

hipError_t launch_attention_decode(const AttnArgs& a, hipStream_t stream) {
    return a.dtype == 0 ? launch_dim<Fp16>(a, stream) : launch_dim<Bf16>(a, stream);
}

}  // namespace slim
