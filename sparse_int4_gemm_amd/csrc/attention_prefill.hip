// slim_attention_prefill: causal attention of many new tokens over the paged
// cache.
//
//   s_j = scale q . k_j,  O = sum_j 2^(c s_j - m) v_j / l,  c = log2 e,
//   m within 2^kLazy of the running maximum of c s_j - kUp, l the sum of the weights.
//
// Bound by the matrix unit (4 head_dim flops for each query, head and key it
// sees) and, nearly as much, by the vector unit (about 6 instructions and an
// exponential for each of those).  A workgroup holds 128 query rows of one key
// head (row r is token r / share, head r % share of the group, so grouped heads
// read each key tile once) and walks the key tiles that any of them sees.
//  - Keys and values go from the pages straight into LDS, 64 keys a tile, two
//    tiles deep, 16 bytes a lane, no registers between, laid out there
//    (kQuad) so that no LDS read below meets a bank twice (counted: none) and
//    nearly all of its address is the instruction's constant.  Rows past the
//    sequence's end, and pages that are none, arrive as zeros.
//  - A wave owns 32 rows.  S^T = K Q^T on 32 x 32 x 16 matrix instructions: a
//    lane holds one query (column lane % 32) and 16 keys of every 32, the lane
//    32 away the other 16, so a row's maximum is 8 instructions and an exchange.
//  - O^T = V^T P^T takes the weights as they lie in registers: its contraction
//    slots are bound to the keys that a lane scored.  V^T comes out of LDS
//    through the transposing read (16 lanes: 4 keys x 16 elements).
//  - The products of the next and the last half tile are issued among the
//    softmax of the current one (half_step), two waves to a SIMD.  Blocks of 64
//    rows a wave halve the LDS traffic, but leave one wave, which cannot
//    issue vector instructions fast enough alone (8192 windowed tokens: 469 us
//    against 424).
//  - The weights are rounded once to the operands' type, as the matrix unit
//    takes them (one unit, averaged over the keys); l sums them in fp32 before that.
//    The maximum is only raised when a row's grows by more than 2^kLazy: a
//    rescale of O costs half as much as the rest of the softmax.
//  - A value that is NaN or infinite in a place that only some rows of a tile
//    see would reach the others as 0 * NaN.  That shows in their results: a
//    wave whose output is not finite is computed again key by key (plain_row),
//    which gives only the rows that do see such a value theirs.
// Measured: 8192 tokens, window 4096, 32 query heads on 8 key heads of 128,
// bf16: 391 to 403 us on different cards, 1.02 to 1.05 PFLOP/s (a library
// product of 8192^3: 1.40 to 1.45); 719 thousand cycles, so 1.8 GHz over the call,
// of which the matrix unit is busy for 57% and the vector unit for 55%.
//
// slim_attention_prefill_q4 is the same kernel over pages of 4 bits (Q4): a
// tile's codes pass through registers, requested a step ahead, are turned into halves by
// one instruction for two, and are written to the places in LDS that the loads
// of halves fill.  A quarter of the bytes, and some 80 vector instructions and
// 32 LDS writes for each of 4 waves and tile more, which two workgroups a CU mostly
// hide: 8192 windowed tokens 392 to 409 us, four prompts of up to 4096 365 to 377 where
// the 16-bit cache takes 367 to 382; not so one wave a SIMD (head size 256: 79 and 66 us) or
// short prompts (2048 tokens of 32 heads: 53 and 49).  The weights are rounded once here
// too: with their low halves as a second operand, as in attention_decode_q4.hip, the error against
// 64 bits falls from 2.3e-3 to 1.7e-3 of the outputs' norm in bf16 and from 2.7e-4 to 2.1e-4 in fp16, where
// the outputs' own rounding puts it, and 8192 windowed tokens take 528 us instead of 398 (four prompts of
// 2000 202 and 161, 61 tokens on 24576 57 and 48).  At head size 64, one group,
// one register more than there are spills (8 bytes a lane).  LDS writes of 16 rows' chunks take 16 cycles,
// 13 with rows taken in another order (no bank met twice), which changed no case's time.
#include "kv_q4.hpp"

namespace slim {
namespace {

constexpr int kKeys = 64;            // keys of a tile
constexpr float kLazy = 8.0f;        // a weight may pass 2^kUp by 2^kLazy
// Query rows of a workgroup: 32 for each of its row waves.
constexpr int kRowWaves = 4, kRowsLog = 7, kRows = 1 << kRowsLog;

// Splits of the keys: kSplitTarget workgroups in all (one a CU), each with at
// least kMinTiles tiles.  One number for the batch, from its rows and the
// longest length: a long sequence among enough short ones is not split (61
// tokens on 24576 alone 49 us, beside 40 single tokens on 200 423).
constexpr int kSplitTarget = 256, kMinTiles = 4;

// A tile lies in LDS as [row of 64 bytes' quads][its rows][64 bytes]: a load of
// 64 lanes brings a quad of 16 rows, and a lane that reads another quad or
// another row of the same residue only changes the instruction's offset.  Of a
// row's four 16-byte chunks of a quad, chunk c of K (and of queries and outputs) is at
// place c ^ k_turn(row), so that 16 consecutive rows' same chunk lie in 16 different bank groups.
constexpr int kQuad = 64;
__device__ __forceinline__ int k_turn(int row) { return (row >> 2) & 3; }

typedef short s4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u2 lds_tr(uint32_t at) {
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                      (__attribute__((address_space(3))) s4v*)(size_t)at));
}

// x of the lane in the lower half and of the one 32 above it.
struct Halves { float lo, hi; };
__device__ __forceinline__ Halves halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, x), __builtin_bit_cast(int, x), false, false);
    const unsigned lo = r[0], hi = r[1];      // a bit_cast of r[1] itself reads element 0
    return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}

// What the launch knows of the grid: key heads x splits x slots (from slot0 on).
struct Grid {
    Divisor kv_heads, splits, share;
    int32_t slots, slot0, chunk, round;
};

// Q4: keys and values lie in the pages as 4 bits each (kv_q4.hpp).
template <class T, int D, int KG, bool Q4>
__global__ __launch_bounds__(64 * kRowWaves * KG, D == 256 ? 1 : D == 64 && KG == 1 ? 3 : 2) void attention_prefill_kernel(
    AttnArgs a, Grid grid) {
    typedef std::conditional_t<Q4, Q4Rows<D>, HalfRows<D>> Rows;
    constexpr int kTileBytes = kKeys * D * 2;
    constexpr int kLoads = D / 32;                       // quads of a row, 64-lane loads of a 16-row block
    __shared__ __align__(1024) unsigned char lds[KG][2][2][kTileBytes];         // [group][buffer][K, V]
    // Waves in KG groups: each group has all the rows, and every KG-th tile.
    const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = any_wave / kRowWaves, wave = any_wave % kRowWaves;
    const int half = lane >> 5, col = lane & 31;

    // Head fastest (a workgroup's XCD is its index mod 8: with 8 or more key
    // heads an XCD's L2 serves its own heads only), then the split, then the
    // slot of rows, last ones first: under the causal mask they have the most keys.
    const int share = grid.share.d, splits = grid.splits.d;
    const int units = grid.kv_heads.quotient(blockIdx.x), kvh = blockIdx.x - units * a.kv_heads;
    const int in_order = grid.splits.quotient(units), split = units - in_order * splits;
    int order = grid.slot0 + in_order;
    if constexpr (KG == 1 && (D == 96 || D == 128)) {
        // Two workgroups share a CU from the start (at D = 64 three, at 256 one): the
        // second 256 in reverse, the shortest of them beside the longest of the first
        // (2048 tokens of 32 heads of 128: 55.8 us in plain order, 54.4 so; of 64: 40.7 and 41.6).
        if (order >= grid.round && order < 2 * grid.round)
            order = grid.round + min(2 * grid.round, grid.slots) - 1 - order;
    }
    const int slot = grid.slots - 1 - order;

    Slot at_slot;
    if (!find_slot(a, share, kRowsLog, slot, at_slot)) return;
    const int b = at_slot.b, len = at_slot.len, row_first = at_slot.row_first, count = at_slot.count;
    const int64_t tile = at_slot.tile;

    // Row r of the block is token (skip + r) / share past `token0`: 32-bit
    // divisions, of small numbers by a product with the reciprocal (exact:
    // (x + 1/2) / share is at least 1 / 2048 away from a whole number).
    const uint32_t r0 = (uint32_t)(tile * kRows);
    const int64_t left = (int64_t)count * share - r0;
    const int rows = left >> kRowsLog ? kRows : (int)left;
    const int token0 = grid.share.quotient(r0), skip = (int)(r0 - (uint32_t)(token0 * share));
    const float per_share = 1.0f / (float)share;
    auto token_of = [&](int r) { return (int)(((float)(skip + r) + 0.5f) * per_share); };
    // Position of the first of them; new tokens before or behind the rows there are
    // count too (held at where all positions are negative: nothing below overflows).
    const int before = max(len - (at_slot.to_row - row_first), -a.tokens);
    const int p_first = before + token0;
    const int p_last = p_first + __builtin_amdgcn_readfirstlane(token_of(rows - 1));
    Span span = key_span(a, p_last);
    span.start = a.window ? max(0, p_first - a.window + 1) : 0;
    const int keys = min(len, a.kv.width << a.kv.page_shift);
    const int32_t* table = a.kv.table + (int64_t)b * a.kv.width;

    const int tiles = span.tiles(kKeys);
    const int per = max(grid.chunk, grid.splits.quotient(tiles + splits - 1));
    // Tiles [begin, end) of the list are this workgroup's; its group's t-th is begin + group + KG t.
    const int begin = min(tiles, split * per), end = min(tiles, begin + per);
    auto tiles_before = [&](int i) { return max(0, (i - begin - group + KG - 1) / KG); };      // of the group's, below i
    constexpr int first = 0;
    const int last = tiles_before(end), steps = (end - begin + KG - 1) / KG;

    constexpr float kUp = T::kTop > kLazy ? T::kTop - kLazy : 0.0f;        // so that no weight passes 2^kTop

    // This lane's query.
    const bool live = 32 * wave + col < rows;
    const int row_in = live ? 32 * wave + col : 0, past = token_of(row_in);
    const int token = row_first + token0 + past, head = kvh * share + skip + row_in - past * share;
    const Span mine = key_span(a, live ? p_first + past : -1);
    // Scores are compared before they are scaled, so the scale's sign goes into the queries (exact).
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    uint32_t keep = a.scale == 0.0f ? 0u : ~0u;
    asm("" : "+v"(keep));                         // one operation with the flip, not a selection after it
    const float scale = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.4426950408889634f;
    // The wave's own tiles [w_begin, w_end): its rows see none of the others.
    // Every row sees all of a 32-key half that begins in [all_from, all_to],
    // and of one that holds sinks only, up to all_to.
    const int w_rows = min(32, rows - 32 * wave);
    const int w_first = p_first + __builtin_amdgcn_readfirstlane(token_of(32 * wave));
    const int w_last = w_rows > 0 ? p_first + __builtin_amdgcn_readfirstlane(token_of(32 * wave + w_rows - 1)) : -1;
    const int sinks = span.sinks, sink_tiles = span.sink_tiles(kKeys), window_tile = span.start / kKeys - sink_tiles;
    const int w_end = w_last < 0 ? 0 : min(last, tiles_before(w_last / kKeys - window_tile + 1));
    const int w_begin = a.window && sinks == 0
                            ? min(w_end, tiles_before(max(0, w_first - a.window + 1) / kKeys - window_tile)) : 0;
    const int all_to = w_rows == 32 ? min(w_first + 1, keys) - kKeys / 2 : -1;
    const int all_from = a.window ? w_last - a.window + 1 : 0;

    // Bookkeeping of a tile: its first key, which of its four 16-key blocks have
    // a page, and of the block that this wave loads its place in the pool
    // and its rows (those before the sequence's end).  Wave w of a group loads
    // block w of K and of V.  Lane j holds it for tile from + j: a table entry looked up for
    // each tile would be waited for each time.
    const int row_mask = (1 << a.kv.page_shift) - 1;
    int at_lo = 0, at_hi = 0, to_scales = 0, blocks = 0, from = first;
    auto base_of = [&](int t) {
        t = begin + group + KG * t;
        return (t < sink_tiles ? t : t + window_tile) * kKeys;
    };
    auto look_up = [&](int t0, auto&& meanwhile) {
        from = t0;
        const int base = base_of(min(t0 + lane, last - 1));
        int page[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            page[i] = table[min(base + 16 * i, keys - 1) >> a.kv.page_shift];       // keys > 0 where there is a tile
        meanwhile();
        blocks = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool is = base + 16 * i < keys && page[i] >= 0 && page[i] < a.kv.pages;
            blocks |= is ? 1 << i : 0;
            if (i == wave) {
                const int key = base + 16 * i;
                int64_t at = ((((int64_t)(is ? page[i] : 0) * a.kv_heads + kvh) << a.kv.page_shift) +
                              (key & row_mask)) * (D * 2);
                if constexpr (Q4) {
                    const Q4Row row(is ? page[i] : 0, a.kv_heads, a.kv.page_shift, D, kvh, key & row_mask);
                    at = row.codes;
                    to_scales = (int)(row.scales - row.codes);
                }
                at_lo = (int)at;
                at_hi = (int)(at >> 32);
                blocks |= is ? max(0, min(16, keys - key)) << 4 : 0;
            }
        }
    };
    struct Place { int base, blocks, lo, hi, to_scales; };
    auto place = [&](int t) {
        Place x;
        x.base = base_of(t);
        x.blocks = __builtin_amdgcn_readlane(blocks, t - from);
        x.lo = __builtin_amdgcn_readlane(at_lo, t - from);
        x.hi = __builtin_amdgcn_readlane(at_hi, t - from);
        if constexpr (Q4) x.to_scales = __builtin_amdgcn_readlane(to_scales, t - from);
        return x;
    };
    // Load j takes quad j of a 16-row block, 4 lanes a row.
    const uint32_t lds0 = lds_u32(&lds[group][0][0][0]);
    const int load_row = lane >> 2, load_chunk = (lane & 3) ^ k_turn(load_row);
    const uint32_t k_from = load_row * (D * 2) + load_chunk * 16, v_from = load_row * (D * 2) + (lane & 3) * 16;
    // The wave's loads of a tile of K or V, kLoads of them, one by one.
    struct Source { u4 rsrc; uint32_t to; };
    auto source_of = [&](bool is_v, int buf, const Place& x, bool any) {
        const unsigned char* pool = reinterpret_cast<const unsigned char*>(is_v ? a.kv.v : a.kv.k);
        Source s;
        s.rsrc = rsrc_words(pool + (int64_t)((uint64_t)(uint32_t)x.lo | (uint64_t)(uint32_t)x.hi << 32),
                            any ? (x.blocks >> 4) * (D * 2) : 0);
        s.to = lds0 + (2 * buf + is_v) * kTileBytes + wave * 16 * kQuad;
        return s;
    };
    auto load_piece = [&](bool is_v, const Source& s, int j) {
        lds_load16_at(s.rsrc, s.to + j * kKeys * kQuad, is_v ? v_from : k_from, j * kQuad);
    };
    auto load = [&](bool is_v, int buf, const Place& x) {
        const Source s = source_of(is_v, buf, x, true);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) load_piece(is_v, s, n);
    };

    // 4 bits: the codes of a 16-row block, lane (row, quad) = (lane % 16, lane / 16)
    // a quad's 16 bytes and its scale (at head size 64 half of them, at 96 the last
    // quad twice, at 256 two quads), pass through registers, and from there into
    // the places that the loads above bring halves to, 16 consecutive lanes' into
    // 16 different bank groups - also those of V, which is turned as K is then.
    constexpr int kQuads = Q4 && D == 256 ? 2 : 1, kWords = Q4 && D == 64 ? 2 : 4;
    constexpr int kPieces = Q4 ? kQuads * kWords : 1;            // dwords of codes, 16-byte chunks of halves
    // (The scale as the byte it is loaded as: widened, it would be waited for before its step.)
    struct Raw { uint32_t codes[kQuads][kWords]; uint8_t scale[kQuads]; };
    Raw raw_k, raw_v;
    const int q4_row = lane & 15, q4_quad = D == 64 ? lane >> 5 : D == 96 ? min(lane >> 4, 2) : lane >> 4;
    const int q4_part = D == 64 ? (lane >> 4 & 1) * 8 : 0;       // of the quad's codes, bytes
    auto fetch = [&](Raw& to, bool is_v, const Place& x, bool any) {
        const unsigned char* pool = reinterpret_cast<const unsigned char*>(is_v ? a.kv.v : a.kv.k) +
                                    (int64_t)((uint64_t)(uint32_t)x.lo | (uint64_t)(uint32_t)x.hi << 32);
        const int rows_of = any ? x.blocks >> 4 : 0;
        const __amdgpu_buffer_rsrc_t codes = make_rsrc(pool, rows_of * (D / 2));
        const __amdgpu_buffer_rsrc_t scales = make_rsrc(pool + x.to_scales, D / 2);
#pragma unroll
        for (int j = 0; j < kQuads; ++j) {
            const int at = q4_row * (D / 2) + (q4_quad + 4 * j) * 16 + q4_part;
            if constexpr (kWords == 2) {
                const u2 w = __builtin_bit_cast(u2, __builtin_amdgcn_raw_buffer_load_b64(codes, at, 0, 0));
                to.codes[j][0] = w[0];
                to.codes[j][1] = w[1];
            } else {
                const u4 w = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(codes, at, 0, 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) to.codes[j][i] = w[i];
            }
            // (Rows past the end: codes of 0, and no scale that makes NaN of them.)
            to.scale[j] = __builtin_amdgcn_raw_buffer_load_b8(scales, q4_row < rows_of ? (q4_quad + 4 * j) * 16 + q4_row : kOOB, 0, 0);
        }
    };
    // Chunk c of a quad is at place c ^ k_turn(row): the lane's address with c's bits turned over.
    const uint32_t q4_to = lds0 + (wave * 16 + q4_row) * kQuad + q4_quad * kKeys * kQuad +
                           ((q4_part / 4) ^ k_turn(q4_row)) * 16;
    auto write_to = [&](bool is_v, int buf) {
        uint32_t at = q4_to + (2 * buf + is_v) * kTileBytes;
        asm("" : "+v"(at));
        return at;
    };
    auto write_piece = [&](const Raw& x, uint32_t to, int i) {
        const int j = i / kWords, c = i % kWords;
        const uint32_t at = (to ^ 16u * c) + 4 * j * kKeys * kQuad;
        *(__attribute__((address_space(3))) u4*)(size_t)at = q4_values<T>(x.codes[j][c], q4_scale(x.scale[j]));
    };
    auto write = [&](const Raw& x, bool is_v, int buf) {
        const uint32_t to = write_to(is_v, buf);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) write_piece(x, to, i);
    };

    // Where this lane reads a tile: K row col, chunk 2 i + half (places 0 or 1, 2 or 3
    // of a quad by i's low bit, turned); V rows 4 half + lane % 16 / 4 (+ 8, + 16 g),
    // elements 32 i + 16 (col / 16) + 4 (lane % 4).
    const uint32_t k_at = lds0 + col * kQuad + (half ^ k_turn(col)) * 16;
    // (4 bits: chunks turned by the row, that of the rows 8 further on by two more.)
    const uint32_t v_at = lds0 + kTileBytes + (4 * half + ((lane & 15) >> 2)) * kQuad +
                          ((32 * (col >> 4) + (lane & 3) * 8) ^ (Q4 ? 16 * half : 0));
    uint32_t v_at8 = (Q4 ? v_at ^ 32u : v_at) + 8 * kQuad;
    if constexpr (Q4) asm("" : "+v"(v_at8));      // a register of its own: offsets are the instruction's
    auto k_read = [&](uint32_t at, int i, int rows_of) { return (at ^ (32u * (i & 1))) + (i >> 1) * rows_of * kQuad; };

    // The wave's queries go through LDS as a key tile does (waves 0 and 1 of the
    // group to K of buffer 1, 2 and 3 to V of it, not in use yet): read straight
    // into the operand layout, every 32 bytes of a load would be another row's.
    // The rows' elements in global memory from the block's first token and head on
    // (at most 128 rows of 2^22: 2^30 bytes):
    auto element = [&](int r, int64_t stride) { return token_of(r) * ((int)stride - share * D) + (skip + r) * D; };
    auto load_queries = [&] {
        const u4 rsrc = rsrc_words(a.q + (int64_t)(row_first + token0) * a.sq + (int64_t)kvh * share * D, kOOB);
        const uint32_t to = lds0 + 2 * kTileBytes + wave * 32 * D * 2;
#pragma unroll
        for (int j = 0; j < 2 * kLoads; ++j) {
            const int in = 32 * wave + 16 * (j & 1) + load_row;
            int at = (element(in, a.sq) + load_chunk * 8) * 2 + (j >> 1) * kQuad;
            asm("" : "+v"(at));                   // without a branch around it
            lds_load16_at(rsrc, to + 1024 * j, in < rows ? at : kOOB, 0);
        }
    };
    u4 qf[D / 16];

    float m = -INFINITY, l = 0.0f;
    f16v o[D / 32];
    // Software pipeline over 32-key halves j of the tiles.  While the softmax
    // of half j runs on the vector unit, the matrix unit has the scores of half
    // j + 1 and the values of half j - 1 to work on, whose operands were read
    // from LDS during half j - 1; so K is needed a tile ahead of V.
    f16v s0, s1;
    u4 kf[D / 16], vf[2][D / 32], w[2] = {};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        vf[0][i] = vf[1][i] = u4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    }
    auto read_k = [&](uint32_t off) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) kf[i] = lds_ld<u4>(k_read(k_at + off, i, kKeys));
    };
    auto score = [&](f16v& s) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s = T::mfma32(kf[i], qf[i], s);
    };
    constexpr int kV = D / 32, kK = D / 16;       // matrix operands of 16 keys of V, of 32 keys of K
    auto add_value = [&](int n) {                 // n of the 2 kV operands of a half
        o[n % kV] = T::mfma32(vf[n / kV][n % kV], w[n / kV], o[n % kV]);
    };
    // Keeps the scores whose key is seen, `seen(e, c)` with element e's c (below).
    // Four comparisons, then four selections: one right after the other would wait.
    auto select = [&](f16v& s, auto&& seen) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            bool is[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) is[e] = seen(4 * g + e, 8 * g + e);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * g + e] = is[e] ? s[4 * g + e] : -INFINITY;
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // A half of the tile, from key `base` on: `cur` holds its scores, `nxt` takes the next half's.
    // The order of the code is the order of issue (the empty barriers hold the
    // compiler to it): vector work between any two matrix instructions, so
    // that neither unit waits for the other.
    auto half_step = [&](f16v& cur, f16v& nxt, int base, int blocks_of, uint32_t k_next, uint32_t v_cur,
                         auto&& between) {
        uint32_t v_base8 = v_at8 + v_cur;
        if constexpr (Q4) asm("" : "+v"(v_base8));
        // Keys that some row does not see: element e's is c + base + 4 half, c a
        // constant, so a limit is compared with constants.  Mostly only one of the two ends cuts.
        if (base > all_to || blocks_of != 3) {
            const int lim = mine.end - base - 4 * half;
            const int lims[2] = {blocks_of & 1 ? lim : -1, blocks_of & 2 ? lim : -1};
            select(cur, [&](int e, int c) { return c < lims[e >> 3]; });
        }
        if (base < all_from && base > sinks - kKeys / 2) {
            const int lim = mine.start - base - 4 * half, sink = mine.sinks - base - 4 * half;
            if (base >= sinks) {
                select(cur, [&](int, int c) { return c >= lim; });
            } else {
                select(cur, [&](int, int c) { return c >= lim || c < sink; });
            }
        }
        asm("" : "+v"(cur));      // one set of registers for both paths
        // A quarter of the products with V: the rows' maxima.
        constexpr int kFirst = kV / 2;
        float top = cur[0];
#pragma unroll
        for (int n = 0; n < kFirst; ++n) {
            __builtin_amdgcn_sched_barrier(0);
            add_value(n);
#pragma unroll
            for (int e = max(1, n * 16 / kFirst); e < (n + 1) * 16 / kFirst; ++e) top = __builtin_elementwise_maximum(top, cur[e]);
        }
        __builtin_amdgcn_sched_barrier(0);
        add_value(kFirst);
        const Halves tops = halves(top);
        top = fmaf(fmaxf(tops.lo, tops.hi), scale, -kUp);
        const bool raise = __any(top > m + kLazy);
        const float was = m;
        m = raise ? fmaxf(m, top) : m;
        const float ms = m == -INFINITY ? 0.0f : m;
        // The others, then the scores of the next half: the weights.  Operands are
        // read for the next half as soon as their registers are free.
#pragma unroll
        for (int e = 0; e < 16; ++e) nxt[e] = 0.0f;
        constexpr int kRest = 2 * kV - kFirst - 1 + kK;
        // Weight pair p of a lane's 8 passes through three chunks: its
        // exponents, the exponentials, their sum and rounding, so that none waits
        // for the one before.
        float ex[16], sum = 0.0f;
        u4 wn[2];
        auto exponents = [&](int n) {
#pragma unroll
            for (int e = n * 8 / kRest * 2; e < (n + 1) * 8 / kRest * 2; ++e) ex[e] = fmaf(cur[e], scale, -ms);
        };
        auto weights = [&](int n) {
#pragma unroll
            for (int p = n * 8 / kRest; p < (n + 1) * 8 / kRest; ++p) {
                sum += ex[2 * p] + ex[2 * p + 1];
                wn[p >> 2][p & 3] = T::pack(ex[2 * p], ex[2 * p + 1]);
            }
        };
        exponents(0);
#pragma unroll
        for (int n = 0; n < kRest; ++n) {
            const int k = n - (kRest - kK);                       // operand of K from 0 on
            __builtin_amdgcn_sched_barrier(0);
            between(n, kRest);
            if (k < 0) {
                add_value(kFirst + 1 + n);
            } else {
                nxt = T::mfma32(kf[k], qf[k], nxt);
                const int g = k / kV, i = k % kV;                 // kK == 2 kV
                const uint32_t at = v_at + v_cur + (i * kKeys + g * 16) * kQuad;
                const uint32_t at8 = Q4 ? v_base8 + (i * kKeys + g * 16) * kQuad : at + 8 * kQuad;
                const u2 x = lds_tr(at), y = lds_tr(at8);
                vf[g][i] = u4{x[0], x[1], y[0], y[1]};
                kf[k] = lds_ld<u4>(k_read(k_at + k_next, k, kKeys));
            }
#pragma unroll
            for (int e = n * 8 / kRest * 2; e < (n + 1) * 8 / kRest * 2; ++e) ex[e] = exp2_fast(ex[e]);
            if (n + 1 < kRest) exponents(n + 1);
            if (n > 0) weights(n - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        weights(kRest - 1);
        w[0] = wn[0];
        w[1] = wn[1];
        asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(sum));      // made among the products above
        if (raise) {
            const float f = m == -INFINITY ? 1.0f : exp2_fast(was - m);
            l *= f;
#pragma unroll
            for (int i = 0; i < kV; ++i) o[i] *= f;
        }
        l += sum;
    };

    // Every wave takes part in every step t of the loads, from first - 1 to
    // last - 1: at the end of `advance` K of tile t + 1 and V of tile t have
    // landed for all waves (in step first - 1 K only), and all are done with K of
    // tile t and V of tile t - 1 (or the queries), so the loads of K of tile t + 2 and
    // V of tile t + 1 may begin.
    // 4 bits: in step t what registers hold of K of tile t + 2 and V of tile t + 1
    // is written, and then K of tile t + 3 and V of tile t + 2 requested.
    Place cur, next, after, later;                // of tiles t, t + 1, t + 2 and t + 3
    if (first < last) {
        look_up(first, load_queries);
        cur = next = place(first);
        after = place(min(first + 1, last - 1));
        if constexpr (Q4) {
            later = place(min(first + 2, last - 1));
            Raw first_k;
            fetch(first_k, false, next, true);
            fetch(raw_v, true, next, true);
            fetch(raw_k, false, after, first + 1 < last);
            wait_vmem_below<0>();                 // the queries too, which the compiler does not know of
            write(first_k, false, 0);
            write(raw_v, true, 0);
        } else {
            load(false, 0, next);
            load(true, 0, next);
        }
    }
    auto advance = [&](int t) {
        if (t >= first) {
            cur = next;
            next = after;
            if constexpr (Q4) after = later;
            else wait_vmem_below<0>();
        } else if constexpr (!Q4) {
            wait_vmem_below<kLoads>();
        }
        __syncthreads();
        constexpr int kAhead = Q4 ? 3 : 2;
        if (t >= first && t + kAhead < last) {
            if (t + kAhead - from == 64) look_up(t + kAhead, [] {});
            (Q4 ? later : after) = place(t + kAhead);
        }
    };
    auto load_all = [&](int t) {
        if constexpr (Q4) {
            if (t + 2 < last) write(raw_k, false, (t - first) & 1);
            if (t >= first && t + 1 < last) write(raw_v, true, (t + 1 - first) & 1);
            if (t + 3 < last) fetch(raw_k, false, later, true);
            if (t + 2 < last) fetch(raw_v, true, after, true);
        } else {
            if (t + 2 < last) load(false, (t - first) & 1, after);
            if (t >= first && t + 1 < last) load(true, (t + 1 - first) & 1, next);
        }
    };
    constexpr uint32_t kHalf = kKeys / 2 * kQuad;
    if (first < last) {
        if constexpr (!Q4) wait_vmem_below<kLoads>();       // the queries; V of the first tile may still be on its way
#pragma unroll
        for (int i = 0; i < kK; ++i)
            qf[i] = (lds_ld<u4>(k_read(k_at + 2 * kTileBytes + wave * 32 * D * 2, i, 32)) ^ flip) & keep;
    }
    // (A group without tiles, or with one fewer, only takes part in the barriers.)
    int t = begin < end ? first - 1 : steps;
    for (; t < w_begin - 1; ++t) {
        advance(t);
        load_all(t);
    }
    if (w_begin < w_end) {
        advance(t);
        load_all(t);
        const uint32_t k_buf = ((t + 1 - first) & 1) * 2 * kTileBytes;
        read_k(k_buf);
        score(s0);
        read_k(k_buf + kHalf);
        for (++t; t < w_end; ++t) {
            advance(t);
            const int odd = (t - first) & 1;
            const uint32_t buf = odd * 2 * kTileBytes, other = 2 * kTileBytes - buf;
            // A workgroup's loads all at once would queue at the address unit
            // (32 of 16 cycles); here each wave spreads its own over the first half.
            // Past the last tile they read nothing (and write zeros nobody reads).
            if constexpr (Q4) {
                const uint32_t to_v = write_to(true, odd ^ 1), to_k = write_to(false, odd);
                half_step(s0, s1, cur.base, cur.blocks & 3, other, buf, [&](int n, int of) {
#pragma unroll
                    for (int i = n * 2 * kPieces / of; i < (n + 1) * 2 * kPieces / of; ++i) {
                        if (i < kPieces) write_piece(raw_v, to_v, i);
                        else write_piece(raw_k, to_k, i - kPieces);
                        if (i == kPieces - 1) fetch(raw_v, true, after, t + 2 < last);
                        if (i == 2 * kPieces - 1) fetch(raw_k, false, later, t + 3 < last);
                    }
                });
                half_step(s1, s0, cur.base + kKeys / 2, cur.blocks >> 2 & 3, other + kHalf, buf + kHalf, [](int, int) {});
                continue;
            }
            const Source k_source = source_of(false, odd, after, t + 2 < last);
            const Source v_source = source_of(true, odd ^ 1, next, t + 1 < last);
            half_step(s0, s1, cur.base, cur.blocks & 3, other, buf, [&](int n, int of) {
#pragma unroll
                for (int i = n * 2 * kLoads / of; i < (n + 1) * 2 * kLoads / of; ++i) {
                    if (i < kLoads) load_piece(true, v_source, i);
                    else load_piece(false, k_source, i - kLoads);
                }
            });
            half_step(s1, s0, cur.base + kKeys / 2, cur.blocks >> 2 & 3, other + kHalf, buf + kHalf, [](int, int) {});
        }
#pragma unroll
        for (int n = 0; n < 2 * kV; ++n) add_value(n);
    }
    for (; t < steps; ++t) {
        advance(t);
        load_all(t);
    }
    wait_vmem_below<0>();                         // no load may write LDS from here on

    constexpr int kRegs = (D / 32) * 16;          // 32-bit results of a lane
    static_assert(kRowWaves * kRegs * 64 * 4 <= (int)sizeof lds, "room for a group's results");
    unsigned char* const mine_lds = &lds[0][0][0][0] + wave * kRegs * 64 * 4;
    __syncthreads();                              // LDS is free
    if constexpr (KG == 2) {
        // The second group leaves its results in LDS, the first joins them.  One
        // group at most has seen nothing (m = -inf), or both.
        float* const at = reinterpret_cast<float*>(mine_lds) + lane;
        if (group == 1) {
#pragma unroll
            for (int i = 0; i < kRegs; ++i) at[i * 64] = o[i / 16][i % 16];
        }
        __shared__ float stats[kRowWaves][2][64];
        if (group == 1) {
            stats[wave][0][lane] = m;
            stats[wave][1][lane] = l;
        }
        __syncthreads();
        if (group == 1) return;
        const float m1 = stats[wave][0][lane], l1 = stats[wave][1][lane], mn = fmaxf(m, m1);
        const float f0 = mn == -INFINITY ? 1.0f : exp2_fast(m - mn), f1 = mn == -INFINITY ? 0.0f : exp2_fast(m1 - mn);
        m = mn;
        l = l * f0 + l1 * f1;
#pragma unroll
        for (int i = 0; i < kRegs; ++i) o[i / 16][i % 16] = o[i / 16][i % 16] * f0 + at[i * 64] * f1;
        asm volatile("" ::: "memory");            // read before the rows go to the same place
    }

    // Lane and the one 32 away hold the two halves of a row's sum.
    const Halves sums = halves(l);
    l = sums.lo + sums.hi;
    const Partials parts(a, D, splits);
    float probe = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) probe = fmaf(o[i][e], 0.0f, probe);
    if (__any(live && !(probe == 0.0f))) {
        for (int r = 32 * wave; r < 32 * wave + w_rows; ++r) {
            const int p = token_of(r), tk = row_first + token0 + p, hd = kvh * share + skip + r - p * share;
            float x[4], mx, lx;
            plain_row<D, kKeys, Rows>(a, span, begin, end, key_span(a, p_first + p), table, kvh,
                                      a.q + tk * a.sq + (int64_t)hd * D, x, mx, lx);
            store_plain_row<T, D>(a, parts, splits > 1, tk, hd, split, x, mx, lx);
        }
        return;
    }
    const int64_t row = (int64_t)token * a.q_heads + head;
    if (splits > 1) {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                parts.put4(row, split, 32 * i + 8 * e + 4 * half,
                           f4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]});
        if (half == 0) parts.mark(row, split, m, l);
        return;
    }
    // The rows leave through LDS too (each wave in its own part, in the order of
    // key rows), whole rows at a time.
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (a.lse && live && half == 0) a.lse[row] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    const uint32_t out = lds_u32(mine_lds);
    typedef __attribute__((address_space(3))) u2* LdsPair;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *(LdsPair)(size_t)(out + (32 * i + col) * kQuad + (e ^ k_turn(col)) * 16 + half * 8) =
                u2{T::pack(o[i][4 * e] * inv, o[i][4 * e + 1] * inv), T::pack(o[i][4 * e + 2] * inv, o[i][4 * e + 3] * inv)};
    asm volatile("" ::: "memory");                // a wave's LDS accesses are served in their order
    uint16_t* const to = a.o + (int64_t)(row_first + token0) * a.so + (int64_t)kvh * share * D;
#pragma unroll
    for (int j = 0; j < 2 * kLoads; ++j) {
        const int in = 32 * wave + 16 * (j & 1) + load_row;
        const u4 x = lds_ld<u4>(out + 1024 * j + lane * 16);
        if (in < rows) *reinterpret_cast<u4*>(to + element(in, a.so) + load_chunk * 8 + (j >> 1) * (kQuad / 2)) = x;
    }
}

// Slots of kRows query rows, enough for every sequence's.
int64_t slots_of(const AttnArgs& a) {
    return (int64_t)a.tokens * (a.q_heads / a.kv_heads) / kRows + a.kv.seqs;
}

template <class T, int D, int KG, bool Q4>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
    const int64_t slots = slots_of(a);
    int64_t most = a.max_len;
    if (a.window && (int64_t)a.window + a.sinks + kRows < most) most = (int64_t)a.window + a.sinks + kRows;
    const int64_t tiles = (most + kKeys - 1) / kKeys, units = slots * a.kv_heads;
    const int64_t want = min(kSplitTarget / units, (tiles + kMinTiles - 1) / kMinTiles);
    const int64_t splits = max((int64_t)1, min(want, kAttnSplitRows / ((int64_t)a.tokens * a.q_heads)));
    const int chunk = (int)max((int64_t)1, (tiles + splits - 1) / splits);
    // A grid holds fewer than 2^32 threads; slots past it go into further launches.
    const int64_t per_slot = a.kv_heads * splits, round = max((int64_t)1, kSplitTarget / per_slot), at_once = ((int64_t(1) << 32) / (64 * kRowWaves * KG) - 1) / per_slot;
    for (int64_t s = 0; s < slots; s += at_once) {
        const int64_t n = min(at_once, slots - s);
        hipLaunchKernelGGL((attention_prefill_kernel<T, D, KG, Q4>), dim3((unsigned)(n * per_slot)), dim3(64 * kRowWaves * KG), 0,
                           stream, a,
                           Grid{Divisor(a.kv_heads), Divisor(splits), Divisor(a.q_heads / a.kv_heads), (int)slots, (int)s,
                                chunk, (int)round});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return splits == 1 ? hipSuccess : launch_attention_join(a, (int)splits, stream);
}

// Two groups of waves on every other tile where one round of workgroups (one
// a CU) holds all row blocks: half the tiles one after another (61 tokens on
// 24576: 73 us in one group, 55 in two; 1024 tokens of 32 heads 28.9 and 25.9).
// With more, two workgroups of one group share a CU and hide each other's
// beginnings and ends (8192 windowed tokens: 427 us in one group, 476 in two;
// 1536 tokens behind 800 50.3 and 52.7, in a window of 1024 27.7 and 30.4) - unless
// the blocks' lengths run from one tile to all of them, as a whole prompt's do: the longest
// is then alone on its CU for most of its time (1100 tokens of 32 heads on 8
// 26.1 us in one group, 23.7 in two; 1536 33.3 and 30.8; 1900 44.2 and 41.3; 1280 behind 320 34.3
// and 33.1; head size 64, 1900 tokens 33.6 and 28.6), up to nearly two rounds (2048 tokens 48.6 and 50.2).
// The same with 4 bits (61 on 24576 55.2 in one group, 49.1 in two; 1100 tokens 32.6 and 29.1; 1536
// behind 800 59.5 and 62.3; four prompts of 2000 167 and 197; 8192 windowed 409 and 457).
template <class T, int D, bool Q4>
hipError_t launch_groups(const AttnArgs& a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.tokens * (a.q_heads / a.kv_heads);
    const int64_t blocks = a.kv.seqs == 1 ? (rows + kRows - 1) / kRows : slots_of(a);
    const bool uneven = a.kv.seqs == 1 && 4 * (int64_t)a.max_len <= 5 * (int64_t)a.tokens &&
                        (a.window == 0 || a.window >= a.tokens);
    const int64_t most = uneven ? 2 * kSplitTarget - kSplitTarget / 8 : kSplitTarget;
    return blocks * a.kv_heads <= most ? launch<T, D, 2, Q4>(a, stream) : launch<T, D, 1, Q4>(a, stream);
}

template <class T, bool Q4>
hipError_t launch_dim(const AttnArgs& a, hipStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_groups<T, 64, Q4>(a, stream);
        case 96: return launch_groups<T, 96, Q4>(a, stream);
        case 128: return launch_groups<T, 128, Q4>(a, stream);
        default: return launch<T, 256, 1, Q4>(a, stream);           // two groups' tiles do not fit LDS
    }
}

}  // namespace

hipError_t launch_attention_prefill(const AttnArgs& a, hipStream_t stream) {
    // One new token of every sequence is the single-token form.
    if (!a.kv.starts) return launch_attention_decode(a, stream);
    return a.dtype == 0 ? launch_dim<Fp16, false>(a, stream) : launch_dim<Bf16, false>(a, stream);
}

hipError_t launch_attention_prefill_q4(const AttnArgs& a, hipStream_t stream) {
    if (!a.kv.starts) return launch_attention_decode_q4(a, stream);
    if (few_rows_q4(a)) return launch_attention_few_q4(a, stream);
    return a.dtype == 0 ? launch_dim<Fp16, true>(a, stream) : launch_dim<Bf16, true>(a, stream);
}

}  // namespace slim
