// C-ABI front end of the paged key-value cache and its attention (declarations
// and the contract of every call are in include/slim.h).  Checks every
// argument before anything is launched; never aborts or throws.
#include <float.h>

#include "api_util.hpp"
#include "attention.hpp"

namespace {

using slim::aligned16;
using slim::fail;
using slim::kMaxDim;

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxPositions = int64_t(1) << 30;   // table_width * page_size
constexpr int64_t kMaxTokens = int64_t(1) << 22;      // a workgroup per token stays within a grid's 2^32 threads
constexpr int64_t kMaxPageBytes = int64_t(1) << 30;
// Elements between rows: the prompt kernel's offsets from a block's first row, of up to
// 128 rows, are 32-bit bytes.
constexpr int64_t kMaxRowStride = int64_t(1) << 22;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool head_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// log2 of a supported page size, -1 otherwise.
int page_shift(int64_t p) {
    for (int s = 4; s <= 10; ++s)
        if (p == int64_t(1) << s) return s;
    return -1;
}

slim_status check_rows(const char* what, const void* p, int64_t stride, int64_t rows, int64_t row) {
    if (!p) return fail(SLIM_EINVAL, "%s is NULL", what);
    if (!aligned16(p)) return fail(SLIM_EINVAL, "%s must be 16-byte aligned", what);
    if (stride % 8 || (rows > 1 && stride < row) || stride < 0 || stride > kMaxRowStride)
        return fail(SLIM_EINVAL, "%s: row stride %lld must be a multiple of 8, at least %lld and at most %lld", what,
                    (long long)stride, (long long)row, (long long)kMaxRowStride);
    return SLIM_OK;
}

// The pool and the sequences' places in it; fills *kv.
slim_status check_cache(int64_t seqs, int64_t kv_heads, int64_t head_dim, const uint16_t* k, const uint16_t* v,
                        int64_t pages, int64_t page_size, const int32_t* table, int64_t table_width,
                        const int32_t* lens, const int32_t* starts, slim::PagedKV* kv) {
    if (page_shift(page_size) < 0)
        return fail(SLIM_EUNSUPPORTED, "page_size must be a power of two from 16 to 1024 (got %lld)",
                    (long long)page_size);
    if (pages <= 0 || pages > kMaxDim)
        return fail(SLIM_EINVAL, "pages out of range (got %lld)", (long long)pages);
    if (table_width <= 0 || table_width > kMaxDim || table_width * page_size > kMaxPositions)
        return fail(SLIM_EINVAL, "table_width must be positive and table_width * page_size at most 2^30 (got %lld)",
                    (long long)table_width);
    if (!k || !v || !table || !lens) return fail(SLIM_EINVAL, "NULL pool, table or lens");
    if (!aligned16(k) || !aligned16(v)) return fail(SLIM_EINVAL, "the pools must be 16-byte aligned");
    if (!aligned4(table) || !aligned4(lens) || !aligned4(starts))
        return fail(SLIM_EINVAL, "table, lens and starts must be 4-byte aligned");
    kv->k = k; kv->v = v;
    kv->table = table; kv->lens = lens; kv->starts = starts;
    kv->pages = (int32_t)pages; kv->width = (int32_t)table_width; kv->seqs = (int32_t)seqs;
    kv->page_shift = page_shift(page_size);
    return SLIM_OK;
}

slim_status check_shape(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int dtype) {
    if (dtype != SLIM_FP16 && dtype != SLIM_BF16) return fail(SLIM_EUNSUPPORTED, "unknown dtype %d", dtype);
    if (!head_dim_ok(head_dim))
        return fail(SLIM_EUNSUPPORTED, "head_dim must be 64, 96, 128 or 256 (got %lld)", (long long)head_dim);
    if (tokens < 0 || tokens > kMaxTokens || seqs < 0 || seqs > kMaxTokens)
        return fail(SLIM_EINVAL, "tokens and seqs must be in [0, 2^22] (got %lld, %lld)", (long long)tokens,
                    (long long)seqs);
    if (kv_heads <= 0 || q_heads <= 0 || q_heads > kMaxHeads || q_heads % kv_heads)
        return fail(SLIM_EINVAL, "q_heads must be a multiple of kv_heads and at most 1024 (got %lld, %lld)",
                    (long long)q_heads, (long long)kv_heads);
    return SLIM_OK;
}

// Everything that both attention calls take.
slim_status check_attention(const uint16_t* Q, int64_t stride_Q, uint16_t* O, int64_t stride_O, float* lse,
                            int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                            int dtype, const uint16_t* Kpool, const uint16_t* Vpool, int64_t pages, int64_t page_size,
                            const int32_t* table, int64_t table_width, const int32_t* lens, const int32_t* starts,
                            int64_t max_len, int64_t window, int64_t sinks, float scale, void* workspace,
                            size_t workspace_bytes, slim::AttnArgs* a) {
    slim_status st = check_rows("Q", Q, stride_Q, tokens, q_heads * head_dim);
    if (st == SLIM_OK) st = check_rows("O", O, stride_O, tokens, q_heads * head_dim);
    if (st != SLIM_OK) return st;
    if (seqs == 0) return fail(SLIM_EINVAL, "tokens without sequences");
    if (!aligned4(lse)) return fail(SLIM_EINVAL, "lse must be 4-byte aligned");
    st = check_cache(seqs, kv_heads, head_dim, Kpool, Vpool, pages, page_size, table, table_width, lens, starts,
                     &a->kv);
    if (st != SLIM_OK) return st;
    if (max_len < 0 || max_len > kMaxPositions) return fail(SLIM_EINVAL, "max_len must be in [0, 2^30]");
    if (window < 0 || window > kMaxPositions || sinks < 0 || sinks > kMaxPositions)
        return fail(SLIM_EINVAL, "window and sinks must be in [0, 2^30]");
    if (!(scale - scale == 0.0f)) return fail(SLIM_EINVAL, "scale must be finite");
    const size_t need = slim::attention_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim);
    if (!workspace) return fail(SLIM_EINVAL, "workspace is NULL but %zu bytes are needed", need);
    if (!aligned16(workspace)) return fail(SLIM_EINVAL, "workspace must be 16-byte aligned");
    if (workspace_bytes < need)
        return fail(SLIM_EINVAL, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
    a->q = Q; a->sq = stride_Q;
    a->o = O; a->so = stride_O;
    a->lse = lse;
    a->tokens = (int32_t)tokens; a->q_heads = (int32_t)q_heads; a->kv_heads = (int32_t)kv_heads;
    a->head_dim = (int32_t)head_dim;
    a->dtype = dtype;
    a->max_len = (int32_t)max_len; a->window = (int32_t)window; a->sinks = (int32_t)sinks;
    a->scale = scale;
    a->ws = static_cast<unsigned char*>(workspace);
    return slim::check_device();
}

// A rotation of heads of head_dim elements; fills *to.
slim_status check_rotation(const slim_rotation* r, int64_t head_dim, slim::Rotation* to) {
    if (!r) return fail(SLIM_EINVAL, "rotation is NULL");
    if (r->rot_dim <= 0 || r->rot_dim % 8 || r->rot_dim > head_dim)
        return fail(SLIM_EINVAL, "rot_dim must be a multiple of 8 from 8 to head_dim (got %lld)", (long long)r->rot_dim);
    if (!r->freqs) return fail(SLIM_EINVAL, "freqs is NULL");
    if (reinterpret_cast<uintptr_t>(r->freqs) & 7u) return fail(SLIM_EINVAL, "freqs must be 8-byte aligned");
    if (r->interleaved != 0 && r->interleaved != 1) return fail(SLIM_EINVAL, "interleaved must be 0 or 1");
    // (Half rows are turned in fp32, with the products of it and the cosines.)
    if (!(r->magnitude >= -(double)FLT_MAX && r->magnitude <= (double)FLT_MAX))
        return fail(SLIM_EINVAL, "magnitude must be finite and within fp32's range");
    to->freqs = r->freqs;
    to->half = (int32_t)(r->rot_dim / 2);
    to->interleaved = r->interleaved;
    to->magnitude = r->magnitude;
    return SLIM_OK;
}

// Output rows that may be the input's.
slim_status check_in_place(const char* what, const void* x, int64_t sx, const void* y, int64_t sy) {
    if (x == y && sx != sy) return fail(SLIM_EINVAL, "%s in place needs one row stride", what);
    return SLIM_OK;
}

// Everything that both appends with a rotation take; fills *a.
slim_status check_append_rope(const uint16_t* Q, int64_t stride_Q, uint16_t* Qout, int64_t stride_Qout, int64_t q_heads,
                              const uint16_t* K, int64_t stride_K, const uint16_t* V, int64_t stride_V, int64_t tokens,
                              int64_t seqs, int64_t kv_heads, int64_t head_dim, const int32_t* table,
                              int64_t table_width, const int32_t* lens, const int32_t* starts, const void* Kpool,
                              const void* Vpool, int64_t pages, int64_t page_size, const slim_rotation* rotation,
                              int dtype, slim::AppendRopeArgs* a) {
    if (seqs == 0) return fail(SLIM_EINVAL, "tokens without sequences");
    if (!Q != !Qout) return fail(SLIM_EINVAL, "Q and Qout must both be given, or neither");
    slim_status st = check_rows("K", K, stride_K, tokens, kv_heads * head_dim);
    if (st == SLIM_OK) st = check_rows("V", V, stride_V, tokens, kv_heads * head_dim);
    if (st == SLIM_OK && Q) {
        if (!rotation) return fail(SLIM_EINVAL, "Q without a rotation");
        st = check_rows("Q", Q, stride_Q, tokens, q_heads * head_dim);
        if (st == SLIM_OK) st = check_rows("Qout", Qout, stride_Qout, tokens, q_heads * head_dim);
        if (st == SLIM_OK) st = check_in_place("Q", Q, stride_Q, Qout, stride_Qout);
    }
    a->by = slim::Rotation{nullptr, 0, 0, 1.0};
    if (st == SLIM_OK && rotation) st = check_rotation(rotation, head_dim, &a->by);
    if (st == SLIM_OK)
        st = check_cache(seqs, kv_heads, head_dim, static_cast<const uint16_t*>(Kpool), static_cast<const uint16_t*>(Vpool),
                         pages, page_size, table, table_width, lens, starts, &a->to.kv);
    if (st != SLIM_OK) return st;
    a->to.k_new = K; a->to.sk = stride_K;
    a->to.v_new = V; a->to.sv = stride_V;
    a->to.tokens = (int32_t)tokens; a->to.kv_heads = (int32_t)kv_heads; a->to.head_dim = (int32_t)head_dim;
    a->q = Q; a->sq = stride_Q;
    a->q_out = Qout; a->sqo = stride_Qout;
    a->q_heads = Q ? (int32_t)q_heads : 0;
    a->dtype = dtype;
    return slim::check_device();
}

}  // namespace

extern "C" {

slim_status slim_kv_append(const uint16_t* K, int64_t stride_K, const uint16_t* V, int64_t stride_V, int64_t tokens,
                           int64_t seqs, int64_t kv_heads, int64_t head_dim, int dtype, const int32_t* table,
                           int64_t table_width, const int32_t* lens, const int32_t* starts, uint16_t* Kpool,
                           uint16_t* Vpool, int64_t pages, int64_t page_size, hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, kv_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs) return fail(SLIM_EINVAL, "slim_kv_append: without starts tokens must equal seqs");
    if (tokens == 0) return slim::done();
    if (seqs == 0) return fail(SLIM_EINVAL, "slim_kv_append: tokens without sequences");
    st = check_rows("K", K, stride_K, tokens, kv_heads * head_dim);
    if (st == SLIM_OK) st = check_rows("V", V, stride_V, tokens, kv_heads * head_dim);
    slim::AppendArgs a;
    if (st == SLIM_OK)
        st = check_cache(seqs, kv_heads, head_dim, Kpool, Vpool, pages, page_size, table, table_width, lens, starts,
                         &a.kv);
    if (st == SLIM_OK) st = slim::check_device();
    if (st != SLIM_OK) return st;
    a.k_new = K; a.sk = stride_K;
    a.v_new = V; a.sv = stride_V;
    a.tokens = (int32_t)tokens; a.kv_heads = (int32_t)kv_heads; a.head_dim = (int32_t)head_dim;
    return slim::launched(slim::launch_kv_append(a, stream), "slim_kv_append launch");
}

slim_status slim_kv_copy_pages(void* Kpool, void* Vpool, int64_t layers, int64_t pages, int64_t page_bytes,
                               const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream) {
    if (layers <= 0 || layers > 4096 || pages <= 0 || pages > kMaxDim || n < 0 || n > kMaxDim)
        return fail(SLIM_EINVAL, "slim_kv_copy_pages: layers, pages or n out of range");
    if (page_bytes <= 0 || page_bytes % 16 || page_bytes > kMaxPageBytes)
        return fail(SLIM_EINVAL, "slim_kv_copy_pages: page_bytes must be a positive multiple of 16, at most 2^30 (got %lld)",
                    (long long)page_bytes);
    if (n == 0) return slim::done();
    if (!Kpool || !Vpool || !src || !dst) return fail(SLIM_EINVAL, "slim_kv_copy_pages: NULL pointer");
    if (!aligned16(Kpool) || !aligned16(Vpool) || !aligned4(src) || !aligned4(dst))
        return fail(SLIM_EINVAL, "slim_kv_copy_pages: pools must be 16-byte aligned, src and dst 4-byte aligned");
    slim_status st = slim::check_device();
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_kv_copy_pages(Kpool, Vpool, layers, pages, page_bytes, src, dst, n, stream),
                          "slim_kv_copy_pages launch");
}

size_t slim_attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                                      int64_t head_dim) {
    if (!head_dim_ok(head_dim) || tokens < 0 || tokens > kMaxTokens || seqs < 0 || seqs > kMaxTokens || kv_heads <= 0 ||
        q_heads <= 0 || q_heads > kMaxHeads || q_heads % kv_heads)
        return 0;
    return slim::attention_workspace_bytes(tokens, seqs, q_heads, kv_heads, head_dim);
}

slim_status slim_attention_decode(const uint16_t* Q, int64_t stride_Q, uint16_t* O, int64_t stride_O, float* lse,
                                  int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int dtype,
                                  const uint16_t* Kpool, const uint16_t* Vpool, int64_t pages, int64_t page_size,
                                  const int32_t* table, int64_t table_width, const int32_t* lens, int64_t max_len,
                                  int64_t window, int64_t sinks, float scale, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
    slim_status st = check_shape(seqs, seqs, q_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (seqs == 0) return slim::done();
    slim::AttnArgs a;
    st = check_attention(Q, stride_Q, O, stride_O, lse, seqs, seqs, q_heads, kv_heads, head_dim, dtype, Kpool, Vpool,
                         pages, page_size, table, table_width, lens, nullptr, max_len, window, sinks, scale, workspace,
                         workspace_bytes, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_attention_decode(a, stream), "slim_attention_decode launch");
}

slim_status slim_attention_prefill(const uint16_t* Q, int64_t stride_Q, uint16_t* O, int64_t stride_O, float* lse,
                                   int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                   int dtype, const uint16_t* Kpool, const uint16_t* Vpool, int64_t pages,
                                   int64_t page_size, const int32_t* table, int64_t table_width, const int32_t* lens,
                                   const int32_t* starts, int64_t max_len, int64_t window, int64_t sinks, float scale,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, q_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs)
        return fail(SLIM_EINVAL, "slim_attention_prefill: without starts tokens must equal seqs");
    if (tokens == 0) return slim::done();
    slim::AttnArgs a;
    st = check_attention(Q, stride_Q, O, stride_O, lse, tokens, seqs, q_heads, kv_heads, head_dim, dtype, Kpool, Vpool,
                         pages, page_size, table, table_width, lens, starts, max_len, window, sinks, scale, workspace,
                         workspace_bytes, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_attention_prefill(a, stream), "slim_attention_prefill launch");
}

slim_status slim_rope(const uint16_t* X, int64_t stride_X, uint16_t* Y, int64_t stride_Y, int64_t tokens, int64_t heads,
                      int64_t head_dim, int dtype, const int32_t* positions, const slim_rotation* rotation,
                      hipStream_t stream) {
    if (dtype != SLIM_FP16 && dtype != SLIM_BF16) return fail(SLIM_EUNSUPPORTED, "unknown dtype %d", dtype);
    if (head_dim <= 0 || head_dim % 8 || head_dim > 1024)
        return fail(SLIM_EUNSUPPORTED, "slim_rope: head_dim must be a multiple of 8 up to 1024 (got %lld)", (long long)head_dim);
    if (tokens < 0 || tokens > kMaxTokens) return fail(SLIM_EINVAL, "tokens must be in [0, 2^22] (got %lld)", (long long)tokens);
    if (heads <= 0 || heads > kMaxHeads) return fail(SLIM_EINVAL, "heads must be in [1, 1024] (got %lld)", (long long)heads);
    slim::RopeArgs a;
    slim_status st = check_rotation(rotation, head_dim, &a.by);
    if (st != SLIM_OK) return st;
    if (tokens == 0) return slim::done();
    st = check_rows("X", X, stride_X, tokens, heads * head_dim);
    if (st == SLIM_OK) st = check_rows("Y", Y, stride_Y, tokens, heads * head_dim);
    if (st == SLIM_OK) st = check_in_place("X", X, stride_X, Y, stride_Y);
    if (st != SLIM_OK) return st;
    if (!positions || !aligned4(positions)) return fail(SLIM_EINVAL, "positions must be given, 4-byte aligned");
    st = slim::check_device();
    if (st != SLIM_OK) return st;
    a.x = X; a.sx = stride_X;
    a.y = Y; a.sy = stride_Y;
    a.positions = positions;
    a.tokens = (int32_t)tokens; a.heads = (int32_t)heads; a.head_dim = (int32_t)head_dim;
    a.dtype = dtype;
    return slim::launched(slim::launch_rope(a, stream), "slim_rope launch");
}

slim_status slim_kv_append_rope(const uint16_t* Q, int64_t stride_Q, uint16_t* Qout, int64_t stride_Qout, int64_t q_heads,
                                const uint16_t* K, int64_t stride_K, const uint16_t* V, int64_t stride_V, int64_t tokens,
                                int64_t seqs, int64_t kv_heads, int64_t head_dim, int dtype, const int32_t* table,
                                int64_t table_width, const int32_t* lens, const int32_t* starts, uint16_t* Kpool,
                                uint16_t* Vpool, int64_t pages, int64_t page_size, const slim_rotation* rotation,
                                hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, Q ? q_heads : kv_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs) return fail(SLIM_EINVAL, "slim_kv_append_rope: without starts tokens must equal seqs");
    if (!rotation) return fail(SLIM_EINVAL, "rotation is NULL");
    if (tokens == 0) return slim::done();
    slim::AppendRopeArgs a;
    st = check_append_rope(Q, stride_Q, Qout, stride_Qout, q_heads, K, stride_K, V, stride_V, tokens, seqs, kv_heads,
                           head_dim, table, table_width, lens, starts, Kpool, Vpool, pages, page_size, rotation, dtype, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_kv_append_rope(a, stream), "slim_kv_append_rope launch");
}

size_t slim_q4_page_bytes(int64_t kv_heads, int64_t page_size, int64_t head_dim) {
    if (kv_heads <= 0 || kv_heads > kMaxHeads || page_shift(page_size) < 0 || !head_dim_ok(head_dim)) return 0;
    return (size_t)(kv_heads * page_size * head_dim * 17 / 32);
}

slim_status slim_kv_append_q4(const uint16_t* Q, int64_t stride_Q, uint16_t* Qout, int64_t stride_Qout, int64_t q_heads,
                              const uint16_t* K, int64_t stride_K, const uint16_t* V, int64_t stride_V, int64_t tokens,
                              int64_t seqs, int64_t kv_heads, int64_t head_dim, int dtype, const int32_t* table,
                              int64_t table_width, const int32_t* lens, const int32_t* starts, uint8_t* Kpool,
                              uint8_t* Vpool, int64_t pages, int64_t page_size, const slim_rotation* rotation,
                              hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, Q ? q_heads : kv_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs) return fail(SLIM_EINVAL, "slim_kv_append_q4: without starts tokens must equal seqs");
    if (tokens == 0) return slim::done();
    slim::AppendRopeArgs a;
    st = check_append_rope(Q, stride_Q, Qout, stride_Qout, q_heads, K, stride_K, V, stride_V, tokens, seqs, kv_heads,
                           head_dim, table, table_width, lens, starts, Kpool, Vpool, pages, page_size, rotation, dtype, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_kv_append_q4(a, stream), "slim_kv_append_q4 launch");
}

slim_status slim_kv_read_q4(uint16_t* K, int64_t stride_K, uint16_t* V, int64_t stride_V, int64_t tokens, int64_t seqs,
                            int64_t kv_heads, int64_t head_dim, int dtype, const int32_t* table, int64_t table_width,
                            const int32_t* lens, const int32_t* starts, const uint8_t* Kpool, const uint8_t* Vpool,
                            int64_t pages, int64_t page_size, hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, kv_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs) return fail(SLIM_EINVAL, "slim_kv_read_q4: without starts tokens must equal seqs");
    if (tokens == 0) return slim::done();
    slim::AppendRopeArgs a;
    st = check_append_rope(nullptr, 0, nullptr, 0, 0, K, stride_K, V, stride_V, tokens, seqs, kv_heads, head_dim, table,
                           table_width, lens, starts, Kpool, Vpool, pages, page_size, nullptr, dtype, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_kv_read_q4(a.to, dtype, stream), "slim_kv_read_q4 launch");
}

slim_status slim_attention_decode_q4(const uint16_t* Q, int64_t stride_Q, uint16_t* O, int64_t stride_O, float* lse,
                                     int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int dtype,
                                     const uint8_t* Kpool, const uint8_t* Vpool, int64_t pages, int64_t page_size,
                                     const int32_t* table, int64_t table_width, const int32_t* lens, int64_t max_len,
                                     int64_t window, int64_t sinks, float scale, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
    slim_status st = check_shape(seqs, seqs, q_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (seqs == 0) return slim::done();
    slim::AttnArgs a;
    st = check_attention(Q, stride_Q, O, stride_O, lse, seqs, seqs, q_heads, kv_heads, head_dim, dtype,
                         reinterpret_cast<const uint16_t*>(Kpool), reinterpret_cast<const uint16_t*>(Vpool), pages,
                         page_size, table, table_width, lens, nullptr, max_len, window, sinks, scale, workspace,
                         workspace_bytes, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_attention_decode_q4(a, stream), "slim_attention_decode_q4 launch");
}

slim_status slim_attention_prefill_q4(const uint16_t* Q, int64_t stride_Q, uint16_t* O, int64_t stride_O, float* lse,
                                      int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                      int dtype, const uint8_t* Kpool, const uint8_t* Vpool, int64_t pages,
                                      int64_t page_size, const int32_t* table, int64_t table_width, const int32_t* lens,
                                      const int32_t* starts, int64_t max_len, int64_t window, int64_t sinks, float scale,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
    slim_status st = check_shape(tokens, seqs, q_heads, kv_heads, head_dim, dtype);
    if (st != SLIM_OK) return st;
    if (!starts && tokens != seqs)
        return fail(SLIM_EINVAL, "slim_attention_prefill_q4: without starts tokens must equal seqs");
    if (tokens == 0) return slim::done();
    slim::AttnArgs a;
    st = check_attention(Q, stride_Q, O, stride_O, lse, tokens, seqs, q_heads, kv_heads, head_dim, dtype,
                         reinterpret_cast<const uint16_t*>(Kpool), reinterpret_cast<const uint16_t*>(Vpool), pages,
                         page_size, table, table_width, lens, starts, max_len, window, sinks, scale, workspace,
                         workspace_bytes, &a);
    if (st != SLIM_OK) return st;
    return slim::launched(slim::launch_attention_prefill_q4(a, stream), "slim_attention_prefill_q4 launch");
}

}  // extern "C"
