// Internal interface of the paged key-value cache and the attention that
// reads it (contract of every call: include/slim.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace slim {

// One layer's pool and the sequences' places in it.
struct PagedKV {
    const uint16_t* k;       // [pages][kv_heads][1 << page_shift][head_dim], or pages of 4 bits (kv_q4.hpp)
    const uint16_t* v;
    const int32_t* table;    // [seqs][width]
    const int32_t* lens;     // [seqs]
    const int32_t* starts;   // [seqs + 1], or NULL: one new token per sequence
    int32_t pages, width, seqs;
    int32_t page_shift;
};

struct AttnArgs {
    PagedKV kv;
    const uint16_t* q;  int64_t sq;
    uint16_t* o;        int64_t so;
    float* lse;              // [tokens][q_heads] or NULL
    int32_t tokens, q_heads, kv_heads, head_dim;
    int32_t dtype;           // slim_dtype
    int32_t max_len;         // expected longest length (split planning only)
    int32_t window, sinks;   // window 0: all positions up to the query's
    float scale;
    unsigned char* ws;
};

struct AppendArgs {
    PagedKV kv;              // k, v: the pools that are written
    const uint16_t* k_new;  int64_t sk;
    const uint16_t* v_new;  int64_t sv;
    int32_t tokens, kv_heads, head_dim;
};

// Rotary positions; half 0: none.
struct Rotation {
    const double* freqs;     // [half], radians a position
    int32_t half;            // pairs of a head
    int32_t interleaved;
    double magnitude;
};

struct RopeArgs {
    const uint16_t* x;  int64_t sx;
    uint16_t* y;        int64_t sy;
    const int32_t* positions;
    int32_t tokens, heads, head_dim;
    int32_t dtype;
    Rotation by;
};

// New keys (turned on the way) and values to their pages, queries beside them.
struct AppendRopeArgs {
    AppendArgs to;
    const uint16_t* q;  int64_t sq;      // NULL: none
    uint16_t* q_out;    int64_t sqo;
    int32_t q_heads;                     // 0 where q is NULL
    int32_t dtype;
    Rotation by;
};

// Workspace: the partial results of split key axes, for at most
// kAttnSplitRows (row, split) pairs: a call splits its rows no further than
// that, whatever its plan would be.
constexpr int64_t kAttnSplitRows = 32768;

size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim);
hipError_t launch_attention_decode(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_prefill(const AttnArgs& a, hipStream_t stream);
// Joins the partial results of a call's rows, `splits` each.
hipError_t launch_attention_join(const AttnArgs& a, int splits, hipStream_t stream);
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream);
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);
hipError_t launch_kv_append_rope(const AppendRopeArgs& a, hipStream_t stream);
// The same calls on pages of 4 bits.
hipError_t launch_kv_append_q4(const AppendRopeArgs& a, hipStream_t stream);
// k_new, v_new are written.
hipError_t launch_kv_read_q4(const AppendArgs& a, int dtype, hipStream_t stream);
hipError_t launch_attention_decode_q4(const AttnArgs& a, hipStream_t stream);
// Prompts of which each has a few new rows on a key head (few_rows_q4).
bool few_rows_q4(const AttnArgs& a);
hipError_t launch_attention_few_q4(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_prefill_q4(const AttnArgs& a, hipStream_t stream);
hipError_t launch_kv_copy_pages(void* k, void* v, int64_t layers, int64_t pages, int64_t page_bytes,
                                const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream);

}  // namespace slim
