// Host-side driver for the sanitizer test of the rotation and the cache of 4
// bits (tests/test_host_sanitizers_rope.py): extreme sizes, strides, rotations
// and pointers that the boundary must reject before any device call.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "slim.h"

static int g_fail = 0;

static void expect(long line, slim_status got, slim_status want) {
    if (got != want || (got != SLIM_OK && strlen(slim_last_error()) == 0)) {
        fprintf(stderr, "FAIL line %ld: status %d (%s), want %d\n", line, (int)got, slim_last_error(), (int)want);
        ++g_fail;
    }
}
#define EXPECT(call, want) expect(__LINE__, (call), (want))

int main() {
    alignas(16) static unsigned char buf[256];
    uint16_t* P = (uint16_t*)buf;
    uint8_t* B = buf;
    int32_t* I = (int32_t*)buf;
    const double* F = (const double*)buf;
    const size_t WS = 1 << 30;
    const slim_rotation R = {F, 128, 0, 1.0f};
    const int64_t BIG = INT64_MAX, NEG = INT64_MIN;
    const int64_t odd[] = {BIG, NEG, -1, 0, BIG - 7};

    for (int64_t x : odd) {
        for (int64_t y : odd)
            if (slim_q4_page_bytes(x, y, 128) || slim_q4_page_bytes(x, 16, y) || slim_q4_page_bytes(1, x, y)) {
                fprintf(stderr, "FAIL size\n");
                ++g_fail;
            }
        const slim_status rows = x == 0 ? SLIM_OK : SLIM_EINVAL;       // no tokens: nothing to do
        const slim_rotation r = {F, x, 0, 1.0f};
        EXPECT(slim_rope(P, 256, P, 256, x, 2, 128, 0, I, &R, 0), rows);
        EXPECT(slim_rope(P, 256, P, 256, 2, x, 128, 0, I, &R, 0), SLIM_EINVAL);
        EXPECT(slim_rope(P, 256, P, 256, 2, 2, x, 0, I, &R, 0), SLIM_EUNSUPPORTED);
        EXPECT(slim_rope(P, x, P, x, 2, 2, 128, 0, I, &R, 0), SLIM_EINVAL);
        EXPECT(slim_rope(P, 256, P, 256, 2, 2, 128, 0, I, &r, 0), SLIM_EINVAL);

        EXPECT(slim_kv_append_rope(P, 512, P, 512, 4, P, 256, P, 256, x, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &R, 0), rows);
        EXPECT(slim_kv_append_rope(P, 512, P, 512, x, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &R, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_rope(P, x, P, x, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &R, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_rope(P, 512, P, 512, 4, P, 256, P, 256, 2, x, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &R, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_rope(P, 512, P, 512, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, x, I, I, P, P, 1, 16, &R, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_rope(P, 512, P, 512, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &r, 0), SLIM_EINVAL);

        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, 256, x, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, 0, 0), rows);
        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, x, 128, 0, I, 1, I, I, B, B, 1, 16, 0, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, x, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, 0, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, x, 16, 0, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, x, 0, 0), SLIM_EUNSUPPORTED);
        EXPECT(slim_kv_append_q4(P, 512, P, 512, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, &r, 0), SLIM_EINVAL);

        EXPECT(slim_kv_read_q4(P, 256, P, 256, x, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, 0), rows);
        EXPECT(slim_kv_read_q4(P, x, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_read_q4(P, 256, P, 256, 2, x, 2, 128, 0, I, 1, I, I, B, B, 1, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_read_q4(P, 256, P, 256, 2, 1, 2, x, 0, I, 1, I, I, B, B, 1, 16, 0), SLIM_EUNSUPPORTED);
        EXPECT(slim_kv_read_q4(P, 256, P, 256, 2, 1, 2, 128, 0, I, x, I, I, B, B, 1, 16, 0), SLIM_EINVAL);

        EXPECT(slim_attention_decode_q4(P, 512, P, 512, 0, x, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, WS, 0), rows);
        EXPECT(slim_attention_decode_q4(P, 512, P, 512, 0, 1, x, 2, 128, 0, B, B, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, WS, 0), SLIM_EINVAL);
        EXPECT(slim_attention_decode_q4(P, 512, P, 512, 0, 1, 4, 2, 128, 0, B, B, x, 16, I, 1, I, 1, 0, 0, 1.0f, P, WS, 0), SLIM_EINVAL);
        if (x != 0) {
            EXPECT(slim_attention_decode_q4(P, 512, P, 512, 0, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, x, 0, 0, 1.0f, P, WS, 0),
                   SLIM_EINVAL);
            EXPECT(slim_attention_prefill_q4(P, 512, P, 512, 0, x, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f, P, WS, 0),
                   SLIM_EINVAL);
            EXPECT(slim_attention_prefill_q4(P, 512, P, 512, 0, 2, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, I, 1, x, 0, 1.0f, P, WS, 0),
                   SLIM_EINVAL);
        }
        EXPECT(slim_attention_prefill_q4(P, 512, P, x, 0, 2, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f, P, WS, 0),
               SLIM_EINVAL);
    }
    // Rotations with parts missing, more positions than 2^30 (width times page), a
    // workspace that is too small.
    const slim_rotation bad[] = {{nullptr, 128, 0, 1.0f}, {F, 12, 0, 1.0f}, {F, 136, 0, 1.0f}, {F, 128, 2, 1.0f},
                                 {F, 128, -1, 1.0f}, {F, 128, 0, NAN}, {F, 128, 0, -INFINITY},
                                 {(const double*)(buf + 4), 128, 0, 1.0f}};
    for (const slim_rotation& r : bad) {
        EXPECT(slim_rope(P, 256, P, 256, 2, 2, 128, 0, I, &r, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_rope(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, &r, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append_q4(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, &r, 0), SLIM_EINVAL);
    }
    EXPECT(slim_rope(P, 256, P, 256, 2, 2, 128, 0, I, nullptr, 0), SLIM_EINVAL);
    EXPECT(slim_kv_append_rope(0, 0, 0, 0, 0, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, nullptr, 0), SLIM_EINVAL);
    EXPECT(slim_kv_append_q4(P, 512, nullptr, 512, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, &R, 0), SLIM_EINVAL);
    EXPECT(slim_kv_append_q4(P, 512, P, 512, 4, P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, B, B, 1, 16, nullptr, 0), SLIM_EINVAL);
    EXPECT(slim_kv_read_q4(P, 256, P, 256, 2, 1, 2, 128, 0, I, 1 << 27, I, I, B, B, 1, 16, 0), SLIM_EINVAL);
    EXPECT(slim_attention_prefill_q4(P, 512, P, 512, 0, 2, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1 << 27, I, I, 1, 0, 0, 1.0f, P, WS, 0),
           SLIM_EINVAL);
    EXPECT(slim_attention_decode_q4(P, 512, P, 512, 0, 1, 4, 2, 128, 0, B, B, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, 1000, 0), SLIM_EINVAL);
    if (g_fail) return 1;
    printf("abi sanitize rope: all checks passed\n");
    return 0;
}
