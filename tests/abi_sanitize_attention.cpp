// Host-side driver for the sanitizer test of the cache and attention entry
// points (tests/test_host_sanitizers_attention.py): extreme sizes, strides and
// pointers that the boundary must reject before any device call.
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
    int32_t* I = (int32_t*)buf;
    const int64_t BIG = INT64_MAX, NEG = INT64_MIN;
    const int64_t odd[] = {BIG, NEG, -1, 0, BIG - 7};

    for (int64_t x : odd) {
        for (int64_t y : odd) {
            if (x != 0 && slim_attention_workspace_bytes(x, y, x, y, 128) != 0) { ++g_fail; fprintf(stderr, "FAIL size\n"); }
            if (slim_attention_workspace_bytes(1, 1, 4, x == 0 ? -1 : x, y) != 0) { ++g_fail; fprintf(stderr, "FAIL size 2\n"); }
        }
        const slim_status rows = x == 0 ? SLIM_OK : SLIM_EINVAL;       // no tokens: nothing to do
        EXPECT(slim_kv_append(P, 256, P, 256, x, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, 0), rows);
        EXPECT(slim_kv_append(P, 256, P, 256, 2, x, 2, 128, 0, I, 1, I, I, P, P, 1, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append(P, x == 0 ? 8 : x, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append(P, 256, P, 256, 2, 1, 2, 128, 0, I, x, I, I, P, P, 1, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append(P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, x, 16, 0), SLIM_EINVAL);
        EXPECT(slim_kv_append(P, 256, P, 256, 2, 1, 2, 128, 0, I, 1, I, I, P, P, 1, x, 0), SLIM_EUNSUPPORTED);
        EXPECT(slim_kv_copy_pages(P, P, x, 1, 16, I, I, 1, 0), SLIM_EINVAL);
        EXPECT(slim_kv_copy_pages(P, P, 1, x, 16, I, I, 1, 0), SLIM_EINVAL);
        EXPECT(slim_kv_copy_pages(P, P, 1, 1, x, I, I, 1, 0), SLIM_EINVAL);
        EXPECT(slim_kv_copy_pages(P, P, 1, 1, 16, I, I, x, 0), rows);
        EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, x, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, 1 << 30, 0),
               rows);
        EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, x, 2, 128, 0, P, P, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, 1 << 30, 0),
               SLIM_EINVAL);
        EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, 4, x, 128, 0, P, P, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, 1 << 30, 0),
               SLIM_EINVAL);
        EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, 4, 2, x, 0, P, P, 1, 16, I, 1, I, 1, 0, 0, 1.0f, P, 1 << 30, 0),
               SLIM_EUNSUPPORTED);
        if (x != 0) {
            EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, x, 0, 0, 1.0f, P, 1 << 30, 0),
                   SLIM_EINVAL);
            EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, 1, x, 0, 1.0f, P, 1 << 30, 0),
                   SLIM_EINVAL);
            EXPECT(slim_attention_decode(P, 512, P, 512, nullptr, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, 1, 0, x, 1.0f, P, 1 << 30, 0),
                   SLIM_EINVAL);
            EXPECT(slim_attention_prefill(P, 512, P, 512, nullptr, x, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f, P,
                                          1 << 30, 0), SLIM_EINVAL);
        }
        EXPECT(slim_attention_prefill(P, 512, P, x == 0 ? 8 : x, nullptr, 2, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f,
                                      P, 1 << 30, 0), SLIM_EINVAL);
        EXPECT(slim_attention_prefill(P, 512, P, 512, nullptr, 2, x, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f, P, 1 << 30,
                                      0), SLIM_EINVAL);
    }
    EXPECT(slim_attention_prefill(P, 512, P, 512, nullptr, 2, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1 << 26, I, I, 1, 0, 0, 1.0f, P, 1 << 30,
                                  0), SLIM_EINVAL);          // more positions than 2^30 (width times page)
    EXPECT(slim_attention_prefill(P, 512, P, 512, nullptr, 2, 1, 4, 2, 128, 0, P, P, 1, 16, I, 1, I, I, 1, 0, 0, 1.0f, P, 1000, 0),
           SLIM_EINVAL);                                     // workspace too small
    if (g_fail) return 1;
    printf("abi sanitize attention: all checks passed\n");
    return 0;
}
