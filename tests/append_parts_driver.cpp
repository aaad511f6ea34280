// Host-side driver for tests/test_append_parts.py: the launches that calls of
// more waves than a grid holds are cut into.  The runtime's entry points below
// take the place of the library's, so nothing is launched: each launch's
// first token, end and grid are written down and joined to the tasks (a slice of a token)
// that its waves work on.  Every task must come up once: queries turned in place
// twice would be turned by twice the angle.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <map>
#include <string>

#include "attention.hpp"

namespace {

// (Filled before main, by what the compiler runs for each source.)
std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> all;
    return all;
}
dim3 g_grid, g_block;
int32_t g_positions[1];

// The call under test: its tasks are [0, g_tasks), those below g_next were taken once.
int64_t g_slices, g_next;
int g_launches, g_fail;

constexpr int kWaves = 4;                     // of a workgroup (256 threads)

// A launch's waves take tasks from token `first` on, those of tokens below `end`.
void took(int64_t first, int64_t end, int64_t slices) {
    const int64_t from = first * slices, waves = (int64_t)g_grid.x * kWaves;
    const int64_t to = from + waves < end * slices ? from + waves : end * slices;
    ++g_launches;
    if (g_block.x != 64 * kWaves || (int64_t)g_grid.x * g_block.x >= int64_t(1) << 32) {
        fprintf(stderr, "FAIL grid %u x %u\n", g_grid.x, g_block.x);
        ++g_fail;
    }
    if ((g_slices && g_slices != slices) || from != g_next) {
        fprintf(stderr, "FAIL launch %d begins with task %lld, %lld follows the last (%lld slices)\n", g_launches,
                (long long)from, (long long)g_next, (long long)slices);
        ++g_fail;
    }
    g_slices = slices;
    g_next = to;
}

void begin() { g_slices = g_next = g_launches = 0; }

void end(const char* what, int64_t tokens, bool parts) {
    if (g_next != tokens * g_slices || (g_launches > 1) != parts) {
        fprintf(stderr, "FAIL %s: %lld of %lld tasks in %d launches\n", what, (long long)g_next,
                (long long)(tokens * g_slices), g_launches);
        ++g_fail;
    }
    printf("%s: %lld tokens of %lld slices, %d launches\n", what, (long long)tokens, (long long)g_slices, g_launches);
}

}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* module; return &module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
    names()[host] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    g_grid = grid;
    g_block = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
    *grid = g_grid;
    *block = g_block;
    *lds = 0;
    *stream = 0;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipLaunchKernel(const void* kernel, dim3, dim3, void** args, size_t, hipStream_t) {
    const std::string& name = names()[kernel];
    auto number = [&](int i) { return (int64_t) * (const int32_t*)args[i]; };
    if (name.find("kv_append_rope_kernel") != std::string::npos)
        took(number(1), ((const slim::AppendRopeArgs*)args[0])->to.tokens, number(4));
    else if (name.find("kv_append_q4_kernel") != std::string::npos)
        took(number(1), ((const slim::AppendRopeArgs*)args[0])->to.tokens, number(6));
    else if (name.find("kv_read_q4_kernel") != std::string::npos)
        took(number(1), ((const slim::AppendArgs*)args[0])->tokens, number(2));
    else if (name.find("rope_kernel") != std::string::npos) {
        const slim::RopeArgs& a = *(const slim::RopeArgs*)args[0];
        const int64_t first = a.positions - g_positions;
        took(first, first + a.tokens, number(2));
    } else {
        fprintf(stderr, "FAIL unknown kernel %s\n", name.c_str());
        ++g_fail;
    }
    return hipSuccess;
}
}

int main() {
    static uint16_t rows[8];
    const int64_t kTokens = int64_t(1) << 22;
    for (int64_t tokens : {kTokens, kTokens - 1, int64_t(1001)})
        for (int half : {64, 12})             // vectors of 8 and of 4 elements
            for (int heads = 1; heads <= 60; ++heads) {
                slim::AppendRopeArgs a;
                memset((void*)&a, 0, sizeof a);
                a.by = slim::Rotation{nullptr, half, 0, 1.0};
                a.q = rows;
                a.q_out = rows;
                a.q_heads = heads;
                a.to.kv_heads = heads % 4 ? 1 : heads;
                a.to.head_dim = 128;
                a.to.tokens = (int32_t)tokens;
                const bool large = tokens > 1001;
                char what[64];
                auto of = [&](const char* call) {
                    snprintf(what, sizeof what, "%s, %d and %d heads, half %d", call, heads, a.to.kv_heads, half);
                    return what;
                };
                begin();
                slim::launch_kv_append_rope(a, 0);
                end(of("append_rope"), tokens, large && g_slices > 8);
                begin();
                slim::launch_kv_append_q4(a, 0);
                end(of("append_q4"), tokens, large && g_slices > 8);
                begin();
                a.to.kv_heads = heads;
                slim::launch_kv_read_q4(a.to, 0, 0);
                end(of("read_q4"), tokens, large && g_slices > 8);
                slim::RopeArgs r;
                memset((void*)&r, 0, sizeof r);
                r.x = rows;
                r.y = rows;
                r.positions = g_positions;
                r.tokens = (int32_t)tokens;
                r.heads = heads;
                r.head_dim = 128;
                r.by = a.by;
                begin();
                slim::launch_rope(r, 0);
                end(of("rope"), tokens, large && g_slices > 8);
            }
    if (g_fail) return 1;
    printf("every task once\n");
    return 0;
}
