// Data movement of the paged key-value cache: writing new keys and values to
// the pages of their positions, and copying whole pages.
#include "attention_util.hpp"
#include "mfma_util.hpp"

namespace slim {
namespace {

constexpr int kThreads = 256;

// One workgroup moves the vectors [kThreads * U * blockIdx.y, ...) of one
// token's new rows: 16-byte vector i < row is of the key, row <= i < 2 row of
// the value (row = kv_heads * head_dim / 8).  Nothing is computed: bound by
// HBM for prompts, by launch and the chain starts -> lens -> table -> store
// for single tokens.  Each wave finds its sequence itself (find_seq), which
// costs one load for up to 64 sequences.  Measured, 32 heads of 128: 8763
// tokens 59 us (4.8 TB/s; a plain copy of a GiB moves 5.7), 64 tokens 3 us.  U vectors a
// thread: 4 where there are workgroups enough (more loads in flight), 1 for up to 512
// tokens.
template <int U>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
    const int t = blockIdx.x;
    const uint32_t dv = (uint32_t)a.head_dim >> 3, row = (uint32_t)a.kv_heads * dv;
    const uint32_t at = blockIdx.y * (kThreads * U) + threadIdx.x;
    u4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = at + u * kThreads;
        if (i < 2 * row) {
            const uint16_t* p = i < row ? a.k_new + t * a.sk + (int64_t)i * 8 : a.v_new + t * a.sv + (int64_t)(i - row) * 8;
            x[u] = *reinterpret_cast<const u4*>(p);
        }
    }
    const int b = find_seq(a.kv, t);
    if (b < 0) return;
    int pos = seq_len(a.kv, b) - 1;
    if (a.kv.starts) pos += 1 + t - a.kv.starts[b + 1];
    const int page_at = pos >> a.kv.page_shift;
    if (pos < 0 || page_at >= a.kv.width) return;
    const int page = a.kv.table[(int64_t)b * a.kv.width + page_at];
    if (page < 0 || page >= a.kv.pages) return;
    const int r = pos & ((1 << a.kv.page_shift) - 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t i = at + u * kThreads;
        if (i < 2 * row) {
            uint16_t* pool = const_cast<uint16_t*>(i < row ? a.kv.k : a.kv.v);
            i = i < row ? i : i - row;
            const uint32_t h = i / dv, e = i - h * dv;
            const int64_t to = ((((int64_t)page * a.kv_heads + h) << a.kv.page_shift) + r) * dv + e;
            *reinterpret_cast<u4*>(pool + to * 8) = x[u];
        }
    }
}

// One workgroup copies kCopyBytes of one page of one layer's K or V, four
// 16-byte loads a lane in flight.  Bound by HBM: 45 pages of 128 KB in 32 layers,
// 755 MB read and written, 145 us, 5.2 TB/s; one page of 32 KB in 32 layers 3.3 us.
constexpr int kCopyU = 4;
constexpr int kCopyBytes = kThreads * kCopyU * 16;

__global__ __launch_bounds__(kThreads) void kv_copy_kernel(unsigned char* k, unsigned char* v, int layers, int pages,
                                                           int64_t page_bytes, const int32_t* src, const int32_t* dst,
                                                           int parts) {
    // blockIdx.x = part of a page, fastest, then the pair; blockIdx.y = layer and array.
    const int pair = blockIdx.x / parts, part = blockIdx.x - pair * parts;
    const int from = src[pair], to = dst[pair];
    if (from < 0 || from >= pages || to < 0 || to >= pages) return;
    unsigned char* pool = (blockIdx.y & 1) ? v : k;
    const int64_t layer = (int64_t)(blockIdx.y >> 1) * pages;
    const unsigned char* s = pool + (layer + from) * page_bytes;
    unsigned char* d = pool + (layer + to) * page_bytes;
    const int64_t at = (int64_t)part * kCopyBytes + threadIdx.x * 16;
    u4 x[kCopyU];
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (at + u * (kThreads * 16) < page_bytes) x[u] = *reinterpret_cast<const u4*>(s + at + u * (kThreads * 16));
#pragma unroll
    for (int u = 0; u < kCopyU; ++u)
        if (at + u * (kThreads * 16) < page_bytes) *reinterpret_cast<u4*>(d + at + u * (kThreads * 16)) = x[u];
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t stream) {
    const int vectors = a.kv_heads * a.head_dim / 8 * 2;
    if (a.tokens <= 512) {
        dim3 grid((unsigned)a.tokens, (unsigned)((vectors + kThreads - 1) / kThreads));
        hipLaunchKernelGGL(kv_append_kernel<1>, grid, dim3(kThreads), 0, stream, a);
    } else {
        dim3 grid((unsigned)a.tokens, (unsigned)((vectors + 4 * kThreads - 1) / (4 * kThreads)));
        hipLaunchKernelGGL(kv_append_kernel<4>, grid, dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_kv_copy_pages(void* k, void* v, int64_t layers, int64_t pages, int64_t page_bytes,
                                const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream) {
    const int64_t parts = (page_bytes + kCopyBytes - 1) / kCopyBytes;
    // A grid's x extent holds fewer than 2^32 threads; pairs past it go into further launches.
    const int64_t most = ((int64_t(1) << 32) / kThreads - 1) / parts;
    for (int64_t at = 0; at < n; at += most) {
        const int64_t count = n - at < most ? n - at : most;
        dim3 grid((unsigned)(count * parts), (unsigned)(2 * layers));
        hipLaunchKernelGGL(kv_copy_kernel, grid, dim3(kThreads), 0, stream, static_cast<unsigned char*>(k),
                           static_cast<unsigned char*>(v), (int)layers, (int)pages, page_bytes, src + at, dst + at,
                           (int)parts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace slim
