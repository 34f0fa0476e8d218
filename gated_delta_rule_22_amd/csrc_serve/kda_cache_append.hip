// Keys and values of new tokens into their slots of the paged cache: a copy
// of rows, 16 bytes a thread, bound by memory. A token's row over all heads is
// contiguous in k and v; in the cache each head's part goes to its own page
// plane. 65,536 tokens of 8 heads of 128 in fp32 (1.07 GB read and written):
// 184 us, 5.8 TB/s.
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
// 1024 pieces a workgroup (4096: 216 us in the call above, 7 instead of 4 us
// for 256 tokens).
constexpr int kPieces = 1024;
// What is moved beyond twice the last-level cache (256 MB) bypasses it:
// 208 -> 184 us above. Less stays in it for the attention that reads it next.
constexpr size_t kStreamBytes = (size_t)512 << 20;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool NT>
__device__ __forceinline__ void move(u32x4* to, const u32x4* from) {
    if (NT) __builtin_nontemporal_store(__builtin_nontemporal_load(from), to);
    else *to = *from;
}

template <bool NT>
__global__ __launch_bounds__(kThreads) void cache_append_kernel(
    const u32x4* __restrict__ k, const u32x4* __restrict__ v, const int* __restrict__ slots,
    u32x4* __restrict__ kc, u32x4* __restrict__ vc, int T, int Hkv, int row16, int page_shift,
    int pool, int tokens) {
    const long t0 = (long)blockIdx.x * tokens;
    const int per_token = Hkv * row16;
    const int here = (int)(T - t0 < tokens ? T - t0 : tokens);
    const int slots_all = pool << page_shift;
    for (int x = threadIdx.x; x < here * per_token; x += kThreads) {
        const int t = x / per_token, y = x - t * per_token;
        const int h = y / row16, piece = y - h * row16;
        const int s = slots[t0 + t];
        if ((unsigned)s >= (unsigned)slots_all) continue;
        const long page = s >> page_shift;
        const int row = s & ((1 << page_shift) - 1);
        const long to = (((page * Hkv + h) << page_shift) + row) * row16 + piece;
        const long from = (t0 + t) * per_token + y;
        move<NT>(kc + to, k + from);
        move<NT>(vc + to, v + from);
    }
}

}  // namespace

hipError_t launch_cache_append(const void* k, const void* v, const int* slots, void* kc,
                               void* vc, int T, int Hkv, int row_bytes, int page_shift,
                               int pool, hipStream_t st) {
    const int row16 = row_bytes / 16;
    const long per_token = (long)Hkv * row16;
    const int tokens = per_token >= kPieces ? 1 : (int)(kPieces / per_token);
    // a grid holds fewer than 2^32 threads
    const long most = ((long)1 << 23) * tokens;
    const auto run = [&](auto kernel) {
        for (long t = 0; t < T; t += most) {
            const int n = (int)(T - t < most ? T - t : most);
            kernel<<<(unsigned)(((long)n + tokens - 1) / tokens), kThreads, 0, st>>>(
                (const u32x4*)k + t * per_token, (const u32x4*)v + t * per_token, slots + t, (u32x4*)kc,
                (u32x4*)vc, n, Hkv, row16, page_shift, pool, tokens);
        }
    };
    if (4 * (size_t)T * Hkv * row_bytes > kStreamBytes) run(cache_append_kernel<true>);
    else run(cache_append_kernel<false>);
    return hipGetLastError();
}

}  // namespace kda
