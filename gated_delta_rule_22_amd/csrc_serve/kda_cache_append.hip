// Keys and values of new tokens into their slots of the paged cache: a copy
// of rows, 16 bytes a thread. A token's row over all heads is contiguous in
// k and v; in the cache each head's part goes to its own page plane.
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void cache_append_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, const int* __restrict__ slots,
    uint4* __restrict__ kc, uint4* __restrict__ vc, int T, int Hkv, int row16, int page_shift,
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
        kc[to] = k[from];
        vc[to] = v[from];
    }
}

}  // namespace

hipError_t launch_cache_append(const void* k, const void* v, const int* slots, void* kc,
                               void* vc, int T, int Hkv, int row_bytes, int page_shift,
                               int pool, hipStream_t st) {
    const int row16 = row_bytes / 16;
    const long per_token = (long)Hkv * row16;
    const int tokens = per_token >= 1024 ? 1 : (int)(1024 / per_token);
    const long grid = ((long)T + tokens - 1) / tokens;
    cache_append_kernel<<<(unsigned)grid, kThreads, 0, st>>>(
        (const uint4*)k, (const uint4*)v, slots, (uint4*)kc, (uint4*)vc, T, Hkv, row16,
        page_shift, pool, tokens);
    return hipGetLastError();
}

}  // namespace kda
