// Queries and keys of new tokens rotated by their positions, keys and values
// into their slots of the paged cache. Bound by memory: every row is read once
// and written once, 16 bytes a lane. 39612 tokens of 32 + 2 * 8 heads of 128, 974 MB:
// 185 us, 5.3 TB/s. (Loads and stores past the caches took 279 us there, where pairs of
// 32 bytes make each store half a line; with halves 139 instead of 146 us at 805 MB: not
// worth a second kernel.) Calls of up to 1024 tokens are a launch, 9.5 us.
#include "kda_rope.h"

namespace kda {
namespace {

template <typename T>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_append_kernel(RopeAppendArgs a, int first) {
    __shared__ float2 cs_all[kRopeWaves][kRopePairs];
    typedef Vec<T> V;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    // A workgroup's waves share a token's rows: as fast as a token a wave up to 4096
    // tokens, and 146 us instead of 154 with 32768 (32 + 2 * 8 heads of 128).
    const long t = first + (long)blockIdx.x;
    const long position = token_position(a.cu, a.kept, a.B, a.T, (int)t);
    if (position < 0) return;
    rope_angles(a.rope, position, cs_all[wave]);
    const int units = a.d / (2 * kVec<T>);           // of a row: 1 .. 16
    const RopeUnit<T> unit(a.rope, lane & (units - 1), cs_all[wave]);
    const int slot = a.Hkv ? a.slots[t] : -1;
    const bool cached = (unsigned)slot < (unsigned)(a.pool << a.page_shift);
    const long page = slot >> a.page_shift;
    const int at = slot & ((1 << a.page_shift) - 1);
    const int step = 64 / units * kRopeWaves, rows = a.Hq + (cached ? 2 * a.Hkv : 0);
    for (int r = wave * (64 / units) + lane / units; r < rows; r += step) {
        const T* from;
        T* to;
        if (r < a.Hq) {
            const long x = (t * a.Hq + r) * a.d;
            from = (const T*)a.q + x;
            to = (T*)a.q_out + x;
        } else {
            const bool key = r < a.Hq + a.Hkv;
            const int h = r - a.Hq - (key ? 0 : a.Hkv);
            from = (const T*)(key ? a.k : a.v) + (t * a.Hkv + h) * a.d;
            to = (T*)(key ? a.kc : a.vc) + (((page * a.Hkv + h) << a.page_shift) + at) * a.d;
        }
        V x = *(const V*)(from + unit.a), y = *(const V*)(from + unit.b);
        if (r < a.Hq + a.Hkv) unit.apply(x, y);
        *(V*)(to + unit.a) = x;
        *(V*)(to + unit.b) = y;
    }
}

}  // namespace

hipError_t launch_rope_append(const RopeAppendArgs& a, hipStream_t st) {
    const auto run = [&](auto kernel) {
        for (long t = 0; t < a.T; t += kRopeGrid) {
            const long n = a.T - t < kRopeGrid ? a.T - t : kRopeGrid;
            kernel<<<(unsigned)n, 64 * kRopeWaves, 0, st>>>(a, (int)t);
        }
    };
    if (a.bf16_io) run(rope_append_kernel<bf16>);
    else run(rope_append_kernel<float>);
    return hipGetLastError();
}

}  // namespace kda
