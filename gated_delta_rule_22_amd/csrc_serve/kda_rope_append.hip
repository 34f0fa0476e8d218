// Queries and keys of new tokens rotated by their positions, keys and values
// into their slots of the paged cache. Bound by memory: every row is read once
// and written once.
#include "kda_rope.h"

namespace kda {
namespace {

template <typename T, bool NT>
__global__ __launch_bounds__(64 * kRopeWaves) void rope_append_kernel(RopeAppendArgs a, int first,
                                                                      int per_token) {
    __shared__ float2 cs_all[kRopeWaves][kRopePairs];
    typedef Vec<T> V;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    // per_token waves share a token's rows
    const int tokens = kRopeWaves / per_token;
    const long t = first + (long)blockIdx.x * tokens + wave / per_token;
    if (t >= a.T) return;
    const long position = token_position(a.cu, a.kept, a.B, a.T, (int)t);
    if (position < 0) return;
    rope_angles(a.rope, position, cs_all[wave]);
    const int units = a.d / (2 * kVec<T>);           // of a row: 1 .. 16
    const RopeUnit<T> unit(a.rope, lane & (units - 1), cs_all[wave]);
    const int slot = a.Hkv ? a.slots[t] : -1;
    const bool cached = (unsigned)slot < (unsigned)(a.pool << a.page_shift);
    const long page = slot >> a.page_shift;
    const int at = slot & ((1 << a.page_shift) - 1);
    const int step = 64 / units * per_token, rows = a.Hq + (cached ? 2 * a.Hkv : 0);
    for (int r = (wave % per_token) * (64 / units) + lane / units; r < rows; r += step) {
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
        V x = load_vec<NT>((const V*)(from + unit.a)), y = load_vec<NT>((const V*)(from + unit.b));
        if (r < a.Hq + a.Hkv) unit.apply(x, y);
        store_vec<NT>((V*)(to + unit.a), x);
        store_vec<NT>((V*)(to + unit.b), y);
    }
}

}  // namespace

hipError_t launch_rope_append(const RopeAppendArgs& a, hipStream_t st) {
    const int per_token = a.T <= 4096 ? kRopeWaves : 1;
    const int tokens = kRopeWaves / per_token;
    const auto run = [&](auto kernel) {
        for (long t = 0; t < a.T; t += kRopeGrid * tokens) {
            const long n = a.T - t < kRopeGrid * tokens ? a.T - t : kRopeGrid * tokens;
            kernel<<<(unsigned)((n + tokens - 1) / tokens), 64 * kRopeWaves, 0, st>>>(a, (int)t, per_token);
        }
    };
    if (a.bf16_io) run(rope_append_kernel<bf16, false>);
    else run(rope_append_kernel<float, false>);
    return hipGetLastError();
}

}  // namespace kda
