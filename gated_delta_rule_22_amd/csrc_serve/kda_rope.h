// Rotation by positions, as the appending kernels do it: a wave has a token,
// finds its request and position, makes the angles' cosines and sines once, a
// pair a lane, and turns the rows of all heads with them.
#pragma once

#include "kda_full_launch.h"

namespace kda {
namespace {

constexpr int kRopeWaves = 4;      // of a workgroup
constexpr int kRopePairs = 64;     // rot is at most 128

// Position of packed row t, or -1 outside all requests: the last i with
// cu[i] <= t, found 64 ways at a time (two steps for up to 4095 requests).
// Offsets that decrease may give any i; it is checked.
__device__ __forceinline__ long token_position(const int* cu, const int* kept, int B, int T, int t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B + 1;         // candidates lo .. lo + n - 1
    while (n > 1) {
        const int step = (int)(((long)n + 63) / 64);
        const bool in = (long)lane * step < n;
        const int x = cu[lo + (in ? lane * step : 0)];
        const unsigned long long below = __ballot(in && x <= t);
        if (!below) return -1;
        const int k = 63 - __builtin_clzll(below);
        lo += k * step;
        n = min(step, n - k * step);
    }
    if (lo >= B || !(cu[lo] <= t && t < cu[lo + 1])) return -1;
    return (long)max(kept[lo], 0) + (t - max(cu[lo], 0));
}

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T> using Vec = T __attribute__((ext_vector_type(16 / sizeof(T))));

// cos and sin of the token's pairs, in the wave's own part of LDS. Angles and
// their functions are fp64: at a position of 2^20 an fp32 angle of the fastest
// pair is off by 2^-5. They cost nothing where a wave has 16 rows or more to
// move; all is bound by memory.
__device__ __forceinline__ void rope_angles(const RopeArgs& r, long position, float2* cs) {
    const int lane = threadIdx.x & 63;
    if (lane < r.rot / 2) {
        double s, c;
        sincos((double)position * r.freqs[lane], &s, &c);
        cs[lane] = make_float2((float)(c * (double)r.factor), (float)(s * (double)r.factor));
    }
    lds_fence_wave();
}

// A lane's part of a row: two vectors of 16 bytes that hold the kVec pairs
// kVec u .. of the rotated channels, or channels behind them.
template <typename T>
struct RopeUnit {
    static constexpr int V = kVec<T>;
    int a, b;                      // channels where the vectors begin
    bool turn, interleaved;
    float c[V], s[V];

    // unit u of a row; the first r.rot channels are rotated
    __device__ __forceinline__ RopeUnit(const RopeArgs& r, int u, const float2* cs) {
        turn = r.freqs && u * 2 * V < r.rot;
        interleaved = r.interleaved;
        const bool halves = turn && !interleaved;
        a = halves ? u * V : u * 2 * V;
        b = a + (halves ? r.rot / 2 : V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 x = turn ? cs[u * V + i] : make_float2(1.f, 0.f);
            c[i] = x.x;
            s[i] = x.y;
        }
    }
    __device__ __forceinline__ void apply(Vec<T>& x, Vec<T>& y) const {
        if (!turn) return;
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float p = to_f32(x[2 * i]), q = to_f32(x[2 * i + 1]);
                x[2 * i] = from_f32<T>(p * c[i] - q * s[i]);
                x[2 * i + 1] = from_f32<T>(q * c[i] + p * s[i]);
                const float u = to_f32(y[2 * i]), w = to_f32(y[2 * i + 1]);
                y[2 * i] = from_f32<T>(u * c[V / 2 + i] - w * s[V / 2 + i]);
                y[2 * i + 1] = from_f32<T>(w * c[V / 2 + i] + u * s[V / 2 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float p = to_f32(x[i]), q = to_f32(y[i]);
                x[i] = from_f32<T>(p * c[i] - q * s[i]);
                y[i] = from_f32<T>(q * c[i] + p * s[i]);
            }
        }
    }
};

// A grid holds fewer than 2^32 threads.
constexpr long kRopeGrid = (long)1 << 23;

}  // namespace
}  // namespace kda
