// Latent rows of new tokens into their slots: c normalised, the positional part
// rotated, and the queries' positional part with it. Bound by memory:
// a token's row stays in registers between the sum of its squares and its scaling. fp32,
// 21414 tokens of 32 heads, 499 MB: 110 us, 4.5 TB/s; calls of up to 1024 tokens are a
// launch, 10.5 us.
#include "kda_rope.h"

namespace kda {
namespace {

// Sum over the 64 lanes, in all of them.
__device__ __forceinline__ double wave_sum(double x) {
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}

template <typename T>
__global__ __launch_bounds__(64 * kRopeWaves) void latent_append_kernel(LatentAppendArgs a, int first) {
    constexpr int V = kVec<T>, kMost = 512 / V / 64;  // vectors of c in a lane
    constexpr int kUnits = kPe / (2 * V);             // of a positional part
    typedef Vec<T> Vt;
    __shared__ float2 cs_all[kRopeWaves][kRopePairs];
    const int wave = wave_id(), lane = threadIdx.x & 63;
    // A token a wave: a workgroup a token is as fast up to 4096 tokens, and 113 us
    // instead of 96 with 32768 (bf16, 32 heads, 512 + 64 channels).
    const long t = first + (long)blockIdx.x * kRopeWaves + wave;
    if (t >= a.T) return;
    const long position = token_position(a.cu, a.kept, a.B, a.T, (int)t);
    if (position < 0) return;
    if (a.rope.freqs) rope_angles(a.rope, position, cs_all[wave]);
    const RopeUnit<T> unit(a.rope, lane % kUnits, cs_all[wave]);
    const int width = a.dc + kPe;
    const T* from = (const T*)a.kv + t * width;
    const int slot = a.slots[t];
    T* to = (unsigned)slot < (unsigned)(a.pool << a.page_shift) ? (T*)a.cache + (long)slot * width
                                                               : nullptr;
    T* out = a.kv_out ? (T*)a.kv_out + t * width : nullptr;
    Vt x[kMost];
    double sum = 0.0;     // fp64: squares of any fp32 values, and no cost next to memory
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int c = (i * 64 + lane) * V;
        x[i] = Vt{};
        if (c < a.dc) x[i] = *(const Vt*)(from + c);
#pragma unroll
        for (int j = 0; j < V; ++j) sum += (double)to_f32(x[i][j]) * (double)to_f32(x[i][j]);
    }
    Vt p = {}, q = {};
    if (lane < kUnits) {
        p = *(const Vt*)(from + a.dc + unit.a);
        q = *(const Vt*)(from + a.dc + unit.b);
        unit.apply(p, q);
    }
    // The factor is inv 2^e, for one of rows of 1e-39 or 1e38 (eps 0) is no normal fp32
    // number. (Products in fp64 instead: 67.3 us, not 65.9, with 21414 tokens in bf16.)
    float inv = 1.f;
    int e = 0;
    if (a.normalise) inv = (float)frexp(1.0 / sqrt(wave_sum(sum) / a.dc + (double)a.eps), &e);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int c = (i * 64 + lane) * V;
        if (c >= a.dc) continue;
        if (a.normalise)
#pragma unroll
            for (int j = 0; j < V; ++j)
                x[i][j] = from_f32<T>(ldexpf(to_f32(x[i][j]), e) * inv * (a.w ? a.w[c + j] : 1.f));
        if (to) *(Vt*)(to + c) = x[i];
        if (out) *(Vt*)(out + c) = x[i];
    }
    if (lane < kUnits) {
        if (to) {
            *(Vt*)(to + a.dc + unit.a) = p;
            *(Vt*)(to + a.dc + unit.b) = q;
        }
        if (out) {
            *(Vt*)(out + a.dc + unit.a) = p;
            *(Vt*)(out + a.dc + unit.b) = q;
        }
    }
    constexpr int kRows = 64 / kUnits;                // heads at a time
    for (int h = lane / kUnits; h < a.Hq; h += kRows) {
        const T* from = (const T*)a.q + (t * a.Hq + h + 1) * a.dq - kPe;
        T* to = (T*)a.q_out + (t * a.Hq + h + 1) * a.dq_out - kPe;
        Vt x = *(const Vt*)(from + unit.a), y = *(const Vt*)(from + unit.b);
        unit.apply(x, y);
        *(Vt*)(to + unit.a) = x;
        *(Vt*)(to + unit.b) = y;
    }
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t st) {
    constexpr int tokens = kRopeWaves;
    const auto run = [&](auto kernel) {
        for (long t = 0; t < a.T; t += kRopeGrid * tokens) {
            const long n = a.T - t < kRopeGrid * tokens ? a.T - t : kRopeGrid * tokens;
            kernel<<<(unsigned)((n + tokens - 1) / tokens), 64 * kRopeWaves, 0, st>>>(a, (int)t);
        }
    };
    if (a.bf16_io) run(latent_append_kernel<bf16>);
    else run(latent_append_kernel<float>);
    return hipGetLastError();
}

}  // namespace kda
