// Causal attention of new tokens over a paged cache.
//
// One wave per (token, query head): 64 keys at a time, one per lane, with the
// running maximum and sum of the softmax in fp32, then the weighted values
// with the head dimension over the lanes.
#include "kda_serve_launch.h"

namespace kda {
namespace {

template <typename T, int D>
__global__ __launch_bounds__(64) void attn_rows_kernel(AttnArgs a) {
    const int t = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x;
    // the request of row t (the first whose rows hold it)
    int req = -1, at = 0;
    for (int i = 0; i < a.B && req < 0; ++i) {
        int lo = a.cu[i], hi = a.cu[i + 1];
        lo = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
        hi = hi < 0 ? 0 : (hi > a.T ? a.T : hi);
        if (t >= lo && t < hi) { req = i; at = t - lo; }
    }
    if (req < 0) return;
    const int h = hq / (a.Hq / a.Hkv);
    const long cap = (long)a.width << a.page_shift;
    long kept = a.kept[req];
    kept = kept < 0 ? 0 : kept;
    const long end = kept + at + 1 < cap ? kept + at + 1 : cap;
    const int page = 1 << a.page_shift;
    const T* q = (const T*)a.q + ((long)t * a.Hq + hq) * D;
    float m = -INFINITY, l = 0.f, acc[(D + 63) / 64] = {};
    for (long k0 = 0; k0 < end; k0 += 64) {
        const long pos = k0 + lane;
        long row = -1;
        if (pos < end) {
            const int pg = a.table[(long)req * a.width + (pos >> a.page_shift)];
            if ((unsigned)pg < (unsigned)a.pool)
                row = (((long)pg * a.Hkv + h) << a.page_shift) + (pos & (page - 1));
        }
        float s = -INFINITY;
        if (row >= 0) {
            s = 0.f;
            const T* k = (const T*)a.kc + row * D;
            for (int i = 0; i < D; ++i) s += to_f32(q[i]) * to_f32(k[i]);
            s *= a.scale;
        }
        float mx = s;
        for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float p = row >= 0 ? __expf(s - mu) : 0.f, c = __expf(m - mu);
        float sum = p;
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
        l = l * c + sum;
        m = mn;
        for (int j = 0; j < (D + 63) / 64; ++j) acc[j] *= c;
        for (int i = 0; i < 64; ++i) {
            const long r = __shfl(row, i);
            const float w = __shfl(p, i);
            if (r < 0) continue;
            for (int j = 0; j < (D + 63) / 64; ++j)
                if (j * 64 + lane < D) acc[j] += w * to_f32(((const T*)a.vc)[r * D + j * 64 + lane]);
        }
    }
    T* o = (T*)a.o + ((long)t * a.Hq + hq) * D;
    for (int j = 0; j < (D + 63) / 64; ++j)
        if (j * 64 + lane < D) o[j * 64 + lane] = from_f32<T>(l > 0.f ? acc[j] / l : (l == 0.f ? 0.f : l));
    if (a.lse && lane == 0) a.lse[(long)t * a.Hq + hq] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename T>
void launch(const AttnArgs& a, hipStream_t st) {
    const dim3 g((unsigned)a.T, (unsigned)a.Hq);
    switch (a.d) {
        case 16: attn_rows_kernel<T, 16><<<g, 64, 0, st>>>(a); break;
        case 32: attn_rows_kernel<T, 32><<<g, 64, 0, st>>>(a); break;
        case 64: attn_rows_kernel<T, 64><<<g, 64, 0, st>>>(a); break;
        default: attn_rows_kernel<T, 128><<<g, 64, 0, st>>>(a); break;
    }
}

}  // namespace

size_t attn_paged_ws(int, int, int, int, int, int, bool) { return 0; }

hipError_t launch_attn_paged(const AttnArgs& a, void*, hipStream_t st) {
    if (a.bf16_io) launch<bf16>(a, st);
    else launch<float>(a, st);
    return hipGetLastError();
}

}  // namespace kda
