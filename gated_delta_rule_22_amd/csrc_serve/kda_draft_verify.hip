// Verification of drafted tokens by rejection sampling.
//
// Token t stays while u_t q_t(x_t) < p_t(x_t): both factors have 24 bits, so
// the product is exact in fp64 and the decision is that of the definition.
// The next token comes from r = max(p_a - q_a, 0) (or p_a) by inversion: the
// least y whose cumulative sum passes u_T sum r. The sums are held in fp64:
// in fp32 the 2^-24 steps of a sum near 1 would be as large as many tokens'
// probabilities.
//
// What bounds it is reading row a of p and q once. The row is cut into parts
// of kPart values, one workgroup each (verify_sums), which finds a for itself
// from the 2 T values that decide; then one workgroup per request finds the
// part whose prefix sum passes the target and walks that part alone
// (verify_pick). A row of a single part needs the second kernel only.
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kEach = 16, kPart = kThreads * kEach;

// Row a of one request: which token comes next is drawn from it.
template <typename T>
struct Row {
    const T* p;
    const T* q;       // null: r = p, but 0 at `zero`
    int zero;         // -1: none
    bool rest;        // r = max(p - q, 0); otherwise r = p
    int V;
    // r of the n-th value and what follows it, kEach of them; 0 behind V. The
    // values need not be aligned: a row starts anywhere for an odd V.
    __device__ void load(long y, double* r) const {
        struct __attribute__((packed)) Vec { T x[16 / sizeof(T)]; };
        constexpr int N = 16 / (int)sizeof(T);
        T a[kEach], b[kEach];
        if (y + kEach <= V) {
#pragma unroll
            for (int i = 0; i < kEach; i += N) {
                const Vec v = *(const Vec*)(p + y + i);
#pragma unroll
                for (int j = 0; j < N; ++j) a[i + j] = v.x[j];
                if (rest && q) {
                    const Vec w = *(const Vec*)(q + y + i);
#pragma unroll
                    for (int j = 0; j < N; ++j) b[i + j] = w.x[j];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const bool in = y + i < V;
                a[i] = in ? p[y + i] : (T)0.f;
                if (rest && q) b[i] = in ? q[y + i] : (T)0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            double x = (double)to_f32(a[i]);
            if (rest) x = q ? x - (double)to_f32(b[i]) : (y + i == zero ? 0.0 : x);
            r[i] = x > 0.0 ? x : 0.0;            // (NaN: 0)
        }
    }
};

__device__ __forceinline__ double wave_sum(double x) {
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}
// Inclusive prefix sum over the workgroup.
__device__ __forceinline__ double block_prefix(double x, double* lds, double& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 63) lds[w] = x;
    __syncthreads();
    double before = 0;
    total = 0;
    for (int i = 0; i < kThreads / 64; ++i) {
        if (i < w) before += lds[i];
        total += lds[i];
    }
    return before + x;
}

// Number of drafted tokens that stay, and the row that decides what follows.
// Every wave finds it, 64 drafted tokens at a time. n < 0: an unused row.
template <typename T>
__device__ int accepted(const VerifyArgs& a, int b, Row<T>& row, int& n) {
    n = a.n_draft ? a.n_draft[b] : a.T;
    n = n < a.T ? n : a.T;
    if (n < 0) return 0;
    const T* p = (const T*)a.p + (long)b * (a.T + 1) * a.V;
    const T* q = a.q ? (const T*)a.q + (long)b * a.T * a.V : nullptr;
    const int* x = a.x + (long)b * a.T;
    const float* u = a.u + (long)b * (a.T + 1);
    const int lane = threadIdx.x & 63;
    int acc = n;
    for (int t0 = 0; t0 < n; t0 += 64) {
        const int t = t0 + lane;
        bool stays = true;
        if (t < n) {
            const int y = x[t];
            stays = (unsigned)y < (unsigned)a.V;
            if (stays) {
                const double pt = (double)to_f32(p[(long)t * a.V + y]);
                const double qt = q ? (double)to_f32(q[(long)t * a.V + y]) : 1.0;
                stays = (double)u[t] * qt < pt;
            }
        }
        const unsigned long long no = __ballot(!stays);
        if (no) {
            acc = t0 + __builtin_ctzll(no);
            break;
        }
    }
    row.p = p + (long)acc * a.V;
    row.q = q ? q + (long)acc * a.V : nullptr;
    row.rest = acc < n;
    row.zero = row.rest && !q ? x[acc] : -1;
    row.V = a.V;
    return acc;
}

// sums[b][part]: the part's share of sum r.
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_sums(VerifyArgs a, double* sums) {
    __shared__ double lds[kThreads / 64];
    const int b = blockIdx.y;
    Row<T> row;
    int n;
    accepted(a, b, row, n);
    if (n < 0) return;
    double r[kEach], s = 0;
    row.load((long)blockIdx.x * kPart + threadIdx.x * kEach, r);
#pragma unroll
    for (int i = 0; i < kEach; ++i) s += r[i];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) sums[(long)b * gridDim.x + blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick(VerifyArgs a, const double* sums, int parts) {
    __shared__ double lds[kThreads / 64];
    __shared__ int sh_part, sh_y, sh_last;
    __shared__ double sh_before;
    const int b = blockIdx.x, tid = threadIdx.x;
    int* tokens = a.tokens + (long)b * (a.T + 1);
    Row<T> row;
    int n;
    const int acc = accepted(a, b, row, n);
    if (n < 0) {
        for (int t = tid; t <= a.T; t += kThreads) tokens[t] = -1;
        if (tid == 0) a.n_commit[b] = 0;
        return;
    }
    const double u = (double)a.u[(long)b * (a.T + 1) + a.T];
    const double* sum = parts > 1 ? sums + (long)b * parts : nullptr;
    if (tid == 0) { sh_part = INT32_MAX; sh_y = INT32_MAX; sh_last = 0; sh_before = 0; }
    __syncthreads();

    // r of a thread's share of a part, and the part's sum
    double r[kEach];
    auto share = [&](int part) {
        row.load((long)part * kPart + tid * kEach, r);
        double s = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) s += r[i];
        return s;
    };
    // sum of part i, for the thread that asks: from the first kernel, or (when
    // r is p after all) from the row itself, by the whole workgroup
    double total = 0, t1;
    if (sum) {
        for (int i = 0; i < parts; i += kThreads) {
            block_prefix(i + tid < parts ? sum[i + tid] : 0.0, lds, t1);
            total += t1;
        }
    } else {
        for (int i = 0; i < parts; ++i) {
            block_prefix(share(i), lds, t1);
            total += t1;
        }
    }
    if (total == 0 && row.rest) {
        row.rest = false;
        sum = nullptr;
        for (int i = 0; i < parts; ++i) {
            block_prefix(share(i), lds, t1);
            total += t1;
        }
    }
    // (u >= 1 passes every border: the last token, whatever the sums round to)
    const double target = u < 1.0 ? u * total : INFINITY;
    // the first part whose prefix sum passes the target
    double before = 0;
    if (sum) {
        int last = -1;                            // last part of this thread with a value
        for (int i = 0; i < parts; i += kThreads) {
            const double s = i + tid < parts ? sum[i + tid] : 0.0;
            const double x = before + block_prefix(s, lds, t1);
            if (s > 0) last = i + tid;
            if (s > 0 && x > target) atomicMin(&sh_part, i + tid);
            __syncthreads();
            if (sh_part == i + tid) sh_before = x - s;
            if (sh_part != INT32_MAX) break;
            before += t1;
        }
        if (sh_part == INT32_MAX) {               // none: the last part that has a value
            if (last >= 0) atomicMax(&sh_last, last);
            __syncthreads();
            if (tid == 0) sh_part = sh_last;
            __syncthreads();
            if (tid == 0) { sh_last = 0; sh_before = total; }
        }
        __syncthreads();
    }
    const int first = sum ? sh_part : 0, end = sum ? first + 1 : parts;
    before = sum ? sh_before : 0.0;
    for (int i = first; i < end; ++i) {
        const double s = share(i);
        double x = before + (block_prefix(s, lds, t1) - s);
        int last = -1, y = INT32_MAX;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            x += r[j];
            if (r[j] > 0) {
                last = i * kPart + tid * kEach + j;
                if (x > target && y == INT32_MAX) y = last;
            }
        }
        if (y != INT32_MAX) atomicMin(&sh_y, y);
        if (last >= 0) atomicMax(&sh_last, last);
        __syncthreads();
        if (sh_y != INT32_MAX) break;
        before += t1;
    }
    const int y = sh_y != INT32_MAX ? sh_y : sh_last;
    for (int t = tid; t <= a.T; t += kThreads)
        tokens[t] = t < acc ? a.x[(long)b * a.T + t] : (t == acc ? y : -1);
    if (tid == 0) a.n_commit[b] = acc + 1;
}

int parts_of(int V) { return (int)(((long)V + kPart - 1) / kPart); }

template <typename T>
void launch(const VerifyArgs& a, double* sums, hipStream_t st) {
    const int parts = parts_of(a.V);
    // at most 65535 requests a launch in the grid's second dimension
    for (int b = 0; parts > 1 && b < a.B; b += 65535) {
        VerifyArgs c = a;
        c.p = (const T*)a.p + (long)b * (a.T + 1) * a.V;
        if (a.q) c.q = (const T*)a.q + (long)b * a.T * a.V;
        c.x = a.x + (long)b * a.T;
        c.u = a.u + (long)b * (a.T + 1);
        if (a.n_draft) c.n_draft = a.n_draft + b;
        const int n = a.B - b < 65535 ? a.B - b : 65535;
        verify_sums<T><<<dim3((unsigned)parts, (unsigned)n), kThreads, 0, st>>>(c, sums + (long)b * parts);
    }
    verify_pick<T><<<(unsigned)a.B, kThreads, 0, st>>>(a, sums, parts);
}

}  // namespace

size_t draft_verify_ws(int B, int, int V) {
    return parts_of(V) > 1 ? (size_t)B * parts_of(V) * sizeof(double) : 0;
}

hipError_t launch_draft_verify(const VerifyArgs& a, void* ws, hipStream_t st) {
    if (a.bf16_io) launch<bf16>(a, (double*)ws, st);
    else launch<float>(a, (double*)ws, st);
    return hipGetLastError();
}

}  // namespace kda
