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
// 256 requests over 131072 tokens, fp32: 36 + 11 us, 201 MB at 5.6 TB/s in
// the first (one workgroup per request: 439 us).
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
    // r of kEach values in pieces of 16 bytes, the i-th from y + i * step on; 0
    // behind V. The values need not be aligned: a row starts anywhere for an
    // odd V.
    __device__ void load(long y, int step, double* r) const {
        struct __attribute__((packed)) Vec { T x[16 / sizeof(T)]; };
        constexpr int N = 16 / (int)sizeof(T);
        T a[kEach], b[kEach];
        const bool both = rest && q;
#pragma unroll
        for (int i = 0; i < kEach / N; ++i) {
            const long at = y + (long)i * step;
            if (at + N <= V) {
                const Vec v = *(const Vec*)(p + at);
#pragma unroll
                for (int j = 0; j < N; ++j) a[i * N + j] = v.x[j];
                if (both) {
                    const Vec w = *(const Vec*)(q + at);
#pragma unroll
                    for (int j = 0; j < N; ++j) b[i * N + j] = w.x[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const bool in = at + j < V;
                    a[i * N + j] = in ? p[at + j] : (T)0.f;
                    if (both) b[i * N + j] = in ? q[at + j] : (T)0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            double x = (double)to_f32(a[i]);
            if (both) x -= (double)to_f32(b[i]);
            else if (rest && y + (long)(i / N) * step + i % N == zero) x = 0.0;
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

// A request's drafted tokens; below 0: an unused row.
__device__ __forceinline__ int drafted(const VerifyArgs& a, int b) {
    const int n = a.n_draft ? a.n_draft[b] : a.T;
    return n < a.T ? n : a.T;
}

// Number of drafted tokens that stay. Every wave finds it, 64 drafted tokens
// at a time.
template <typename T>
__device__ int accepted(const VerifyArgs& a, int b, int n) {
    const T* p = (const T*)a.p + (long)b * (a.T + 1) * a.V;
    const T* q = a.q ? (const T*)a.q + (long)b * a.T * a.V : nullptr;
    const int* x = a.x + (long)b * a.T;
    const float* u = a.u + (long)b * (a.T + 1);
    const int lane = threadIdx.x & 63;
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
        if (no) return t0 + __builtin_ctzll(no);
    }
    return n;
}

// The row that decides what follows the acc tokens that stay.
template <typename T>
__device__ __forceinline__ Row<T> row_of(const VerifyArgs& a, int b, int n, int acc) {
    Row<T> row;
    row.p = (const T*)a.p + ((long)b * (a.T + 1) + acc) * a.V;
    row.rest = acc < n;
    row.q = a.q && row.rest ? (const T*)a.q + ((long)b * a.T + acc) * a.V : nullptr;
    row.zero = row.rest && !a.q ? a.x[(long)b * a.T + acc] : -1;
    row.V = a.V;
    return row;
}

// sums[b][part]: the part's share of sum r; accs[b]: the tokens that stay. (Two
// parts a workgroup took as long, four longer.)
template <typename T>
__global__ __launch_bounds__(kThreads) void verify_sums(VerifyArgs a, double* sums, int* accs) {
    __shared__ double lds[kThreads / 64];
    constexpr int kVec = 16 / (int)sizeof(T);
    const int b = blockIdx.y;
    const int n = drafted(a, b);
    if (n < 0) return;
    const int acc = accepted<T>(a, b, n);
    const Row<T> row = row_of<T>(a, b, n, acc);
    if (blockIdx.x == 0 && threadIdx.x == 0) accs[b] = acc;
    double r[kEach], s = 0;
    row.load((long)blockIdx.x * kPart + threadIdx.x * kVec, kThreads * kVec, r);
#pragma unroll
    for (int i = 0; i < kEach; ++i) s += r[i];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) sums[(long)b * gridDim.x + blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void verify_pick(VerifyArgs a, const double* sums, const int* accs,
                                                        int parts) {
    __shared__ double lds[kThreads / 64];
    __shared__ int sh_part, sh_y, sh_last;
    __shared__ double sh_before;
    const int b = blockIdx.x, tid = threadIdx.x;
    int* tokens = a.tokens + (long)b * (a.T + 1);
    const int n = drafted(a, b);
    const double* sum = parts > 1 ? sums + (long)b * parts : nullptr;
    const double sum0 = sum && tid < parts ? sum[tid] : 0.0;
    const double u = (double)a.u[(long)b * (a.T + 1) + a.T];
    if (n < 0) {
        for (int t = tid; t <= a.T; t += kThreads) tokens[t] = -1;
        if (tid == 0) a.n_commit[b] = 0;
        return;
    }
    const int acc = parts > 1 ? accs[b] : accepted<T>(a, b, n);
    Row<T> row = row_of<T>(a, b, n, acc);
    if (tid == 0) { sh_part = INT32_MAX; sh_y = INT32_MAX; sh_last = 0; sh_before = 0; }
    __syncthreads();

    // r of a thread's share of a part, and the part's sum
    double r[kEach];
    auto share = [&](int part) {
        row.load((long)part * kPart + tid * kEach, 16 / (int)sizeof(T), r);
        double s = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) s += r[i];
        return s;
    };
    // sum of part i, for the thread that asks: from the first kernel, or (when
    // r is p after all) from the row itself, by the whole workgroup
    double total = 0, t1;
    double p0 = 0, t0 = 0;                        // of the first parts' sums
    if (sum) {
        p0 = block_prefix(sum0, lds, t0);
        total = t0;
        for (int i = kThreads; i < parts; i += kThreads) {
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
            const double s = i == 0 ? sum0 : i + tid < parts ? sum[i + tid] : 0.0;
            double x = p0;
            t1 = t0;
            if (i > 0) x = before + block_prefix(s, lds, t1);
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
    int* accs = (int*)(sums + (size_t)a.B * parts);
    // requests of a launch: at most 65535 in the grid's second dimension, and fewer
    // than 2^32 threads in a grid
    const long most = parts > 1 ? 65535 : 1 << 23;
    for (long b = 0; b < a.B; b += most) {
        const int n = (int)(a.B - b < most ? a.B - b : most);
        VerifyArgs c = a;
        c.p = (const T*)a.p + b * (a.T + 1) * a.V;
        if (a.q) c.q = (const T*)a.q + b * a.T * a.V;
        c.x = a.x + b * a.T;
        c.u = a.u + b * (a.T + 1);
        if (a.n_draft) c.n_draft = a.n_draft + b;
        c.n_commit = a.n_commit + b;
        c.tokens = a.tokens + b * (a.T + 1);
        if (parts > 1)
            verify_sums<T><<<dim3((unsigned)parts, (unsigned)n), kThreads, 0, st>>>(
                c, sums + b * parts, accs + b);
        verify_pick<T><<<(unsigned)n, kThreads, 0, st>>>(c, sums + b * parts, accs + b, parts);
    }
}

}  // namespace

size_t draft_verify_ws(int B, int V) {
    return parts_of(V) > 1 ? (size_t)B * (parts_of(V) * sizeof(double) + sizeof(int)) : 0;
}

hipError_t launch_draft_verify(const VerifyArgs& a, void* ws, hipStream_t st) {
    if (a.bf16_io) launch<bf16>(a, (double*)ws, st);
    else launch<float>(a, (double*)ws, st);
    return hipGetLastError();
}

}  // namespace kda
