// Verification of drafted tokens by rejection sampling.
//
// Token t stays while u_t q_t(x_t) < p_t(x_t): both factors have 24 bits, so
// the product is exact in fp64 and the decision is that of the definition.
// The next token comes from r = max(p_a - q_a, 0) (or p_a) by inversion: the
// least y whose cumulative sum passes u_T sum r. The sums are held in fp64:
// in fp32 the 2^-24 steps of a sum near 1 would be as large as many tokens'
// probabilities.
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Row a of one request: which token comes next is drawn from it.
template <typename T>
struct Row {
    const T* p;
    const T* q;       // null: r = p, but 0 at `zero`
    int zero;         // -1: none
    bool rest;        // r = max(p - q, 0); otherwise r = p
    __device__ double operator()(int y) const {
        const double x = (double)to_f32(p[y]);
        double r = x;
        if (rest) r = q ? x - (double)to_f32(q[y]) : (y == zero ? 0.0 : x);
        return r > 0.0 ? r : 0.0;
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void draft_verify_kernel(VerifyArgs a) {
    __shared__ double part[kThreads];
    __shared__ int sh_a, sh_y, sh_last;
    const int b = blockIdx.x, tid = threadIdx.x;
    int n = a.n_draft ? a.n_draft[b] : a.T;
    if (n > a.T) n = a.T;
    if (n < 0) {
        for (int t = tid; t <= a.T; t += kThreads) a.tokens[(long)b * (a.T + 1) + t] = -1;
        if (tid == 0) a.n_commit[b] = 0;
        return;
    }
    const T* p = (const T*)a.p + (long)b * (a.T + 1) * a.V;
    const T* q = a.q ? (const T*)a.q + (long)b * a.T * a.V : nullptr;
    const int* x = a.x + (long)b * a.T;
    const float* u = a.u + (long)b * (a.T + 1);
    if (tid == 0) {
        int t = 0;
        for (; t < n; ++t) {
            if ((unsigned)x[t] >= (unsigned)a.V) break;
            const double pt = (double)to_f32(p[(long)t * a.V + x[t]]);
            const double qt = q ? (double)to_f32(q[(long)t * a.V + x[t]]) : 1.0;
            if (!((double)u[t] * qt < pt)) break;
        }
        sh_a = t;
    }
    __syncthreads();
    const int acc = sh_a;
    Row<T> row{p + (long)acc * a.V, q ? q + (long)acc * a.V : nullptr, -1, acc < n};
    if (row.rest && !q) row.zero = x[acc];
    const int span = (a.V + kThreads - 1) / kThreads;
    const long lo0 = (long)tid * span;
    const int lo = (int)(lo0 < a.V ? lo0 : a.V);
    const int hi = lo + span < a.V ? lo + span : a.V;
    double total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        double s = 0;
        for (int y = lo; y < hi; ++y) s += row(y);
        __syncthreads();
        part[tid] = s;
        __syncthreads();
        total = 0;
        for (int i = 0; i < kThreads; ++i) total += part[i];
        if (total > 0 || !row.rest) break;
        row.rest = false;
    }
    double before = 0;
    for (int i = 0; i < tid; ++i) before += part[i];
    const double target = (double)u[a.T] * total;
    if (tid == 0) { sh_y = a.V; sh_last = 0; }
    __syncthreads();
    double s = 0;
    int last = -1;
    for (int y = lo; y < hi; ++y) {
        const double r = row(y);
        if (r > 0) last = y;
        s += r;
        if (before + s > target) { atomicMin(&sh_y, y); break; }
    }
    if (last >= 0) atomicMax(&sh_last, last);
    __syncthreads();
    const int y = sh_y < a.V ? sh_y : sh_last;
    for (int t = tid; t <= a.T; t += kThreads)
        a.tokens[(long)b * (a.T + 1) + t] = t < acc ? x[t] : (t == acc ? y : -1);
    if (tid == 0) a.n_commit[b] = acc + 1;
}

}  // namespace

size_t draft_verify_ws(int, int, int) { return 0; }

hipError_t launch_draft_verify(const VerifyArgs& a, void*, hipStream_t st) {
    if (a.bf16_io) draft_verify_kernel<bf16><<<a.B, kThreads, 0, st>>>(a);
    else draft_verify_kernel<float><<<a.B, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace kda
