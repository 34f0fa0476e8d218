// Block tables and slot maps of a serving step, from request lengths.
//
// With need_i = ceil((kept_i + new_i) / page) and have_i pages held, request i
// takes max(need_i - have_i, 0) pages from the pool's ring and gives
// max(have_i - need_i, 0) back; their exclusive prefix sums over the requests
// place every moved page, and the prefix sum of new_i (cu) every new token.
//
// One workgroup checks the inputs, decides the status and scans
// (page_plan_scan); what is left are three flat lists (slots, pages taken,
// pages given back), each entry of which finds its request by a binary search
// in the list's prefix sums (page_plan_fill).
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 1024;

// Workspace of B requests: pages held before the call (the caller's array
// may be overwritten in place), prefix sums of pages taken and given back,
// and the ring as it was.
struct PlanWs {
    int *have, *taken, *given, *ring;   // [B], [B + 1], [B + 1], [2]
    __host__ __device__ PlanWs(void* ws, int B)
        : have((int*)ws), taken(have + B), given(taken + B + 1), ring(given + B + 1) {}
};

// Inclusive prefix sums of v over the workgroup, and the total.
template <typename T>
__device__ T block_scan(T v, T* lds, T& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int o = 1; o < 64; o <<= 1) {
        const T x = __shfl_up(v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();                     // lds free of an earlier call's reads
    if (lane == 63) lds[w] = v;
    __syncthreads();
    T before = 0, all = 0;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
        if (i < w) before += lds[i];
        all += lds[i];
    }
    total = all;
    return v + before;
}

// Largest i with off[i] <= x, for off[0] = 0 <= x < off[n].
__device__ __forceinline__ int find(const int* off, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (off[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ void fill(const PlanArgs& a, const PlanWs& w, long first, long step) {
    const int B = a.B, mask = (1 << a.page_shift) - 1;
    const int head = w.ring[0], count = w.ring[1];
    const int tokens = a.cu[B], taken = w.taken[B], given = w.given[B];
    const long all = (long)a.n_slots + taken + given;
    for (long j = first; j < all; j += step) {
        if (j < a.n_slots) {
            const int t = (int)j;
            int slot = -1;
            if (t < tokens) {
                const int i = find(a.cu, B, t);
                const int pos = a.kept[i] + (t - a.cu[i]), pg = pos >> a.page_shift;
                const int page = pg < w.have[i]
                    ? a.table[(long)i * a.width + pg]
                    : a.ring[((long)head + w.taken[i] + pg - w.have[i]) % a.pool];
                slot = (page << a.page_shift) + (pos & mask);
            }
            a.slots[t] = slot;
        } else if (j < (long)a.n_slots + taken) {
            const int x = (int)(j - a.n_slots), i = find(w.taken, B, x);
            a.table[(long)i * a.width + w.have[i] + (x - w.taken[i])] =
                a.ring[((long)head + x) % a.pool];
        } else {
            const int x = (int)(j - a.n_slots - taken), i = find(w.given, B, x);
            a.ring[((long)head + count + x) % a.pool] =
                a.table[(long)i * a.width + a.pages_out[i] + (x - w.given[i])];
        }
    }
}

__global__ __launch_bounds__(kThreads) void page_plan_scan(PlanArgs a, void* ws, bool fill_too) {
    __shared__ long lds_l[kThreads / 64];
    __shared__ int lds_i[kThreads / 64];
    const PlanWs w(ws, a.B);
    const int head = a.ring_in[0], count = a.ring_in[1];
    const long page = 1l << a.page_shift;
    long tokens = 0, taken = 0, given = 0;
    int bad = 0;
    for (int i = threadIdx.x; i < a.B; i += kThreads) {
        const long kept = a.kept[i], fresh = a.fresh[i], have = a.pages_in[i];
        const long need = (kept + fresh + page - 1) >> a.page_shift;
        bad |= kept < 0 || fresh < 0 || have < 0 || have > a.width || need > a.width;
        tokens += fresh;
        taken += need > have ? need - have : 0;
        given += have > need ? have - need : 0;
    }
    long n_tokens, n_taken, n_given, n_bad;
    block_scan<long>(tokens, lds_l, n_tokens);
    block_scan<long>(taken, lds_l, n_taken);
    block_scan<long>(given, lds_l, n_given);
    block_scan<long>((long)bad, lds_l, n_bad);
    // Given-back entries land behind the free ones and never on an entry that
    // is taken in this call, because free and given-back pages together fit
    // the ring; more of them means that a page is held twice.
    int status = KDA_PLAN_OK;
    if (n_bad || head < 0 || count < 0 || count > a.pool || head >= (a.pool > 0 ? a.pool : 1) ||
        count + n_given > a.pool)
        status = KDA_PLAN_INVALID;
    else if (n_tokens > a.n_slots)
        status = KDA_PLAN_NO_SLOTS;
    else if (n_taken > count)
        status = n_taken - count > INT32_MAX ? INT32_MAX : (int)(n_taken - count);
    const bool ok = status == KDA_PLAN_OK;
    int cu0 = 0, taken0 = 0, given0 = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int i = base + (int)threadIdx.x;
        int fresh = 0, plus = 0, minus = 0, have = 0, need = 0;
        if (i < a.B) {
            have = a.pages_in[i];
            need = have;
            if (ok) {
                fresh = a.fresh[i];
                need = (int)(((long)a.kept[i] + fresh + page - 1) >> a.page_shift);
                plus = need > have ? need - have : 0;
                minus = have > need ? have - need : 0;
            }
        }
        int t_fresh, t_plus, t_minus;
        const int s_fresh = block_scan<int>(fresh, lds_i, t_fresh);
        const int s_plus = block_scan<int>(plus, lds_i, t_plus);
        const int s_minus = block_scan<int>(minus, lds_i, t_minus);
        if (i < a.B) {
            w.have[i] = have;
            w.taken[i] = taken0 + s_plus - plus;
            w.given[i] = given0 + s_minus - minus;
            a.cu[i] = cu0 + s_fresh - fresh;
            a.pages_out[i] = need;
        }
        cu0 += t_fresh;
        taken0 += t_plus;
        given0 += t_minus;
    }
    if (threadIdx.x == 0) {
        w.taken[a.B] = taken0;
        w.given[a.B] = given0;
        w.ring[0] = head;
        w.ring[1] = count;
        a.cu[a.B] = cu0;
        a.ring_out[0] = taken0 ? (int)(((long)head + taken0) % a.pool) : head;
        a.ring_out[1] = count - taken0 + given0;
        a.status[0] = status;
    }
    if (fill_too) {
        __syncthreads();
        fill(a, w, threadIdx.x, kThreads);
    }
}

__global__ __launch_bounds__(256) void page_plan_fill(PlanArgs a, void* ws) {
    fill(a, PlanWs(ws, a.B), (long)blockIdx.x * 256 + threadIdx.x, (long)gridDim.x * 256);
}

}  // namespace

size_t page_plan_ws(int B) { return (3 * (size_t)B + 4) * sizeof(int); }

hipError_t launch_page_plan(const PlanArgs& a, void* ws, hipStream_t st) {
    const bool one = a.n_slots <= 4096;
    page_plan_scan<<<1, kThreads, 0, st>>>(a, ws, one);
    if (!one) {
        const int grid = (int)(((long)a.n_slots + 255) / 256 < 2048 ? ((long)a.n_slots + 255) / 256
                                                                    : 2048);
        page_plan_fill<<<grid, 256, 0, st>>>(a, ws);
    }
    return hipGetLastError();
}

}  // namespace kda
