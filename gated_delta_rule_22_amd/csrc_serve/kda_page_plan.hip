// Block tables and slot maps of a serving step, from request lengths.
//
// With need_i = ceil((kept_i + new_i) / page) and have_i pages held, request i
// takes max(need_i - have_i, 0) pages from the pool's ring and gives
// max(have_i - need_i, 0) back; their exclusive prefix sums over the requests
// place every moved page, and the prefix sum of new_i (cu) every new token.
//
// One workgroup checks the inputs, decides the status and scans
// (page_plan_scan); what are left are three flat lists (slots, pages taken,
// pages given back), each entry of which finds its request in the list's prefix
// sums. For small steps the same workgroup fills them, for others a second
// launch (page_plan_fill): the counts may be updated in place, so everything
// has to be read before anything is written. Memory latencies bound both: 256
// requests of up to 8 tokens 7 us, 1024 requests with 276,000 slots in pages of
// 16 4.1 + 6 us.
#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 1024;
// One launch up to so many slots and table entries, of which any number may be
// given back: 256 requests over 259 pages 8.2 us with one, 7.7 with two and
// another 3 us on the host; 512 over 259 13 and 9; 1024 over 1900, 30% of them
// ended, 75 and 9.
constexpr int kOneSlots = 4096;
constexpr long kOneEntries = 1l << 17;

// Workspace of B requests: pages held before the call (the caller's array
// may be overwritten in place), prefix sums of pages taken and given back,
// and the ring as it was.
struct PlanWs {
    int *have, *taken, *given, *ring;   // [B], [B + 1], [B + 1], [2]
    __host__ __device__ PlanWs(void* ws, int B)
        : have((int*)ws), taken(have + B), given(taken + B + 1), ring(given + B + 1) {}
};

// Inclusive prefix sum over the wave: shifts inside each 16-lane row, then
// the last lane of row 0 (2) into row 1 (3) and of row 1 into rows 2 and 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ long dpp_add(long x) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, false);
    return x + (long)((unsigned long)(unsigned)lo | (unsigned long)(unsigned)hi << 32);
}
__device__ __forceinline__ long wave_prefix(long x) {
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    return dpp_add<0x143, 0xC>(x);
}

// Tokens, pages taken and pages given back of some requests; bad: one of
// them has a value outside its range.
struct Counts {
    long tokens, taken, given;
    int bad;
};
// Inclusive prefix sums over the workgroup, and the totals. 64 bits: the
// inputs are anything.
__device__ __forceinline__ Counts block_prefix(Counts c, Counts* lds, Counts& total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    c.tokens = wave_prefix(c.tokens);
    c.taken = wave_prefix(c.taken);
    c.given = wave_prefix(c.given);
    c.bad = __any(c.bad);
    __syncthreads();                     // lds free of an earlier call's reads
    if (lane == 63) lds[w] = c;
    __syncthreads();
    // the waves' sums, one a lane, and their prefix
    Counts t = lds[lane < kThreads / 64 ? lane : 0];
    if (lane >= kThreads / 64) t = Counts{0, 0, 0, 0};
    const Counts own = t;
    t.tokens = wave_prefix(t.tokens);
    t.taken = wave_prefix(t.taken);
    t.given = wave_prefix(t.given);
    total.tokens = __shfl(t.tokens, 63);
    total.taken = __shfl(t.taken, 63);
    total.given = __shfl(t.given, 63);
    total.bad = __any(t.bad);
    c.tokens += __shfl(t.tokens - own.tokens, w);
    c.taken += __shfl(t.taken - own.taken, w);
    c.given += __shfl(t.given - own.given, w);
    return c;
}

// A request: what it holds and needs.
struct Request { int have, need; Counts c; };
__device__ __forceinline__ Request request(const PlanArgs& a, int i) {
    Request r{0, 0, {0, 0, 0, 0}};
    if (i >= a.B) return r;
    const long kept = a.kept[i], fresh = a.fresh[i], have = a.pages_in[i];
    const long need = (kept + fresh + (1l << a.page_shift) - 1) >> a.page_shift;
    r.c.bad = kept < 0 || fresh < 0 || have < 0 || have > a.width || need > a.width ||
              kept + fresh > INT32_MAX;
    r.have = (int)have;
    r.need = (int)need;
    r.c.tokens = fresh;
    r.c.taken = need > have ? need - have : 0;
    r.c.given = have > need ? have - need : 0;
    return r;
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
// The same for 64 neighbouring x of a wave (x of lane 0 is the least, and
// inside): the wave narrows the range of the first by 64 a step, and the
// others look among the 63 offsets that follow; only x of more requests than
// that search by themselves. Two or three memory latencies instead of ten.
__device__ __forceinline__ int find_wave(const int* off, int n, int x, bool in) {
    const int lane = threadIdx.x & 63;
    const int x0 = __builtin_amdgcn_readfirstlane(x);
    int lo = 0, hi = n;                  // off[lo] <= x0 < off[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int at = lo + lane * step;
        const unsigned long long le = __ballot(at < hi && off[at < hi ? at : lo] <= x0);
        // lanes that hold: 0 .. k
        const int k = 63 - __builtin_clzll(le);
        const int next = lo + (k + 1) * step;
        lo += k * step;
        hi = next < hi ? next : hi;
    }
    const int at = lo + 1 + lane;
    const int border = at < n ? off[at] : INT32_MAX;   // of the requests behind
    int i = 0;
    for (int bit = 32; bit; bit >>= 1)                 // borders <= x among them
        if (__shfl(border, i + bit - 1) <= x) i += bit;
    if (in && i == 63 && lo + 64 < n && off[lo + 64] <= x) return find(off, n, x);
    return lo + i;
}

// Entry x of the ring from head, x <= pool.
__device__ __forceinline__ int ring_at(const PlanArgs& a, int head, int x) {
    const unsigned i = (unsigned)head + (unsigned)x;
    return (int)(i >= (unsigned)a.pool ? i - (unsigned)a.pool : i);
}

// `first` counts threads: whole waves are consecutive and aligned.
__device__ void fill(const PlanArgs& a, const PlanWs& w, long first, long step) {
    const int B = a.B, mask = (1 << a.page_shift) - 1;
    const int head = w.ring[0], count = w.ring[1];
    const int tokens = a.cu[B], taken = w.taken[B], given = w.given[B];
    // each list fills whole waves, so that the lanes of a wave search together
    const auto waves = [](int n) { return ((long)n + 63) & ~63l; };
    const long taken0 = waves(a.n_slots), given0 = taken0 + waves(taken);
    const long all = given0 + waves(given);
    for (long j = first; j < all; j += step) {
        if (j < taken0) {
            const int t = (int)j;
            int slot = -1, i = 0;
            // the wave's first slot has a token if any of them has
            if (__builtin_amdgcn_readfirstlane(t) < tokens) i = find_wave(a.cu, B, t, t < tokens);
            if (t < tokens) {
                const int pos = a.kept[i] + (t - a.cu[i]), pg = pos >> a.page_shift;
                const int page = pg < w.have[i]
                    ? a.table[(long)i * a.width + pg]
                    : a.ring[ring_at(a, head, w.taken[i] + pg - w.have[i])];
                // (a page id that is none gives no slot rather than another page's)
                if ((unsigned)page < (unsigned)a.pool) slot = (page << a.page_shift) + (pos & mask);
            }
            if (t < a.n_slots) a.slots[t] = slot;
        } else if (j < given0) {
            const int x = (int)(j - taken0), i = find_wave(w.taken, B, x, x < taken);
            if (x < taken)
                a.table[(long)i * a.width + w.have[i] + (x - w.taken[i])] = a.ring[ring_at(a, head, x)];
        } else {
            const int x = (int)(j - given0), i = find_wave(w.given, B, x, x < given);
            if (x < given)
                a.ring[ring_at(a, head, count + x)] =
                    a.table[(long)i * a.width + a.pages_out[i] + (x - w.given[i])];
        }
    }
}

__global__ __launch_bounds__(kThreads) void page_plan_scan(PlanArgs a, void* ws, bool fill_too) {
    __shared__ Counts lds[kThreads / 64];
    const PlanWs w(ws, a.B);
    const int head = a.ring_in[0], count = a.ring_in[1];
    // up to kThreads requests are read and summed once; more are summed first
    Request r = request(a, threadIdx.x);
    Counts all, p = block_prefix(r.c, lds, all);
    for (int base = kThreads; base < a.B; base += kThreads) {
        Counts t;
        block_prefix(request(a, base + (int)threadIdx.x).c, lds, t);
        all.tokens += t.tokens;
        all.taken += t.taken;
        all.given += t.given;
        all.bad |= t.bad;
    }
    // Given-back entries land behind the free ones and never on an entry that
    // is taken in this call, because free and given-back pages together fit
    // the ring; more of them means that a page is held twice.
    int status = KDA_PLAN_OK;
    if (all.bad || head < 0 || count < 0 || count > a.pool || head >= (a.pool > 0 ? a.pool : 1) ||
        count + all.given > a.pool)
        status = KDA_PLAN_INVALID;
    else if (all.tokens > a.n_slots)
        status = KDA_PLAN_NO_SLOTS;
    else if (all.taken > count)
        status = all.taken - count > INT32_MAX ? INT32_MAX : (int)(all.taken - count);
    const bool ok = status == KDA_PLAN_OK;
    int tokens0 = 0, taken0 = 0, given0 = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int i = base + (int)threadIdx.x;
        Counts t = all;
        if (a.B > kThreads) {
            r = request(a, i);
            p = block_prefix(r.c, lds, t);
        }
        if (i < a.B) {
            w.have[i] = r.have;
            w.taken[i] = ok ? taken0 + (int)(p.taken - r.c.taken) : 0;
            w.given[i] = ok ? given0 + (int)(p.given - r.c.given) : 0;
            a.cu[i] = ok ? tokens0 + (int)(p.tokens - r.c.tokens) : 0;
            a.pages_out[i] = ok ? r.need : r.have;
        }
        tokens0 += (int)t.tokens;
        taken0 += (int)t.taken;
        given0 += (int)t.given;
    }
    if (threadIdx.x == 0) {
        const int taken = ok ? (int)all.taken : 0, given = ok ? (int)all.given : 0;
        w.taken[a.B] = taken;
        w.given[a.B] = given;
        w.ring[0] = head;
        w.ring[1] = count;
        a.cu[a.B] = ok ? (int)all.tokens : 0;
        a.ring_out[0] = taken ? ring_at(a, head, taken) : head;
        a.ring_out[1] = count - taken + given;
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
    const bool one = a.n_slots <= kOneSlots && (long)a.B * a.width <= kOneEntries;
    page_plan_scan<<<1, kThreads, 0, st>>>(a, ws, one);
    if (!one) {
        // a thread per slot, and per page up to 2^17 of them, at most 2^19
        const long entries = (long)a.B * a.width;
        long n = (long)a.n_slots + (entries < kOneEntries ? entries : kOneEntries);
        n = (n + 255) / 256;
        const int grid = (int)(n < 2048 ? n : 2048);
        page_plan_fill<<<grid, 256, 0, st>>>(a, ws);
    }
    return hipGetLastError();
}

}  // namespace kda
