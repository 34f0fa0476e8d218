// Work split of the paged attention, computed by every workgroup for itself.
//
// The n new tokens of a request and the G query heads of a KV head form n * G
// rows (row r: token r / G, head r % G), cut into tiles of R rows. A tile's
// keys are cut into parts of C keys, C such that all tiles of the call make
// some hundreds of parts: one part per tile when there are tiles enough, many
// when few long requests have to fill the card. Lengths are on the
// device, so the first wave of each workgroup reads them, four requests a
// lane, sums the work and finds its part in the prefix sums, in registers:
// about 300 instructions, where a kernel that writes the list first would cost
// every call a launch. (All four waves doing it spent
// more time on it than on small calls' keys.) The grid is what the host can
// bound; workgroups behind the last part end at once.
//
// The KV heads of a tile are neighbours in the order of parts: with 8 of them
// each of the 8 XCDs, which take workgroups in turn, keeps to one head, and
// the tiles that run there together find its keys in the XCD's own cache.
#pragma once

#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kAttnThreads = 256;
// Starting a part costs about as much as 1024 of its keys: more parts than
// there is room for on the card balance uneven lengths, but are not made
// shorter than this for it (a ragged fp32 batch of few keys: 45 us with up to
// 2048 parts, 32 us with 256).
constexpr int kLongPart = 1024;
// Requests that a wave holds, four a lane. With more of them a launch of its
// own (attn_list) sums the blocks of this many once, and a workgroup reads the
// sums instead of going through all requests: 1024 requests of one token over
// 1000 positions 675 -> 4.8 + 643 us.
constexpr int kBlock = 256;
// Granularity and least length of a part: a step of the bf16 streams, two of
// the other kernels.
constexpr int kUnit = 128;

// What a launch works on, besides AttnArgs.
struct AttnSplit {
    int R, R_log2;      // rows of a tile, a power of two
    int min_rows;       // only requests of at least min_rows rows ...
    int max_rows;       // ... and at most max_rows of them
    int most_log2;      // parts over the whole call: about as many as tiles, but not
    int some_log2;      // more than 2^most_log2, not fewer than 2^some_log2, and as few
    int few_log2;       // as 2^few_log2 rather than parts shorter than kLongPart
    long far;           // keys of all tiles above which the cache is read past the last
                        // level (see far_keys)
    int slots;          // partial results that the workspace holds
    int* table;         // of more than kBlock requests: see AttnTable; null otherwise
    float* ml;          // [slots][R][2]: running maximum (log2 domain), sum
    float* acc;         // [slots][R][d]: unnormalised rows
};

struct AttnItem {
    int req, h, tile, part, parts, tiles;
    int row0;           // first packed row of the request
    int n;              // its new tokens
    int kept;           // its tokens before them
    int C;              // keys of a part
    int slot;           // partial result of part 0, tile 0, head 0
    bool far;           // its keys and values are read once, and more than a cache holds
    bool found;
};

struct AttnReq { int n, kv, tiles, row0, kept; bool back; };

// A request from its offsets and length as they are stored; in = false: none.
template <typename A>
__device__ __forceinline__ AttnReq attn_req(const A& a, const AttnSplit& s, bool in, int lo,
                                            int hi, int kept) {
    AttnReq r;
    lo = min(max(lo, 0), a.T);
    hi = min(max(hi, 0), a.T);
    const int cap = a.width << a.page_shift;         // at most 2^30, as T is
    r.row0 = lo;
    r.n = in ? max(hi - lo, 0) : 0;
    r.back = in && hi < lo;
    r.kept = min(max(kept, A::kLeastKept), cap);
    r.kv = r.kept + min(r.n, cap - r.kept);
    if constexpr (A::kLeastKept < 0) r.kv = max(r.kv, 0);
    const int rows = r.n * (a.Hq / a.Hkv);           // at most T Hq
    r.tiles = rows >= s.min_rows && rows <= s.max_rows ? (rows + s.R - 1) >> s.R_log2 : 0;
    return r;
}

// Inclusive prefix sum over the wave: shifts inside each 16-lane row, then
// the last lane of row 0 (2) into row 1 (3) and of row 1 into rows 2 and 3.
__device__ __forceinline__ int wave_prefix(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

// Sum over the wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ long dpp_add(long x) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, false);
    return x + (long)((unsigned long)(unsigned)lo | (unsigned long)(unsigned)hi << 32);
}
__device__ __forceinline__ long wave_total(long x) {
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    x = dpp_add<0x143, 0xC>(x);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)x, 63);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(x >> 32), 63);
    return (long)((unsigned long)lo | (unsigned long)hi << 32);
}

// 256 requests of one wave, four a lane: what they were cut into. UNITS
// counts the tiles that were cut (for joining them), otherwise the parts.
template <bool UNITS>
struct AttnBlock {
    AttnReq r0, r1, r2, r3;
    int p0, p1, p2, p3;      // parts of a tile
    int f1, f2, f3, mine, p; // items before the 2nd .. 4th request, in all, and the prefix
    int c1, c2, c3, cut, q;  // the same for partial results

    template <typename A>
    __device__ void load(const A& a, const AttnSplit& s, int base) {
        // no branch between the loads: one memory latency for all of them
        const int i = base + 4 * (threadIdx.x & 63), last = a.B - 1;
        const int u0 = a.cu[min(i, a.B)], u1 = a.cu[min(i + 1, a.B)], u2 = a.cu[min(i + 2, a.B)],
                  u3 = a.cu[min(i + 3, a.B)], u4 = a.cu[min(i + 4, a.B)];
        const int k0 = a.kept_of(min(i, last)), k1 = a.kept_of(min(i + 1, last)),
                  k2 = a.kept_of(min(i + 2, last)), k3 = a.kept_of(min(i + 3, last));
        r0 = attn_req(a, s, i <= last, u0, u1, k0);
        r1 = attn_req(a, s, i + 1 <= last, u1, u2, k1);
        r2 = attn_req(a, s, i + 2 <= last, u2, u3, k2);
        r3 = attn_req(a, s, i + 3 <= last, u3, u4, k3);
    }
    __device__ int tiles() const { return r0.tiles + r1.tiles + (r2.tiles + r3.tiles); }
    // Rows that the requests claim. More than T of them in a call (some twice,
    // which takes offsets that decrease) would be more tiles than the grid and
    // the workspace are made for: such a call has no items.
    __device__ bool back() const { return r0.back || r1.back || r2.back || r3.back; }
    __device__ long claims() const { return (long)r0.n + r1.n + ((long)r2.n + r3.n); }
    __device__ long cost() const {
        return (long)r0.tiles * r0.kv + (long)r1.tiles * r1.kv +
               ((long)r2.tiles * r2.kv + (long)r3.tiles * r3.kv);
    }
    // ceil(kv / C) in fp32. C is above the call's work over 2^16 (2^most_log2, where the
    // parts are not kda_attn_even.h's units), and kv is part of that work: the quotient is
    // at most 2^16, and three roundings of 2^-24 move it by less than 0.012. Cut to a
    // whole number it may then be two too few, where the quotient is just above a whole
    // number (from 2^23 keys on), or one too many. (A request without tiles has no part
    // in the work, and its parts count for nothing.)
    static __device__ int parts(int kv, int C, float rC) {
        int n = max((int)((float)kv * rC), 1);
        // (fits 32 bits: two parts or less, and one where a part is more than 2^28 keys)
        const int rest = (int)((unsigned)kv - (unsigned)n * (unsigned)C);
        if (rest > 0) n += rest > C ? 2 : 1;
        if (rest <= -C && n > 1) --n;
        return n;
    }
    __device__ void split(const AttnArgs& a, int C) {
        const float rC = 1.f / (float)C;
        p0 = parts(r0.kv, C, rC);
        p1 = parts(r1.kv, C, rC);
        p2 = parts(r2.kv, C, rC);
        p3 = parts(r3.kv, C, rC);
        const int t0 = r0.tiles * a.Hkv, t1 = r1.tiles * a.Hkv, t2 = r2.tiles * a.Hkv,
                  t3 = r3.tiles * a.Hkv;
        const auto items = [](int t, int n) { return UNITS ? (n == 1 ? 0 : t) : t * n; };
        const auto cuts = [](int t, int n) { return n == 1 ? 0 : t * n; };
        f1 = items(t0, p0);
        f2 = f1 + items(t1, p1);
        f3 = f2 + items(t2, p2);
        mine = f3 + items(t3, p3);
        c1 = cuts(t0, p0);
        c2 = c1 + cuts(t1, p1);
        c3 = c2 + cuts(t2, p2);
        cut = c3 + cuts(t3, p3);
        p = wave_prefix(mine);
        q = wave_prefix(cut);
    }
    __device__ int items() const { return __builtin_amdgcn_readlane(p, 63); }
    __device__ int slots() const { return __builtin_amdgcn_readlane(q, 63); }
    // Item y of these, 0 <= y < items(): the lane that has it writes it down.
    __device__ void find(const AttnArgs& a, int base, int y, int slot0, int C, bool far,
                         AttnItem* to) const {
        const int local = y - (p - mine);
        if (local < 0 || local >= mine) return;
        // (a request without items begins where the next one does)
        const bool b1 = local >= f1, b2 = local >= f2, b3 = local >= f3;
        const auto of = [&](int x0, int x1, int x2, int x3) { return b3 ? x3 : b2 ? x2 : b1 ? x1 : x0; };
        const int tiles = of(r0.tiles, r1.tiles, r2.tiles, r3.tiles), n = of(p0, p1, p2, p3);
        const unsigned k = (unsigned)(local - of(0, f1, f2, f3)), rest = k / (unsigned)a.Hkv;
        const unsigned part = rest / (unsigned)max(tiles, 1);
        to->req = base + 4 * (int)(threadIdx.x & 63) + of(0, 1, 2, 3);
        to->h = (int)(k - rest * (unsigned)a.Hkv);
        // the last tile first: it sees the most keys
        to->tile = tiles - 1 - (int)(rest - part * (unsigned)tiles);
        to->part = (int)part;
        to->parts = n;
        to->tiles = tiles;
        to->row0 = of(r0.row0, r1.row0, r2.row0, r3.row0);
        to->n = of(r0.n, r1.n, r2.n, r3.n);
        to->kept = of(r0.kept, r1.kept, r2.kept, r3.kept);
        to->C = C;
        to->slot = slot0 + q - cut + of(0, c1, c2, c3);
        to->far = far && tiles == 1;
        to->found = tiles > 0 && (int)part < n;
    }
};

// What attn_list writes down: C, the call's parts and cut tiles, whether its
// keys are more than a cache holds, and for every block of kBlock requests what
// lies before it, with the totals at the end.
struct AttnTable {
    int *head, *items, *slots, *units;
    __host__ __device__ static int blocks(int B) { return (B + kBlock - 1) / kBlock; }
    __host__ __device__ static size_t ints(int B) {
        return (size_t)(4 + 3 * ((long)blocks(B) + 1) + 3) & ~(size_t)3;
    }
    __device__ AttnTable(int* t, int B)
        : head(t), items(t + 4), slots(items + blocks(B) + 1), units(slots + blocks(B) + 1) {}
};

// Keys of a part from the call's work and tiles. What follows the sums (whole
// numbers) has no product that one compiled kernel could fuse with a sum and
// another not: every workgroup of every kernel of a call gets the same C. The
// bounds below leave room for its rounding.
__device__ __forceinline__ int attn_part(const AttnArgs& a, const AttnSplit& s, long cost, int tiles) {
    const float total = (float)(cost * a.Hkv), all = (float)(tiles * a.Hkv);
    const float parts = fminf(fmaxf(all, (float)(1 << s.some_log2)), (float)(1 << s.most_log2));
    const float most = total / parts;
    const float few = total * __builtin_bit_cast(float, (127 - s.few_log2) << 23);
    const float want = fmaxf(most, fminf(few, (float)kLongPart));
    // a part covers at most all positions
    return __builtin_amdgcn_readfirstlane(((int)fminf(want, 1073741824.f) & ~(kUnit - 1)) + kUnit);
}

// The first wave's view of the call: one block of requests at a time, the only
// one of a call of up to kBlock.
template <bool UNITS>
struct AttnSched {
    AttnBlock<UNITS> block;
    int C, items;
    bool far;

    template <typename A>
    __device__ void init(const A& a, const AttnSplit& s) {
        if (s.table) {
            C = __builtin_amdgcn_readfirstlane(s.table[0]);
            items = __builtin_amdgcn_readfirstlane(s.table[UNITS ? 2 : 1]);
            far = __builtin_amdgcn_readfirstlane(s.table[3]) != 0;
            return;
        }
        block.load(a, s, 0);
        const long cost = wave_total(block.cost());
        C = attn_part(a, s, cost, __builtin_amdgcn_readlane(wave_prefix(block.tiles()), 63));
        far = cost > s.far;
        block.split(a, C);
        items = block.items();
        if (__any(block.back()) && wave_total(block.claims()) > a.T) items = 0;
    }
    // The y-th item of the call into LDS; found = false behind the last.
    template <typename A>
    __device__ void find(const A& a, const AttnSplit& s, int y, AttnItem* to) {
        if (threadIdx.x == 0) to->found = false;
        if (y >= items) return;
        int base = 0, before = 0, slot0 = 0;
        if (s.table) {
            const AttnTable t(s.table, a.B);
            const int* list = UNITS ? t.units : t.items;
            const int n = AttnTable::blocks(a.B), lane = threadIdx.x & 63;
            // the block whose successor begins behind y
            int k = 0;
            unsigned long long behind = 0;
            for (; k < n; k += 64) {
                behind = __ballot(list[min(k + lane, n - 1) + 1] > y);
                if (behind) break;
            }
            if (!behind) return;
            k += __builtin_ctzll(behind);
            base = k * kBlock;
            before = list[k];
            slot0 = t.slots[k];
            block.load(a, s, base);
            block.split(a, C);
        }
        block.find(a, base, y - before, slot0, C, far, to);
    }
};

// The item that the first wave wrote down, for the whole workgroup.
__device__ __forceinline__ AttnItem attn_shared(const AttnItem& lds) {
    __syncthreads();
    AttnItem it = lds;
    it.req = __builtin_amdgcn_readfirstlane(it.req);
    it.h = __builtin_amdgcn_readfirstlane(it.h);
    it.tile = __builtin_amdgcn_readfirstlane(it.tile);
    it.part = __builtin_amdgcn_readfirstlane(it.part);
    it.parts = __builtin_amdgcn_readfirstlane(it.parts);
    it.tiles = __builtin_amdgcn_readfirstlane(it.tiles);
    it.row0 = __builtin_amdgcn_readfirstlane(it.row0);
    it.n = __builtin_amdgcn_readfirstlane(it.n);
    it.kept = __builtin_amdgcn_readfirstlane(it.kept);
    it.C = __builtin_amdgcn_readfirstlane(it.C);
    it.slot = __builtin_amdgcn_readfirstlane(it.slot);
    it.far = __builtin_amdgcn_readfirstlane((int)it.far) != 0;
    it.found = __builtin_amdgcn_readfirstlane((int)it.found) != 0;
    return it;
}

// The x-th part of the call.
template <typename A>
__device__ __forceinline__ AttnItem attn_item(const A& a, const AttnSplit& s, int x,
                                              AttnItem& lds) {
    if (wave_id() == 0) {
        AttnSched<false> sched;
        sched.init(a, s);
        sched.find(a, s, x, &lds);
    }
    return attn_shared(lds);
}

// Bounds of the host: parts of a call whose tiles number at most `tiles`
// (KV heads included), and partial results.
inline long attn_max_items(long tiles, long target) { return tiles + target + 16; }
// (a tile that is cut has two parts or more, and fewer than twice its keys / C)
inline long attn_max_slots(long tiles, long target) {
    return (tiles < target ? tiles : target) + target + 16;
}
inline long attn_max_tiles(long T, long B, long G, long Hkv, long R) {
    return (T * G / R + (B < T ? B : T)) * Hkv;
}

}  // namespace
}  // namespace kda
