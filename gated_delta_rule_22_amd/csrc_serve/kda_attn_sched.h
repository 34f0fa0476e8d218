// Work split of the paged attention, computed by every workgroup for itself.
//
// The n new tokens of a request and the G query heads of a KV head form n * G
// rows (row r: token r / G, head r % G), cut into tiles of R rows. A tile's
// keys are cut into parts of C keys, C such that all tiles of the call make
// about `target` parts: one part per tile when there are tiles enough,
// many when few long requests have to fill the card. Lengths are on the
// device, so each workgroup reads them (B of each, coalesced), sums the work
// and finds its part in the prefix sums: about 2 us, most of it hidden by the
// other workgroups of its compute unit, against about 5 us for a kernel of
// its own that writes the list. The grid is what the host can bound.
#pragma once

#include "kda_serve_launch.h"

namespace kda {
namespace {

constexpr int kAttnThreads = 256;

// What a launch works on, besides AttnArgs.
struct AttnSplit {
    int R;              // rows of a tile
    int min_rows;       // only requests of at least min_rows rows ...
    int max_rows;       // ... and at most max_rows of them
    int unit;           // granularity and least length of a part, a power of two
    int target_log2;    // parts wanted over the whole call: 2^target_log2
    int slots;          // partial results that the workspace holds
    float* ml;          // [slots][R][2]: running maximum (log2 domain), sum
    float* acc;         // [slots][R][d]: unnormalised rows
};

struct AttnItem {
    int req, h, tile, part, parts, tiles;
    int row0;           // first packed row of the request
    int n;              // its new tokens
    int kept;           // its tokens before them
    int C;              // keys of a part
    long slot;          // partial result of part 0, tile 0, head 0
    bool found;
};

struct AttnReq { int n, kv, tiles, row0, kept; };

__device__ __forceinline__ AttnReq attn_req(const AttnArgs& a, const AttnSplit& s, int i) {
    AttnReq r{0, 0, 0, 0, 0};
    if (i >= a.B) return r;
    int lo = a.cu[i], hi = a.cu[i + 1];
    lo = min(max(lo, 0), a.T);
    hi = min(max(hi, 0), a.T);
    const int cap = a.width << a.page_shift;
    r.row0 = lo;
    r.n = max(hi - lo, 0);
    r.kept = min(max(a.kept[i], 0), cap);
    r.kv = min(r.kept + (long)r.n, (long)cap);
    const long rows = (long)r.n * (a.Hq / a.Hkv);
    r.tiles = rows >= s.min_rows && rows <= s.max_rows ? (int)((rows + s.R - 1) / s.R) : 0;
    return r;
}

struct AttnSchedLds { long wave[2][kAttnThreads / 64]; AttnItem item; long cost; };

// Exclusive prefix and total of two counters over the workgroup.
__device__ __forceinline__ void attn_scan(long& x, long& y, long& tx, long& ty, AttnSchedLds& lds) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    long ix = x, iy = y;
    for (int o = 1; o < 64; o <<= 1) {
        const long px = __shfl_up(ix, o), py = __shfl_up(iy, o);
        if (lane >= o) { ix += px; iy += py; }
    }
    __syncthreads();
    if (lane == 63) { lds.wave[0][w] = ix; lds.wave[1][w] = iy; }
    __syncthreads();
    tx = ty = 0;
    x = ix - x;
    y = iy - y;
    for (int i = 0; i < kAttnThreads / 64; ++i) {
        if (i < w) { x += lds.wave[0][i]; y += lds.wave[1][i]; }
        tx += lds.wave[0][i];
        ty += lds.wave[1][i];
    }
}

// The x-th part of the call (UNITS = false), or the x-th tile of those that
// were cut into several parts (UNITS = true: for joining them).
template <bool UNITS>
__device__ __forceinline__ AttnItem attn_item(const AttnArgs& a, const AttnSplit& s, long x,
                                              AttnSchedLds& lds) {
    const int tid = threadIdx.x;
    AttnReq first = attn_req(a, s, tid);
    long cost = (long)first.tiles * first.kv;
    for (int i = tid + kAttnThreads; i < a.B; i += kAttnThreads) {
        const AttnReq r = attn_req(a, s, i);
        cost += (long)r.tiles * r.kv;
    }
    long zero = 0, total, none;
    attn_scan(cost, zero, total, none, lds);
    // a part covers at most all positions, which fit 31 bits
    const long want = (total * a.Hkv) >> s.target_log2;
    const int C = (int)min((want & ~(long)(s.unit - 1)) + s.unit, (long)INT32_MAX);
    if (tid == 0) lds.item.found = false;
    long at = 0, slot0 = 0;
    for (int base = 0; base < a.B; base += kAttnThreads) {
        const AttnReq r = base == 0 ? first : attn_req(a, s, base + tid);
        const unsigned parts = r.kv > C ? ((unsigned)r.kv + (unsigned)C - 1) / (unsigned)C : 1;
        const long tiles = (long)r.tiles * a.Hkv;
        const long here = parts * tiles;
        const long mine = UNITS ? (parts > 1 ? tiles : 0) : here;
        long p = mine, q = parts > 1 ? here : 0, tp, tq;
        attn_scan(p, q, tp, tq, lds);
        if (x >= at + p && x < at + p + mine) {
            const unsigned local = (unsigned)(x - at - p), rest = local / (unsigned)a.Hkv;
            AttnItem it;
            it.req = base + tid;
            it.h = (int)(local % (unsigned)a.Hkv);
            // the last tile first: it sees the most keys
            it.tile = r.tiles - 1 - (int)(rest % (unsigned)r.tiles);
            it.part = (int)(rest / (unsigned)r.tiles);
            it.parts = (int)parts;
            it.tiles = r.tiles;
            it.row0 = r.row0;
            it.n = r.n;
            it.kept = r.kept;
            it.C = C;
            it.slot = slot0 + q;
            it.found = true;
            lds.item = it;
        }
        at += tp;
        slot0 += tq;
        if (x < at) break;                 // the same for every thread
    }
    __syncthreads();
    return lds.item;
}

// Bounds of the host: parts of a call whose tiles number at most `tiles`
// (KV heads included), and partial results.
inline long attn_max_items(long tiles, long target) { return tiles + target; }
inline long attn_max_slots(long target) { return 2 * target; }
inline long attn_max_tiles(long T, long B, long G, long Hkv, long R) {
    return (T * G / R + (B < T ? B : T)) * Hkv;
}

}  // namespace
}  // namespace kda
