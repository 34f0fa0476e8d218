// Work split for attention kernels that fill the card with one launch: G groups of
// workgroups, as many as its compute units hold (one or two each), and each an even share of
// the call's keys.
//
// The rows of a request are cut into tiles of R times `side` rows as in
// kda_attn_sched.h (one KV head). A tile is a number of units: its keys in Cs, behind
// `start` units without keys that stand for what beginning it costs. The units of all
// tiles in a row, cut into G ranges of equal length, are the groups' work: whole
// tiles, and at either end of a range a piece of one that neighbours have the rest of.
// (Parts of one length, dealt out to the compute units in turn, left some of them a third
// more to do than others.) Every workgroup finds its range from the lengths on the device.
//
// A group is `side` workgroups, each with R rows of its tiles: they read the same keys
// at the same time, on the same XCD, in whose cache all but the first find them.
//
// A piece's rows go to the workspace, at most two pieces a workgroup, and a second
// kernel joins them. The workgroup that has a tile's second piece describes the
// tile to it.
#pragma once

#include <type_traits>

#include "kda_attn_rows.h"

namespace kda {
namespace {

struct EvenSplit {
    int R;              // rows of a workgroup; AttnSplit has those of a tile
    int side;           // workgroups side by side
    int G;              // groups of them
    int* table;         // of more than kBlock requests: see AttnTable; null otherwise
    int* pieces;        // [G side][4]: first row, tile of R rows, new tokens, pieces (0: none) of
                        // the tile whose second piece this workgroup has
    float* ml;          // [2 G side][R][2]: running maximum (log2 domain), sum
    float* acc;         // [2 G side][R][d]: unnormalised rows
};

// Keys of a unit: 64, or what makes the call some 2^16 units. (cost: tiles times keys,
// and a key more for each tile, so that there are never 2^31 units.)
constexpr int kUnitKeys = 64;
__device__ __forceinline__ int even_unit(long cost) {
    const float want = (float)cost * 0x1p-16f;
    return __builtin_amdgcn_readfirstlane(((int)fminf(want, 1073741824.f) & ~(kUnitKeys - 1)) + kUnitKeys);
}
// Units without keys: a tile's start costs about what 128 of its keys do.
__device__ __forceinline__ int even_start(int C) { return C == 64 ? 2 : C == 128 ? 1 : 0; }

// A tile, or a request's place among the units.
struct EvenItem {
    int req, tile;
    int row0, n, kept;  // of the request: first packed row, new tokens, tokens before them
    int unit, units;    // the unit asked for, in its tile, and the tile's number of them
    int C, start;
    int total;          // units of the call
    bool found;
};

// 256 requests of one wave, four a lane.
struct EvenBlock : AttnBlock<false> {
    __device__ void split_even(int C) {
        const float rC = 1.f / (float)C;
        const int start = even_start(C);
        p0 = parts(r0.kv, C, rC) + start;
        p1 = parts(r1.kv, C, rC) + start;
        p2 = parts(r2.kv, C, rC) + start;
        p3 = parts(r3.kv, C, rC) + start;
        f1 = r0.tiles * p0;
        f2 = f1 + r1.tiles * p1;
        f3 = f2 + r2.tiles * p2;
        mine = f3 + r3.tiles * p3;
        p = wave_prefix(mine);
    }
    // Unit y of these: the lane that has it writes it down.
    __device__ void find_even(int base, int y, int C, EvenItem* to) const {
        const int local = y - (p - mine);
        if (local < 0 || local >= mine) return;
        const bool b1 = local >= f1, b2 = local >= f2, b3 = local >= f3;
        const auto of = [&](int x0, int x1, int x2, int x3) { return b3 ? x3 : b2 ? x2 : b1 ? x1 : x0; };
        const int tiles = of(r0.tiles, r1.tiles, r2.tiles, r3.tiles);
        const unsigned units = (unsigned)of(p0, p1, p2, p3), k = (unsigned)(local - of(0, f1, f2, f3));
        const int t = (int)(k / units);
        to->req = base + 4 * (int)(threadIdx.x & 63) + of(0, 1, 2, 3);
        // early tiles of a prompt see few keys, late ones many: in turn from both ends
        to->tile = t & 1 ? tiles - 1 - t / 2 : t / 2;
        to->row0 = of(r0.row0, r1.row0, r2.row0, r3.row0);
        to->n = of(r0.n, r1.n, r2.n, r3.n);
        to->kept = of(r0.kept, r1.kept, r2.kept, r3.kept);
        to->unit = (int)(k - t * units);
        to->units = (int)units;
        to->C = C;
        to->start = even_start(C);
        to->found = tiles > 0;
    }
};

// Units [even_begin(w), even_begin(w + 1)) are workgroup w's; of a call of fewer units
// than workgroups, only as many of these have one.
__device__ __forceinline__ int even_groups(const EvenSplit& e, int total) { return min(e.G, total); }
__device__ __forceinline__ int even_begin(const EvenSplit& e, int total, int w) {
    const int G = even_groups(e, total);
    return w < G ? (int)((long)w * total / G) : total;
}

// The runs from unit y of the call, or workgroup w's first one (y < 0), up to that
// workgroup's last unit, into LDS; by one wave. found = false: there are no more. Several
// at once, for each alone would wait for the lengths again (a call of more than kBlock
// requests: one, the others may be in other blocks).
constexpr int kEvenRuns = 4;
__device__ __forceinline__ int even_at_once(const EvenSplit& e) { return e.table ? 1 : kEvenRuns; }
template <typename A>
__device__ __forceinline__ void even_find(const A& a, const AttnSplit& s, const EvenSplit& e, int y, int w,
                                          EvenItem* to) {
    const int lane = threadIdx.x & 63;
    EvenBlock block;
    int C, total, base = 0, before = 0;
    if (e.table) {
        const AttnTable t(e.table, a.B);
        const int n = AttnTable::blocks(a.B);
        C = __builtin_amdgcn_readfirstlane(t.head[0]);
        total = __builtin_amdgcn_readfirstlane(t.head[1]);
        if (y < 0) y = even_begin(e, total, w);
        int k = 0;
        unsigned long long behind = 0;
        for (; k < n; k += 64) {
            behind = __ballot(t.items[min(k + lane, n - 1) + 1] > y);
            if (behind) break;
        }
        if (behind) {
            k += __builtin_ctzll(behind);
            base = k * kBlock;
            before = t.items[k];
        }
        block.load(a, s, base);
        block.split_even(C);
    } else {
        block.load(a, s, 0);
        C = even_unit(wave_total(block.cost() + block.tiles()));
        block.split_even(C);
        total = __builtin_amdgcn_readlane(block.p, 63);
        if (__any(block.back()) && wave_total(block.claims()) > a.T) total = 0;
        if (y < 0) y = even_begin(e, total, w);
    }
    const int y1 = even_begin(e, total, w + 1);
    for (int k = 0; k < even_at_once(e); ++k) {
        if (lane == 0) {
            to[k].found = false;
            to[k].total = total;
        }
        if (y >= y1) continue;
        block.find_even(base, y - before, C, to + k);
        lds_fence_wave();
        y += min(uniform(to[k].units) - uniform(to[k].unit), y1 - y);
    }
}

// What a workgroup has of a tile.
struct EvenRun {
    int req, tile, row0, n, kept;
    int begin, end;     // keys (end: not cut at the request's length)
    int piece, pieces;
    int slot;           // of a piece: the group's first run has even ones, its last odd ones
    int units;          // the run's
};
__device__ __forceinline__ EvenRun even_run(const EvenItem& lds, const EvenSplit& e, int w, int y, int y1) {
    const auto u = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    EvenRun r;
    r.req = u(lds.req);
    r.tile = u(lds.tile);
    r.row0 = u(lds.row0);
    r.n = u(lds.n);
    r.kept = u(lds.kept);
    const int unit = u(lds.unit), units = u(lds.units), C = u(lds.C), start = u(lds.start), total = u(lds.total);
    r.units = min(units - unit, y1 - y);
    r.begin = max(unit - start, 0) * C;
    r.end = (int)min((long)max(unit + r.units - start, 0) * C, (long)1 << 30);
    // workgroups of the first and the last unit that have keys
    const long first = (long)y - unit + start, last = (long)y - unit + units - 1;
    const long G = even_groups(e, total);
    const int w0 = (int)(((first + 1) * G - 1) / total), w1 = (int)(((last + 1) * G - 1) / total);
    r.piece = w - w0;   // below 0: of this tile only units without keys
    r.pieces = w1 - w0 + 1;
    r.slot = r.piece > 0 ? 0 : 1;
    return r;
}

// The keys of a run, and what of them needs a mask.
__device__ __forceinline__ Keys run_keys(const AttnArgs& a, const EvenRun& it, int R) {
    const int cap = a.width << a.page_shift;
    const int rows = it.n * a.Hq, r0 = it.tile * R, r1 = min(r0 + R, rows) - 1;
    Keys k;
    k.begin = it.begin;
    const int last = (int)((unsigned)r1 / (unsigned)a.Hq), first = (int)((unsigned)r0 / (unsigned)a.Hq);
    k.end = (int)min(min((long)it.end, (long)it.kept + last + 1), (long)cap);
    k.all = (int)min((long)it.kept + first + 1, (long)cap);
    return k;
}

// Row r of the run's request: packed row and query head.
__device__ __forceinline__ RowAt run_row(const AttnArgs& a, const EvenRun& it, int r) {
    AttnItem x{};
    x.row0 = it.row0;
    x.n = it.n;
    return row_at(a, x, a.Hq, r);
}

// A workgroup's runs in turn, each with what is left in LDS free to use.
template <typename A, typename F>
__device__ __forceinline__ void even_runs(const A& a, const AttnSplit& s, const EvenSplit& e, EvenItem* items, F run) {
    // workgroups go to the 8 XCDs in turn: neighbours in the units on the same one
    const int n = gridDim.x, b = blockIdx.x, v = n % 8 ? b : b % 8 * (n / 8) + b / 8;
    const int w = v / e.side, side = v - w * e.side;
    int y = -1, y1 = 0;
    for (;;) {
        if (wave_id() == 0) even_find(a, s, e, y, w, items);
        __syncthreads();
        for (int k = 0; k < even_at_once(e); ++k) {
            const EvenItem& item = items[k];
            const bool first = y < 0;
            if (first) {
                const int total = uniform(item.total);
                y = even_begin(e, total, w);
                y1 = even_begin(e, total, w + 1);
            }
            const bool more = y < y1 && uniform((int)item.found) != 0;
            EvenRun it{};
            if (more) it = even_run(item, e, w, y, y1);
            it.tile = it.tile * e.side + side;
            it.slot += 2 * v;
            const bool rows = it.tile * e.R < it.n * a.Hq;
            if (first && threadIdx.x == 0) {
                int* x = e.pieces + 4 * v;
                x[0] = it.row0;
                x[1] = it.tile;
                x[2] = it.n;
                x[3] = more && rows && it.piece == 1 ? it.pieces : 0;
            }
            if (!more) return;
            y += it.units;
            if (it.piece >= 0 && rows) run(it);
            __syncthreads();                         // the run's last reads of LDS are done
        }
    }
}

// The list of a call of more than kBlock requests: the units in front of each block.
template <typename A>
__global__ __launch_bounds__(64 * kListWaves) void even_list(A a, AttnSplit s, EvenSplit e) {
    __shared__ long cost_of[kListWaves], claims_of[kListWaves];
    const AttnTable t(e.table, a.B);
    const int n = AttnTable::blocks(a.B), wave = wave_id(), lane = threadIdx.x & 63;
    long cost = 0, claims = 0;
    for (int k = wave; k < n; k += kListWaves) {
        EvenBlock b;
        b.load(a, s, k * kBlock);
        cost += b.cost() + b.tiles();
        claims += b.claims();
    }
    cost = wave_total(cost);
    claims = wave_total(claims);
    if (lane == 0) {
        cost_of[wave] = cost;
        claims_of[wave] = claims;
    }
    __syncthreads();
    cost = claims = 0;
    for (int w = 0; w < kListWaves; ++w) {
        cost += cost_of[w];
        claims += claims_of[w];
    }
    const int C = even_unit(cost);
    for (int k = wave; k < n; k += kListWaves) {
        EvenBlock b;
        b.load(a, s, k * kBlock);
        b.split_even(C);
        const int items = __builtin_amdgcn_readlane(b.p, 63);
        if (lane == 0) t.items[k] = items;
    }
    __syncthreads();
    if (wave != 0) return;
    int items = 0;
    for (int k = 0; k < n; k += 64) {
        const bool in = k + lane < n;
        const int x = in ? t.items[k + lane] : 0, px = wave_prefix(x);
        if (in) t.items[k + lane] = items + px - x;
        items += __builtin_amdgcn_readlane(px, 63);
    }
    if (lane == 0) {
        t.items[n] = items;
        t.head[0] = C;
        t.head[1] = claims > a.T ? 0 : items;
    }
}

// What joins from a piece, or from the pieces that some lanes have joined. Without weights
// (scores of -infinity alone) its values are 0, or NaN where a position's are not finite:
// that has to reach the row.
__device__ __forceinline__ Joined with_odd(Joined x) {
    if (x.l == 0.f) x.l = (x.v[0] + x.v[1]) + (x.v[2] + x.v[3]);
    return x;
}

// Joins the pieces of the tiles that were cut, their rows shared evenly by the
// workgroups. Every workgroup reads the descriptions of all G and puts the tiles in
// order. Up to 16 pieces a group of D / 4 lanes has a row; with more the groups share
// one row, each takes its share of the pieces, and the shares join through LDS.
constexpr int kEvenMost = 512;       // workgroups G of a call
constexpr int kEvenJoins = 1024;
template <typename T, int D, typename A>
__global__ __launch_bounds__(kAttnThreads) void even_join(A a, EvenSplit e) {
    constexpr int kLanes = D / 4, kGroups = kAttnThreads / kLanes;
    __shared__ int rows_to[kEvenMost];               // rows of the tiles up to workgroup w's
    __shared__ int wave_rows[4];
    __shared__ __align__(16) float lds_v[kGroups][D];
    __shared__ float lds_ml[kGroups][2];
    const int group = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    {
        // two neighbours a thread
        int mine[2];
        for (int i = 0; i < 2; ++i) {
            const int w = 2 * (int)threadIdx.x + i;
            mine[i] = 0;
            if (w >= e.G * e.side) continue;
            const i32x4 x = *(const i32x4*)(e.pieces + 4 * w);
            if (x[3] > 0) mine[i] = max(min(e.R, x[2] * a.Hq - x[1] * e.R), 0);
        }
        const int p = wave_prefix(mine[0] + mine[1]);
        if ((threadIdx.x & 63) == 63) wave_rows[threadIdx.x >> 6] = p;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < 4; ++w) before += w < (int)(threadIdx.x >> 6) ? wave_rows[w] : 0;
        rows_to[2 * threadIdx.x] = before + p - mine[1];
        rows_to[2 * threadIdx.x + 1] = before + p;
        __syncthreads();
    }
    const int all = rows_to[kEvenMost - 1];
    const int r0 = (int)((long)all * blockIdx.x / gridDim.x), r1 = (int)((long)all * (blockIdx.x + 1) / gridDim.x);
    if (r0 >= r1) return;
    int w = 0;
    {
        int lo = 0, hi = kEvenMost - 1;              // the first with rows_to > r0
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (rows_to[mid] > r0) hi = mid;
            else lo = mid + 1;
        }
        w = lo;
    }
    for (int r = r0; r < r1; ++w) {
        const int end = min(rows_to[w], r1), from = w ? rows_to[w - 1] : 0;
        if (end <= r) continue;                      // (a workgroup without a tile to describe)
        const i32x4 x = *(const i32x4*)(e.pieces + 4 * w);
        const int row_a = r - from, have = end - r, pieces = x[3];
        r = end;
        // pieces of the group before this one (its last run), this one's, the next one's, ...
        // (their first ones)
        const int v0 = w - e.side;
        if (v0 < 0 || v0 + (pieces - 1) * e.side >= e.G * e.side) continue;   // (a guard)
        const auto part = [&](int row, int p) {
            const bool in = p < pieces;
            const int slot = !in || p == 0 ? 2 * v0 + 1 : 2 * (v0 + p * e.side);
            const long at = (long)slot * e.R + row;
            Joined y;
            y.m = e.ml[at * 2];
            y.l = e.ml[at * 2 + 1];
            y.v = *(const f32x4*)(e.acc + at * D + d);
            y = with_odd(y);
            if (!in) y.l = 0.f;
            return y;
        };
        const auto write = [&](const Joined& y, int row) {
            AttnItem it{};
            it.row0 = x[0];
            it.n = x[2];
            const RowAt to = row_at(a, it, a.Hq, x[1] * e.R + row);
            const float inv = y.l == 0.f ? 0.f : 1.f / y.l;
            T* o = (T*)a.o + to.q * D + d;
            for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(y.v[i] * inv);
            if (a.lse && d == 0) a.lse[to.q] = y.l == 0.f ? -INFINITY : (y.m + __log2f(y.l)) * kLn2;
        };
        // N pieces of each of M rows in flight
        const auto few = [&](auto n, auto m) {
            constexpr int N = decltype(n)::value, M = decltype(m)::value;
            for (int row = group; row < have; row += M * kGroups) {
                Joined z[M][N];
#pragma unroll
                for (int r = 0; r < M; ++r)
#pragma unroll
                    for (int p = 0; p < N; ++p) z[r][p] = part(row_a + min(row + r * kGroups, have - 1), p);
#pragma unroll
                for (int r = 0; r < M; ++r) {
                    Joined y;
#pragma unroll
                    for (int p = 0; p < N; ++p) y.add(z[r][p]);
                    if (row + r * kGroups < have) write(y, row_a + row + r * kGroups);
                }
            }
        };
        if (pieces <= 2) {
            few(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
            continue;
        }
        if (pieces <= 4) {
            few(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
            continue;
        }
        if (pieces <= 16) {                          // eight pieces in flight
            for (int row = group; row < have; row += kGroups) {
                Joined y;
                for (int p = 0; p < pieces; p += 8) {
                    Joined z[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = part(row_a + row, p + i);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y.add(z[i]);
                }
                write(y, row_a + row);
            }
            continue;
        }
        for (int row = 0; row < have; ++row) {
            Joined y;
            for (int p = group; p < pieces; p += 8 * kGroups) {
                Joined z[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = part(row_a + row, p + i * kGroups);
#pragma unroll
                for (int i = 0; i < 8; ++i) y.add(z[i]);
            }
            __syncthreads();                         // the last row's shares are read
            *(f32x4*)&lds_v[group][d] = y.v;
            if (d == 0) { lds_ml[group][0] = y.m; lds_ml[group][1] = y.l; }
            __syncthreads();
            if (group == 0) {
                Joined z;
                for (int g = 0; g < kGroups; ++g) {
                    Joined x1;
                    x1.m = lds_ml[g][0];
                    x1.l = lds_ml[g][1];
                    x1.v = *(const f32x4*)&lds_v[g][d];
                    z.add(with_odd(x1));
                }
                write(z, row_a + row);
            }
        }
    }
}

}  // namespace
}  // namespace kda
