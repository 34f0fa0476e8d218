// What the attention kernels share: rows and keys of a part, the softmax
// weights' two terms, loads to LDS, and the kernels that list the parts of many
// requests and join those of cut tiles.
#pragma once

#include "kda_attn_sched.h"

namespace kda {
namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr int kKeepAll = 1 << 30;

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ bool finite_bits(float x) {
    return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) != 0x7f800000u;
}
// x with 0 for its values that are not finite; odd is set if there is one.
__device__ __forceinline__ bf16x8 only_finite(bf16x8 x, bool& odd) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 w = __builtin_bit_cast(u32x4, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = w[j];
        const uint32_t lo = (u & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
        const uint32_t hi = (u & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
        odd |= (lo | hi) != 0;
        w[j] = u & ~(lo | hi);
    }
    return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ f32x4 mma4(float a, float b, f32x4 c) {
    // D(16x16) += A(16x4) B(4x16), fp32: lane l holds A[l%16][l/16], B[l/16][l%16]
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Eight weights p >= 0 as two bf16 terms each: the leading bits cut off, and what
// is left of p (1 + 2^-20). One term would lose up to 2^-8 of a weight, as much
// as the result's own rounding does (2.0e-3 to 2.3e-3 from fp64 in all instead of
// 1.7e-3); two lose 2^-15 (1.7e-3 in all). The second one's products cost the
// streams nothing and prompts a quarter to a third: 8192 tokens over 24576
// positions, 32 heads over 8 of 128, 4.0 -> 5.3 ms, 4096 over 12000 of width 64
// 0.66 -> 0.83 ms. The 2^-20 keeps the second term of p > 0 above 0, so
// that both have the sign of p and an infinite value stays infinite.
__device__ __forceinline__ void two_terms(const float (&p)[8], bf16x8& hi, bf16x8& lo) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 h;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint32_t a = __builtin_bit_cast(uint32_t, p[j]), b = __builtin_bit_cast(uint32_t, p[j + 1]);
        h[j / 2] = __builtin_amdgcn_perm(b, a, 0x07060302);      // upper halves
        lo[j] = (bf16)__builtin_fmaf(p[j], 1.f + 0x1p-20f, -__builtin_bit_cast(float, a & 0xffff0000u));
        lo[j + 1] = (bf16)__builtin_fmaf(p[j + 1], 1.f + 0x1p-20f, -__builtin_bit_cast(float, b & 0xffff0000u));
    }
    hi = __builtin_bit_cast(bf16x8, h);
}

// The same for four.
__device__ __forceinline__ void two_terms(const float (&p)[4], bf16x4& hi, bf16x4& lo) {
    const float q[8] = {p[0], p[1], p[2], p[3], 0.f, 0.f, 0.f, 0.f};
    bf16x8 h, l;
    two_terms(q, h, l);
    hi = __builtin_shufflevector(h, h, 0, 1, 2, 3);
    lo = __builtin_shufflevector(l, l, 0, 1, 2, 3);
}

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Largest over the four lanes l % 16 + {0, 16, 32, 48}.
__device__ __forceinline__ float max_quarters(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float sum_quarters(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Row r of a request: packed row and query head.
struct RowAt { bool in; long q; int t; };
__device__ __forceinline__ RowAt row_at(const AttnArgs& a, const AttnItem& it, int G, int r) {
    const unsigned t = (unsigned)r / (unsigned)G;
    RowAt x;
    x.in = (int)t < it.n;
    x.t = (int)t;
    x.q = (long)(it.row0 + (x.in ? (int)t : 0)) * a.Hq + it.h * G + (int)((unsigned)r - t * (unsigned)G);
    return x;
}
// Range of keys of a part, and what of it needs a mask.
struct Keys {
    int begin, end;      // the part's positions
    int all;             // positions below are visible to every row of the tile
};
__device__ __forceinline__ Keys part_keys(const AttnArgs& a, const AttnSplit& s,
                                          const AttnItem& it, int G) {
    const int cap = a.width << a.page_shift;
    const int rows = it.n * G, r0 = it.tile * s.R, r1 = min(r0 + s.R, rows) - 1;
    Keys k;
    k.begin = it.part * it.C;
    const int last = (int)((unsigned)r1 / (unsigned)G), first = (int)((unsigned)r0 / (unsigned)G);
    k.end = (int)min(min((long)k.begin + it.C, (long)it.kept + last + 1), (long)cap);
    k.all = (int)min((long)it.kept + first + 1, (long)cap);
    return k;
}

// A request's row of the block table. Nothing writes it while the kernel runs,
// so its entries are read as constants: scalar loads, which do not wait for
// the keys and values in flight as vector loads would.
typedef const __attribute__((address_space(4))) int const_int;
__device__ __forceinline__ const_int* table_row(const AttnArgs& a, int req) {
    return (const_int*)(uintptr_t)(a.table + (long)req * a.width);
}
// Page id of the 16 positions at pos (a multiple of 16), -1 when there is none.
// Behind the end (end > 0) the last page's entry is read instead: no branch,
// so that several loads are in flight at once.
__device__ __forceinline__ int page_at(const AttnArgs& a, const_int* table, int pos, int end) {
    const int p = table[min(pos, end - 1) >> a.page_shift];
    return pos < end && (unsigned)p < (unsigned)a.pool ? p : -1;
}
// Which 16-byte piece of a row of D values LDS holds in place of piece c, so
// that the reads of 16 lanes (16 bytes each) or 32 (8 bytes) cover the 64
// banks once. Rows are 2 D bytes, 256 / (2 D) of them cover the banks.
// K: 16 lanes read piece c of 16 keys.
template <int D> __device__ __forceinline__ int k_piece(int key, int c) {
    return D >= 128 ? c ^ (key & 15) : c ^ (key >> 1 & 7);
}
// V, transposing reads: 32 lanes take 64 bytes of four consecutive keys, ...
template <int D> __device__ __forceinline__ int v_piece4(int key, int c) {
    return D >= 128 ? c ^ 4 * (key & 3) : c ^ 4 * (key >> 1 & 1);
}
// ... or 32 bytes of eight.
template <int D> __device__ __forceinline__ int v_piece8(int key, int c) {
    return D >= 128 ? c ^ 2 * (key & 7) : D == 64 ? c ^ 2 * (key >> 1 & 3)
         : D == 32 ? c ^ 2 * (key >> 2 & 1) : c;
}

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// D(32x32) += A(32x16) B(16x32): lane l holds A[l%32][8(l/32)..+7],
// B[8(l/32)..+7][l%32], D[8(i/4) + 4(l/32) + i%4][l%32] in element i.
__device__ __forceinline__ f32x16 mma_big(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float max_halves(float x) { return fmaxf(x, __shfl_xor(x, 32)); }

// 16 bytes a lane from base + off (bytes, per lane) to LDS at the wave's
// address `to`, in the order of the lanes. As inline assembly, because the
// compiler otherwise waits for all of them before it reads any LDS with a
// transposing load; there is no result register, and the kernel waits itself.
__device__ __forceinline__ void load_to_lds(uint32_t to, uint32_t off, const void* base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 ::"s"(to), "v"(off), "s"(base) : "memory", "m0");
}

// The lists of a call of many requests (AttnTable), a workgroup for each of
// its launches: sixteen waves sum the work and then the parts of their blocks,
// the first one puts the blocks' sums in order. 4096 requests of one token over
// 300 positions, 8 KV heads of 128: 8.0 us (1024 requests: 5.0), memory
// latencies of two passes over the lengths, which stay in the cache for the second.
constexpr int kListWaves = 16;
template <typename A>
__global__ __launch_bounds__(64 * kListWaves) void attn_list(A a, AttnSplit s0, AttnSplit s1) {
    __shared__ long cost_of[kListWaves], claims_of[kListWaves];
    __shared__ int tiles_of[kListWaves];
    const AttnSplit& s = blockIdx.x == 0 ? s0 : s1;
    const AttnTable t(s.table, a.B);
    const int n = AttnTable::blocks(a.B), wave = wave_id(), lane = threadIdx.x & 63;
    long cost = 0, claims = 0;
    int tiles = 0;
    for (int k = wave; k < n; k += kListWaves) {
        AttnBlock<false> b;
        b.load(a, s, k * kBlock);
        cost += b.cost();
        claims += b.claims();
        tiles += b.tiles();
    }
    cost = wave_total(cost);
    claims = wave_total(claims);
    tiles = __builtin_amdgcn_readlane(wave_prefix(tiles), 63);
    if (lane == 0) {
        cost_of[wave] = cost;
        claims_of[wave] = claims;
        tiles_of[wave] = tiles;
    }
    __syncthreads();
    cost = claims = 0;
    tiles = 0;
    for (int w = 0; w < kListWaves; ++w) {
        cost += cost_of[w];
        claims += claims_of[w];
        tiles += tiles_of[w];
    }
    const int C = attn_part(a, s, cost, tiles);
    for (int k = wave; k < n; k += kListWaves) {
        AttnBlock<false> b;
        b.load(a, s, k * kBlock);
        b.split(a, C);
        AttnBlock<true> u = __builtin_bit_cast(AttnBlock<true>, b);
        u.split(a, C);
        // (read from lane 63 by the whole wave: the sum's last step must not be
        // moved to where only lane 0 is active)
        const int items = b.items(), slots = b.slots(), units = u.items();
        if (lane == 0) {
            t.items[k] = items;
            t.slots[k] = slots;
            t.units[k] = units;
        }
    }
    __syncthreads();
    if (wave != 0) return;
    // in place: each block's own count -> what lies before it
    int items = 0, slots = 0, units = 0;
    for (int k = 0; k < n; k += 64) {
        const bool in = k + lane < n;
        const int x = in ? t.items[k + lane] : 0, y = in ? t.slots[k + lane] : 0,
                  z = in ? t.units[k + lane] : 0;
        const int px = wave_prefix(x), py = wave_prefix(y), pz = wave_prefix(z);
        if (in) {
            t.items[k + lane] = items + px - x;
            t.slots[k + lane] = slots + py - y;
            t.units[k + lane] = units + pz - z;
        }
        items += __builtin_amdgcn_readlane(px, 63);
        slots += __builtin_amdgcn_readlane(py, 63);
        units += __builtin_amdgcn_readlane(pz, 63);
    }
    if (lane == 0) {
        t.items[n] = items;
        t.slots[n] = slots;
        t.units[n] = units;
        t.head[0] = C;
        t.head[1] = claims > a.T ? 0 : items;
        t.head[2] = claims > a.T ? 0 : units;
        t.head[3] = cost > s.far;
    }
}
// Joins the parts of tiles that were cut, rows shared evenly by the workgroups.
// A group of D / 4 lanes holds four columns each of a row. Up to 16 parts every
// group has a row of its own. With more the groups share one row, each takes
// its share of the parts, and the shares join through LDS. A part without a key
// of the row has l = 0 (and NaN scores leave m at -infinity, but not l at 0).
struct Joined {
    float m = -INFINITY, l = 0.f;
    f32x4 v = zero4();
    __device__ void add(const Joined& x) {
        const bool none = x.l == 0.f;
        const float mn = none ? m : fmaxf(m, x.m);
        const float c = m == -INFINITY ? 1.f : exp2_f(m - mn);
        const float c1 = none ? 0.f : x.m == -INFINITY ? 1.f : exp2_f(x.m - mn);
        l = l * c + x.l * c1;
        for (int i = 0; i < 4; ++i) v[i] = v[i] * c + (none ? 0.f : x.v[i] * c1);
        m = mn;
    }
};

template <typename T, int D, typename A>
__global__ __launch_bounds__(kAttnThreads) void attn_join(A a, AttnSplit s0, AttnSplit s1, int n0) {
    constexpr int kLanes = D / 4, kGroups = kAttnThreads / kLanes;
    __shared__ __align__(16) float lds_v[kGroups][D];
    __shared__ float lds_ml[kGroups][2];
    const int G = a.Hq / a.Hkv;
    const int group = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
    // the first n0 workgroups join the first launch's parts
    const bool one = (int)blockIdx.x < n0;
    const AttnSplit& s = one ? s0 : s1;
    const unsigned block = one ? blockIdx.x : blockIdx.x - n0, blocks = one ? n0 : gridDim.x - n0;
    __shared__ AttnItem shared_item;
    __shared__ int shared_units;
    AttnSched<true> sched;
    if (wave_id() == 0) {
        sched.init(a, s);
        if (threadIdx.x == 0) shared_units = sched.items;
    }
    __syncthreads();
    // an even share of the rows of all cut tiles, of which the partial results
    // are two or more each
    const unsigned all = (unsigned)min(max(uniform(shared_units), 0), s.slots) << s.R_log2;
    const unsigned share = (all + blocks - 1) / blocks;
    const unsigned row_end = min(all, share * (block + 1));
    for (unsigned r = share * block; r < row_end;) {
        const int x = (int)(r >> s.R_log2), row0 = (int)(r & (s.R - 1));
        __syncthreads();                             // the last item is read
        if (wave_id() == 0) sched.find(a, s, x, &shared_item);
        const AttnItem it = attn_shared(shared_item);
        const int rows = (int)min((unsigned)(s.R - row0), row_end - r);
        r += rows;
        const int step = it.tiles * a.Hkv, slot = it.slot + it.tile * a.Hkv + it.h;
        // (a guard)
        if (!it.found || slot < 0 || slot + (long)step * (it.parts - 1) >= s.slots) continue;
        const int have = min(rows, it.n * G - (it.tile * s.R + row0));   // rows that exist
        auto part = [&](int row, int p) {
            const bool in = p < it.parts;
            const long from = (long)(slot + step * (in ? p : 0)) * s.R + row;
            Joined y;
            y.m = s.ml[from * 2];
            y.l = in ? s.ml[from * 2 + 1] : 0.f;
            y.v = *(const f32x4*)(s.acc + from * D + d);
            return y;
        };
        auto write = [&](const Joined& y, int row) {
            const RowAt to = row_at(a, it, G, it.tile * s.R + row);
            const float inv = y.l == 0.f ? 0.f : 1.f / y.l;
            T* o = (T*)a.o + to.q * D + d;
            for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(y.v[i] * inv);
            if (a.lse && d == 0) a.lse[to.q] = y.l == 0.f ? -INFINITY : (y.m + __log2f(y.l)) * kLn2;
        };
        if (it.parts <= 4) {                         // two rows in flight
            for (int row = group; row < have; row += 2 * kGroups) {
                const int other = min(row + kGroups, have - 1);
                Joined y[8], z, z1;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    y[p] = part(row0 + row, p);
                    y[4 + p] = part(row0 + other, p);
                }
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    z.add(y[p]);
                    z1.add(y[4 + p]);
                }
                write(z, row0 + row);
                if (row + kGroups < have) write(z1, row0 + other);
            }
            continue;
        }
        if (it.parts <= 16) {                        // eight parts in flight
            for (int row = group; row < have; row += kGroups) {
                Joined y;
                for (int p = 0; p < it.parts; p += 8) {
                    Joined z[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = part(row0 + row, p + i);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y.add(z[i]);
                }
                write(y, row0 + row);
            }
            continue;
        }
        for (int row = 0; row < have; ++row) {
            Joined y;
            for (int p = group; p < it.parts; p += 8 * kGroups) {
                Joined z[8];                         // eight parts in flight
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = part(row0 + row, p + i * kGroups);
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
                    z.add(x1);
                }
                write(z, row0 + row);
            }
        }
    }
}

struct Launch {
    AttnSplit split;
    long items, joins;     // workgroups
};
Launch launch_of(long T, long B, long G, long Hkv, int R, int most_log2, int some_log2,
                 int few_log2, int max_rows) {
    Launch l{};
    l.split.R = R;
    l.split.R_log2 = __builtin_ctz((unsigned)R);
    l.split.min_rows = 1;
    l.split.max_rows = max_rows;
    l.split.most_log2 = most_log2;
    l.split.some_log2 = some_log2;
    l.split.few_log2 = few_log2;
    // requests of no more rows than a tile are a tile each
    const long target = 1l << most_log2;
    const long tiles = max_rows <= R ? (B < T ? B : T) * Hkv : attn_max_tiles(T, B, G, Hkv, R);
    l.items = attn_max_items(tiles, target);
    l.split.slots = (int)attn_max_slots(tiles, target);
    // the joining's: a row or more each, at most 1024 for each of a call's splits
    // (2048 for one: 7 to 9 us more where there is little to join, no less where
    // there is much)
    const long rows = (tiles < target ? tiles : target) * R;
    l.joins = rows < 1024 ? rows : 1024;
    return l;
}

// Workgroups of a launch, of up to 512 threads: a grid holds fewer than 2^32 of them, and
// the calls that are accepted make up to 2^31 parts (one each for T Hq of 2^30).
constexpr unsigned kGrid = 1u << 22;
template <typename F>
void in_grids(unsigned n, F launch) {
    for (unsigned first = 0; first < n; first += kGrid) launch(n - first < kGrid ? n - first : kGrid, first);
}
}  // namespace
}  // namespace kda
