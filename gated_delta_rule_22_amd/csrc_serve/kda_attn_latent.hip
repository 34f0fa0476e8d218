// Causal attention over a paged latent cache: every position's row (c, pe) is the
// key of all query heads, and c its value. Online softmax as in the paged
// attention of grouped heads (kda_attn_paged.hip).
//
// A request's rows are its new tokens times all query heads, cut into tiles of R = 32 or
// 64 rows. The call's tiles times keys are shared out evenly between as many workgroups
// as the card holds (kda_attn_even.h): parts of whole tiles left compute units idle for a
// third to a half of the time, since a tile has few rows and a long request many keys.
// The keys go through LDS 32 at a time, where they serve as keys and as values.
//
// bf16 weights are two terms, a leading part and its rest, so that only the result is
// rounded: 2^-16 of a weight is lost. Per row and key 2 (dc + 64) + 4 dc flops.
//
// What bounds it, and what it measured with 512 + 64 channels:
//   256 single tokens, 16 heads, 2.7 GB of cache: 495 us, 5.5 TB/s, the memory's rate;
//   128 single tokens, 128 heads, 199 GF: 335 us. Each 64 rows of a request read its keys
//     again, from their XCD's cache if they do it at the same time (`side`);
//   4 drafts of 8 tokens over up to 262144 keys, 32 heads, 353 GF: 490 us, 720 TF/s, and
//     1060 with the weights' second terms;
//   one token over 1000 keys, 32 heads: 20.5 us, of which two launches are 10, and the rest
//     one chain of memory latencies: lengths, pages, queries and keys, pieces.
// 64 rows need 256 registers a lane with 512 channels. Some of them are spilled outside of
// the products' loops; tiles of 128 rows spill in them (390 -> 700 us).
#include "kda_attn_even.h"
#include "kda_full_launch.h"

#include <limits.h>

namespace kda {
namespace {

// Wait until at most N of the wave's vector memory accesses are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
}

// Piece of 16 bytes that LDS holds in place of piece c of a key's row. bf16:
// the rows' stride is 32 banks modulo 64; 16 lanes in a row that read one piece of 16
// keys, and 32 lanes that read two pieces of 8 keys, cover the banks once. The latter
// (the values) have no conflicts; the former do: SQ_LDS_BANK_CONFLICT counts 320 cycles a
// step of 32 rows and 352 of 64, 4 for each of its 72 reads of keys and 4 for each store of
// weights. That is what groups of the lanes 0-3, 12-15, 20-27 and of the others of each 32
// would cost instead of 16 lanes in a row.
__device__ __forceinline__ int latent_piece(int key, int c) {
    return c ^ (2 * (key >> 1 & 3) + (key >> 3 & 1));
}

// x as a value that is not known to be the same in every step: what is made from it
// is made where it is used, not kept in registers that the rows' sums need. (Spilled
// ones would be read back behind the loads in flight.)
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

constexpr int kLatentThreads = 512;

// Largest over the lanes l % 16 + {0, 16, 32, 48}, without LDS.
__device__ __forceinline__ float max_of_quarters(float x) {
    const auto u = [](float y) { return __builtin_bit_cast(unsigned, y); };
    const auto f = [](unsigned y) { return __builtin_bit_cast(float, y); };
    const auto a = __builtin_amdgcn_permlane16_swap(u(x), u(x), false, false);
    x = fmaxf(f(a[0]), f(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(u(x), u(x), false, false);
    return fmaxf(f(b[0]), f(b[1]));
}

// The keys of a run on their way to LDS: steps of 32 keys, buffers taken in turn. Each
// wave loads a part of 16 keys of a step, which one page holds.
template <int DC, int BUF>
struct KeySteps {
    static constexpr int W = DC + kPe, KT = 32, kPieces = W / 8;
    static constexpr int kLoads16 = 16 * kPieces / 64, LD = (kLoads16 + 3) / 4;
    static constexpr bool kUneven = kLoads16 % 4 != 0;
    const AttnArgs& a;
    const Keys keys;
    const int* table;
    bf16* const tiles;
    int wave, lane;
    int half, load0;             // which 16 keys, and the first of the wave's loads of them
    bool fewer;                  // LD - 1 loads
    uint32_t off[LD];            // where in the keys' rows the lane's bytes are
    int fetched, buf;            // the next step's position and buffer
    // Pages of the 64 sixteens of keys from `pages_from` on, one a lane (behind the end the
    // last key's). Scalar loads would share their counter with LDS, whose reads would
    // wait for them.
    int pages, pages_from;
    // of the b-th step from the next one to be waited for: whether loads are in flight (a
    // page that does not exist has none), and its sixteens without a page
    bool have[BUF];
    int gaps[BUF];

    __device__ __forceinline__ KeySteps(const AttnArgs& args, const Keys& k, const int* t, bf16* to)
        : a(args), keys(k), table(t), tiles(to), wave(wave_id()), lane(threadIdx.x & 63) {
        half = wave >> 2;
        load0 = kLoads16 * (wave & 3) / 4;
        fewer = kUneven && kLoads16 * ((wave & 3) + 1) / 4 - load0 < LD;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            int key, byte;
            piece_at(i, lane, key, byte);
            off[i] = key * (2 * W) + byte;
        }
        fetched = keys.begin;
        buf = 0;
#pragma unroll
        for (int b = 0; b < BUF; ++b) {
            have[b] = false;
            gaps[b] = 0;
        }
        pages = -1;
        pages_from = keys.begin;
        if (keys.begin < keys.end) look_up();
    }
    __device__ __forceinline__ void piece_at(int i, int l, int& key, int& byte) const {
        const int x = (load0 + i) * 64 + l;
        key = x / kPieces;
        byte = 16 * latent_piece(key, x - key * kPieces);
    }
    __device__ __forceinline__ void look_up() {
        pages_from = fetched;
        const int page = table[min(fetched + 16 * fresh(lane), keys.end - 1) >> a.page_shift];
        pages = (unsigned)page < (unsigned)a.pool ? page : -1;
    }
    // The next step, b steps behind the next one to be waited for. Positions behind the
    // end are read from the last one, which some row of the tile sees: nothing else of
    // an unused row gets here.
    __device__ __forceinline__ void fetch(int b) {
        if (fetched >= keys.end) return;
        if (fetched - pages_from >= 1024) look_up();
        const int at16 = (fetched - pages_from) >> 4;
        const int p0 = __builtin_amdgcn_readlane(pages, at16), p1 = __builtin_amdgcn_readlane(pages, at16 + 1);
        const int pg = half ? p1 : p0;
        have[b] = pg >= 0;
        gaps[b] = (p0 < 0) | (p1 < 0) << 1;
        bf16* to = tiles + (buf * KT + 16 * half) * W + load0 * 512;
        if (pg >= 0) {
            const int at = uniform(min(fetched + 16 * half, keys.end - 1)), most = keys.end - 1 - at;
            const int row = at & ((1 << a.page_shift) - 1);
            const bf16* from = (const bf16*)a.kc + (((long)pg << a.page_shift) + row) * W;
            const uint32_t l0 = uniform((int)(uint32_t)(uintptr_t)(lds_void*)to);
            if (most >= 15) {
#pragma unroll
                for (int i = 0; i < LD; ++i)
                    if (i < LD - 1 || !fewer) load_to_lds(l0 + i * 1024, off[i], from);
            } else {
                const int l = fresh(lane);
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    if (i == LD - 1 && fewer) continue;
                    int key, byte;
                    piece_at(i, l, key, byte);
                    load_to_lds(l0 + i * 1024, min(key, most) * (2 * W) + byte, from);
                }
            }
        } else {
            for (int i = 0; i < LD; ++i)
                if (i < LD - 1 || !fewer) *(bf16x8*)(to + i * 512 + 8 * lane) = bf16x8{};
        }
        fetched += KT;
        buf = buf + 1 == BUF ? 0 : buf + 1;
    }
    // Waits for this wave's part of the oldest step, behind which there may be another one.
    __device__ __forceinline__ void wait() {
        if (BUF > 3 && have[1]) {
            if (fewer) wait_loads<LD - 1>();
            else wait_loads<LD>();
        } else {
            wait_loads<0>();
        }
    }
    // The oldest step is in use; which sixteens of it have no page.
    __device__ __forceinline__ int take() {
        const int missing = gaps[0];
#pragma unroll
        for (int b = 0; b + 1 < BUF; ++b) {
            have[b] = have[b + 1];
            gaps[b] = gaps[b + 1];
        }
        have[BUF - 1] = false;
        return missing;
    }
    __device__ __forceinline__ bf16* tile(int b) const { return tiles + b * KT * W; }
    // Positions that only some rows see: a value there that is not finite must not meet
    // the weight 0 of the others in a product. It counts 0, and the scores of the rows
    // that see its position become NaN. By all waves, with barriers.
    __device__ __forceinline__ void clear_odd(bf16* t, int* odd_keys) const {
        if (threadIdx.x < KT) odd_keys[threadIdx.x] = 0;
        __syncthreads();
        for (int i = 0; i < LD; ++i) {
            int key, byte;
            piece_at(i, fresh(lane), key, byte);
            if ((i == LD - 1 && fewer) || byte >= 2 * DC) continue;
            bool odd = false;
            bf16x8* v = (bf16x8*)(t + 16 * half * W + ((load0 + i) * 64 + lane) * 8);
            *v = only_finite(*v, odd);
            if (odd) odd_keys[16 * half + key] = 1;
        }
        __syncthreads();
    }
};

// Tiles of 32 and 64 rows: waves 0 to 3 make the weights, waves 4 to 7 the values of
// the step before, so that each SIMD has one of both and a step has one barrier. Score
// wave rg + 2 kg has half of the rows and 16 keys. The rows' reference is their maximum
// up to the step before, or less than that by up to kFollow. Where a step's maximum is
// above it by more than kJump (in the first step of a run, for one), the step's weights
// are made again behind the barrier. So a weight is at most 2^8, as in the other
// attention kernels: it costs nothing in fp32 and bf16, and the sums of n keys stay
// inside fp32 with values up to 2^119 / n. (Following from 8 on and making weights again
// from 24 on took as long: 16 heads 479 us, 128 heads 332 to 336, drafts 500 to 510.)
template <int DC, int R> struct NarrowLds {
    static constexpr int W = DC + kPe, RP = R / 16;
    static constexpr int BUF = R == 64 && DC == 512 ? 3 : 4;     // what LDS holds
    __align__(128) bf16 tile[BUF * 32 * W];
    __align__(16) bf16 p[2][2 * RP * 512];
    float top[2][2][R], factor[2][R], sum[2][R], ref[R];
    __align__(16) int jump[2][4];
    int moved[2][2], odd[32];
    EvenItem items[kEvenRuns];
};
constexpr float kFollow = 4.f, kJump = 8.f;      // log2

template <int DC, int R>
__device__ __forceinline__ void narrow_run(const AttnArgs& a, const EvenSplit& e, const EvenRun& it,
                                           NarrowLds<DC, R>& lds) {
    constexpr int W = DC + kPe, KT = 32, RP = R / 16, RTW = R / 32, KS = W / 32, CT = DC / 64;
    constexpr int BUF = NarrowLds<DC, R>::BUF;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const Keys keys = run_keys(a, it, R);
    KeySteps<DC, BUF> ks(a, keys, a.table + (long)it.req * a.width, lds.tile);
#pragma unroll
    for (int b = 0; b < BUF - 2; ++b) ks.fetch(b);
    const int steps = keys.end > keys.begin ? (keys.end - keys.begin + KT - 1) / KT : 0;
    // (both kinds of waves go through the same barriers)
    const auto begin_step = [&](int j, bool& partial) {
        int missing = 0;
        if (j < steps) {
            ks.wait();
            missing = ks.take();
        }
        __syncthreads();                             // the step has landed, the weights of the last are there
        partial = j < steps && keys.all < keys.end && keys.begin + (j + 1) * KT > keys.all;
        return missing;
    };
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const auto jumped = [&](i32x4 x) { return uniform(x[0] | x[1] | x[2] | x[3]) != 0; };

    if (wave < 4) {
        const int rg = wave & 1, kg = wave >> 1, row0 = rg * 16 * RTW + c16;
        bf16x8 qf[RTW][KS];
        int limit[RTW];                              // last visible position
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt) {
            const RowAt x = run_row(a, it, it.tile * R + row0 + rt * 16);
            limit[rt] = x.in ? (int)min((long)it.kept + x.t, (long)kKeepAll) : -1;
            // (rows behind the request's read its first token's)
            const bf16* q = (const bf16*)a.q + x.q * W + 8 * g4;
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[rt][k] = *(const bf16x8*)(q + 32 * k);
        }
        const float scale = a.scale * kLog2e;
        float m[RTW], l[RTW], l_before[RTW], factor[RTW];
        f32x4 st[RTW];
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt) {
            m[rt] = -INFINITY;
            l[rt] = l_before[rt] = 0.f;
            factor[rt] = 1.f;
            st[rt] = zero4();
        }
        const auto weights = [&](int j) {
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) {
                const float mu = m[rt] == -INFINITY ? 0.f : m[rt];
                float p[4];
                l_before[rt] = l[rt];
                for (int i = 0; i < 4; ++i) {
                    p[i] = exp2_f(st[rt][i] - mu);
                    l[rt] += p[i];
                }
                bf16x4 hi, lo;
                two_terms(p, hi, lo);
                bf16* to = lds.p[j & 1] + ((rg * RTW + rt) * 64 + lane) * 8 + 4 * kg;
                *(bf16x4*)to = hi;
                *(bf16x4*)(to + RP * 512) = lo;
            }
        };
        // The rows' largest score of step j, of both key groups.
        const auto top_of = [&](int j, int rt) {
            return fmaxf(lds.top[j & 1][0][row0 + rt * 16], lds.top[j & 1][1][row0 + rt * 16]);
        };
        const auto follow = [&](int rt, float top) {
            const float mn = fmaxf(m[rt], top), c = mn == -INFINITY ? 1.f : exp2_f(m[rt] - mn);
            m[rt] = mn;
            l[rt] *= c;
            factor[rt] *= c;
        };
        const auto publish = [&](int j, bool moved) {
            if (kg != 0) return;
            if (moved && g4 == 0)
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) lds.factor[j & 1][row0 + rt * 16] = factor[rt];
            if (lane == 0) lds.moved[j & 1][rg] = moved;
        };
        int buf = 0;
        for (int j = 0; j <= steps; ++j) {
            bool partial;
            const int missing = begin_step(j, partial);
            // What is in LDS is read first, and the fetch is behind it. Fragments of keys
            // stay in flight ahead of their products. (Pieces 4 i + g4: the order of LDS
            // repeats every eight.)
            const bf16* from = ks.tile(buf) + (16 * kg + c16) * W;
            const bf16* k[2] = {from + 8 * latent_piece(c16, g4), from + 8 * latent_piece(c16, 4 + g4)};
            const auto read = [&](int i) { return *(const bf16x8*)(k[i & 1] + 64 * (i / 2)); };
            constexpr int kAhead = KS < 6 ? KS : RTW > 1 ? 4 : 6;
            bf16x8 kf[kAhead];
            float top[RTW];
            const i32x4 flags = *(const i32x4*)lds.jump[(j - 1) & 1];
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) top[rt] = top_of(j - 1, rt);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kf[i] = read(i);
            __builtin_amdgcn_sched_barrier(0);
            ks.fetch(BUF - 3);
            __builtin_amdgcn_sched_barrier(0);
            if (j > 0 && jumped(flags)) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) {
                    l[rt] = l_before[rt];
                    follow(rt, top[rt]);
                }
                publish(j - 1, true);
                weights(j - 1);
                __syncthreads();
            }
            if (partial) {
                ks.clear_odd(ks.tile(buf), lds.odd);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) kf[i] = read(i);
            }
            if (j == steps) break;
            // The reference may stay behind the maximum by up to kFollow.
            bool ahead = false;
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) {
                factor[rt] = 1.f;
                if (j == 0) top[rt] = -INFINITY;
                ahead |= top[rt] > m[rt] + kFollow;
            }
            const bool moved = __any(ahead);
            if (moved) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) follow(rt, top[rt]);
            }
            publish(j, moved);

#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) st[rt] = zero4();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < KS; ++i) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) st[rt] = mma32(kf[i % kAhead], qf[rt][i], st[rt]);
                if (i + kAhead < KS) kf[i % kAhead] = read(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            const int pos = keys.begin + j * KT;
            bool jump = false;
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) {
                for (int i = 0; i < 4; ++i) st[rt][i] *= scale;
                if (pos + KT > keys.all || missing) {
                    for (int i = 0; i < 4; ++i) {
                        const int y = 16 * kg + 4 * g4 + i;
                        if (partial && lds.odd[y]) st[rt][i] = NAN;
                        if (pos + y >= keys.end || (missing >> kg & 1) || pos + y > limit[rt]) st[rt][i] = -INFINITY;
                    }
                }
                const float mx = max_of_quarters(fmaxf(fmaxf(st[rt][0], st[rt][1]), fmaxf(st[rt][2], st[rt][3])));
                if (g4 == 0) lds.top[j & 1][kg][row0 + rt * 16] = mx;
                jump |= mx > m[rt] + kJump;
            }
            jump = __any(jump);
            if (lane == 0) lds.jump[j & 1][wave] = jump;
            weights(j);
            buf = buf + 1 == BUF ? 0 : buf + 1;
        }
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt) {
            const float sum = sum_quarters(l[rt]);
            if (g4 == 0) {
                lds.sum[kg][row0 + rt * 16] = sum;
                if (kg == 0) lds.ref[row0 + rt * 16] = m[rt];
            }
        }
        __syncthreads();
        return;
    }

    const int vw = wave - 4;
    f32x4 acc[RP][CT];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = zero4();
    int buf = 0, back = 0;
    for (int j = 0; j <= steps; ++j) {
        bool partial;
        begin_step(j, partial);
        if (j > 0) {
            const int x = (j - 1) & 1;
            const bf16* tile = ks.tile(back);
            const int key = 4 * g4 + c16 / 4;        // (and 16 behind it: the same order in LDS)
            const i32x4 flags = *(const i32x4*)lds.jump[x];
            int moved[2] = {lds.moved[x][0], lds.moved[x][1]};
            bf16x8 va[CT], pf[RP], pr[RP];
#pragma unroll
            for (int b = 0; b < CT; ++b) {
                // pieces of four b are in four orders, those behind them in the same
                const int c = 2 * (vw * CT + b % 4) + (c16 & 3) / 2;
                const bf16* v = tile + key * W + 8 * latent_piece(key, c) + 4 * (c16 & 1) + 64 * (b / 4);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + 16 * W));
                va[b] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
            const bf16* p = lds.p[x] + lane * 8;
            const auto read = [&]() {
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    pf[r] = *(const bf16x8*)(p + r * 512);
                    pr[r] = *(const bf16x8*)(p + (RP + r) * 512);
                }
            };
            read();
            __builtin_amdgcn_sched_barrier(0);
            ks.fetch(BUF - 3);
            __builtin_amdgcn_sched_barrier(0);
            if (jumped(flags)) {
                __syncthreads();                     // the weights are made again
                read();
                moved[0] = lds.moved[x][0];
                moved[1] = lds.moved[x][1];
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!uniform(moved[g])) continue;
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) {
                    const float c = lds.factor[x][(g * RTW + rt) * 16 + c16];
#pragma unroll
                    for (int b = 0; b < CT; ++b) acc[g * RTW + rt][b] *= c;
                }
            }
#pragma unroll
            for (int r = 0; r < RP; ++r) {
#pragma unroll
                for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pf[r], acc[r][b]);
#pragma unroll
                for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pr[r], acc[r][b]);
            }
        } else {
            ks.fetch(BUF - 3);
        }
        if (partial) ks.clear_odd(ks.tile(buf), lds.odd);
        back = buf;
        buf = buf + 1 == BUF ? 0 : buf + 1;
    }
    __syncthreads();                                 // the rows' sums and references are there
    const int col = vw * (16 * CT) + 4 * g4;
#pragma unroll
    for (int r = 0; r < RP; ++r) {
        const int y = 16 * r + c16;
        const float sum = lds.sum[0][y] + lds.sum[1][y], ref = lds.ref[y];
        if (it.pieces > 1) {
            const long at = (long)it.slot * R + y;
            // (a row without a key in this piece has sums of 0)
#pragma unroll
            for (int b = 0; b < CT; ++b) *(f32x4*)(e.acc + at * DC + col + 16 * b) = acc[r][b];
            if (vw == 0 && g4 == 0) {
                e.ml[at * 2] = ref;
                e.ml[at * 2 + 1] = sum;
            }
            continue;
        }
        const RowAt x = run_row(a, it, it.tile * R + y);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (!x.in) continue;
#pragma unroll
        for (int b = 0; b < CT; ++b) {
            bf16x4 z;
            for (int i = 0; i < 4; ++i) z[i] = (bf16)(acc[r][b][i] * inv);
            *(bf16x4*)((bf16*)a.o + x.q * DC + col + 16 * b) = z;
        }
        if (a.lse && vw == 0 && g4 == 0) a.lse[x.q] = sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * kLn2;
    }
}

template <int DC, int R>
__global__ __launch_bounds__(kLatentThreads, 2) void attn_latent_narrow(AttnArgs a, AttnSplit s, EvenSplit e) {
    __shared__ NarrowLds<DC, R> lds;
    even_runs(a, s, e, lds.items, [&](const EvenRun& it) { narrow_run<DC, R>(a, e, it, lds); });
}

// fp32: 32 rows, 32 keys a step. Scores: a wave takes 16 rows and 16 keys, lane
// quarter g the channels g W / 4 .. of both, so that its reads are 16 bytes.
// Values as above; the 16 columns of a product's block are VW apart, so that a
// lane reads VW neighbours.
template <int DC> struct LatentLdsF {
    static constexpr int W = DC + kPe, KT = 32;
    __align__(128) float tile[2 * KT * W];
    __align__(16) float p[2 * 2 * 64 * 4];
    float top[2][32], factor[32], sum[2][32];
    int moved[2], odd[KT];
    EvenItem items[kEvenRuns];
};
constexpr int kRowsF = 32;

template <int DC>
__device__ __forceinline__ void latent_run_f32(const AttnArgs& a, const EvenSplit& e, const EvenRun& it,
                                               LatentLdsF<DC>& lds) {
    constexpr int W = DC + kPe, KT = 32, KQ = W / 16;   // pieces of a lane's channels
    constexpr int CT = DC / 64, VW = CT < 4 ? CT : 4;
    constexpr int kPieces = W / 4, kKeys = KT / 4, LD = kKeys * kPieces / 64;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const int rg = wave & 1, kg = wave >> 1;
    const Keys keys = run_keys(a, it, kRowsF);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;
    auto piece = [](int key, int c) { return c ^ (key & 15); };

    f32x4 qf[KQ];
    const RowAt at_row = run_row(a, it, it.tile * kRowsF + rg * 16 + c16);
    const int limit = at_row.in ? (int)min((long)it.kept + at_row.t, (long)kKeepAll) : -1;
    for (int k = 0; k < KQ; ++k) {
        f32x4 z = zero4();
        if (at_row.in) z = *(const f32x4*)((const float*)a.q + at_row.q * W + 4 * (g4 * KQ + k));
        qf[k] = z;
    }
    float m = -INFINITY, l = 0.f;
    f32x4 acc[2][CT];
    for (int r = 0; r < 2; ++r)
        for (int c = 0; c < CT; ++c) acc[r][c] = zero4();

    auto fkey = [&](int i) { return (i * 64 + lane) / kPieces; };
    auto fcol = [&](int i) {
        const int x = i * 64 + lane, r = x / kPieces;
        return 16 * piece(wave * kKeys + r, x - r * kPieces);
    };
    auto fetch = [&](int buf, int pos) {
        const int at = min(pos + wave * kKeys, keys.end - 1);
        const int page = page_at(a, table, at, keys.end);
        float* to = lds.tile + (buf * KT + wave * kKeys) * W;
        if (page >= 0) {
            const float* from = (const float*)a.kc + (((long)page << a.page_shift) + (at & row_mask)) * W;
            const int most = keys.end - 1 - at;
            const uint32_t l0 = uniform((int)(uint32_t)(uintptr_t)(lds_void*)to);
            for (int i = 0; i < LD; ++i)
                load_to_lds(l0 + i * 1024, min(fkey(i), most) * (4 * W) + fcol(i), from);
        } else {
            for (int i = 0; i < LD; ++i) *(f32x4*)(to + i * 256 + 4 * lane) = zero4();
        }
    };

    if (keys.begin < keys.end) fetch(0, keys.begin);
    int buf = 0;
    for (int pos = keys.begin; pos < keys.end; pos += KT, buf ^= 1) {
        wait_loads<0>();
        __syncthreads();
        if (pos + KT < keys.end) fetch(buf ^ 1, pos + KT);
        int missing = 0;
        for (int u = 0; u < 2; ++u)
            missing |= (page_at(a, table, min(pos + 16 * u, keys.end - 1), keys.end) < 0) << u;
        float* tile = lds.tile + buf * KT * W;
        const bool partial = keys.all < keys.end && pos + KT > keys.all;
        if (partial) {
            float* x = tile + wave * kKeys * W;
            if (lane < kKeys) lds.odd[wave * kKeys + lane] = 0;
            lds_fence_wave();
            for (int i = 0; i < LD; ++i) {
                if (fcol(i) >= 4 * DC) continue;
                bool odd = false;
                f32x4* v = (f32x4*)(x + i * 256 + 4 * lane);
                f32x4 y = *v;
                for (int j = 0; j < 4; ++j)
                    if (!finite_bits(y[j])) {
                        y[j] = 0.f;
                        odd = true;
                    }
                *v = y;
                if (odd) lds.odd[wave * kKeys + fkey(i)] = 1;
            }
            __syncthreads();
        }
        f32x4 st = zero4();
        {
            const float* k = tile + (16 * kg + c16) * W;
#pragma unroll
            for (int i = 0; i < KQ; ++i) {
                const f32x4 kf = *(const f32x4*)(k + 4 * piece(c16, g4 * KQ + i));
                for (int j = 0; j < 4; ++j) st = mma4(kf[j], qf[i][j], st);
            }
        }
        for (int i = 0; i < 4; ++i) st[i] *= scale;
        if (pos + KT > keys.all || missing) {
            for (int i = 0; i < 4; ++i) {
                const int y = 16 * kg + 4 * g4 + i;
                if (partial && lds.odd[y]) st[i] = NAN;
                if (pos + y >= keys.end || (missing >> kg & 1) || pos + y > limit) st[i] = -INFINITY;
            }
        }
        float mx = max_quarters(fmaxf(fmaxf(st[0], st[1]), fmaxf(st[2], st[3])));
        if (g4 == 0) lds.top[kg][rg * 16 + c16] = mx;
        __syncthreads();
        mx = fmaxf(lds.top[0][rg * 16 + c16], lds.top[1][rg * 16 + c16]);
        const bool moved = __any(mx > m);
        if (moved) {
            const float mn = fmaxf(m, mx);
            const float c = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            l *= c;
            if (kg == 0 && g4 == 0) lds.factor[rg * 16 + c16] = c;
        }
        if (kg == 0 && lane == 0) lds.moved[rg] = moved;
        const float mu = m == -INFINITY ? 0.f : m;
        f32x4 p;
        for (int i = 0; i < 4; ++i) {
            p[i] = exp2_f(st[i] - mu);
            l += p[i];
        }
        *(f32x4*)(lds.p + ((rg * 2 + kg) * 64 + lane) * 4) = p;
        __syncthreads();
        for (int r = 0; r < 2; ++r) {
            if (!uniform(lds.moved[r])) continue;
            const float c = lds.factor[r * 16 + c16];
            for (int b = 0; b < CT; ++b) acc[r][b] *= c;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 p0 = *(const f32x4*)(lds.p + (t * 64 + lane) * 4);
            const f32x4 p1 = *(const f32x4*)(lds.p + ((2 + t) * 64 + lane) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 16 * t + 4 * g4 + i;
#pragma unroll
                for (int g = 0; g < CT / VW; ++g) {
                    const int col = wave * (DC / 4) + 16 * VW * g + VW * c16;
                    const float* x = tile + key * W + 4 * piece(key, col / 4) + col % 4;
#pragma unroll
                    for (int j = 0; j < VW; ++j) {
                        acc[0][g * VW + j] = mma4(x[j], p0[i], acc[0][g * VW + j]);
                        acc[1][g * VW + j] = mma4(x[j], p1[i], acc[1][g * VW + j]);
                    }
                }
            }
        }
    }
    const float part_sum = sum_quarters(l);
    if (g4 == 0) {
        lds.sum[kg][rg * 16 + c16] = part_sum;
        if (kg == 0) lds.top[0][rg * 16 + c16] = m;
    }
    __syncthreads();
    for (int r = 0; r < 2; ++r) {
        const int row = 16 * r + c16;
        const float sum = lds.sum[0][row] + lds.sum[1][row], top = lds.top[0][row];
        const bool cut = it.pieces > 1;
        const long at = (long)it.slot * kRowsF + row;
        const RowAt x = run_row(a, it, it.tile * kRowsF + row);
        if (!cut && !x.in) continue;
        const float inv = cut ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        float* to = cut ? e.acc + at * DC : (float*)a.o + x.q * DC;
        for (int g = 0; g < CT / VW; ++g)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < VW; ++j)
                    to[wave * (DC / 4) + 16 * VW * g + VW * (4 * g4 + i) + j] = acc[r][g * VW + j][i] * inv;
        if (wave != 0 || g4 != 0) continue;
        if (cut) {
            e.ml[at * 2] = top;
            e.ml[at * 2 + 1] = sum;
        } else if (a.lse) {
            a.lse[x.q] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
        }
    }
}

template <int DC>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_latent_f32(AttnArgs a, AttnSplit s, EvenSplit e) {
    __shared__ LatentLdsF<DC> lds;
    even_runs(a, s, e, lds.items, [&](const EvenRun& it) { latent_run_f32<DC>(a, e, it, lds); });
}

// Kernel and work split of a call, from sizes alone.
struct LatentPlan {
    AttnSplit split;
    EvenSplit even;
    int groups;            // workgroups
    size_t bytes;
};
LatentPlan plan_of(int T, int B, int Hq, int dc, int max_new, bool bf16_io) {
    const long most = (long)(max_new > 0 && max_new < T ? max_new : T) * Hq;
    LatentPlan p{};
    const int R = !bf16_io || most <= 32 ? 32 : 64;
    // Requests that are all of the same length have their rows side by side.
    const long tiles = (most + R - 1) / R;
    const bool same = max_new > 0 && (long)B * max_new == T;
    const int side_log2 = !same ? 0 : tiles % 4 == 0 ? 2 : tiles % 2 == 0 ? 1 : 0;
    p.even.R = R;
    p.even.side = 1 << side_log2;
    p.split.R = R << side_log2;
    p.split.R_log2 = __builtin_ctz((unsigned)p.split.R);
    p.split.min_rows = 1;
    p.split.max_rows = INT32_MAX;
    // as many workgroups as the card's 256 compute units hold
    p.groups = dc == 128 ? 512 : 256;
    p.even.G = p.groups >> side_log2;
    p.bytes = (size_t)p.groups * (2 * R * (dc + 2) + 4) * sizeof(float);
    if (B > kBlock) p.bytes += AttnTable::ints(B) * sizeof(int);
    return p;
}

template <int DC>
hipError_t launch(const AttnArgs& a, const LatentPlan& p, hipStream_t st) {
    if (a.B > kBlock) even_list<<<1, 64 * kListWaves, 0, st>>>(a, p.split, p.even);
    const auto run = [&](auto kernel, int threads) { kernel<<<p.even.G * p.even.side, threads, 0, st>>>(a, p.split, p.even); };
    if (!a.bf16_io) run(attn_latent_f32<DC>, kAttnThreads);
    else if (p.even.R == 32) run(attn_latent_narrow<DC, 32>, kLatentThreads);
    else run(attn_latent_narrow<DC, 64>, kLatentThreads);
    // no more workgroups than rows of cut tiles
    const long rows = (long)(p.even.G - 1) * p.split.R;
    const int n = (int)(rows < kEvenJoins ? rows : kEvenJoins);
    if (n && a.bf16_io) even_join<bf16, DC><<<n, kAttnThreads, 0, st>>>(a, p.even);
    else if (n) even_join<float, DC><<<n, kAttnThreads, 0, st>>>(a, p.even);
    return hipGetLastError();
}

}  // namespace

size_t attn_latent_ws(int T, int B, int Hq, int dc, int max_new, bool bf16_io) {
    return plan_of(T, B, Hq, dc, max_new, bf16_io).bytes;
}

hipError_t launch_attn_latent(const AttnArgs& a, void* ws, hipStream_t st) {
    LatentPlan p = plan_of(a.T, a.B, a.Hq, a.d, a.max_new, a.bf16_io);
    EvenSplit& e = p.even;
    e.pieces = (int*)ws;
    e.ml = (float*)(e.pieces + 4 * p.groups);
    e.acc = e.ml + (size_t)4 * p.groups * e.R;
    if (a.B > kBlock) e.table = (int*)(e.acc + (size_t)2 * p.groups * e.R * a.d);
    // a call of few keys has fewer units than that
    const long tiles = ((long)a.T * a.Hq >> p.split.R_log2) + (a.B < a.T ? a.B : a.T);
    const long units = tiles * (((long)a.width << a.page_shift) / kUnitKeys + 1 + 2);
    if (units < e.G) e.G = (int)units;
    switch (a.d) {
        case 128: return launch<128>(a, p, st);
        case 256: return launch<256>(a, p, st);
        default: return launch<512>(a, p, st);
    }
}

}  // namespace kda
