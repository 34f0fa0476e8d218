// Causal attention over a paged latent cache: every position's row (c, pe) is the
// key of all query heads, and c its value. Online softmax as in the paged
// attention of grouped heads (kda_attn_paged.hip).
//
// A request's rows are its new tokens times all query heads, cut into tiles of
// 32 RT rows; a workgroup of four waves takes a tile and a part of its keys
// (kda_attn_sched.h). The keys go through LDS, KT at a time, where they serve as
// keys and as values. The waves divide a step's work twice:
//   scores  wave w takes 32 rows (their queries stay in its registers) and a
//           quarter, half or all of the step's keys, S^T = K Q^T;
//   values  each wave takes a quarter of the value channels for all rows,
//           O^T += V^T P^T, so that V is read from LDS once, not by every wave.
// The weights P pass through LDS in between, in the order of the second product's
// operand.
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
// the rows' stride is 32 banks modulo 64; 16 lanes that read one piece of 16
// keys, and 32 lanes that read two pieces of 8 keys, cover the banks once.
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

// What a step needs of the request's pages: the 16 keys at pos + 16 u.
template <int KT> struct StepPages {
    int id[KT / 16];
    // bit u: positions of a page that does not exist
    __device__ int missing() const {
        int m = 0;
        for (int u = 0; u < KT / 16; ++u) m |= (id[u] < 0) << u;
        return m;
    }
};

// How eight waves share a tile of R rows: row groups of RTW row tiles of 16 (RGN),
// key groups (KG) and, where a wave takes two row tiles, halves of the contraction
// (HV): such a wave makes half the sums of both and adds the other half to one.
template <int DC, int R_> struct LatentShape {
    static constexpr int W = DC + kPe, R = R_, RP = R / 16;
    static constexpr int KT = 32;                    // keys of a step
    static constexpr int BUF = R == 128 ? 3 : 4;     // steps in LDS
    static constexpr int HV = R == 128 ? 2 : 1, RTW = HV;
    static constexpr int RGN = RP / RTW, KG = R == 128 ? 1 : 2;
    static constexpr int SW = RGN * KG * HV;         // waves that make scores: 4 or all 8
    static constexpr int NU = KT / 16 / KG;          // key tiles of a wave's scores
    static constexpr int KS = W / 32 / HV;           // steps of their contraction
    static constexpr int CT = DC / 128;              // value columns of a wave, in 16s
    static constexpr bool kPipe = R > 32;            // see the kernel's loops
    // Loads of 1 KB: of 16 keys, which one page holds, and the most of a wave. LW waves
    // share 16 keys: wave x of them has the loads from load_of(x) on.
    static constexpr int LW = 4, kLoads16 = 16 * (W / 8) / 64, LD = (kLoads16 + LW - 1) / LW;
    static constexpr bool kUneven = kLoads16 % LW != 0;
    __device__ static int load_of(int x) { return kLoads16 * x / LW; }
};
constexpr int kLatentThreads = 512;

template <int DC, int R> struct LatentLds {
    typedef LatentShape<DC, R> S;
    __align__(128) bf16 tile[S::BUF * S::KT * S::W];
    __align__(16) bf16 p[2 * S::RP * 64 * 8];
    f32x4 half[S::HV > 1 ? 8 * S::NU * 64 : 1];
    float top[S::KG][R], factor[R], sum[S::KG][R];
    int moved[S::RP], odd[S::KT];
    EvenItem item;
};

// Largest over the lanes l % 16 + {0, 16, 32, 48}, without LDS.
__device__ __forceinline__ float max_of_quarters(float x) {
    const auto u = [](float y) { return __builtin_bit_cast(unsigned, y); };
    const auto f = [](unsigned y) { return __builtin_bit_cast(float, y); };
    const auto a = __builtin_amdgcn_permlane16_swap(u(x), u(x), false, false);
    x = fmaxf(f(a[0]), f(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(u(x), u(x), false, false);
    return fmaxf(f(b[0]), f(b[1]));
}

// One run: a piece of a tile's keys, or all of them.
template <int DC, int R>
__device__ __forceinline__ void latent_run(const AttnArgs& a, const EvenSplit& e, const EvenRun& it,
                                           LatentLds<DC, R>& lds) {
    typedef LatentShape<DC, R> S;
    constexpr int W = S::W, KT = S::KT, NU = S::NU, BUF = S::BUF, CT = S::CT, LD = S::LD, RTW = S::RTW;
    constexpr int KS = S::KS, kPieces = W / 8;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const int rg = wave % S::RGN, kg = S::HV > 1 ? 0 : wave / S::RGN % S::KG, hv = S::HV > 1 ? wave / S::RGN : 0;
    const bool scores = S::SW == 8 || wave < S::SW;
    const Keys keys = run_keys(a, it, R);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;
    const int row0 = (rg * RTW + hv) * 16, row = row0 + c16;   // the lane's row of the tile

    bf16x8 qf[RTW][KS];
#pragma unroll
    for (int rt = 0; rt < RTW; ++rt) {
        const RowAt x = run_row(a, it, it.tile * R + (rg * RTW + rt) * 16 + c16);
        // (rows behind the request's read its first token's)
        const bf16* q = (const bf16*)a.q + x.q * W + 32 * KS * hv + 8 * g4;
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[rt][k] = *(const bf16x8*)(q + 32 * k);
    }
    const RowAt own = run_row(a, it, it.tile * R + row);
    const int limit = own.in ? (int)min((long)it.kept + own.t, (long)kKeepAll) : -1;   // last visible position
    float m = -INFINITY, l = 0.f;
    f32x4 acc[S::RP][CT];
#pragma unroll
    for (int r = 0; r < S::RP; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = zero4();

    // This wave's loads of a step: 16 keys (those at 16 u), some of their pieces of 16
    // bytes in the order of LDS. Where in the keys' rows the lane's are is made anew in
    // every step of the widest tiles, whose sums need the registers.
    const int u = wave / S::LW, load0 = S::load_of(wave % S::LW);
    const bool fewer = S::kUneven && S::load_of(wave % S::LW + 1) - load0 < LD;
    const auto piece_at = [&](int i, int l, int& key, int& byte) {
        const int x = (load0 + i) * 64 + l;
        key = x / kPieces;
        byte = 16 * latent_piece(key, x - key * kPieces);
    };
    constexpr bool kKeep = R < 128;
    uint32_t foff[kKeep ? LD : 1];
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            int key, byte;
            piece_at(i, lane, key, byte);
            foff[i] = key * (2 * W) + byte;
        }
    }
    // Positions behind the end are read from the last one, which some row of the tile
    // sees: nothing else of an unused row gets here.
    const auto fetch = [&](int buf, int pos, int page) {
        bf16* to = lds.tile + (buf * KT + 16 * u) * W + load0 * 512;
        if (page >= 0) {
            const int at = uniform(min(pos + 16 * u, keys.end - 1)), most = keys.end - 1 - at;
            const bf16* from = (const bf16*)a.kc + (((long)page << a.page_shift) + (at & row_mask)) * W;
            const uint32_t l0 = uniform((int)(uint32_t)(uintptr_t)(lds_void*)to);
            if (kKeep && most >= 15) {
#pragma unroll
                for (int i = 0; i < LD; ++i)
                    if (i < LD - 1 || !fewer) load_to_lds(l0 + i * 1024, foff[i], from);
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
    };
    const auto own_page = [&](const StepPages<KT>& p) {
        int x = p.id[0];
#pragma unroll
        for (int i = 1; i < KT / 16; ++i) x = u == i ? p.id[i] : x;
        return uniform(x);
    };
    // Pages of 16 keys of which the first is behind the end: those of the last key.
    const auto pages_at = [&](int pos) {
        StepPages<KT> p;
#pragma unroll
        for (int u = 0; u < KT / 16; ++u)
            p.id[u] = page_at(a, table, min(pos + 16 * u, keys.end - 1), keys.end);
        return p;
    };

    // Steps are fetched in turn; their pages are looked up a fetch earlier. have[b]: of
    // the b-th step from the next one to be waited for, whether this wave's loads are in
    // flight (a page that does not exist has none); gaps[b]: its keys without a page.
    StepPages<KT> next{};
    if (keys.begin < keys.end) next = pages_at(keys.begin);
    int fetched = keys.begin, fetch_buf = 0;
    bool have[BUF] = {};
    int gaps[BUF] = {};
    const auto fetch_next = [&](int b) {
        if (fetched >= keys.end) return;
        const int page = own_page(next);
        have[b] = page >= 0;
        gaps[b] = next.missing();
        next = pages_at(fetched + KT);
        fetch(fetch_buf, fetched, page);
        fetched += KT;
        fetch_buf = fetch_buf + 1 == BUF ? 0 : fetch_buf + 1;
    };
    // Waits for this wave's part of the oldest step; `after` of them are behind it.
    const auto wait_step = [&](int after) {
        int n = 0;
#pragma unroll
        for (int b = 1; b < BUF - 1; ++b) n += b <= after && n == b - 1 && have[b];
        if (n == 2) {
            if (fewer) wait_loads<2 * LD - 2>();
            else wait_loads<2 * LD>();
        } else if (n == 1) {
            if (fewer) wait_loads<LD - 1>();
            else wait_loads<LD>();
        } else {
            wait_loads<0>();
        }
    };
    const auto step_done = [&]() {                   // the oldest step is in use
#pragma unroll
        for (int b = 0; b + 1 < BUF; ++b) {
            have[b] = have[b + 1];
            gaps[b] = gaps[b + 1];
        }
        have[BUF - 1] = false;
    };

    // Positions that only some rows see: a value there that is not finite must not meet
    // the weight 0 of the others in a product. It counts 0, and the scores of the rows
    // that see its position become NaN.
    const auto clear_odd = [&](bf16* tile) {
        if (threadIdx.x < KT) lds.odd[threadIdx.x] = 0;
        __syncthreads();
        for (int i = 0; i < LD; ++i) {
            int key, byte;
            piece_at(i, fresh(lane), key, byte);
            if ((i == LD - 1 && fewer) || byte >= 2 * DC) continue;
            bool odd = false;
            bf16x8* v = (bf16x8*)(tile + 16 * u * W + ((load0 + i) * 64 + lane) * 8);
            *v = only_finite(*v, odd);
            if (odd) lds.odd[16 * u + key] = 1;
        }
        __syncthreads();
    };

    // (what is made from it is made in the step: see fresh)
    const auto lane_in_step = [&]() { return R < 64 ? lane : fresh(lane); };
    // Scores of a step, in three parts with a barrier between the first two: products;
    // what the other waves have of the rows; weights. kAhead fragments of keys are in
    // flight ahead of their products.
    f32x4 st[NU];
    float mx = -INFINITY;
    const auto mask = [&](int pos, int missing, bool partial) {
        const int g4 = lane_in_step() >> 4;
#pragma unroll
        for (int x = 0; x < NU; ++x)
            for (int i = 0; i < 4; ++i) st[x][i] *= scale;
        if (pos + KT > keys.all || missing) {
            for (int x = 0; x < NU; ++x)
                for (int i = 0; i < 4; ++i) {
                    const int y = 16 * (kg * NU + x) + 4 * g4 + i;
                    if (partial && lds.odd[y]) st[x][i] = NAN;
                    if (pos + y >= keys.end || (missing >> (kg * NU + x) & 1) || pos + y > limit) st[x][i] = -INFINITY;
                }
        }
        mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < NU; ++x)
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, st[x][i]);
        mx = max_of_quarters(mx);
    };
    const auto products = [&](const bf16* tile, int pos, int missing, bool partial) {
        if (!scores) return;
        constexpr int kAhead = KS < 6 ? KS : RTW > 1 ? 4 : 6;
        const int lane = lane_in_step(), c16 = lane & 15, g4 = lane >> 4;
#pragma unroll
        for (int x = 0; x < NU; ++x) {
            const bf16* from = tile + (16 * (kg * NU + x) + c16) * W;
            // pieces first + 4 i + g4: the order of LDS repeats every eight
            const int first = 4 * KS * hv;
            const bf16* k[2] = {from + 8 * latent_piece(c16, first + g4), from + 8 * latent_piece(c16, first + 4 + g4)};
            const auto read = [&](int i) { return *(const bf16x8*)(k[i & 1] + 64 * (i / 2)); };
            f32x4 sc[RTW];
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) sc[rt] = zero4();
            bf16x8 kf[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kf[i] = read(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < KS; ++i) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) sc[rt] = mma32(kf[i % kAhead], qf[rt][i], sc[rt]);
                if (i + kAhead < KS) kf[i % kAhead] = read(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            st[x] = sc[0];
            if constexpr (S::HV > 1) {
                // to the other half's wave its row tile's sums
                lds.half[(wave * NU + x) * 64 + lane] = hv ? sc[0] : sc[1];
                if (hv) st[x] = sc[1];
            }
        }
        if constexpr (S::KG > 1) {
            mask(pos, missing, partial);
            if (g4 == 0) lds.top[kg][row0 + c16] = mx;
        }
    };
    const auto weights = [&](int pos, int missing, bool partial) {
        if (!scores) return;
        const int lane = lane_in_step(), c16 = lane & 15, g4 = lane >> 4;
        if constexpr (S::HV > 1) {
#pragma unroll
            for (int x = 0; x < NU; ++x) st[x] += lds.half[((wave ^ 4) * NU + x) * 64 + lane];
            mask(pos, missing, partial);
        } else {
#pragma unroll
            for (int k = 0; k < S::KG; ++k) mx = fmaxf(mx, lds.top[k][row0 + c16]);
        }
        // The reference may stay behind the maximum by up to 8 in the log2 domain.
        const bool moved = __any(mx > m + 8.f);
        if (moved) {
            const float mn = fmaxf(m, mx);
            const float c = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            l *= c;
            if (kg == 0 && g4 == 0) lds.factor[row0 + c16] = c;
        }
        if (kg == 0 && lane == 0) lds.moved[rg * RTW + hv] = moved;
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int x = 0; x < NU; ++x) {
            float p[4];
            for (int i = 0; i < 4; ++i) {
                p[i] = exp2_f(st[x][i] - mu);
                l += p[i];
            }
            bf16x4 hi, lo;
            two_terms(p, hi, lo);
            const int t = kg * NU + x, r = rg * RTW + hv;
            bf16* to = lds.p + (r * 64 + lane) * 8 + 4 * t;
            *(bf16x4*)to = hi;
            *(bf16x4*)(to + S::RP * 512) = lo;
        }
    };
    const auto values = [&](const bf16* tile) {
        const int lane = lane_in_step(), c16 = lane & 15, g4 = lane >> 4;
        int any_moved = 0;
        for (int r = 0; r < S::RP; ++r) any_moved |= lds.moved[r];
        if (uniform(any_moved)) {
#pragma unroll
            for (int r = 0; r < S::RP; ++r) {
                const float c = lds.moved[r] ? lds.factor[r * 16 + c16] : 1.f;
#pragma unroll
                for (int b = 0; b < CT; ++b) acc[r][b] *= c;
            }
        }
        const int key = 4 * g4 + c16 / 4;            // (and 16 behind it: the same order in LDS)
        bf16x8 va[CT];
#pragma unroll
        for (int b = 0; b < CT; ++b) {
            const int c = 2 * (wave * CT + b) + (c16 & 3) / 2;
            const bf16* x = tile + key * W + 8 * latent_piece(key, c) + 4 * (c16 & 1);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)x);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(x + 16 * W));
            va[b] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        // the weights of the next rows are read ahead of these rows' products
        const bf16* p = lds.p + lane * 8;
        bf16x8 pf = *(const bf16x8*)p, pr = *(const bf16x8*)(p + S::RP * 512);
#pragma unroll
        for (int r = 0; r < S::RP; ++r) {
            const bf16* x = p + (r + 1 < S::RP ? r + 1 : r) * 512;
            const bf16x8 nf = *(const bf16x8*)x, nr = *(const bf16x8*)(x + S::RP * 512);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pf, acc[r][b]);
#pragma unroll
            for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pr, acc[r][b]);
            pf = nf;
            pr = nr;
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    const auto tile_of = [&](int b) { return lds.tile + b * KT * W; };
    if constexpr (S::kPipe) {
        // The scores of a step are made in front of the values of the one before it, with
        // no barrier in between: there is always something to multiply. Steps in LDS: two
        // in use, the others in flight.
#pragma unroll
        for (int b = 0; b < BUF - 2; ++b) fetch_next(b);
        int buf = 0, back = 0;
        for (int pos = keys.begin; pos < keys.end + KT; pos += KT) {
            const bool front = pos < keys.end;
            const bool partial = keys.all < keys.end && pos + KT > keys.all;
            int missing = 0;
            if (front) {
                wait_step(BUF - 3);
                missing = gaps[0];
                step_done();
            }
            __syncthreads();                         // the step has landed, the weights of the last are there
            fetch_next(BUF - 3);
            if (front) {
                if (partial) clear_odd(tile_of(buf));
                products(tile_of(buf), pos, missing, partial);
            }
            if (pos > keys.begin) values(tile_of(back));
            lds_barrier();
            if (front) weights(pos, missing, partial);
            back = buf;
            buf = buf + 1 == BUF ? 0 : buf + 1;
        }
    } else {
#pragma unroll
        for (int b = 0; b < BUF - 1; ++b) fetch_next(b);
        int buf = 0;
        for (int pos = keys.begin; pos < keys.end; pos += KT) {
            const bool partial = keys.all < keys.end && pos + KT > keys.all;
            wait_step(BUF - 2);
            const int missing = gaps[0];
            step_done();
            __syncthreads();                         // the step has landed, the last one is done with
            fetch_next(BUF - 2);
            if (partial) clear_odd(tile_of(buf));
            products(tile_of(buf), pos, missing, partial);
            lds_barrier();
            weights(pos, missing, partial);
            lds_barrier();
            values(tile_of(buf));
            buf = buf + 1 == BUF ? 0 : buf + 1;
        }
    }

    // the rows' sums and references, to all waves
    const float part_sum = sum_quarters(l);
    if (scores && g4 == 0) {
        lds.sum[kg][row] = part_sum;
        if (kg == 0) lds.factor[row] = m;
    }
    __syncthreads();
    const int col = wave * (16 * CT) + 4 * g4;
    if (it.pieces > 1) {
        float* to = e.acc + ((long)it.slot * R + c16) * DC + col;
        // (a row without a key in this piece has l = 0, and its values are not used)
#pragma unroll
        for (int r = 0; r < S::RP; ++r)
#pragma unroll
            for (int b = 0; b < CT; ++b) *(f32x4*)(to + r * 16 * DC + 16 * b) = acc[r][b];
        if (const int r = threadIdx.x; r < R) {
            float sum = 0.f;
            for (int k = 0; k < S::KG; ++k) sum += lds.sum[k][r];
            e.ml[((long)it.slot * R + r) * 2] = lds.factor[r];
            e.ml[((long)it.slot * R + r) * 2 + 1] = sum;
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < S::RP; ++r) {
        const int y = 16 * r + c16;
        float sum = 0.f;
        for (int k = 0; k < S::KG; ++k) sum += lds.sum[k][y];
        const RowAt x = run_row(a, it, it.tile * R + y);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        bf16* to = (bf16*)a.o + x.q * DC + col;
        if (x.in) {
#pragma unroll
            for (int b = 0; b < CT; ++b) {
                bf16x4 z;
                for (int i = 0; i < 4; ++i) z[i] = (bf16)(acc[r][b][i] * inv);
                *(bf16x4*)(to + 16 * b) = z;
            }
            if (a.lse && wave == 0 && g4 == 0)
                a.lse[x.q] = sum == 0.f ? -INFINITY : (lds.factor[y] + __log2f(sum)) * kLn2;
        }
    }
}

template <int DC, int R>
__global__ __launch_bounds__(kLatentThreads, 2) void attn_latent_bf16(
    AttnArgs a, AttnSplit s, EvenSplit e) {
    __shared__ LatentLds<DC, R> lds;
    even_runs(a, s, e, lds.item, [&](const EvenRun& it) { latent_run<DC, R>(a, e, it, lds); });
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
    const_int* table;
    bf16* const tiles;
    int wave, lane;
    int half, load0;             // which 16 keys, and the first of the wave's loads of them
    bool fewer;                  // LD - 1 loads
    uint32_t off[LD];            // where in the keys' rows the lane's bytes are
    int fetched, buf;            // the next step's position and buffer
    int page[2];                 // and pages
    // of the b-th step from the next one to be waited for: whether loads are in flight (a
    // page that does not exist has none), and its sixteens without a page
    bool have[BUF];
    int gaps[BUF];

    __device__ __forceinline__ KeySteps(const AttnArgs& args, const Keys& k, const_int* t, bf16* to)
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
        if (keys.begin < keys.end) look_up();
    }
    __device__ __forceinline__ void piece_at(int i, int l, int& key, int& byte) const {
        const int x = (load0 + i) * 64 + l;
        key = x / kPieces;
        byte = 16 * latent_piece(key, x - key * kPieces);
    }
    // (sixteens behind the end: the last key's page)
    __device__ __forceinline__ void look_up() {
        page[0] = page_at(a, table, min(fetched, keys.end - 1), keys.end);
        page[1] = page_at(a, table, min(fetched + 16, keys.end - 1), keys.end);
    }
    // The next step, b steps behind the next one to be waited for. Positions behind the
    // end are read from the last one, which some row of the tile sees: nothing else of
    // an unused row gets here.
    __device__ __forceinline__ void fetch(int b) {
        if (fetched >= keys.end) return;
        const int pg = uniform(half ? page[1] : page[0]);
        have[b] = pg >= 0;
        gaps[b] = (page[0] < 0) | (page[1] < 0) << 1;
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
        look_up();
    }
    // Waits for this wave's part of the oldest step, of `after` that may be behind it.
    __device__ __forceinline__ void wait(int after) {
        int n = 0;
#pragma unroll
        for (int b = 1; b < BUF - 1; ++b) n += b <= after && n == b - 1 && have[b];
        if (n == 2) {
            if (fewer) wait_loads<2 * LD - 2>();
            else wait_loads<2 * LD>();
        } else if (n == 1) {
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
// wave rg + 2 kg has half of the rows and 16 keys. The rows' reference is what all
// their keys' maxima were up to the step before: a weight may be up to 2^60 then, which
// costs nothing in fp32 and bf16. Where a maximum jumps further (the first step of a
// run, for one), the step's weights are made again behind the barrier.
template <int DC, int R> struct NarrowLds {
    static constexpr int W = DC + kPe, RP = R / 16;
    static constexpr int BUF = R == 64 && DC == 512 ? 3 : 4;     // what LDS holds
    __align__(128) bf16 tile[BUF * 32 * W];
    __align__(16) bf16 p[2][2 * RP * 512];
    float top[2][2][R], factor[2][R], sum[2][R], ref[R];
    int moved[2][2], jump[2][4], odd[32];
    EvenItem item;
};
constexpr float kJump = 60.f;

template <int DC, int R>
__device__ __forceinline__ void narrow_run(const AttnArgs& a, const EvenSplit& e, const EvenRun& it,
                                           NarrowLds<DC, R>& lds) {
    constexpr int W = DC + kPe, KT = 32, RP = R / 16, RTW = R / 32, KS = W / 32, CT = DC / 64;
    constexpr int BUF = NarrowLds<DC, R>::BUF;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const Keys keys = run_keys(a, it, R);
    KeySteps<DC, BUF> ks(a, keys, table_row(a, it.req), lds.tile);
#pragma unroll
    for (int b = 0; b < BUF - 2; ++b) ks.fetch(b);
    const int steps = keys.end > keys.begin ? (keys.end - keys.begin + KT - 1) / KT : 0;
    // (both kinds of waves go through the same barriers)
    const auto begin_step = [&](int j, bool& partial) {
        int missing = 0;
        if (j < steps) {
            ks.wait(BUF - 3);
            missing = ks.take();
        }
        __syncthreads();                             // the step has landed, the weights of the last are there
        partial = j < steps && keys.all < keys.end && keys.begin + (j + 1) * KT > keys.all;
        return missing;
    };
    const auto jumped = [&](int j) {
        const int* x = lds.jump[j & 1];
        return j >= 0 && uniform(x[0] | x[1] | x[2] | x[3]) != 0;
    };

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
            if (jumped(j - 1)) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) {
                    l[rt] = l_before[rt];
                    follow(rt, top_of(j - 1, rt));
                }
                publish(j - 1, true);
                weights(j - 1);
                __syncthreads();
            }
            ks.fetch(BUF - 3);
            if (partial) ks.clear_odd(ks.tile(buf), lds.odd);
            if (j == steps) break;
            // The reference may stay behind the maximum by up to 8 in the log2 domain.
            float top[RTW];
            bool ahead = false;
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) {
                factor[rt] = 1.f;
                top[rt] = j > 0 ? top_of(j - 1, rt) : -INFINITY;
                ahead |= top[rt] > m[rt] + 8.f;
            }
            const bool moved = __any(ahead);
            if (moved) {
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) follow(rt, top[rt]);
            }
            publish(j, moved);

            // products: fragments of keys are in flight ahead of them
            const bf16* from = ks.tile(buf) + (16 * kg + c16) * W;
            // (pieces 4 i + g4: the order of LDS repeats every eight)
            const bf16* k[2] = {from + 8 * latent_piece(c16, g4), from + 8 * latent_piece(c16, 4 + g4)};
            const auto read = [&](int i) { return *(const bf16x8*)(k[i & 1] + 64 * (i / 2)); };
            constexpr int kAhead = KS < 6 ? KS : 6;
            bf16x8 kf[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) kf[i] = read(i);
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
        if (jumped(j - 1)) __syncthreads();          // the weights are made again
        ks.fetch(BUF - 3);
        if (partial) ks.clear_odd(ks.tile(buf), lds.odd);
        if (j > 0) {
            const int x = (j - 1) & 1;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!uniform(lds.moved[x][g])) continue;
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) {
                    const float c = lds.factor[x][(g * RTW + rt) * 16 + c16];
#pragma unroll
                    for (int b = 0; b < CT; ++b) acc[g * RTW + rt][b] *= c;
                }
            }
            const bf16* tile = ks.tile(back);
            const int key = 4 * g4 + c16 / 4;        // (and 16 behind it: the same order in LDS)
            bf16x8 va[CT];
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
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const bf16x8 pf = *(const bf16x8*)(p + r * 512), pr = *(const bf16x8*)(p + (RP + r) * 512);
#pragma unroll
                for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pf, acc[r][b]);
#pragma unroll
                for (int b = 0; b < CT; ++b) acc[r][b] = mma32(va[b], pr, acc[r][b]);
            }
        }
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
            // (a row without a key in this piece has l = 0, and its values are not used)
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
    even_runs(a, s, e, lds.item, [&](const EvenRun& it) { narrow_run<DC, R>(a, e, it, lds); });
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
    EvenItem item;
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
        for (int g = 0; (!cut || sum != 0.f) && g < CT / VW; ++g)
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
    even_runs(a, s, e, lds.item, [&](const EvenRun& it) { latent_run_f32<DC>(a, e, it, lds); });
}

// Kernel and work split of a call, from sizes alone.
struct LatentPlan {
    AttnSplit split;
    EvenSplit even;
    size_t bytes;
};
LatentPlan plan_of(int T, int B, int Hq, int dc, int max_new, bool bf16_io) {
    const long most = (long)(max_new > 0 && max_new < T ? max_new : T) * Hq;
    LatentPlan p{};
    const int R = !bf16_io || most <= 32 ? 32 : most <= 64 ? 64 : 128;
    p.split.R = p.even.R = R;
    p.split.R_log2 = p.even.R_log2 = __builtin_ctz((unsigned)R);
    p.split.min_rows = 1;
    p.split.max_rows = INT32_MAX;
    // as many workgroups as the card's 256 compute units hold
    p.even.G = dc == 128 ? 512 : 256;
    p.bytes = (size_t)p.even.G * (2 * R * (dc + 2) + 4) * sizeof(float);
    if (B > kBlock) p.bytes += AttnTable::ints(B) * sizeof(int);
    return p;
}

template <int DC>
hipError_t launch(const AttnArgs& a, const LatentPlan& p, hipStream_t st) {
    if (a.B > kBlock) even_list<<<1, 64 * kListWaves, 0, st>>>(a, p.split, p.even);
    const auto run = [&](auto kernel, int threads) { kernel<<<p.even.G, threads, 0, st>>>(a, p.split, p.even); };
    if (!a.bf16_io) run(attn_latent_f32<DC>, kAttnThreads);
    else if (p.split.R == 32) run(attn_latent_narrow<DC, 32>, kLatentThreads);
    else if (p.split.R == 64) run(attn_latent_narrow<DC, 64>, kLatentThreads);
    else run(attn_latent_bf16<DC, 128>, kLatentThreads);
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
    e.ml = (float*)(e.pieces + 4 * e.G);
    e.acc = e.ml + (size_t)4 * e.G * e.R;
    if (a.B > kBlock) e.table = (int*)(e.acc + (size_t)2 * e.G * e.R * a.d);
    // a call of few keys has fewer units than that
    const long tiles = ((long)a.T * a.Hq >> e.R_log2) + (a.B < a.T ? a.B : a.T);
    const long units = tiles * (((long)a.width << a.page_shift) / kUnitKeys + 1 + 2);
    if (units < e.G) e.G = (int)units;
    switch (a.d) {
        case 128: return launch<128>(a, p, st);
        case 256: return launch<256>(a, p, st);
        default: return launch<512>(a, p, st);
    }
}

}  // namespace kda
