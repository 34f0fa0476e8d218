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
#include "kda_attn_rows.h"
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

template <int DC, int RT> struct LatentShape {
    static constexpr int W = DC + kPe;
    static constexpr int KG = 4 / RT;                // waves that share a row group
    static constexpr int KT = RT == 1 ? 64 : 32;     // keys of a step
    static constexpr int NU = KT / 16 / KG;          // key tiles of a wave's scores
    static constexpr int BUF = RT == 1 ? 2 : 3;      // steps in LDS
    static constexpr int CT = DC / 64;               // value columns of a wave, in 16s
    static constexpr int RP = 2 * RT;                // row tiles of 16
    static constexpr int KS2 = KT / 32;
    static constexpr int kKeys = KT / 4;             // keys that a wave fetches
    static constexpr int LD = kKeys * (W / 8) / 64;  // its loads
};

template <int DC, int RT> struct LatentLds {
    typedef LatentShape<DC, RT> S;
    __align__(128) bf16 tile[S::BUF * S::KT * S::W];
    __align__(16) bf16 p[2 * S::RP * S::KS2 * 64 * 8];
    float top[S::KG][32 * RT];
    float factor[32 * RT], sum[S::KG][32 * RT];
    int moved[4], odd[S::KT];
    AttnItem item;
};

template <int DC, int RT>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_latent_bf16(AttnArgs a, AttnSplit s,
                                                                    unsigned first_block) {
    typedef LatentShape<DC, RT> S;
    constexpr int W = S::W, KT = S::KT, NU = S::NU, BUF = S::BUF, CT = S::CT, LD = S::LD;
    constexpr int KS = W / 32;                       // steps of the scores' contraction
    constexpr int kPieces = W / 8;
    __shared__ LatentLds<DC, RT> lds;
    const AttnItem it = attn_item(a, s, (int)(first_block + blockIdx.x), lds.item);
    if (!it.found) return;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const int rg = wave % RT, kg = wave / RT;
    const Keys keys = part_keys(a, s, it, a.Hq);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;

    // queries of the wave's 32 rows
    bf16x8 qf[2][KS];
    int limit[2];                                    // last visible position
    for (int rt = 0; rt < 2; ++rt) {
        const RowAt x = row_at(a, it, a.Hq, it.tile * s.R + rg * 32 + rt * 16 + c16);
        limit[rt] = x.in ? (int)min((long)it.kept + x.t, (long)kKeepAll) : -1;
        const bf16* q = (const bf16*)a.q + x.q * W + 8 * g4;
        for (int k = 0; k < KS; ++k) {
            bf16x8 z = {};
            if (x.in) z = *(const bf16x8*)(q + 32 * k);
            qf[rt][k] = z;
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    f32x4 acc[S::RP][CT];
    for (int r = 0; r < S::RP; ++r)
        for (int c = 0; c < CT; ++c) acc[r][c] = zero4();

    // The lane's i-th 16 bytes of the wave's keys of a step: key fkey(i) of them,
    // byte fcol(i) of its row.
    auto fkey = [&](int i) { return (i * 64 + lane) / kPieces; };
    auto fcol = [&](int i) {
        const int x = i * 64 + lane, r = x / kPieces;
        return 16 * latent_piece(wave * S::kKeys + r, x - r * kPieces);
    };
    // A step's keys of this wave. Positions behind the end are read from the last
    // one, which some row of the tile sees: nothing else of an unused row gets here.
    auto fetch = [&](int buf, int pos, int page) {
        const int base = pos + wave * S::kKeys;
        bf16* to = lds.tile + (buf * KT + wave * S::kKeys) * W;
        if (page >= 0) {
            const int at = min(base, keys.end - 1);
            const bf16* from = (const bf16*)a.kc + (((long)page << a.page_shift) + (at & row_mask)) * W;
            const int most = keys.end - 1 - at;
            const uint32_t l0 = uniform((int)(uint32_t)(uintptr_t)(lds_void*)to);
            for (int i = 0; i < LD; ++i)
                load_to_lds(l0 + i * 1024, min(fkey(i), most) * (2 * W) + fcol(i), from);
        } else {
            for (int i = 0; i < LD; ++i) *(bf16x8*)(to + i * 512 + 8 * lane) = bf16x8{};
        }
    };
    const auto own_page = [&](const StepPages<KT>& p) {
        int x = p.id[0];
        for (int u = 1; u < KT / 16; ++u) x = wave * S::kKeys / 16 == u ? p.id[u] : x;
        return uniform(x);
    };
    // Pages of 16 keys of which the first is behind the end: those of the last key.
    const auto pages_at = [&](int pos) {
        StepPages<KT> p;
        for (int u = 0; u < KT / 16; ++u)
            p.id[u] = page_at(a, table, min(pos + 16 * u, keys.end - 1), keys.end);
        return p;
    };

    StepPages<KT> pg[BUF];                           // of this step and those in flight
    if (keys.begin < keys.end) {
        for (int b = 0; b < BUF - 1; ++b) {
            pg[b] = pages_at(keys.begin + b * KT);
            if (keys.begin + b * KT < keys.end) fetch(b, keys.begin + b * KT, own_page(pg[b]));
        }
        pg[BUF - 1] = pages_at(keys.begin + (BUF - 1) * KT);
    }
    int buf = 0;
    for (int pos = keys.begin; pos < keys.end; pos += KT) {
        // this wave's part of the step has landed; with three buffers the next
        // step's loads may be in flight, if it has any
        if (BUF == 3 && pos + KT < keys.end && own_page(pg[1]) >= 0) wait_loads<LD>();
        else wait_loads<0>();
        __syncthreads();                             // everybody's, and the last step is done with
        const int last_buf = buf == 0 ? BUF - 1 : buf - 1;
        if (pos + (BUF - 1) * KT < keys.end)
            fetch(last_buf, pos + (BUF - 1) * KT, own_page(pg[BUF - 1]));
        const int missing = pg[0].missing();
        for (int b = 0; b < BUF - 1; ++b) pg[b] = pg[b + 1];
        pg[BUF - 1] = pages_at(pos + BUF * KT);
        bf16* tile = lds.tile + buf * KT * W;
        const bool partial = keys.all < keys.end && pos + KT > keys.all;
        if (partial) {
            // Positions that only some rows see: a value there that is not finite must
            // not meet the weight 0 of the others in a product. It counts 0, and the
            // scores of the rows that see its position become NaN.
            bf16* x = tile + wave * S::kKeys * W;
            if (lane < S::kKeys) lds.odd[wave * S::kKeys + lane] = 0;
            lds_fence_wave();
            for (int i = 0; i < LD; ++i) {
                if (fcol(i) >= 2 * DC) continue;
                bool odd = false;
                bf16x8* v = (bf16x8*)(x + i * 512 + 8 * lane);
                *v = only_finite(*v, odd);
                if (odd) lds.odd[wave * S::kKeys + fkey(i)] = 1;
            }
            __syncthreads();
        }

        // scores
        f32x4 st[2][NU];
        for (int u = 0; u < NU; ++u) {
            const bf16* k = tile + (16 * (kg * NU + u) + c16) * W;
            st[0][u] = st[1][u] = zero4();
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const bf16x8 kf = *(const bf16x8*)(k + 8 * latent_piece(c16, 4 * i + g4));
                st[0][u] = mma32(kf, qf[0][i], st[0][u]);
                st[1][u] = mma32(kf, qf[1][i], st[1][u]);
            }
        }
        for (int rt = 0; rt < 2; ++rt)
            for (int u = 0; u < NU; ++u)
                for (int i = 0; i < 4; ++i) st[rt][u][i] *= scale;
        if (pos + KT > keys.all || missing) {
            for (int u = 0; u < NU; ++u)
                for (int i = 0; i < 4; ++i) {
                    const int y = 16 * (kg * NU + u) + 4 * g4 + i;
                    const bool none = pos + y >= keys.end || (missing >> (kg * NU + u) & 1);
                    const bool odd = partial && lds.odd[y];
                    for (int rt = 0; rt < 2; ++rt) {
                        if (odd) st[rt][u][i] = NAN;
                        if (none || pos + y > limit[rt]) st[rt][u][i] = -INFINITY;
                    }
                }
        }
        float mx[2];
        for (int rt = 0; rt < 2; ++rt) {
            mx[rt] = -INFINITY;
            for (int u = 0; u < NU; ++u)
                for (int i = 0; i < 4; ++i) mx[rt] = fmaxf(mx[rt], st[rt][u][i]);
            mx[rt] = max_quarters(mx[rt]);
        }
        if constexpr (S::KG > 1) {
            if (g4 == 0)
                for (int rt = 0; rt < 2; ++rt) lds.top[kg][rg * 32 + rt * 16 + c16] = mx[rt];
            __syncthreads();
            for (int rt = 0; rt < 2; ++rt)
                for (int k = 0; k < S::KG; ++k)
                    mx[rt] = fmaxf(mx[rt], lds.top[k][rg * 32 + rt * 16 + c16]);
        }
        // The reference may stay behind the maximum by up to 8 in the log2 domain.
        const bool moved = __any(mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f);
        if (moved) {
            for (int rt = 0; rt < 2; ++rt) {
                const float mn = fmaxf(m[rt], mx[rt]);
                const float c = mn == -INFINITY ? 1.f : exp2_f(m[rt] - mn);
                m[rt] = mn;
                l[rt] *= c;
                if (kg == 0 && g4 == 0) lds.factor[rg * 32 + rt * 16 + c16] = c;
            }
        }
        if (kg == 0 && lane == 0) lds.moved[rg] = moved;
        for (int rt = 0; rt < 2; ++rt) {
            const float mu = m[rt] == -INFINITY ? 0.f : m[rt];
            for (int u = 0; u < NU; ++u) {
                float p[4];
                for (int i = 0; i < 4; ++i) {
                    p[i] = exp2_f(st[rt][u][i] - mu);
                    l[rt] += p[i];
                }
                bf16x4 hi, lo;
                two_terms(p, hi, lo);
                const int t = kg * NU + u, r = rg * 2 + rt;
                bf16* to = lds.p + ((r * S::KS2 + t / 2) * 64 + lane) * 8 + 4 * (t & 1);
                *(bf16x4*)to = hi;
                *(bf16x4*)(to + S::RP * S::KS2 * 512) = lo;
            }
        }
        __syncthreads();

        // values
        for (int g = 0; g < RT; ++g) {
            if (!uniform(lds.moved[g])) continue;
            for (int rt = 0; rt < 2; ++rt) {
                const float c = lds.factor[g * 32 + rt * 16 + c16];
                for (int b = 0; b < CT; ++b) acc[2 * g + rt][b] *= c;
            }
        }
#pragma unroll
        for (int ks = 0; ks < S::KS2; ++ks) {
            bf16x8 pf[S::RP], pr[S::RP];
            for (int r = 0; r < S::RP; ++r) {
                const bf16* x = lds.p + ((r * S::KS2 + ks) * 64 + lane) * 8;
                pf[r] = *(const bf16x8*)x;
                pr[r] = *(const bf16x8*)(x + S::RP * S::KS2 * 512);
            }
            const int key = 32 * ks + 4 * g4 + c16 / 4;
#pragma unroll
            for (int b = 0; b < CT; ++b) {
                const int c = 2 * (wave * CT + b) + (c16 & 3) / 2;
                const bf16* x = tile + key * W + 8 * latent_piece(key, c) + 4 * (c16 & 1);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)x);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(x + 16 * W));
                const bf16x8 va = __builtin_bit_cast(
                    bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                for (int r = 0; r < S::RP; ++r) {
                    acc[r][b] = mma32(va, pf[r], acc[r][b]);
                    acc[r][b] = mma32(va, pr[r], acc[r][b]);
                }
            }
        }
        buf = buf + 1 == BUF ? 0 : buf + 1;
    }

    // the rows' sums and references, to all waves
    for (int rt = 0; rt < 2; ++rt) {
        const float sum = sum_quarters(l[rt]);
        if (g4 == 0) {
            lds.sum[kg][rg * 32 + rt * 16 + c16] = sum;
            if (kg == 0) lds.top[0][rg * 32 + rt * 16 + c16] = m[rt];
        }
    }
    __syncthreads();
    for (int r = 0; r < S::RP; ++r) {
        const int row = 16 * r + c16;
        float sum = 0.f;
        for (int k = 0; k < S::KG; ++k) sum += lds.sum[k][row];
        const float top = lds.top[0][row];
        const int col = wave * (DC / 4) + 4 * g4;
        if (it.parts > 1) {
            const long slot = (long)it.slot + (long)it.part * it.tiles + it.tile;
            if ((unsigned long)slot >= (unsigned long)s.slots) return;   // (a guard)
            const long at = slot * s.R + row;
            // (a row without a key in this part has l = 0, and its values are not read)
            for (int b = 0; sum != 0.f && b < CT; ++b)
                *(f32x4*)(s.acc + at * DC + col + 16 * b) = acc[r][b];
            if (wave == 0 && g4 == 0) { s.ml[at * 2] = top; s.ml[at * 2 + 1] = sum; }
            continue;
        }
        const RowAt x = row_at(a, it, a.Hq, it.tile * s.R + row);
        if (!x.in) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int b = 0; b < CT; ++b) {
            bf16x4 y;
            for (int i = 0; i < 4; ++i) y[i] = (bf16)(acc[r][b][i] * inv);
            *(bf16x4*)((bf16*)a.o + x.q * DC + col + 16 * b) = y;
        }
        if (a.lse && wave == 0 && g4 == 0)
            a.lse[x.q] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
    }
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
    AttnItem item;
};

template <int DC>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_latent_f32(AttnArgs a, AttnSplit s,
                                                                   unsigned first_block) {
    constexpr int W = DC + kPe, KT = 32, KQ = W / 16;   // pieces of a lane's channels
    constexpr int CT = DC / 64, VW = CT < 4 ? CT : 4;
    constexpr int kPieces = W / 4, kKeys = KT / 4, LD = kKeys * kPieces / 64;
    __shared__ LatentLdsF<DC> lds;
    const AttnItem it = attn_item(a, s, (int)(first_block + blockIdx.x), lds.item);
    if (!it.found) return;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const int rg = wave & 1, kg = wave >> 1;
    const Keys keys = part_keys(a, s, it, a.Hq);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;
    auto piece = [](int key, int c) { return c ^ (key & 15); };

    f32x4 qf[KQ];
    const RowAt at_row = row_at(a, it, a.Hq, it.tile * s.R + rg * 16 + c16);
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
        const bool cut = it.parts > 1;
        const long slot = (long)it.slot + (long)it.part * it.tiles + it.tile;
        if (cut && (unsigned long)slot >= (unsigned long)s.slots) return;   // (a guard)
        const long at = slot * s.R + row;
        const RowAt x = row_at(a, it, a.Hq, it.tile * s.R + row);
        if (!cut && !x.in) continue;
        const float inv = cut ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        float* to = cut ? s.acc + at * DC : (float*)a.o + x.q * DC;
        for (int g = 0; (!cut || sum != 0.f) && g < CT / VW; ++g)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < VW; ++j)
                    to[wave * (DC / 4) + 16 * VW * g + VW * (4 * g4 + i) + j] = acc[r][g * VW + j][i] * inv;
        if (wave != 0 || g4 != 0) continue;
        if (cut) {
            s.ml[at * 2] = top;
            s.ml[at * 2 + 1] = sum;
        } else if (a.lse) {
            a.lse[x.q] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
        }
    }
}

// Kernel and work split of a call, from sizes alone.
struct LatentPlan {
    int RT;
    Launch l;
    size_t bytes;
};
LatentPlan plan_of(int T, int B, int Hq, int dc, int max_new, bool bf16_io) {
    const long most = (long)(max_new > 0 && max_new < T ? max_new : T) * Hq;
    LatentPlan p{};
    p.RT = !bf16_io || most <= 32 ? 1 : most <= 64 ? 2 : 4;
    p.l = launch_of(T, B, Hq, 1, 32 * p.RT, 10, 9, 8, INT32_MAX);
    p.bytes = (size_t)p.l.split.slots * p.l.split.R * (dc + 2) * sizeof(float);
    if (B > kBlock) p.bytes += AttnTable::ints(B) * sizeof(int);
    return p;
}

template <int DC>
hipError_t launch(const AttnArgs& a, const LatentPlan& p, hipStream_t st) {
    const AttnSplit& s = p.l.split;
    if (a.B > kBlock) attn_list<<<1, 64 * kListWaves, 0, st>>>(a, s, s);
    const auto run = [&](auto kernel) {
        in_grids((unsigned)p.l.items, [&](unsigned grid, unsigned first) {
            kernel<<<grid, kAttnThreads, 0, st>>>(a, s, first);
        });
    };
    if (!a.bf16_io) run(attn_latent_f32<DC>);
    else if (p.RT == 1) run(attn_latent_bf16<DC, 1>);
    else if (p.RT == 2) run(attn_latent_bf16<DC, 2>);
    else run(attn_latent_bf16<DC, 4>);
    const int n = (int)p.l.joins;
    if (a.bf16_io) attn_join<bf16, DC><<<(unsigned)n, kAttnThreads, 0, st>>>(a, s, s, n);
    else attn_join<float, DC><<<(unsigned)n, kAttnThreads, 0, st>>>(a, s, s, n);
    return hipGetLastError();
}

}  // namespace

size_t attn_latent_ws(int T, int B, int Hq, int dc, int max_new, bool bf16_io) {
    return plan_of(T, B, Hq, dc, max_new, bf16_io).bytes;
}

hipError_t launch_attn_latent(const AttnArgs& a, void* ws, hipStream_t st) {
    LatentPlan p = plan_of(a.T, a.B, a.Hq, a.d, a.max_new, a.bf16_io);
    AttnSplit& s = p.l.split;
    s.far = LONG_MAX;
    s.ml = (float*)ws;
    s.acc = s.ml + (size_t)s.slots * s.R * 2;
    if (a.B > kBlock) s.table = (int*)(s.acc + (size_t)s.slots * s.R * a.d);
    switch (a.d) {
        case 128: return launch<128>(a, p, st);
        case 256: return launch<256>(a, p, st);
        default: return launch<512>(a, p, st);
    }
}

}  // namespace kda
