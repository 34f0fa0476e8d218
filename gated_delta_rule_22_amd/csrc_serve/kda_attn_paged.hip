// Causal attention of new tokens over a paged cache.
//
// With s_j = scale q.k_j over a row's visible positions, m = max s_j and
// l = sum exp(s_j - m): o = sum exp(s_j - m) v_j / l. One pass over the keys
// keeps m, l and the unnormalised row; a new maximum m' scales l and the row
// by exp(m - m'). Results over disjoint parts of the keys join by the same
// rule. Scores are kept in the log2 domain (s log2 e), so that the
// exponential is one v_exp_f32.
//
// attn_stream_*: decode steps and drafts, up to 32 rows per KV head. What
// bounds them is reading K and V once. A workgroup takes one tile of 16 RT
// rows and a part of its keys (kda_attn_sched.h); its four waves take 32
// (fp32: 16) keys each in turn and run free of each other, so that every wave
// has its next keys and values in flight while it computes. Their rows are
// joined through LDS at the end. bf16, 32 query heads over 8 of 128: one token
// of 256 requests over 1024 to 16384 positions (5.8 GB) 970 + 7 us, 6.0 TB/s;
// 8 tokens of 4 over 65536 to 262144 (2.6 GB) 425 + 8 us, 6.2 TB/s; one token
// over 1000 positions 8.2 + 4.5 us: memory latencies, and 2072
// workgroups started of which 64 have a part. fp32, 16 heads over 4:
// 64 tokens over 4096 positions (1.1 GB) 193 us, 5.6 TB/s; 1024 tokens over
// 1024 of width 64 80 us, half of the fp32 matrix rate. Widths 32 and 16, bf16, 32
// heads over 8: one token of 256 requests over 1024 to 8192 positions 172 and 94
// us, 5.2 and 4.8 TB/s; 2048 tokens over 2048, in tiles of 32 rows that read the
// keys again each, 102 and 98 us, where width 64 in tiles of 128 takes 109.
#include "kda_attn_rows.h"

#include <limits.h>

namespace kda {
namespace {

constexpr int kTileRows = 128;

template <bool NT>
__device__ __forceinline__ bf16x8 load16(const bf16* p) {
    return NT ? __builtin_nontemporal_load((const bf16x8*)p) : *(const bf16x8*)p;
}
// Result of a row, from its unnormalised values: 8 (bf16) or 4 (fp32) of them.
__device__ __forceinline__ void store_row(bf16* o, const float* v, float inv) {
    bf16x8 x;
    for (int i = 0; i < 8; ++i) x[i] = (bf16)(v[i] * inv);
    *(bf16x8*)o = x;
}
__device__ __forceinline__ void store_row(float* o, const float* v, float inv) {
    for (int j = 0; j < 8; j += 4) {
        f32x4 x;
        for (int i = 0; i < 4; ++i) x[i] = v[j + i] * inv;
        *(f32x4*)(o + j) = x;
    }
}

// Joins the four waves' rows: ml[wave][16][2] and acc[wave][16][D + 4] in LDS
// hold 16 rows of each; writes the rows themselves, or a partial result.
template <typename T, int D>
__device__ __forceinline__ void join_waves(const AttnArgs& a, const AttnSplit& s,
                                           const AttnItem& it, int G, int r0, const float* ml,
                                           const float* acc) {
    constexpr int kPer = 8, kLanes = D / kPer;      // 2 .. 16 threads per row
    const int row = threadIdx.x / kLanes, d = threadIdx.x % kLanes * kPer;
    if (row >= 16) return;
    float m = -INFINITY, l = 0.f, v[kPer] = {};
    for (int w = 0; w < 4; ++w) m = fmaxf(m, ml[(w * 16 + row) * 2]);
    for (int w = 0; w < 4; ++w) {
        const float mw = ml[(w * 16 + row) * 2], lw = ml[(w * 16 + row) * 2 + 1];
        if (lw == 0.f) continue;                    // that wave saw no key of this row
        const float c = mw == -INFINITY ? 1.f : exp2_f(mw - m);   // (all scores NaN: lw is)
        l += c * lw;
        const float* x = acc + (w * 16 + row) * (D + 4) + d;
        for (int i = 0; i < kPer; ++i) v[i] += c * x[i];
    }
    const int r = it.tile * s.R + r0 + row;
    if (it.parts > 1) {
        const long slot = (long)it.slot + ((long)it.part * it.tiles + it.tile) * a.Hkv + it.h;
        if ((unsigned long)slot >= (unsigned long)s.slots) return;   // (a guard)
        const long at = slot * s.R + r0 + row;
        // (a row without a key in this part has l = 0, and its values are not read)
        for (int i = 0; l != 0.f && i < kPer; i += 4)
            *(f32x4*)(s.acc + at * D + d + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        if (d == 0) { s.ml[at * 2] = m; s.ml[at * 2 + 1] = l; }
        return;
    }
    const RowAt x = row_at(a, it, G, r);
    if (!x.in) return;
    store_row((T*)a.o + x.q * D + d, v, l == 0.f ? 0.f : 1.f / l);
    if (a.lse && d == 0) a.lse[x.q] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

// The running maximum, sum and rows of 16 RT rows in one wave. Lane l holds
// row l % 16 of each group of 16 throughout; the sum stays one over the lane's
// own keys until the end.
//
// bf16, 32 keys a step. S^T = K Q^T leaves lane l with the scores of its
// row against keys 16 sub + 4 (l / 16) + i; as the second operand of
// O^T += V^T P^T they stay in place when the contraction runs over the keys in
// that same order, which the transposing LDS read gives V.
template <int D> struct StreamLds {
    static constexpr int kJoin = 4 * 16 * (D + 4), kStage = 4 * 32 * D / 2;
    __align__(16) float join[kJoin > kStage ? kJoin : kStage];   // first the waves' V stages
    float join_ml[4 * 16 * 2];
    AttnItem item;
};
template <int D, int RT, bool NT>
__device__ __forceinline__ void stream_part(const AttnArgs& a, const AttnSplit& s,
                                            const AttnItem& it, StreamLds<D>& lds) {
    constexpr int KS = D < 32 ? 1 : D / 32;          // steps of 32 over the head
    constexpr int NB = D / 16;                       // value columns in 16s
    constexpr int VL = D / 16;                       // 16-byte loads per lane for 32 rows of V
    constexpr int CH = D / 8;                        // 16-byte pieces of a row
    const int G = a.Hq / a.Hkv, wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const Keys keys = part_keys(a, s, it, G);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    bf16* stage = (bf16*)lds.join + wave * (32 * D);     // V of this wave's 32 keys

    bf16x8 qf[RT][KS];
    int limit[RT];                                   // last visible position of the lane's row
    for (int rt = 0; rt < RT; ++rt) {
        const RowAt x = row_at(a, it, G, it.tile * s.R + rt * 16 + c16);
        limit[rt] = x.in ? (int)min((long)it.kept + x.t, (long)kKeepAll) : -1;
        const bf16* q = (const bf16*)a.q + x.q * D;
        for (int k = 0; k < KS; ++k) {
            const int d = 32 * k + 8 * g4;
            bf16x8 z = {};
            if (x.in && d < D) z = *(const bf16x8*)(q + d);
            qf[rt][k] = z;
        }
    }

    float m[RT], l[RT];
    f32x4 acc[RT][NB];
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY;
        l[rt] = 0.f;
        for (int b = 0; b < NB; ++b) acc[rt][b] = zero4();
    }

    bf16x8 kf[2][KS], vf[VL];
    // pages of the 32 keys at hand and, a step ahead of their loads, of the next
    int page[2] = {-1, -1}, page_next[2] = {-1, -1};
    const int row_mask = (1 << a.page_shift) - 1;
    auto base_of = [&](int p, int pos) {             // row of the plane of head h
        return (((long)p * a.Hkv + it.h) << a.page_shift) + (pos & row_mask);
    };
    auto load_k = [&](int pos) {
        for (int u = 0; u < 2; ++u) {
            if (page[u] >= 0) {
                const bf16* k = (const bf16*)a.kc + (base_of(page[u], pos + 16 * u) + c16) * D;
                for (int i = 0; i < KS; ++i)
                    if (D >= 32 || g4 < 2) kf[u][i] = load16<NT>(k + 32 * i + 8 * g4);
            } else {
                for (int i = 0; i < KS; ++i) kf[u][i] = bf16x8{};
            }
        }
    };
    // piece i * 64 + lane of the 32 rows; a half (16 rows) is VL / 2 loads,
    // but one load for D = 16
    auto load_v = [&](int pos) {
        for (int i = 0; i < VL; ++i) {
            const int x = i * 64 + lane, key = x / CH, c = x % CH;
            if (VL > 1) {
                const int u = i >= VL / 2;
                if (page[u] >= 0)
                    vf[i] = load16<NT>((const bf16*)a.vc +
                                       (base_of(page[u], pos + 16 * u) + (key & 15)) * D + 8 * c);
                else
                    vf[i] = bf16x8{};
            } else {
                const int p = key < 16 ? page[0] : page[1];
                vf[i] = bf16x8{};
                if (p >= 0)
                    vf[i] = *(const bf16x8*)((const bf16*)a.vc +
                                             (base_of(p, pos + (key & 16)) + (key & 15)) * D + 8 * c);
            }
        }
    };
    if (D == 16)
        for (int u = 0; u < 2; ++u) kf[u][0] = bf16x8{};

    int pos = keys.begin + wave * 32;
    if (pos < keys.end) {
        page[0] = page_at(a, table, pos, keys.end);
        page[1] = page_at(a, table, pos + 16, keys.end);
        page_next[0] = page_at(a, table, pos + 128, keys.end);
        page_next[1] = page_at(a, table, pos + 144, keys.end);
        load_k(pos);
        load_v(pos);
    }
    for (; pos < keys.end; pos += 128) {
        const int next = pos + 128;
        const int page_2 = page_at(a, table, next + 128, keys.end);
        const int page_3 = page_at(a, table, next + 144, keys.end);
        const bool gap0 = page[0] < 0, gap1 = page[1] < 0;
        f32x4 st[RT][2];
        for (int rt = 0; rt < RT; ++rt)
            for (int u = 0; u < 2; ++u) {
                f32x4 x = zero4();
                for (int k = 0; k < KS; ++k) x = mma32(kf[u][k], qf[rt][k], x);
                st[rt][u] = x;
            }
        // V rows that no row of the tile sees hold anything: they count 0
        if (pos + 32 > keys.end) {
            for (int i = 0; i < VL; ++i)
                if (pos + (i * 64 + lane) / CH >= keys.end) vf[i] = bf16x8{};
        }
        // Positions that only some rows see: a value there that is not finite
        // must not meet the weight 0 of the others in a product. It counts 0
        // here and is added below for the rows that see it.
        bool odd = false;
        if (pos + 32 > keys.all) {
            for (int i = 0; i < VL; ++i) vf[i] = only_finite(vf[i], odd);
            odd = __any(odd);
        }
        lds_fence_wave();                            // last step's reads of the stage are done
        for (int i = 0; i < VL; ++i) {
            const int x = i * 64 + lane, key = x / CH, c = x % CH;
            *(bf16x8*)(stage + key * D + 8 * v_piece8<D>(key, c)) = vf[i];
        }
        const int p0 = page[0], p1 = page[1];
        page[0] = page_next[0];
        page[1] = page_next[1];
        if (next < keys.end) {
            load_k(next);
            load_v(next);
        }
        page_next[0] = page_2;
        page_next[1] = page_3;
        bf16x8 pf[RT], pr[RT];
        float pe[RT][2][4];
        for (int rt = 0; rt < RT; ++rt) {
            float x[2][4];
            for (int u = 0; u < 2; ++u)
                for (int i = 0; i < 4; ++i) x[u][i] = st[rt][u][i] * scale;
            if (pos + 32 > keys.all || gap0 || gap1) {
                for (int u = 0; u < 2; ++u)
                    for (int i = 0; i < 4; ++i) {
                        const int key = pos + 16 * u + 4 * g4 + i;
                        if (key > limit[rt] || key >= keys.end || (u ? gap1 : gap0)) x[u][i] = -INFINITY;
                    }
            }
            float mx = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                             fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
            mx = max_quarters(mx);
            if (__any(mx > m[rt])) {
                const float mn = fmaxf(m[rt], mx);
                const float c = mn == -INFINITY ? 1.f : exp2_f(m[rt] - mn);
                m[rt] = mn;
                l[rt] *= c;
                for (int b = 0; b < NB; ++b) acc[rt][b] *= c;
            }
            const float mu = m[rt] == -INFINITY ? 0.f : m[rt];
            float sum = 0.f;
            for (int u = 0; u < 2; ++u)
                for (int i = 0; i < 4; ++i) {
                    const float p = exp2_f(x[u][i] - mu);
                    sum += p;
                    pe[rt][u][i] = p;
                }
            l[rt] += sum;
            two_terms({pe[rt][0][0], pe[rt][0][1], pe[rt][0][2], pe[rt][0][3], pe[rt][1][0],
                       pe[rt][1][1], pe[rt][1][2], pe[rt][1][3]}, pf[rt], pr[rt]);
        }
        lds_fence_wave();                            // the stage is written
        for (int b = 0; b < NB; ++b) {
            s16x4 lo, hi;
            {
                const int key = 4 * g4 + c16 / 4, c = 2 * b + (c16 & 3) / 2;
                const bf16* x = stage + key * D + 8 * v_piece8<D>(key, c) + 4 * (c16 & 1);
                lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)x);
                hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(x + 16 * D));
            }
            const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            for (int rt = 0; rt < RT; ++rt) {
                acc[rt][b] = mma32(va, pf[rt], acc[rt][b]);
                acc[rt][b] = mma32(va, pr[rt], acc[rt][b]);
            }
        }
        if (odd) {
            // the values left out above, for the rows that see them
            for (int key = 0; key < 32; ++key) {
                const int p = key < 16 ? p0 : p1;
                if (p < 0 || pos + key >= keys.end) continue;
                const bf16* v = (const bf16*)a.vc + base_of(p, pos + (key & 16)) * D + (long)(key & 15) * D;
                for (int rt = 0; rt < RT; ++rt) {
                    float w = 0.f;
                    for (int u = 0; u < 2; ++u)
                        for (int i = 0; i < 4; ++i)
                            if (u == key / 16 && i == (key & 3)) w = pe[rt][u][i];
                    w = __shfl(w, c16 + 16 * ((key & 15) / 4));
                    const bool sees = pos + key <= limit[rt];
                    for (int b = 0; b < NB; ++b)
                        for (int i = 0; i < 4; ++i) {
                            const float x = (float)v[16 * b + 4 * g4 + i];
                            if (sees && !finite_bits(x)) acc[rt][b][i] += w * x;
                        }
                }
            }
        }
    }

    for (int rt = 0; rt < RT; ++rt) {
        const float sum = sum_quarters(l[rt]);
        __syncthreads();                             // stage and the last group's rows are free
        if (g4 == 0) {
            lds.join_ml[(wave * 16 + c16) * 2] = m[rt];
            lds.join_ml[(wave * 16 + c16) * 2 + 1] = sum;
        }
        for (int b = 0; b < NB; ++b)
            *(f32x4*)(lds.join + (wave * 16 + c16) * (D + 4) + 16 * b + 4 * g4) = acc[rt][b];
        __syncthreads();
        join_waves<bf16, D>(a, s, it, G, rt * 16, lds.join_ml, lds.join);
    }
}
// Keys and values that are read once, and are more than the last-level cache
// holds, are read past it (see far_keys).
template <int D, int RT>
__device__ __forceinline__ void stream_bf16(const AttnArgs& a, const AttnSplit& s, int block,
                                            StreamLds<D>& lds) {
    const AttnItem it = attn_item(a, s, block, lds.item);
    if (!it.found) return;
    if constexpr (D >= 64) {
        if (it.far) {
            stream_part<D, RT, true>(a, s, it, lds);
            return;
        }
    }
    stream_part<D, RT, false>(a, s, it, lds);
}
template <int D, int RT>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_stream_bf16(AttnArgs a, AttnSplit s,
                                                                    unsigned first) {
    __shared__ StreamLds<D> lds;
    stream_bf16<D, RT>(a, s, (int)(first + blockIdx.x), lds);
}

// fp32, 16 keys a step. The contraction over the head takes element
// g D / 4 + s of the lane quarter g in step s, so that a lane's part of a key
// is contiguous; O^T's row 4 g + i of block c is value column (4 g + i) D / 16
// + c, so that a lane's part of a value row is contiguous too.
template <int D, int RT>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_stream_f32(AttnArgs a, AttnSplit s,
                                                                   unsigned first) {
    constexpr int KD = D / 4, NB = D / 16;
    __shared__ __align__(16) float join[4 * 16 * (D + 4)];
    __shared__ float join_ml[4 * 16 * 2];
    __shared__ AttnItem shared_item;
    const AttnItem it = attn_item(a, s, (int)(first + blockIdx.x), shared_item);
    if (!it.found) return;
    const int G = a.Hq / a.Hkv, wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const Keys keys = part_keys(a, s, it, G);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;

    f32x4 qf[RT][KD / 4];
    int limit[RT];
    for (int rt = 0; rt < RT; ++rt) {
        const RowAt x = row_at(a, it, G, it.tile * s.R + rt * 16 + c16);
        limit[rt] = x.in ? (int)min((long)it.kept + x.t, (long)kKeepAll) : -1;
        const float* q = (const float*)a.q + x.q * D + g4 * KD;
        for (int k = 0; k < KD / 4; ++k) {
            f32x4 z = zero4();
            if (x.in) z = *(const f32x4*)(q + 4 * k);
            qf[rt][k] = z;
        }
    }
    float m[RT], l[RT];
    f32x4 acc[RT][NB];
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY;
        l[rt] = 0.f;
        for (int b = 0; b < NB; ++b) acc[rt][b] = zero4();
    }

    f32x4 kf[KD / 4];
    float vf[4][NB];
    auto base_of = [&](int p, int pos) {
        return (((long)p * a.Hkv + it.h) << a.page_shift) + (pos & row_mask);
    };
    auto load_k = [&](int p, int pos) {
        if (p >= 0) {
            const float* k = (const float*)a.kc + (base_of(p, pos) + c16) * D + g4 * KD;
            for (int i = 0; i < KD / 4; ++i) kf[i] = *(const f32x4*)(k + 4 * i);
        } else {
            for (int i = 0; i < KD / 4; ++i) kf[i] = zero4();
        }
    };
    auto load_v = [&](int p, int pos) {
        for (int i = 0; i < 4; ++i) {
            const float* v = (const float*)a.vc + (base_of(p >= 0 ? p : 0, pos) + 4 * g4 + i) * D + c16 * NB;
            for (int b = 0; b < NB; b += (NB < 4 ? NB : 4)) {
                if (p < 0) {
                    for (int j = 0; j < (NB < 4 ? NB : 4); ++j) vf[i][b + j] = 0.f;
                } else if (NB >= 4) {
                    const f32x4 x = *(const f32x4*)(v + b);
                    for (int j = 0; j < 4; ++j) vf[i][b + j] = x[j];
                } else {
                    for (int j = 0; j < NB; ++j) vf[i][b + j] = v[b + j];
                }
            }
        }
    };

    int pos = keys.begin + wave * 16;
    int page = -1, page_next = -1;
    if (pos < keys.end) {
        page = page_at(a, table, pos, keys.end);
        page_next = page_at(a, table, pos + 64, keys.end);
        load_k(page, pos);
        load_v(page, pos);
    }
    for (; pos < keys.end; pos += 64) {
        const int next = pos + 64;
        const int page_2 = page_at(a, table, next + 64, keys.end);
        f32x4 st[RT];
        for (int rt = 0; rt < RT; ++rt) {
            f32x4 x = zero4();
            for (int k = 0; k < KD / 4; ++k)
                for (int j = 0; j < 4; ++j) x = mma4(kf[k][j], qf[rt][k][j], x);
            st[rt] = x;
        }
        if (next < keys.end) load_k(page_next, next);
        float pe[RT][4];
        for (int rt = 0; rt < RT; ++rt) {
            float x[4];
            for (int i = 0; i < 4; ++i) {
                x[i] = st[rt][i] * scale;
                const int key = pos + 4 * g4 + i;
                if (key > limit[rt] || key >= keys.end || page < 0) x[i] = -INFINITY;
            }
            const float mx = max_quarters(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
            if (__any(mx > m[rt])) {
                const float mn = fmaxf(m[rt], mx);
                const float c = mn == -INFINITY ? 1.f : exp2_f(m[rt] - mn);
                m[rt] = mn;
                l[rt] *= c;
                for (int b = 0; b < NB; ++b) acc[rt][b] *= c;
            }
            const float mu = m[rt] == -INFINITY ? 0.f : m[rt];
            for (int i = 0; i < 4; ++i) {
                pe[rt][i] = exp2_f(x[i] - mu);
                l[rt] += pe[rt][i];
            }
        }
        bool odd = false;
        if (pos + 16 > keys.all) {
            for (int i = 0; i < 4; ++i) {
                const bool out = pos + 4 * g4 + i >= keys.end;
                for (int b = 0; b < NB; ++b) {
                    if (out) vf[i][b] = 0.f;         // no row sees it: it holds anything
                    odd |= !finite_bits(vf[i][b]);
                }
            }
            odd = __any(odd);
        }
        if (odd) {
            // positions that only some rows see, with a value that is not
            // finite: it must not meet the weight 0 of the other rows
            for (int i = 0; i < 4; ++i)
                for (int b = 0; b < NB; ++b)
                    if (!finite_bits(vf[i][b])) vf[i][b] = 0.f;
            for (int key = 0; key < 16; ++key) {
                if (page < 0 || pos + key >= keys.end) continue;
                const float* v = (const float*)a.vc + (base_of(page, pos) + key) * D;
                for (int rt = 0; rt < RT; ++rt) {
                    float w = 0.f;
                    for (int i = 0; i < 4; ++i)
                        if (i == (key & 3)) w = pe[rt][i];
                    w = __shfl(w, c16 + 16 * (key / 4));
                    const bool sees = pos + key <= limit[rt];
                    for (int b = 0; b < NB; ++b)
                        for (int i = 0; i < 4; ++i) {
                            const float x = v[(4 * g4 + i) * NB + b];
                            if (sees && !finite_bits(x)) acc[rt][b][i] += w * x;
                        }
                }
            }
        }
        for (int i = 0; i < 4; ++i)
            for (int b = 0; b < NB; ++b)
                for (int rt = 0; rt < RT; ++rt) acc[rt][b] = mma4(vf[i][b], pe[rt][i], acc[rt][b]);
        if (next < keys.end) load_v(page_next, next);
        page = page_next;
        page_next = page_2;
    }

    for (int rt = 0; rt < RT; ++rt) {
        const float sum = sum_quarters(l[rt]);
        __syncthreads();
        if (g4 == 0) {
            join_ml[(wave * 16 + c16) * 2] = m[rt];
            join_ml[(wave * 16 + c16) * 2 + 1] = sum;
        }
        for (int b = 0; b < NB; ++b)
            for (int i = 0; i < 4; ++i)
                join[(wave * 16 + c16) * (D + 4) + (4 * g4 + i) * NB + b] = acc[rt][b][i];
        __syncthreads();
        join_waves<float, D>(a, s, it, G, rt * 16, join_ml, join);
    }
}

// Prompts: tiles of 128 rows, 32 per wave, against 64 keys at a time that all
// waves share in LDS. What bounds it is the matrix cores, 6 D flops per row
// and key (4 D of the definition and 2 D of the weights' second terms), the LDS
// reads that feed them (each wave reads all 64 keys and values for its 32
// rows), and the exponentials.
//
// As above S^T = K Q^T and O^T += V^T P^T, with the 32x32x16 product: the
// scores of row l % 32 stay in lanes l and l + 32 and are the second operand
// of the next product as they are. K and V of the next 64 keys are fetched while
// these are computed on, two buffers each and one barrier a step.
//
// 8192 tokens over 24576 positions, 32 heads over 8 of 128: 5.2 to 5.4 ms
// from card to card, 5.8 TFLOP of products at 1.07 to 1.11 PFLOP/s with the matrix
// cores busy 55% of the cycles at 1.9 GHz: the clock falls as they fill, and a
// library product of 8192^3 reaches 1.20 PFLOP/s there. (Before the second terms: scores of the next 64 keys made while
// the exponentials of these run, K fetched two steps ahead: the same at width
// 128, 8% longer at 64, where the registers leave a workgroup less.)
//
// K and V go from memory to LDS directly, 16 bytes a lane in the lanes' order;
// which 16 bytes of the row each lane fetches is permuted (k_piece, v_piece4):
// with 8 lanes' worth of banks in mind instead of 16, half of the LDS cycles
// were conflicts.
template <int D> struct TileLds {
    __align__(128) bf16 k[2 * 64 * D], v[2 * 64 * D];
    int gap_wave[4][4], odd_wave[4];
    AttnItem item;
};
template <int D>
__device__ __forceinline__ void tile_bf16(const AttnArgs& a, const AttnSplit& s, int block,
                                          TileLds<D>& lds) {
    constexpr int KS = D / 16, NB = D / 32, CH = D / 8, LD = 16 * CH / 64;
    constexpr int kTile = 64 * D;                    // of K or V
    bf16 *const kbuf = lds.k, *const vbuf = lds.v;
    int (&gap_wave)[4][4] = lds.gap_wave;
    int (&odd_wave)[4] = lds.odd_wave;
    const AttnItem it = attn_item(a, s, block, lds.item);
    if (!it.found) return;
    const int G = a.Hq / a.Hkv, wave = wave_id(), lane = threadIdx.x & 63;
    const int c32 = lane & 31, half = lane >> 5;
    const Keys keys = part_keys(a, s, it, G);
    const_int* table = table_row(a, it.req);
    const float scale = a.scale * kLog2e;
    const int row_mask = (1 << a.page_shift) - 1;

    bf16x8 qf[KS];
    const RowAt at = row_at(a, it, G, it.tile * s.R + wave * 32 + c32);
    const int limit = at.in ? (int)min((long)it.kept + at.t, (long)kKeepAll) : -1;
    for (int k = 0; k < KS; ++k) {
        bf16x8 z = {};
        if (at.in) z = *(const bf16x8*)((const bf16*)a.q + at.q * D + 8 * half + 16 * k);
        qf[k] = z;
    }
    float m = -INFINITY, l = 0.f;
    f32x16 acc[NB];
    for (int b = 0; b < NB; ++b) acc[b] = f32x16{};

    // where the lane's 16 bytes of the wave's 16 keys come from
    uint32_t koff[LD], voff[LD];
    for (int i = 0; i < LD; ++i) {
        const int x = i * 64 + lane, r = x / CH, c = x % CH;
        koff[i] = 2 * (r * D + 8 * k_piece<D>(r, c));
        voff[i] = 2 * (r * D + 8 * v_piece4<D>(r, c));
    }
    auto page_of = [&](int pos) { return page_at(a, table, pos + 16 * wave, keys.end); };
    // This wave's 16 keys (values) of the step at pos, from page p; zeros where
    // there is none.
    auto fetch = [&](const void* cache, bf16* buf, const uint32_t* off, int pos, int p) {
        bf16* to = buf + 16 * wave * D;
        if (p >= 0) {
            const long row = (((long)p * a.Hkv + it.h) << a.page_shift) + ((pos + 16 * wave) & row_mask);
            const bf16* from = (const bf16*)cache + row * D;
            const uint32_t lds = uniform((int)(uint32_t)(uintptr_t)(lds_void*)to);
            for (int i = 0; i < LD; ++i) load_to_lds(lds + i * 1024, off[i], from);
        } else {
            for (int i = 0; i < LD; ++i) *(bf16x8*)(to + i * 512 + 8 * lane) = bf16x8{};
        }
    };
    // Scores of the step whose keys are in kt.
    auto scores = [&](const bf16* kt, f32x16 (&st)[2]) {
        bf16x8 kf[2][KS];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < KS; ++k)
                kf[u][k] = *(const bf16x8*)(kt + (32 * u + c32) * D + 8 * k_piece<D>(c32, 2 * k + half));
        st[0] = f32x16{};
        st[1] = f32x16{};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < KS; ++k) st[u] = mma_big(kf[u][k], qf[k], st[u]);
        // the first half's reads, then a read behind every product: left to
        // itself the compiler reads into one register and waits each time
        __builtin_amdgcn_sched_group_barrier(0x100, KS, 0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, KS, 0);
    };
    auto missing_of = [&](int step) {
        int missing = 0;
        for (int w = 0; w < 4; ++w) missing |= uniform(gap_wave[step & 3][w]) << w;
        return missing;
    };
    // Masks the scores of the step at pos and moves the reference m. It may
    // stay behind the maximum by up to 8 in the log2 domain: weights up to 2^8
    // lose nothing, and the rows are rescaled a few times instead of with
    // every new maximum.
    auto settle = [&](f32x16 (&st)[2], int pos, int missing) {
        if (pos + 64 > keys.all || missing) {
            for (int u = 0; u < 2; ++u)
                for (int i = 0; i < 16; ++i) {
                    const int y = 32 * u + 8 * (i / 4) + 4 * half + i % 4;
                    if (pos + y > limit || pos + y >= keys.end || (missing >> (y / 16) & 1))
                        st[u][i] = -INFINITY;
                }
        }
        float mx = -INFINITY;
        for (int u = 0; u < 2; ++u)
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, st[u][i]);
        mx = max_halves(mx) * scale;
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx);
            const float c = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            l *= c;
            for (int b = 0; b < NB; ++b) acc[b] *= c;
        }
    };

    // One step: the 64 keys at pos, the step-th of the part.
    int page_next = 0;                   // of this wave's 16 keys of the next step
    auto advance = [&](int pos, int step) {
        const int buf = step & 1;
        const bf16* kt = kbuf + buf * kTile;
        f32x16 st[2];
        bf16* vt = vbuf + buf * kTile;
        // pages missing in the next step's keys: known to the wave that fetches
        // them. Three sets of flags are in use before the barrier: the next step's
        // are set, this step's are, and a slower wave still reads the last one's.
        // (Four, for the mask.)
        if (lane == 0) gap_wave[(step + 1) & 3][wave] = page_next < 0;
        __builtin_amdgcn_s_waitcnt(0x0f70);          // vmcnt(0): this wave's part has landed
        __syncthreads();
        const bool more = pos + 64 < keys.end;
        if (more) fetch(a.kc, kbuf + (buf ^ 1) * kTile, koff, pos + 64, page_next);
        if (more) fetch(a.vc, vbuf + (buf ^ 1) * kTile, voff, pos + 64, page_next);
        page_next = page_of(pos + 128);
        bool odd = false;
        const int missing = missing_of(step);
        if (pos + 64 > keys.all || missing) {
            // Keys that no row of the tile sees hold anything: they count 0. Of the
            // others a value that is not finite must not meet the weight 0 of the
            // rows that do not see it: it counts 0 here and is added below.
            for (int i = 0; i < LD; ++i) {
                bf16* v = vt + (16 * wave) * D + i * 512 + 8 * lane;
                bf16x8 x = *(const bf16x8*)v;
                if (pos + 16 * wave + (i * 64 + lane) / CH >= keys.end) x = bf16x8{};
                *(bf16x8*)v = only_finite(x, odd);
            }
            odd = __any(odd);
            if (lane == 0) odd_wave[wave] = odd;
            __syncthreads();                         // the values are cleared, the flags set
            odd = uniform(odd_wave[0] | odd_wave[1] | odd_wave[2] | odd_wave[3]);
            __syncthreads();                         // and read
        }
        scores(kt, st);
        settle(st, pos, missing);
        const float mu = m == -INFINITY ? 0.f : m;
        bf16x8 pf[4], pr[4];
        float sum = 0.f;
        for (int u = 0; u < 2; ++u)
            for (int i = 0; i < 16; ++i) {
                const float p = exp2_f(__builtin_fmaf(st[u][i], scale, -mu));
                sum += p;
                st[u][i] = p;
            }
        l += sum;
        for (int ks = 0; ks < 4; ++ks) {
            float p[8];
            for (int j = 0; j < 8; ++j) p[j] = st[ks / 2][8 * (ks % 2) + j];
            two_terms(p, pf[ks], pr[ks]);
        }
        for (int ks = 0; ks < 4; ++ks)
            for (int b = 0; b < NB; ++b) {
                s16x4 x[2];
                for (int j = 0; j < 2; ++j) {
                    const int key = 16 * ks + 8 * j + 4 * half + (lane & 15) / 4;
                    const int dv = 32 * b + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    const int c = v_piece4<D>(key, dv / 8);
                    x[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_s16x4*)(vt + key * D + 8 * c + dv % 8));
                }
                const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
                acc[b] = mma_big(va, pf[ks], acc[b]);
                acc[b] = mma_big(va, pr[ks], acc[b]);
            }
        if (odd) {
            // the values left out above, for the rows that see them
            for (int y = 0; y < 64; ++y) {
                const int p = page_at(a, table, pos + (y & 48), keys.end);
                if (p < 0 || pos + y >= keys.end) continue;
                const bf16* gv = (const bf16*)a.vc +
                    ((((long)p * a.Hkv + it.h) << a.page_shift) + ((pos + y) & row_mask)) * D;
                float w = 0.f;
                for (int u = 0; u < 2; ++u)
                    for (int i = 0; i < 16; ++i)
                        if (y / 32 == u && (y & 31) / 8 == i / 4 && y % 4 == i % 4) w = st[u][i];
                w = __shfl(w, c32 + 32 * ((y / 4) & 1));
                const bool sees = pos + y <= limit;
                for (int b = 0; b < NB; ++b)
                    for (int i = 0; i < 16; ++i) {
                        const float v = (float)gv[32 * b + 8 * (i / 4) + 4 * half + i % 4];
                        if (sees && !finite_bits(v)) acc[b][i] += w * v;
                    }
            }
        }
    };

    if (keys.begin < keys.end) {
        const int p0 = page_of(keys.begin);
        page_next = page_of(keys.begin + 64);
        if (lane == 0) gap_wave[0][wave] = p0 < 0;
        fetch(a.kc, kbuf, koff, keys.begin, p0);
        fetch(a.vc, vbuf, voff, keys.begin, p0);
        for (int pos = keys.begin, step = 0; pos < keys.end; pos += 64, ++step) advance(pos, step);
    }

    // (a score past fp32, whose difference to the infinite maximum gave the weight 0)
    const float sum = m == INFINITY ? NAN : l + __shfl_xor(l, 32);
    const int row = wave * 32 + c32;
    if (it.parts > 1) {
        const long slot = (long)it.slot + ((long)it.part * it.tiles + it.tile) * a.Hkv + it.h;
        if ((unsigned long)slot >= (unsigned long)s.slots) return;   // (a guard)
        float* x = s.acc + (slot * s.R + row) * D;
        // (a row without a key in this part has l = 0, and its values are not read)
        for (int b = 0; sum != 0.f && b < NB; ++b)
            for (int i = 0; i < 16; i += 4)
                *(f32x4*)(x + 32 * b + 2 * i + 4 * half) =
                    f32x4{acc[b][i], acc[b][i + 1], acc[b][i + 2], acc[b][i + 3]};
        if (half == 0) {
            s.ml[(slot * s.R + row) * 2] = m;
            s.ml[(slot * s.R + row) * 2 + 1] = sum;
        }
        return;
    }
    if (!at.in) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    bf16* o = (bf16*)a.o + at.q * D;
    for (int b = 0; b < NB; ++b)
        for (int i = 0; i < 16; i += 4) {
            bf16x4 x;
            for (int j = 0; j < 4; ++j) x[j] = (bf16)(acc[b][i + j] * inv);
            *(bf16x4*)(o + 32 * b + 2 * i + 4 * half) = x;
        }
    if (a.lse && half == 0) a.lse[at.q] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
}

template <int D>
__global__ __launch_bounds__(kAttnThreads, D == 64 ? 3 : 2) void attn_tile_bf16(AttnArgs a, AttnSplit s,
                                                                               unsigned first) {
    __shared__ TileLds<D> lds;
    tile_bf16<D>(a, s, (int)(first + blockIdx.x), lds);
}

// Long and short requests of a call at once: the first n0 workgroups are the
// tiles', the others the streams'. Two launches took the longer of the two
// plus the other (25 + 13 us in a ragged batch).
template <int D>
__global__ __launch_bounds__(kAttnThreads, D == 64 ? 3 : 2) void attn_both_bf16(AttnArgs a, AttnSplit s0,
                                                                  AttnSplit s1, unsigned n0,
                                                                  unsigned first) {
    union Lds {
        TileLds<D> tile;
        StreamLds<D> stream;
        __device__ Lds() {}
    };
    __shared__ Lds lds;
    const unsigned block = first + blockIdx.x;
    if (block < n0) tile_bf16<D>(a, s0, (int)block, lds.tile);
    else stream_bf16<D, 2>(a, s1, (int)(block - n0), lds.stream);
}

// Kernels of a call, from sizes alone. Rows of a request are at most
// max_new * G (T * G when the largest is not known).
//
// Up to kStreamRows rows a request is the stream kernels'; of a call with
// larger ones (bf16, d of 64 and 128) those are the tile kernel's. At 64: 64
// requests of 64 rows over 4000 positions 229 -> 247 us, 32 of 48 rows of width
// 64 over 2000 77 -> 66. Parts: see AttnSplit. Streams, at most 2048 and at least
// 1024 of them (4 long contexts: 480 us with 2048, 425 with 1024), 256 short ones
// (with 512: 31 + 13 us in a ragged fp32 batch instead of 28 + 5). Tiles, 512,
// what the card holds at once (256: 512 tokens over 3000 positions 66 instead of
// 55 us, 1024: 65). Units of 128 keys (64: 528 tokens of 4 heads 15 instead of 12 us,
// 512: 19).
constexpr int kStreamRows = 32;

struct Plan {
    int n;                 // launches
    bool tiles;            // the first is the tile kernel
    int RT;                // row groups of the stream kernel
    Launch l[2];
    size_t bytes;          // workspace
};
Plan plan_of(int T, int B, int Hq, int Hkv, int d, int max_new, bool bf16_io) {
    const long G = Hq / Hkv, most = (max_new > 0 && max_new < T ? max_new : T) * G;
    Plan p{};
    p.tiles = bf16_io && d >= 64 && most > kStreamRows;
    p.RT = most <= 16 ? 1 : 2;
    if (p.tiles) {
        p.l[p.n] = launch_of(T, B, G, Hkv, kTileRows, 9, 9, 9, INT32_MAX);
        p.l[p.n].split.min_rows = kStreamRows + 1;
        ++p.n;
    }
    if (!p.tiles || B > 1) {
        p.l[p.n] = launch_of(T, B, G, Hkv, 16 * p.RT, 11, 10, 8, p.tiles ? kStreamRows : INT32_MAX);
        ++p.n;
    }
    // a single request is the tile kernel's whatever its length
    if (p.tiles && B == 1) p.l[0].split.min_rows = 1;
    for (int i = 0; i < p.n; ++i) {
        p.bytes += (size_t)p.l[i].split.slots * p.l[i].split.R * (d + 2) * sizeof(float);
        if (B > kBlock) p.bytes += AttnTable::ints(B) * sizeof(int);
    }
    return p;
}

// Keys of a call (times tiles that read them) above which the stream kernel for
// bf16, d of 64 and 128 reads K and V non-temporally, where a request is one
// tile and so reads them once: 512 MB of them, twice what the last-level cache
// could still hold from an earlier call, and only of a pool that is larger
// itself (requests may share pages). Decode batch over 5.8 GB 1017 -> 971 us.
// 201 MB that repeated calls find in the cache, of a pool of 17 GB, read so: 42
// -> 51 us (16 requests of one token over 3000 positions, 32 heads over 8 of 128).
long far_keys(const AttnArgs& a) {
    constexpr size_t kFarBytes = (size_t)512 << 20;
    const size_t key = (size_t)a.Hkv * a.d * 4;      // bytes of K and V
    if (!a.bf16_io || a.d < 64 || ((size_t)a.pool << a.page_shift) * key <= kFarBytes) return LONG_MAX;
    return (long)(kFarBytes / key);
}

template <int D>
void launch_stream(const AttnArgs& a, const Plan& p, const Launch& l, hipStream_t st) {
    const auto run = [&](auto kernel) {
        in_grids((unsigned)l.items, [&](unsigned grid, unsigned first) {
            kernel<<<grid, kAttnThreads, 0, st>>>(a, l.split, first);
        });
    };
    if (a.bf16_io) {
        if (p.RT == 1) run(attn_stream_bf16<D, 1>);
        else run(attn_stream_bf16<D, 2>);
    } else {
        if (p.RT == 1) run(attn_stream_f32<D, 1>);
        else run(attn_stream_f32<D, 2>);
    }
}

template <int D>
hipError_t launch(const AttnArgs& a, const Plan& p, hipStream_t st) {
    const Launch &l0 = p.l[0], &l1 = p.l[p.n - 1];
    if (a.B > kBlock) attn_list<<<(unsigned)p.n, 64 * kListWaves, 0, st>>>(a, l0.split, l1.split);
    if constexpr (D >= 64) {
        const unsigned n0 = (unsigned)l0.items;
        if (p.n == 2) {
            in_grids(n0 + (unsigned)l1.items, [&](unsigned grid, unsigned first) {
                attn_both_bf16<D><<<grid, kAttnThreads, 0, st>>>(a, l0.split, l1.split, n0, first);
            });
        } else if (p.tiles) {
            in_grids(n0, [&](unsigned grid, unsigned first) {
                attn_tile_bf16<D><<<grid, kAttnThreads, 0, st>>>(a, l0.split, first);
            });
        }
    }
    if (!p.tiles) launch_stream<D>(a, p, l0, st);
    const int n0 = (int)l0.joins, n = n0 + (p.n > 1 ? (int)l1.joins : 0);
    if (a.bf16_io) attn_join<bf16, D><<<(unsigned)n, kAttnThreads, 0, st>>>(a, l0.split, l1.split, n0);
    else attn_join<float, D><<<(unsigned)n, kAttnThreads, 0, st>>>(a, l0.split, l1.split, n0);
    return hipGetLastError();
}

}  // namespace

size_t attn_paged_ws(int T, int B, int Hq, int Hkv, int d, int max_new, bool bf16_io) {
    return plan_of(T, B, Hq, Hkv, d, max_new, bf16_io).bytes;
}

hipError_t launch_attn_paged(const AttnArgs& a, void* ws, hipStream_t st) {
    Plan p = plan_of(a.T, a.B, a.Hq, a.Hkv, a.d, a.max_new, a.bf16_io);
    float* at = (float*)ws;
    for (int i = 0; i < p.n; ++i) {
        AttnSplit& s = p.l[i].split;
        s.far = far_keys(a);
        s.ml = at;
        s.acc = s.ml + (size_t)s.slots * s.R * 2;
        at = s.acc + (size_t)s.slots * s.R * a.d;
        if (a.B > kBlock) {
            s.table = (int*)at;
            at += AttnTable::ints(a.B);
        }
    }
    switch (a.d) {
        case 16: return launch<16>(a, p, st);
        case 32: return launch<32>(a, p, st);
        case 64: return launch<64>(a, p, st);
        default: return launch<128>(a, p, st);
    }
}

}  // namespace kda
