// Causal attention of packed prompts over keys and values that were expanded from
// latents: every head has keys of its own, whose last 64 channels are shared.
// Online softmax and work split as in kda_attn_paged.hip, with a head's queries
// as the rows and the requests' keys as they are packed.
//
// bf16: 32 rows a wave, against 64 keys at a time that all waves share in LDS, two
// buffers, one barrier a step; eight waves a workgroup, or four and three workgroups a
// compute unit for heads of 64 (ragged prompts 65 -> 59 us together with shorter parts).
// What bounds it is the matrix cores: per row and key 2 (dn + 64) + 4 dv flops, of which
// 2 dv are the weights' second terms (2^-16 of a weight is lost, not 2^-9).
//   8192 tokens over 16384 before them, 32 heads of 128: 3.9 to 4.1 ms from card to card,
//     1.18 to 1.24 PFLOP/s with the second terms, which is what a library product reaches;
//   21 prompts of 1 to 1526 tokens, 12 heads of 64: 44 + 12 us, starting and joining parts.
// Half of the waves a product late, or the last values' products between the next weights,
// leave fewer registers for reads ahead of the products: 4.2 to 4.9 ms.
#include "kda_attn_rows.h"
#include "kda_full_launch.h"

#include <limits.h>

namespace kda {
namespace {

// A wave's share of the loads of a step: KEYS rows of 16 P bytes, key by key as they
// lie in LDS.
template <int KEYS, int P>
struct KeyLoads {
    static constexpr int LD = KEYS * P / 64;
    const char* base;            // the wave's first key of the step ahead
    long stride;                 // bytes from one key to the next, at most 2^28
    uint32_t off[LD];            // the lane's bytes

    static __device__ __forceinline__ int key(int i) { return (i * 64 + (threadIdx.x & 63)) / P; }
    // `place`: the 16 bytes of a key's row that lie in its piece c
    template <typename F>
    __device__ __forceinline__ void init(const char* from, long bytes, F place) {
        base = from;
        stride = bytes;
        for (int i = 0; i < LD; ++i)
            off[i] = (uint32_t)(key(i) * stride) + 16 * place(key(i), (int)(threadIdx.x & 63) % P);
    }
    // of a step of which `have` of the wave's keys exist (others read the last one that
    // does, which may be another wave's), to LDS at `to`
    __device__ __forceinline__ void issue(uint32_t to, int have, int step) {
        if (have >= KEYS) {
#pragma unroll
            for (int i = 0; i < LD; ++i) load_to_lds(to + i * 1024, off[i], base);
        } else {
            const char* from = base + min(have - 1, 0) * stride;
            const int last = max(have - 1, 0);
#pragma unroll
            for (int i = 0; i < LD; ++i)
                load_to_lds(to + i * 1024, off[i] - (uint32_t)((key(i) - min(key(i), last)) * stride), from);
        }
        base += stride * step;
    }
};

template <int DV> struct ExpandedShape {
    static constexpr int DK = DV + kPe;
    static constexpr int kWaves = DV == 64 ? 4 : 8, kRows = 32 * kWaves, KT = 64;
    static constexpr int kPerSimd = DV == 64 ? 3 : 2;    // waves, by their registers
    static constexpr int kKeys = KT / kWaves;        // that a wave fetches
};

template <int DV> struct ExpandedLds {
    typedef ExpandedShape<DV> S;
    __align__(128) bf16 k[2 * S::KT * DV], pe[2 * S::KT * kPe], v[2 * S::KT * DV];
    int odd_wave[2][S::kWaves];
    AttnItem item;
};

// LDS order of a key's pieces of D channels: reads of one piece of 16 keys cover the banks.
template <int D> __device__ __forceinline__ int expanded_piece(int key, int c) {
    return D == 128 ? c ^ (key & 15) : c ^ (key >> 1 & 7);
}

template <int DV>
__global__ __launch_bounds__(64 * ExpandedShape<DV>::kWaves, ExpandedShape<DV>::kPerSimd) void attn_expanded_bf16(
    ExpandedArgs a, AttnSplit s, unsigned first_block) {
    typedef ExpandedShape<DV> S;
    constexpr int DK = S::DK, KT = S::KT, KS = DK / 16, NB = DV / 32, kKeys = S::kKeys;
    constexpr int LV = kKeys * DV / 512;
    __shared__ ExpandedLds<DV> lds;
    const AttnItem it = attn_item(a, s, (int)(first_block + blockIdx.x), lds.item);
    if (!it.found) return;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c32 = lane & 31, half = lane >> 5;
    const Keys keys = part_keys(a, s, it, 1);
    const float scale = a.scale * kLog2e;
    const long k0 = uniform(a.row_of(it.req));
    const long kv_row = (long)a.Hq * 2 * DV;         // dn = dv
    const bf16* kv = (const bf16*)a.kc + k0 * kv_row + (long)it.h * 2 * DV;
    const bf16* pe = (const bf16*)a.vc + k0 * a.pe_stride;

    bf16x8 qf[KS];
    const RowAt at = row_at(a, it, 1, it.tile * s.R + wave * 32 + c32);
    // last of the part's positions that the lane's row sees
    const int limit = at.in ? (int)min((long)it.kept + at.t, (long)keys.end - 1) : -1;
    // last position that a row of this wave sees
    const int first_row = it.tile * s.R + wave * 32;
    const int wave_limit = first_row < it.n ? uniform((int)min((long)it.kept + first_row + 31, (long)kKeepAll)) : -1;
    for (int k = 0; k < KS; ++k) {
        bf16x8 z = {};
        if (at.in) z = *(const bf16x8*)((const bf16*)a.q + at.q * DK + 8 * half + 16 * k);
        qf[k] = z;
    }
    float m = -INFINITY, l = 0.f;
    f32x16 acc[NB];
    for (int b = 0; b < NB; ++b) acc[b] = f32x16{};

    const int k_first = wave * kKeys;                // of the keys that this wave fetches
    const char* kv_at = (const char*)(kv + (long)(keys.begin + k_first) * kv_row);
    KeyLoads<kKeys, DV / 8> kl, vl;
    KeyLoads<kKeys, kPe / 8> pl;
    kl.init(kv_at, 2 * kv_row, [&](int r, int c) { return expanded_piece<DV>(k_first + r, c); });
    pl.init((const char*)(pe + (long)(keys.begin + k_first) * a.pe_stride), 2 * a.pe_stride,
            [&](int r, int c) { return expanded_piece<kPe>(k_first + r, c); });
    vl.init(kv_at + 2 * DV, 2 * kv_row, [&](int r, int c) { return v_piece4<DV>(k_first + r, c); });
    const auto address = [&](bf16* p) { return (uint32_t)uniform((int)(uint32_t)(uintptr_t)(lds_void*)p); };
    const auto fetch = [&](int buf, int pos) {
        const int have = keys.end - (pos + k_first);
        kl.issue(address(lds.k + (buf * KT + k_first) * DV), have, KT);
        pl.issue(address(lds.pe + (buf * KT + k_first) * kPe), have, KT);
        vl.issue(address(lds.v + (buf * KT + k_first) * DV), have, KT);
    };

    if (keys.begin < keys.end) fetch(0, keys.begin);
    int buf = 0;
    for (int pos = keys.begin; pos < keys.end; pos += KT, buf ^= 1) {
        __builtin_amdgcn_s_waitcnt(0x0f70);          // vmcnt(0): this wave's part has landed
        // Positions that only some rows see: a value there that is not finite must not
        // meet the weight 0 of the others in a product. The wave that fetched it clears it,
        // and it is added below for the rows that see it.
        const bool some = pos + KT > keys.all;
        if (some) {
            bool odd = false;
            for (int i = 0; i < LV; ++i) {
                bf16* v = lds.v + (buf * KT + k_first) * DV + i * 512 + 8 * lane;
                *(bf16x8*)v = only_finite(*(const bf16x8*)v, odd);
            }
            odd = __any(odd);
            if (lane == 0) lds.odd_wave[buf][wave] = odd;
        }
        __syncthreads();
        if (pos + KT < keys.end) fetch(buf ^ 1, pos + KT);
        const bf16 *kt = lds.k + buf * KT * DV, *pt = lds.pe + buf * KT * kPe, *vt = lds.v + buf * KT * DV;
        if (pos > wave_limit) continue;              // no row of this wave sees these keys
        f32x16 st[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            st[u] = f32x16{};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const bf16x8 kf = k < DV / 16
                    ? *(const bf16x8*)(kt + (32 * u + c32) * DV + 8 * expanded_piece<DV>(c32, 2 * k + half))
                    : *(const bf16x8*)(pt + (32 * u + c32) * kPe + 8 * expanded_piece<kPe>(c32, 2 * k - DV / 8 + half));
                st[u] = mma_big(kf, qf[k], st[u]);
            }
        }
        if (pos + KT - 1 > limit) {
            const int seen = limit - pos - 4 * half;
            for (int u = 0; u < 2; ++u)
                for (int i = 0; i < 16; ++i)
                    if (32 * u + 8 * (i / 4) + i % 4 > seen) st[u][i] = -INFINITY;
        }
        float mx = -INFINITY;
        for (int u = 0; u < 2; ++u)
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, st[u][i]);
        mx *= scale;
        // the reference may stay behind the maximum by up to 8 in the log2 domain
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, max_halves(mx));
            const float c = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            l *= c;
            for (int b = 0; b < NB; ++b) acc[b] *= c;
        }
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
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                s16x4 x[2];
                for (int j = 0; j < 2; ++j) {
                    const int key = 16 * ks + 8 * j + 4 * half + (lane & 15) / 4;
                    const int dv = 32 * b + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    const int c = v_piece4<DV>(key, dv / 8);
                    x[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_s16x4*)(vt + key * DV + 8 * c + dv % 8));
                }
                const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
                acc[b] = mma_big(va, pf[ks], acc[b]);
                acc[b] = mma_big(va, pr[ks], acc[b]);
            }
        bool odd = false;
        for (int w = 0; some && w < S::kWaves; ++w) odd |= lds.odd_wave[buf][w] != 0;
        if (uniform((int)odd)) {
            // the values left out above, for the rows that see them
            for (int y = 0; y < KT && pos + y < keys.end; ++y) {
                const bf16* gv = kv + (long)(pos + y) * kv_row + DV;
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
    }

    // (a score past fp32, whose difference to the infinite maximum gave the weight 0)
    const float sum = m == INFINITY ? NAN : l + __shfl_xor(l, 32);
    const int row = wave * 32 + c32;
    if (it.parts > 1) {
        const long slot = (long)it.slot + ((long)it.part * it.tiles + it.tile) * a.Hkv + it.h;
        if ((unsigned long)slot >= (unsigned long)s.slots) return;   // (a guard)
        float* x = s.acc + (slot * s.R + row) * DV;
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
    bf16* o = (bf16*)a.o + at.q * DV;
    for (int b = 0; b < NB; ++b)
        for (int i = 0; i < 16; i += 4) {
            bf16x4 x;
            for (int j = 0; j < 4; ++j) x[j] = (bf16)(acc[b][i + j] * inv);
            *(bf16x4*)(o + 32 * b + 2 * i + 4 * half) = x;
        }
    if (a.lse && half == 0) a.lse[at.q] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
}

// fp32: 16 rows a wave, 64 a workgroup, 16 keys at a time. The contraction over a
// key takes the channels g DK / 4 .. in lane quarter g, so that reads are 16 bytes;
// the 16 columns of a product's block of values are 4 apart.
template <int DV> struct ExpandedLdsF {
    static constexpr int DK = DV + kPe, KT = 16;
    __align__(128) float k[2 * KT * DV], pe[2 * KT * kPe], v[2 * KT * DV];
    int odd_wave[2][4];
    AttnItem item;
};
constexpr int kRowsF = 64;

template <int DV>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_expanded_f32(ExpandedArgs a, AttnSplit s,
                                                                     unsigned first_block) {
    constexpr int DK = DV + kPe, KT = 16, KQ = DK / 16, CT = DV / 16, kKeys = KT / 4;
    constexpr int LV = kKeys * DV / 256;
    __shared__ ExpandedLdsF<DV> lds;
    const AttnItem it = attn_item(a, s, (int)(first_block + blockIdx.x), lds.item);
    if (!it.found) return;
    const int wave = wave_id(), lane = threadIdx.x & 63;
    const int c16 = lane & 15, g4 = lane >> 4;
    const Keys keys = part_keys(a, s, it, 1);
    const float scale = a.scale * kLog2e;
    const long k0 = uniform(a.row_of(it.req));
    const long kv_row = (long)a.Hq * 2 * DV;
    const float* kv = (const float*)a.kc + k0 * kv_row + (long)it.h * 2 * DV;
    const float* pe = (const float*)a.vc + k0 * a.pe_stride;
    auto piece = [](int key, int c) { return c ^ (key & 15); };

    f32x4 qf[KQ];
    const RowAt at = row_at(a, it, 1, it.tile * s.R + wave * 16 + c16);
    const int limit = at.in ? (int)min((long)it.kept + at.t, (long)keys.end - 1) : -1;
    const int wave_limit = uniform((int)min((long)it.kept + it.tile * s.R + wave * 16 + 15, (long)kKeepAll));
    for (int k = 0; k < KQ; ++k) {
        f32x4 z = zero4();
        if (at.in) z = *(const f32x4*)((const float*)a.q + at.q * DK + 4 * (g4 * KQ + k));
        qf[k] = z;
    }
    float m = -INFINITY, l = 0.f;
    f32x4 acc[CT];
    for (int b = 0; b < CT; ++b) acc[b] = zero4();

    const int k_first = wave * kKeys;
    const char* kv_at = (const char*)(kv + (long)(keys.begin + k_first) * kv_row);
    KeyLoads<kKeys, DV / 4> kl, vl;
    KeyLoads<kKeys, kPe / 4> pl;
    kl.init(kv_at, 4 * kv_row, [&](int r, int c) { return piece(k_first + r, c); });
    pl.init((const char*)(pe + (long)(keys.begin + k_first) * a.pe_stride), 4 * a.pe_stride,
            [&](int r, int c) { return piece(k_first + r, c); });
    vl.init(kv_at + 4 * DV, 4 * kv_row, [](int, int c) { return c; });
    const auto address = [&](float* p) { return (uint32_t)uniform((int)(uint32_t)(uintptr_t)(lds_void*)p); };
    const auto fetch = [&](int buf, int pos) {
        const int have = keys.end - (pos + k_first);
        kl.issue(address(lds.k + (buf * KT + k_first) * DV), have, KT);
        pl.issue(address(lds.pe + (buf * KT + k_first) * kPe), have, KT);
        vl.issue(address(lds.v + (buf * KT + k_first) * DV), have, KT);
    };

    if (keys.begin < keys.end) fetch(0, keys.begin);
    int buf = 0;
    for (int pos = keys.begin; pos < keys.end; pos += KT, buf ^= 1) {
        __builtin_amdgcn_s_waitcnt(0x0f70);
        const bool some = pos + KT > keys.all;
        if (some) {
            bool odd = false;
            for (int i = 0; i < LV; ++i) {
                f32x4* v = (f32x4*)(lds.v + (buf * KT + k_first) * DV + i * 256 + 4 * lane);
                f32x4 x = *v;
                for (int j = 0; j < 4; ++j)
                    if (!finite_bits(x[j])) {
                        x[j] = 0.f;
                        odd = true;
                    }
                *v = x;
            }
            odd = __any(odd);
            if (lane == 0) lds.odd_wave[buf][wave] = odd;
        }
        __syncthreads();
        if (pos + KT < keys.end) fetch(buf ^ 1, pos + KT);
        const float *kt = lds.k + buf * KT * DV, *pt = lds.pe + buf * KT * kPe, *vt = lds.v + buf * KT * DV;
        if (pos > wave_limit) continue;
        f32x4 st = zero4();
#pragma unroll
        for (int i = 0; i < KQ; ++i) {
            // (the last lane quarters' channels are partly of the shared part)
            const int c = g4 * KQ + i;
            const float* k = c < DV / 4 ? kt + c16 * DV + 4 * piece(c16, c) : pt + c16 * kPe + 4 * piece(c16, c - DV / 4);
            const f32x4 kf = *(const f32x4*)k;
            for (int j = 0; j < 4; ++j) st = mma4(kf[j], qf[i][j], st);
        }
        for (int i = 0; i < 4; ++i) {
            st[i] *= scale;
            if (pos + 4 * g4 + i > limit) st[i] = -INFINITY;
        }
        const float mx = max_quarters(fmaxf(fmaxf(st[0], st[1]), fmaxf(st[2], st[3])));
        if (__any(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float c = mn == -INFINITY ? 1.f : exp2_f(m - mn);
            m = mn;
            l *= c;
            for (int b = 0; b < CT; ++b) acc[b] *= c;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        for (int i = 0; i < 4; ++i) {
            st[i] = exp2_f(st[i] - mu);
            l += st[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < CT / 4; ++g) {
                const f32x4 x = *(const f32x4*)(vt + (4 * g4 + i) * DV + 64 * g + 4 * c16);
                for (int j = 0; j < 4; ++j) acc[4 * g + j] = mma4(x[j], st[i], acc[4 * g + j]);
            }
        bool odd = false;
        for (int w = 0; some && w < 4; ++w) odd |= lds.odd_wave[buf][w] != 0;
        if (uniform((int)odd)) {
            for (int y = 0; y < KT && pos + y < keys.end; ++y) {
                const float* gv = kv + (long)(pos + y) * kv_row + DV;
                float w = 0.f;
                for (int i = 0; i < 4; ++i)
                    if (i == (y & 3)) w = st[i];
                w = __shfl(w, c16 + 16 * (y / 4));
                const bool sees = pos + y <= limit;
                for (int b = 0; b < CT; ++b)
                    for (int i = 0; i < 4; ++i) {
                        const float v = gv[64 * (b / 4) + 4 * (4 * g4 + i) + b % 4];
                        if (sees && !finite_bits(v)) acc[b][i] += w * v;
                    }
            }
        }
    }

    const float sum = sum_quarters(l);
    const int row = wave * 16 + c16;
    const bool cut = it.parts > 1;
    const long slot = (long)it.slot + ((long)it.part * it.tiles + it.tile) * a.Hkv + it.h;
    if (cut ? (unsigned long)slot >= (unsigned long)s.slots : !at.in) return;   // (the first: a guard)
    const float inv = cut ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
    float* to = cut ? s.acc + (slot * s.R + row) * DV : (float*)a.o + at.q * DV;
    for (int g = 0; (!cut || sum != 0.f) && g < CT / 4; ++g)
        for (int i = 0; i < 4; ++i) {
            f32x4 x;
            for (int j = 0; j < 4; ++j) x[j] = acc[4 * g + j][i] * inv;
            *(f32x4*)(to + 64 * g + 4 * (4 * g4 + i)) = x;
        }
    if (g4 != 0) return;
    if (cut) {
        s.ml[(slot * s.R + row) * 2] = m;
        s.ml[(slot * s.R + row) * 2 + 1] = sum;
    } else if (a.lse) {
        a.lse[at.q] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
    }
}

struct ExpandedPlan {
    Launch l;
    size_t bytes;
};
ExpandedPlan plan_of(int T, int B, int H, int dv, int max_q, bool bf16_io) {
    ExpandedPlan p{};
    // Heads of 64 have room for 768 workgroups on the card, and shorter parts of ragged
    // prompts pay: 64 -> 58 us with up to 2^11 parts, and 2^10 rather than parts shorter
    // than kLongPart (2^11 of them 63, 2^12 69). Others have room for 256.
    const bool small = bf16_io && dv == 64;
    const int rows = !bf16_io ? kRowsF : small ? ExpandedShape<64>::kRows : ExpandedShape<128>::kRows;
    const int most = small ? 11 : 9, few = small ? 10 : 9;
    p.l = launch_of(T, B, 1, H, rows, most, most, few, INT32_MAX);
    p.bytes = (size_t)p.l.split.slots * p.l.split.R * (dv + 2) * sizeof(float);
    if (B > kBlock) p.bytes += AttnTable::ints(B) * sizeof(int);
    return p;
}

template <int DV>
hipError_t launch(const ExpandedArgs& a, const ExpandedPlan& p, hipStream_t st) {
    const AttnSplit& s = p.l.split;
    if (a.B > kBlock) attn_list<<<1, 64 * kListWaves, 0, st>>>(a, s, s);
    in_grids((unsigned)p.l.items, [&](unsigned grid, unsigned first) {
        if (a.bf16_io) attn_expanded_bf16<DV><<<grid, 64 * ExpandedShape<DV>::kWaves, 0, st>>>(a, s, first);
        else attn_expanded_f32<DV><<<grid, kAttnThreads, 0, st>>>(a, s, first);
    });
    const int n = (int)p.l.joins;
    if (a.bf16_io) attn_join<bf16, DV><<<(unsigned)n, kAttnThreads, 0, st>>>(a, s, s, n);
    else attn_join<float, DV><<<(unsigned)n, kAttnThreads, 0, st>>>(a, s, s, n);
    return hipGetLastError();
}

}  // namespace

size_t attn_expanded_ws(int T, int B, int H, int dv, int max_q, bool bf16_io) {
    return plan_of(T, B, H, dv, max_q, bf16_io).bytes;
}

hipError_t launch_attn_expanded(const ExpandedArgs& a, void* ws, hipStream_t st) {
    ExpandedPlan p = plan_of(a.T, a.B, a.Hq, a.d, a.max_new, a.bf16_io);
    AttnSplit& s = p.l.split;
    s.far = LONG_MAX;
    s.ml = (float*)ws;
    s.acc = s.ml + (size_t)s.slots * s.R * 2;
    if (a.B > kBlock) s.table = (int*)(s.acc + (size_t)s.slots * s.R * a.d);
    return a.d == 64 ? launch<64>(a, p, st) : launch<128>(a, p, st);
}

}  // namespace kda
