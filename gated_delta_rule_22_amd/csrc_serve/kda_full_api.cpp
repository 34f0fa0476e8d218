// C ABI of the full-attention layers: argument validation on the host, then
// dispatch to the HIP kernels on the caller's stream. Nothing here allocates,
// synchronises or keeps state between calls.
#include "kda_full.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_full_launch.h"
#include "kda_serve_checks.h"

namespace {

bool rope_ok(const kda_rope* r, int most) {
    return r->freqs && aligned(r->freqs, 8) && r->rot >= 16 && r->rot <= most && r->rot % 16 == 0 &&
           isfinite(r->factor);
}
kda::RopeArgs rope_args(const kda_rope* r) {
    return r ? kda::RopeArgs{r->freqs, r->rot, r->interleaved != 0, r->factor}
             : kda::RopeArgs{nullptr, 0, false, 1.f};
}
bool latent_ok(int dc, int dr) { return dr == kda::kPe && (dc == 128 || dc == 256 || dc == 512); }

}  // namespace

extern "C" {

kda_status kda_rope_append(const void* q, const void* k, const void* v, const int* slot_map,
                           const int* kept_len, const int* cu_new, void* q_out, void* k_cache,
                           void* v_cache, int T, int B, int Hq, int Hkv, int d, int page_size,
                           int n_pool, const kda_rope* rope, kda_dtype dtype, void* stream) {
    if (T < 0 || B < 0 || Hq < 0 || Hkv < 0 || n_pool < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!dim_ok(d) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size)) return KDA_ERR_INVALID_ARG;
    if (!rope || !rope_ok(rope, d)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || (Hq == 0 && Hkv == 0)) return KDA_OK;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4;
    const size_t nq = product(T, Hq, d, elt), nk = product(T, Hkv, d, elt);
    const size_t cache = product(n_pool, Hkv, page_size, d, elt);
    if (nq > kMaxBytes || nk > kMaxBytes || cache > kMaxBytes || (size_t)B > kMaxRows ||
        product(T, (size_t)Hq + 2 * (size_t)Hkv) > kMaxRows)
        return KDA_ERR_INVALID_ARG;
    if (!kept_len || !cu_new || (nq && (!q || !q_out)) || (nk && (!k || !v || !slot_map)) ||
        (cache && (!k_cache || !v_cache)))
        return KDA_ERR_INVALID_ARG;
    const void* p16[] = {q, k, v, q_out, k_cache, v_cache};
    for (const void* p : p16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {slot_map, kept_len, cu_new};
    for (const void* p : p4)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{q == q_out ? nullptr : q, nq}, {k, nk}, {v, nk},
                        {nk ? slot_map : nullptr, (size_t)T * 4}, {kept_len, (size_t)B * 4},
                        {cu_new, (size_t)B * 4 + 4}, {rope->freqs, (size_t)rope->rot * 4}};
    const Range out[] = {{q_out, nq}, {k_cache, cache}, {v_cache, cache}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::RopeAppendArgs a{};
    a.q = q; a.k = k; a.v = v; a.slots = slot_map; a.kept = kept_len; a.cu = cu_new;
    a.q_out = q_out; a.kc = k_cache; a.vc = v_cache;
    a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.page_shift = log2i(page_size);
    a.pool = n_pool; a.rope = rope_args(rope); a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_rope_append(a, (hipStream_t)stream));
}

kda_status kda_latent_append(const void* kv, const float* w, const int* slot_map,
                             const int* kept_len, const int* cu_new, void* cache, void* kv_out,
                             const void* q, void* q_out, int T, int B, int Hq, int dq, int dq_out,
                             int dc, int dr, int page_size, int n_pool, int normalise, float eps,
                             const kda_rope* rope, kda_dtype dtype, void* stream) {
    if (T < 0 || B < 0 || Hq < 0 || n_pool < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!latent_ok(dc, dr) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size)) return KDA_ERR_INVALID_ARG;
    if (Hq && (dq < dr || dq_out < dr || dq % 8 || dq_out % 8)) return KDA_ERR_INVALID_ARG;
    if (normalise ? !(eps >= 0.f) || !isfinite(eps) : w != nullptr) return KDA_ERR_INVALID_ARG;
    if (rope && (!rope_ok(rope, dr) || rope->rot != dr)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return KDA_OK;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4, width = (size_t)dc + dr;
    const size_t rows = product(T, width, elt), pages = product(n_pool, page_size, width, elt);
    const size_t nq = product(T, Hq, dq > 0 ? dq : 0, elt);
    const size_t no = product(T, Hq, dq_out > 0 ? dq_out : 0, elt);
    if (rows > kMaxBytes || pages > kMaxBytes || nq > kMaxBytes || no > kMaxBytes ||
        (size_t)B > kMaxRows || product(T, (size_t)Hq + 1) > kMaxRows)
        return KDA_ERR_INVALID_ARG;
    if (!kv || !slot_map || !kept_len || !cu_new || (pages && !cache) || (Hq && (!q || !q_out)))
        return KDA_ERR_INVALID_ARG;
    const void* p16[] = {kv, w, cache, kv_out, q, q_out};
    for (const void* p : p16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {slot_map, kept_len, cu_new};
    for (const void* p : p4)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    if (Hq && q == q_out && dq != dq_out) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{kv == kv_out ? nullptr : kv, rows}, {w, (size_t)dc * 4},
                        {slot_map, (size_t)T * 4}, {kept_len, (size_t)B * 4},
                        {cu_new, (size_t)B * 4 + 4},
                        {rope ? rope->freqs : nullptr, (size_t)dr * 4},
                        {q == q_out ? nullptr : q, nq}};
    const Range out[] = {{cache, pages}, {kv_out, rows}, {q_out, no}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::LatentAppendArgs a{};
    a.kv = kv; a.w = w; a.slots = slot_map; a.kept = kept_len; a.cu = cu_new; a.cache = cache;
    a.kv_out = kv_out; a.q = q; a.q_out = q_out;
    a.T = T; a.B = B; a.Hq = Hq; a.dq = dq; a.dq_out = dq_out; a.dc = dc;
    a.page_shift = log2i(page_size); a.pool = n_pool; a.normalise = normalise != 0; a.eps = eps;
    a.rope = rope_args(rope); a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_latent_append(a, (hipStream_t)stream));
}

size_t kda_attn_latent_workspace_size(int T, int B, int Hq, int dc, int dr, int max_new,
                                      kda_dtype dtype) {
    if (T <= 0 || B <= 0 || Hq <= 0 || !latent_ok(dc, dr) || max_new < 0) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    if (product(T, Hq) > kMaxRows || (size_t)B > kMaxRows) return 0;
    return kda::attn_latent_ws(T, B, Hq, dc, max_new, dtype == KDA_BF16);
}

kda_status kda_attn_latent(const void* q, const void* cache, const int* block_table,
                           const int* kept_len, const int* cu_new, void* o, float* lse, int T,
                           int B, int Hq, int dc, int dr, int page_size, int n_pool, int max_pages,
                           int max_new, float scale, kda_dtype dtype, void* ws, size_t ws_bytes,
                           void* stream) {
    if (T < 0 || B < 0 || Hq < 0 || n_pool < 0 || max_pages < 0 || max_new < 0)
        return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > kMaxScale) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!latent_ok(dc, dr) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || Hq == 0) return KDA_OK;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4, width = (size_t)dc + dr;
    const size_t rows = product(T, Hq, width, elt), pages = product(n_pool, page_size, width, elt);
    const size_t outs = product(T, Hq, dc, elt), table = product(B, max_pages, 4);
    if (rows > kMaxBytes || pages > kMaxBytes || table > kMaxBytes || product(T, Hq) > kMaxRows ||
        product(max_pages, page_size) > kMaxRows || (size_t)B > kMaxRows)
        return KDA_ERR_INVALID_ARG;
    if (!q || !o || !kept_len || !cu_new || (table && !block_table) || (pages && !cache))
        return KDA_ERR_INVALID_ARG;
    const void* p16[] = {q, cache, o};
    for (const void* p : p16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {block_table, kept_len, cu_new, lse};
    for (const void* p : p4)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attn_latent_workspace_size(T, B, Hq, dc, dr, max_new, dtype);
    if (need && (!ws || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if (need && !aligned(ws, 16)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{q, rows}, {cache, pages}, {block_table, table},
                        {kept_len, (size_t)B * 4}, {cu_new, (size_t)B * 4 + 4}};
    const Range out[] = {{o, outs}, {lse, product(T, Hq, 4)}, {ws, need}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a{};
    a.q = q; a.kc = cache; a.table = block_table; a.kept = kept_len; a.cu = cu_new;
    a.o = o; a.lse = lse;
    a.T = T; a.B = B; a.Hq = Hq; a.Hkv = 1; a.d = dc; a.page_shift = log2i(page_size);
    a.pool = n_pool; a.width = max_pages; a.max_new = max_new; a.scale = scale;
    a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_attn_latent(a, ws, (hipStream_t)stream));
}

// Channels of one key of kda_attn_expanded, or between two shared parts.
static constexpr int kMaxKeyRow = 1 << 26;

size_t kda_attn_expanded_workspace_size(int T, int B, int H, int dn, int dr, int dv, int max_q,
                                        kda_dtype dtype) {
    if (T <= 0 || B <= 0 || H <= 0 || max_q < 0) return 0;
    if (dr != kda::kPe || dn != dv || (dv != 64 && dv != 128)) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    if (product(T, H) > kMaxRows || (size_t)B > kMaxRows) return 0;
    return kda::attn_expanded_ws(T, B, H, dv, max_q, dtype == KDA_BF16);
}

kda_status kda_attn_expanded(const void* q, const void* kv, const void* k_pe, const int* cu_q,
                             const int* cu_k, void* o, float* lse, int T, int N, int B, int H,
                             int dn, int dr, int dv, int pe_stride, int max_q, float scale,
                             kda_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
    if (T < 0 || N < 0 || B < 0 || H < 0 || max_q < 0) return KDA_ERR_INVALID_ARG;
    if (!(scale >= 0.f) || scale > kMaxScale) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (dr != kda::kPe || dn != dv || (dv != 64 && dv != 128)) return KDA_ERR_UNSUPPORTED;
    if (pe_stride < dr || pe_stride % 8) return KDA_ERR_INVALID_ARG;
    // (the kernels' offsets, in bytes over the 16 keys or fewer that a wave fetches, have 32 bits)
    if (pe_stride > kMaxKeyRow || product(H, (size_t)dn + dv) > (size_t)kMaxKeyRow) return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || H == 0) return KDA_OK;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4;
    const size_t rows = product(T, H, (size_t)dn + dr, elt), outs = product(T, H, dv, elt);
    const size_t keys = product(N, H, (size_t)dn + dv, elt);
    const size_t stride = product(N, pe_stride, elt);
    if (rows > kMaxBytes || keys > kMaxBytes || stride > kMaxBytes || product(T, H) > kMaxRows ||
        (size_t)N > kMaxRows || (size_t)B > kMaxRows)
        return KDA_ERR_INVALID_ARG;
    // the last row of k_pe ends after dr channels
    const size_t pe = N ? stride - ((size_t)pe_stride - dr) * elt : 0;
    if (!q || !o || !cu_q || !cu_k || (N && (!kv || !k_pe))) return KDA_ERR_INVALID_ARG;
    const void* p16[] = {q, kv, k_pe, o};
    for (const void* p : p16)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {cu_q, cu_k, lse};
    for (const void* p : p4)
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attn_expanded_workspace_size(T, B, H, dn, dr, dv, max_q, dtype);
    if (need && (!ws || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if (need && !aligned(ws, 16)) return KDA_ERR_INVALID_ARG;
    const size_t nb = (size_t)B * 4 + 4;
    const Range in[] = {{q, rows}, {kv, keys}, {k_pe, pe}, {cu_q, nb}, {cu_k, nb}};
    const Range out[] = {{o, outs}, {lse, product(T, H, 4)}, {ws, need}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::ExpandedArgs a{};
    a.q = q; a.kc = kv; a.vc = k_pe; a.cu = cu_q; a.cu_k = cu_k; a.o = o; a.lse = lse;
    a.T = T; a.N = N; a.B = B; a.Hq = H; a.Hkv = H; a.d = dv; a.page_shift = 0;
    a.width = 1 << 30; a.pool = 0; a.max_new = max_q; a.pe_stride = pe_stride;
    a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)(dn + dr));
    a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_attn_expanded(a, ws, (hipStream_t)stream));
}

}  // extern "C"
