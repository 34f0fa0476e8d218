// C ABI of the serving step: argument validation on the host, then dispatch
// to the HIP kernels on the caller's stream. Nothing here allocates,
// synchronises or keeps state between calls.
#include "kda_serve.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_serve_launch.h"

namespace {

constexpr size_t kMaxBytes = SIZE_MAX >> 3;
// query rows, positions, requests of a plan or an attention: 32-bit indices with room
constexpr size_t kMaxRows = (size_t)1 << 30;

constexpr float kMaxScale = 0x1p127f;          // scores are held times log2 e

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool page_ok(int p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
bool pool_ok(int pool, int page) { return (long)pool * page <= INT32_MAX; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int log2i(int x) { return __builtin_ctz((unsigned)x); }

// Product of sizes (each >= 0), or kMaxBytes + 1 when it would be larger.
template <typename... Ts>
size_t product(Ts... xs) {
    size_t acc = 1;
    bool zero = false, over = false;
    for (const size_t x : {(size_t)xs...}) {
        if (x == 0) zero = true;
        else if (acc > kMaxBytes / x) over = true;
        else acc *= x;
    }
    return zero ? 0 : (over ? kMaxBytes + 1 : acc);
}

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
    Range(const void* p, size_t bytes) : lo((uintptr_t)p), hi(p ? (uintptr_t)p + bytes : lo) {}
};
bool overlap(const Range& a, const Range& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// Whether an output overlaps an input or an output before it.
template <int NI, int NO>
bool clash(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Range& r : in)
            if (overlap(out[i], r)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

kda_status done(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace

extern "C" {

size_t kda_page_plan_workspace_size(int B) {
    return B < 0 || (size_t)B > kMaxRows ? 0 : kda::page_plan_ws(B);
}

kda_status kda_page_plan(const int* kept_len, const int* n_new, const int* n_pages_in,
                         int* n_pages_out, int* block_table, int* free_ring,
                         const int* ring_in, int* ring_out, int* cu_new, int* slot_map,
                         int* status, int B, int max_pages, int page_size, int n_pool,
                         int n_slots, void* ws, size_t ws_bytes, void* stream) {
    if (B < 0 || max_pages < 0 || n_pool < 0 || n_slots < 0) return KDA_ERR_INVALID_ARG;
    if (!page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size) || (size_t)B > kMaxRows) return KDA_ERR_INVALID_ARG;
    const size_t table = product(B, max_pages, 4);
    if (table > kMaxBytes) return KDA_ERR_INVALID_ARG;
    if (B && (!kept_len || !n_new || !n_pages_in || !n_pages_out)) return KDA_ERR_INVALID_ARG;
    if (!ring_in || !ring_out || !cu_new || !status || (table && !block_table) || (n_pool && !free_ring) || (n_slots && !slot_map))
        return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {kept_len, n_new, n_pages_in, n_pages_out, block_table, free_ring,
                          ring_in, ring_out, cu_new, slot_map, status, ws};
    for (const void* p : ptrs)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_page_plan_workspace_size(B);
    if (!ws || ws_bytes < need) return KDA_ERR_WORKSPACE;
    const size_t n = (size_t)B * 4;
    const Range in[] = {{kept_len, n}, {n_new, n},
                        // the counts may be updated in place
                        {n_pages_in == n_pages_out ? nullptr : n_pages_in, n},
                        {ring_in == ring_out ? nullptr : ring_in, 8}};
    const Range out[] = {{n_pages_out, n}, {block_table, table}, {free_ring, (size_t)n_pool * 4},
                         {ring_out, 8}, {cu_new, n + 4}, {slot_map, (size_t)n_slots * 4},
                         {status, 4}, {ws, need}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::PlanArgs a{};
    a.kept = kept_len; a.fresh = n_new; a.pages_in = n_pages_in; a.pages_out = n_pages_out;
    a.table = block_table; a.ring = free_ring; a.ring_in = ring_in; a.ring_out = ring_out;
    a.cu = cu_new; a.slots = slot_map; a.status = status;
    a.B = B; a.width = max_pages; a.page_shift = log2i(page_size); a.pool = n_pool;
    a.n_slots = n_slots;
    return done(kda::launch_page_plan(a, ws, (hipStream_t)stream));
}

kda_status kda_cache_append(const void* k, const void* v, const int* slot_map,
                            void* k_cache, void* v_cache, int T, int Hkv, int d,
                            int page_size, int n_pool, kda_dtype dtype, void* stream) {
    if (T < 0 || Hkv < 0 || n_pool < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!dim_ok(d) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || Hkv == 0 || n_pool == 0) return KDA_OK;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4;
    const size_t rows = product(T, Hkv, d, elt), cache = product(n_pool, Hkv, page_size, d, elt);
    // one token's rows are indexed in 32 bits
    if (rows > kMaxBytes || cache > kMaxBytes || product(Hkv, d, elt) > ((size_t)1 << 30))
        return KDA_ERR_INVALID_ARG;
    if (!k || !v || !slot_map || !k_cache || !v_cache) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {k, v, k_cache, v_cache};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(slot_map, 4)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{k, rows}, {v, rows}, {slot_map, (size_t)T * 4}};
    const Range out[] = {{k_cache, cache}, {v_cache, cache}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    return done(kda::launch_cache_append(k, v, slot_map, k_cache, v_cache, T, Hkv,
                                         (int)(d * elt), log2i(page_size), n_pool,
                                         (hipStream_t)stream));
}

size_t kda_attn_paged_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_new,
                                     kda_dtype dtype) {
    if (T <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || !dim_ok(d) || max_new < 0) return 0;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
    if (product(T, Hq, d, 4) > kMaxBytes || product(T, Hq) > kMaxRows || (size_t)B > kMaxRows)
        return 0;
    return kda::attn_paged_ws(T, B, Hq, Hkv, d, max_new, dtype == KDA_BF16);
}

kda_status kda_attn_paged(const void* q, const void* k_cache, const void* v_cache,
                          const int* block_table, const int* kept_len, const int* cu_new,
                          void* o, float* lse, int T, int B, int Hq, int Hkv, int d,
                          int page_size, int n_pool, int max_pages, int max_new, float scale,
                          kda_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
    if (T < 0 || B < 0 || Hq < 0 || Hkv < 0 || n_pool < 0 || max_pages < 0 || max_new < 0)
        return KDA_ERR_INVALID_ARG;
    if (!(scale >= 0.f) || scale > kMaxScale) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (!dim_ok(d) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!pool_ok(n_pool, page_size)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0 || Hq == 0) return KDA_OK;
    if (Hkv == 0 || Hq % Hkv) return KDA_ERR_INVALID_ARG;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4;
    const size_t rows = product(T, Hq, d, elt), cache = product(n_pool, Hkv, page_size, d, elt);
    const size_t table = product(B, max_pages, 4);
    if (rows > kMaxBytes || cache > kMaxBytes || table > kMaxBytes ||
        product(T, Hq) > kMaxRows || product(max_pages, page_size) > kMaxRows || (size_t)B > kMaxRows)
        return KDA_ERR_INVALID_ARG;
    if (!q || !o || !kept_len || !cu_new || (table && !block_table) ||
        (cache && (!k_cache || !v_cache)))
        return KDA_ERR_INVALID_ARG;
    const void* p16[] = {q, k_cache, v_cache, o};
    for (const void* p : p16)
        if (p && !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {block_table, kept_len, cu_new, lse};
    for (const void* p : p4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attn_paged_workspace_size(T, B, Hq, Hkv, d, max_new, dtype);
    if (need && (!ws || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if (need && !aligned(ws, 16)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{q, rows}, {k_cache, cache}, {v_cache, cache}, {block_table, table},
                        {kept_len, (size_t)B * 4}, {cu_new, (size_t)B * 4 + 4}};
    const Range out[] = {{o, rows}, {lse, product(T, Hq, 4)}, {ws, need}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::AttnArgs a{};
    a.q = q; a.kc = k_cache; a.vc = v_cache; a.table = block_table; a.kept = kept_len;
    a.cu = cu_new; a.o = o; a.lse = lse;
    a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.page_shift = log2i(page_size);
    a.pool = n_pool; a.width = max_pages; a.max_new = max_new;
    a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)d);
    a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_attn_paged(a, ws, (hipStream_t)stream));
}

size_t kda_draft_verify_workspace_size(int B, int T, int V) {
    return B <= 0 || T < 0 || V <= 0 ? 0 : kda::draft_verify_ws(B, V);
}

kda_status kda_draft_verify(const void* target_probs, const void* draft_probs,
                            const int* draft_tokens, const float* u, const int* n_draft,
                            int* n_commit, int* tokens, int B, int T, int V, kda_dtype dtype,
                            void* ws, size_t ws_bytes, void* stream) {
    if (B < 0 || T < 0 || V < 0) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED;
    if (B == 0) return KDA_OK;
    if (V == 0) return KDA_ERR_INVALID_ARG;
    const size_t elt = dtype == KDA_BF16 ? 2 : 4;
    const size_t np = product(B, (size_t)T + 1, V, elt), nq = product(B, T, V, elt);
    const size_t nx = product(B, T, 4), nt = product(B, (size_t)T + 1, 4);
    if (np > kMaxBytes || T == INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (!target_probs || !u || !n_commit || !tokens || (T && !draft_tokens))
        return KDA_ERR_INVALID_ARG;
    if (!aligned(target_probs, 16) || !aligned(draft_probs, 16)) return KDA_ERR_INVALID_ARG;
    const void* p4[] = {draft_tokens, u, n_draft, n_commit, tokens};
    for (const void* p : p4)
        if (p && !aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda_draft_verify_workspace_size(B, T, V);
    if (need && (!ws || ws_bytes < need)) return KDA_ERR_WORKSPACE;
    if (need && !aligned(ws, 16)) return KDA_ERR_INVALID_ARG;
    const Range in[] = {{target_probs, np}, {draft_probs, nq}, {draft_tokens, nx}, {u, nt},
                        {n_draft, (size_t)B * 4}};
    const Range out[] = {{n_commit, (size_t)B * 4}, {tokens, nt}, {ws, need}};
    if (clash(in, out)) return KDA_ERR_INVALID_ARG;
    kda::VerifyArgs a{};
    a.p = target_probs; a.q = draft_probs; a.x = draft_tokens; a.u = u; a.n_draft = n_draft;
    a.n_commit = n_commit; a.tokens = tokens; a.B = B; a.T = T; a.V = V;
    a.bf16_io = dtype == KDA_BF16;
    return done(kda::launch_draft_verify(a, ws, (hipStream_t)stream));
}

}  // extern "C"
