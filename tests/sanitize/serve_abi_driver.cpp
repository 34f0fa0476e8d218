// Host sanitizer run of the serving C ABI's validation (kda_serve_api.cpp built
// with AddressSanitizer and UndefinedBehaviorSanitizer for the host by
// tests/test_sanitizers_serve.py). Every call below is rejected, or is a no-op
// or a size query, before any HIP call, so it runs without a GPU. Exit status 0
// = every status as expected (the sanitizers abort on their own findings).
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "kda_serve.h"

static int fails = 0;
static void expect(const char* what, int got, int want) {
    if (got != want) {
        std::printf("FAIL %s: status %d, expected %d\n", what, got, want);
        ++fails;
    }
}

// Made-up, well spaced device addresses, never dereferenced.
template <typename T = void>
static T* P(int i, size_t off = 0) {
    return reinterpret_cast<T*>((uintptr_t(1) << 40) + (uintptr_t(i) << 36) + off);
}
static const int OK = KDA_OK, INV = KDA_ERR_INVALID_ARG, UNS = KDA_ERR_UNSUPPORTED, WS = KDA_ERR_WORKSPACE;

struct Plan {
    int *kept = P<int>(0), *fresh = P<int>(1), *in = P<int>(2), *out = P<int>(3), *table = P<int>(4),
        *ring = P<int>(5), *ring_in = P<int>(6), *ring_out = P<int>(7), *cu = P<int>(8),
        *slots = P<int>(9), *status = P<int>(10);
    int B = 8, width = 16, page = 64, pool = 100, n_slots = 50;
    void* ws = P(11);
    size_t bytes = 1 << 20;
    int run() const {
        return kda_page_plan(kept, fresh, in, out, table, ring, ring_in, ring_out, cu, slots, status,
                             B, width, page, pool, n_slots, ws, bytes, nullptr);
    }
};
struct Append {
    void *k = P(0), *v = P(1);
    int* slots = P<int>(2);
    void *kc = P(3), *vc = P(4);
    int T = 8, H = 2, d = 64, page = 64, pool = 10;
    kda_dtype dtype = KDA_BF16;
    int run() const {
        return kda_cache_append(k, v, slots, kc, vc, T, H, d, page, pool, dtype, nullptr);
    }
};
struct Attn {
    void *q = P(0), *kc = P(1), *vc = P(2);
    int *table = P<int>(3), *kept = P<int>(4), *cu = P<int>(5);
    void* o = P(6);
    float* lse = P<float>(7);
    int T = 40, B = 4, Hq = 8, Hkv = 2, d = 64, page = 64, pool = 100, width = 16, max_new = 0;
    float scale = 0.f;
    kda_dtype dtype = KDA_BF16;
    void* ws = P(8);
    size_t bytes = size_t(1) << 34;
    int run() const {
        return kda_attn_paged(q, kc, vc, table, kept, cu, o, lse, T, B, Hq, Hkv, d, page, pool, width,
                              max_new, scale, dtype, ws, bytes, nullptr);
    }
};
struct Verify {
    void *p = P(0), *q = P(1);
    int* x = P<int>(2);
    float* u = P<float>(3);
    int *n = P<int>(4), *commit = P<int>(5), *tokens = P<int>(6);
    int B = 4, T = 7, V = 10001;
    kda_dtype dtype = KDA_F32;
    void* ws = P(7);
    size_t bytes = size_t(1) << 34;
    int run() const {
        return kda_draft_verify(p, q, x, u, n, commit, tokens, B, T, V, dtype, ws, bytes,
                                nullptr);
    }
};
template <typename C, typename F>
static void with(const char* what, int want, F change) {
    C c;
    change(c);
    expect(what, c.run(), want);
}

int main() {
    // size queries: huge and negative sizes must not overflow
    for (int B : {INT_MIN, -1, 0, 1, 1 << 30, (1 << 30) + 1, INT_MAX})
        for (int T : {INT_MIN, -1, 0, 1, 1 << 30, INT_MAX})
            for (int H : {-1, 0, 1, 7, INT_MAX})
                for (int n : {INT_MIN, 0, 1, INT_MAX})
                    std::printf("%zu %zu %zu\n", kda_page_plan_workspace_size(B),
                                kda_attn_paged_workspace_size(T, B, H, H > 0 ? H : 1, 128, n, KDA_BF16),
                                kda_draft_verify_workspace_size(B, T, n));

    with<Plan>("plan huge", INV, [](Plan& c) { c.B = c.width = INT_MAX; });
    with<Plan>("plan requests", INV, [](Plan& c) { c.B = (1 << 30) + 1; c.bytes = SIZE_MAX; });
    with<Plan>("plan negative", INV, [](Plan& c) { c.n_slots = INT_MIN; });
    with<Plan>("plan pool", INV, [](Plan& c) { c.pool = INT_MAX; });
    with<Plan>("plan page", UNS, [](Plan& c) { c.page = INT_MIN; });
    with<Plan>("plan misaligned", INV, [](Plan& c) { c.cu = P<int>(8, 2); });
    with<Plan>("plan null", INV, [](Plan& c) { c.ring_in = nullptr; });
    with<Plan>("plan overlap", INV, [](Plan& c) { c.out = P<int>(2, 4); });
    with<Plan>("plan outputs", INV, [](Plan& c) { c.status = P<int>(9, 8); });
    with<Plan>("plan no ws", WS, [](Plan& c) { c.ws = nullptr; });
    with<Plan>("plan small ws", WS, [](Plan& c) { c.bytes = kda_page_plan_workspace_size(8) - 1; });

    with<Append>("append huge", INV, [](Append& c) { c.T = c.H = INT_MAX; });
    with<Append>("append heads", INV, [](Append& c) { c.H = INT_MAX; c.T = c.pool = 1; });
    with<Append>("append negative", INV, [](Append& c) { c.pool = INT_MIN; });
    with<Append>("append pool", INV, [](Append& c) { c.pool = INT_MAX; });
    with<Append>("append d", UNS, [](Append& c) { c.d = INT_MIN; });
    with<Append>("append misaligned", INV, [](Append& c) { c.vc = P(4, 8); });
    with<Append>("append overlap", INV, [](Append& c) { c.kc = P(0, 1024); });
    with<Append>("append nothing", OK, [](Append& c) { c = Append{}; c.T = 0; c.k = nullptr; });

    with<Attn>("attn huge", INV, [](Attn& c) { c.T = c.Hq = c.Hkv = INT_MAX; });
    with<Attn>("attn rows", INV, [](Attn& c) { c.T = INT_MAX; });
    with<Attn>("attn requests", INV, [](Attn& c) { c.B = INT_MAX; c.width = 1; c.bytes = SIZE_MAX; });
    with<Attn>("attn table", INV, [](Attn& c) { c.width = INT_MAX; });
    with<Attn>("attn negative", INV, [](Attn& c) { c.max_new = INT_MIN; });
    with<Attn>("attn heads", INV, [](Attn& c) { c.Hkv = 3; });
    with<Attn>("attn no KV head", INV, [](Attn& c) { c.Hkv = 0; });
    with<Attn>("attn d", UNS, [](Attn& c) { c.d = 256; });
    for (float s : {-1.f, 2.5e38f, INFINITY, -INFINITY, NAN})
        with<Attn>("attn scale", INV, [&](Attn& c) { c.scale = s; });
    with<Attn>("attn null", INV, [](Attn& c) { c.kc = nullptr; });
    with<Attn>("attn misaligned", INV, [](Attn& c) { c.q = P(0, 4); });
    with<Attn>("attn in place", INV, [](Attn& c) { c.o = c.q; });
    with<Attn>("attn lse", INV, [](Attn& c) { c.lse = P<float>(6, 16); });
    with<Attn>("attn no ws", WS, [](Attn& c) { c.ws = nullptr; });
    with<Attn>("attn ws misaligned", INV, [](Attn& c) { c.ws = P(8, 4); });
    with<Attn>("attn nothing", OK, [](Attn& c) { c.B = 0; c.q = nullptr; });

    with<Verify>("verify huge", INV, [](Verify& c) { c.B = c.T = c.V = INT_MAX; });
    with<Verify>("verify tokens", INV, [](Verify& c) { c.T = INT_MAX; c.B = c.V = 1; });
    with<Verify>("verify negative", INV, [](Verify& c) { c.T = INT_MIN; });
    with<Verify>("verify no vocabulary", INV, [](Verify& c) { c.V = 0; });
    with<Verify>("verify null", INV, [](Verify& c) { c.u = nullptr; });
    with<Verify>("verify misaligned", INV, [](Verify& c) { c.p = P(0, 8); });
    with<Verify>("verify overlap", INV, [](Verify& c) { c.tokens = c.x; });
    with<Verify>("verify no ws", WS, [](Verify& c) { c.ws = nullptr; });
    with<Verify>("verify small ws", WS,
                 [](Verify& c) { c.bytes = kda_draft_verify_workspace_size(4, 7, 10001) - 1; });
    with<Verify>("verify nothing", OK, [](Verify& c) { c.B = 0; c.p = nullptr; });

    std::printf("%d failures\n", fails);
    return fails != 0;
}
