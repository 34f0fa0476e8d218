// Host sanitizer run of the validation of the full-attention layers' C ABI
// (kda_full_api.cpp built with AddressSanitizer and UndefinedBehaviorSanitizer for
// the host by tests/test_sanitizers_full.py). Every call below is rejected, or is a
// no-op or a size query, before any HIP call, so it runs without a GPU. Exit status 0
// = every status as expected (the sanitizers abort on their own findings).
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "kda_full.h"

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
static const int MANY[] = {INT_MIN, -1, INT_MAX};

struct Rope {
    const void *q = P(0), *k = P(1), *v = P(2);
    const int *slots = P<int>(3), *kept = P<int>(4), *cu = P<int>(5);
    void *qo = P(6), *kc = P(7), *vc = P(8);
    int T = 8, B = 4, Hq = 4, Hkv = 2, d = 64, page = 64, pool = 10;
    kda_rope rope = {P<double>(20), 64, 0, 1.f};
    kda_dtype dtype = KDA_BF16;
    int run() const {
        return kda_rope_append(q, k, v, slots, kept, cu, qo, kc, vc, T, B, Hq, Hkv, d, page, pool, &rope, dtype,
                               nullptr);
    }
};
struct Latent {
    const void* kv = P(0);
    const float* w = P<float>(1);
    const int *slots = P<int>(2), *kept = P<int>(3), *cu = P<int>(4);
    void *cache = P(5), *kvo = P(6);
    const void* q = P(7);
    void* qo = P(8);
    int T = 8, B = 4, Hq = 4, dq = 192, dqo = 576, dc = 512, dr = 64, page = 64, pool = 10, norm = 1;
    float eps = 1e-6f;
    kda_rope rope = {P<double>(20), 64, 0, 1.f};
    kda_dtype dtype = KDA_BF16;
    int run() const {
        return kda_latent_append(kv, w, slots, kept, cu, cache, kvo, q, qo, T, B, Hq, dq, dqo, dc, dr, page, pool,
                                 norm, eps, &rope, dtype, nullptr);
    }
};
struct Attn {
    const void *q = P(0), *cache = P(1);
    const int *table = P<int>(2), *kept = P<int>(3), *cu = P<int>(4);
    void* o = P(5);
    float* lse = P<float>(6);
    int T = 40, B = 4, Hq = 8, dc = 512, dr = 64, page = 64, pool = 100, width = 16, max_new = 0;
    float scale = 0.1f;
    kda_dtype dtype = KDA_BF16;
    void* ws = P(7);
    size_t bytes = 0;
    int run() const {
        return kda_attn_latent(q, cache, table, kept, cu, o, lse, T, B, Hq, dc, dr, page, pool, width, max_new,
                               scale, dtype, ws, bytes, nullptr);
    }
};
struct Expanded {
    const void *q = P(0), *kv = P(1), *pe = P(2);
    const int *cq = P<int>(3), *ck = P<int>(4);
    void* o = P(5);
    float* lse = P<float>(6);
    int T = 40, N = 90, B = 4, H = 8, dn = 128, dr = 64, dv = 128, ld = 576, max_q = 0;
    float scale = 0.f;
    kda_dtype dtype = KDA_BF16;
    void* ws = P(7);
    size_t bytes = 0;
    int run() const {
        return kda_attn_expanded(q, kv, pe, cq, ck, o, lse, T, N, B, H, dn, dr, dv, ld, max_q, scale, dtype, ws,
                                 bytes, nullptr);
    }
};

template <typename S, typename V>
static int with(V S::*field, V value) {
    S s;
    s.*field = value;
    return s.run();
}

int main() {
    for (int x : MANY) {
        // sizes at the ends of int: refused, or nothing to do, never an overflow
        if (x < 0) {
            expect("rope T", with(&Rope::T, x), INV);
            expect("rope B", with(&Rope::B, x), INV);
            expect("rope Hq", with(&Rope::Hq, x), INV);
            expect("rope Hkv", with(&Rope::Hkv, x), INV);
            expect("latent T", with(&Latent::T, x), INV);
            expect("latent Hq", with(&Latent::Hq, x), INV);
            expect("latent dq", with(&Latent::dq, x), INV);
            expect("latent dqo", with(&Latent::dqo, x), INV);
            expect("attn T", with(&Attn::T, x), INV);
            expect("attn width", with(&Attn::width, x), INV);
            expect("expanded N", with(&Expanded::N, x), INV);
            expect("expanded ld", with(&Expanded::ld, x), INV);
        } else {
            expect("rope T", with(&Rope::T, x), INV);
            expect("rope B", with(&Rope::B, x), INV);
            expect("rope Hq", with(&Rope::Hq, x), INV);
            expect("rope Hkv", with(&Rope::Hkv, x), INV);
            expect("latent T", with(&Latent::T, x), INV);
            expect("latent Hq", with(&Latent::Hq, x), INV);
            expect("latent dq", with(&Latent::dq, x), INV);
            expect("attn T", with(&Attn::T, x), INV);
            expect("attn B", with(&Attn::B, x), INV);
            expect("attn Hq", with(&Attn::Hq, x), INV);
            expect("attn width", with(&Attn::width, x), INV);
            expect("attn pool", with(&Attn::pool, x), INV);
            expect("expanded T", with(&Expanded::T, x), INV);
            expect("expanded N", with(&Expanded::N, x), INV);
            expect("expanded H", with(&Expanded::H, x), INV);
            expect("expanded ld", with(&Expanded::ld, x), INV);
        }
        expect("attn workspace", (int)kda_attn_latent_workspace_size(x, x, x, 512, 64, 0, KDA_BF16), 0);
        expect("expanded workspace", (int)kda_attn_expanded_workspace_size(x, x, x, 128, 64, 128, 0, KDA_F32), 0);
    }
    expect("rope d", with(&Rope::d, 96), UNS);
    expect("rope page", with(&Rope::page, INT_MIN), UNS);
    expect("rope freqs", with(&Rope::rope, kda_rope{nullptr, 64, 0, 1.f}), INV);
    expect("rope rot", with(&Rope::rope, kda_rope{P<double>(20), INT_MIN, 0, 1.f}), INV);
    expect("rope factor", with(&Rope::rope, kda_rope{P<double>(20), 64, 0, NAN}), INV);
    expect("rope empty", with(&Rope::T, 0), OK);
    expect("latent dc", with(&Latent::dc, INT_MAX), UNS);
    expect("latent dr", with(&Latent::dr, INT_MIN), UNS);
    expect("latent eps", with(&Latent::eps, -1.f), INV);
    expect("latent empty", with(&Latent::B, 0), OK);
    expect("attn workspace missing", with(&Attn::ws, (void*)nullptr), WS);
    expect("attn workspace short", with(&Attn::bytes, (size_t)16), WS);
    expect("attn scale", with(&Attn::scale, 0.f), INV);
    expect("attn empty", with(&Attn::Hq, 0), OK);
    expect("expanded workspace short", with(&Expanded::bytes, (size_t)16), WS);
    expect("expanded dv", with(&Expanded::dv, 64), UNS);
    expect("expanded scale", with(&Expanded::scale, -1.f), INV);
    expect("expanded empty", with(&Expanded::H, 0), OK);
    std::printf("\n%d failures\n", fails);
    return fails != 0;
}
