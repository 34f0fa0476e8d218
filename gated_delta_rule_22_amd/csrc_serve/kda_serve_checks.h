// Checks of arguments that the C ABIs of the serving step and of the
// full-attention layers share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

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
