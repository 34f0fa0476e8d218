// Internal launchers behind the serving C ABI (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_common.h"
#include "kda_serve.h"

namespace kda {

struct PlanArgs {
    const int *kept, *fresh, *pages_in;
    int *pages_out, *table, *ring;
    const int* ring_in;
    int *ring_out, *cu, *slots, *status;
    int B, width, page_shift, pool, n_slots;
};
// ws: page_plan_ws(B) bytes
size_t page_plan_ws(int B);
hipError_t launch_page_plan(const PlanArgs& a, void* ws, hipStream_t st);

// Rows of row_bytes (a multiple of 16) bytes per token and head.
hipError_t launch_cache_append(const void* k, const void* v, const int* slots, void* kc,
                               void* vc, int T, int Hkv, int row_bytes, int page_shift,
                               int pool, hipStream_t st);

struct AttnArgs {
    const void *q, *kc, *vc;
    const int *table, *kept, *cu;
    void* o;
    float* lse;           // or null
    int T, B, Hq, Hkv, d, page_shift, pool, width;
    int max_new;          // a hint, 0 = unknown
    float scale;
    bool bf16_io;
    static constexpr int kLeastKept = 0;
    __device__ int kept_of(int i) const { return kept[i]; }
};
size_t attn_paged_ws(int T, int B, int Hq, int Hkv, int d, int max_new, bool bf16_io);
hipError_t launch_attn_paged(const AttnArgs& a, void* ws, hipStream_t st);

struct VerifyArgs {
    const void *p, *q;    // q or null
    const int* x;
    const float* u;
    const int* n_draft;   // or null
    int *n_commit, *tokens;
    int B, T, V;
    bool bf16_io;
};
size_t draft_verify_ws(int B, int V);
hipError_t launch_draft_verify(const VerifyArgs& a, void* ws, hipStream_t st);

}  // namespace kda
