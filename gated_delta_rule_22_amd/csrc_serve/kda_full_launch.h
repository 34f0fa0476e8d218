// Internal launchers behind the C ABI of the full-attention layers (arguments
// already validated).
#pragma once

#include "kda_full.h"
#include "kda_serve_launch.h"

namespace kda {

struct RopeArgs {
    const double* freqs;   // or null: no rotation
    int rot;
    bool interleaved;
    float factor;
};

struct RopeAppendArgs {
    const void *q, *k, *v;
    const int *slots, *kept, *cu;
    void *q_out, *kc, *vc;
    int T, B, Hq, Hkv, d, page_shift, pool;
    RopeArgs rope;
    bool bf16_io;
};
hipError_t launch_rope_append(const RopeAppendArgs& a, hipStream_t st);

struct LatentAppendArgs {
    const void* kv;
    const float* w;        // or null
    const int *slots, *kept, *cu;
    void *cache, *kv_out;  // kv_out or null
    const void* q;
    void* q_out;
    int T, B, Hq, dq, dq_out, dc, page_shift, pool;
    bool normalise;
    float eps;
    RopeArgs rope;
    bool bf16_io;
};
hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t st);

// Channels of a latent row's positional part.
constexpr int kPe = 64;

// AttnArgs of the latent cache: kc is the cache, Hkv is 1, d is dc.
size_t attn_latent_ws(int T, int B, int Hq, int dc, int max_new, bool bf16_io);
hipError_t launch_attn_latent(const AttnArgs& a, void* ws, hipStream_t st);

// Expanded keys: every head its own, request i's tokens before its new ones
// counted from its keys. kc is kv, vc is k_pe, Hkv is Hq, d is dv; a cache of 2^30
// pages of one token, so that no length is cut.
struct ExpandedArgs : AttnArgs {
    const int* cu_k;
    int N;
    long pe_stride;
    static constexpr int kLeastKept = -(1 << 30);
    __device__ int row_of(int i) const { return min(max(cu_k[i], 0), N); }
    __device__ int kept_of(int i) const {
        const int n = min(max(cu[i + 1], 0), T) - min(max(cu[i], 0), T);
        return max(row_of(i + 1) - row_of(i), 0) - max(n, 0);
    }
};
size_t attn_expanded_ws(int T, int B, int H, int dv, int max_q, bool bf16_io);
hipError_t launch_attn_expanded(const ExpandedArgs& a, void* ws, hipStream_t st);

}  // namespace kda
