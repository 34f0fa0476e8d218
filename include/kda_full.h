/*
 * kda_full.h — C ABI of the full-attention layers of a hybrid stack (gfx950).
 *
 * Next to its KDA layers such a stack has layers of grouped heads, whose
 * queries and keys are rotated by their positions, or layers whose keys and
 * values are one latent vector a token, shared by all heads:
 *   kda_rope_append    queries and keys rotated, keys and values into the pages
 *                      that kda_attn_paged reads
 *   kda_latent_append  latents normalised, their positional part rotated, into
 *                      the pages of a latent cache; the queries' part rotated
 *   kda_attn_latent    attention over that cache, with the up-projections
 *                      absorbed into the queries and the output projection
 *   kda_attn_expanded  attention of prompts over keys and values that were
 *                      expanded from the latents
 * slot_map, cu_new and block_table are kda_page_plan's. The rules of
 * kda_serve.h hold here too (ownership, streams, alignment, overlaps, graphs,
 * values on the device that are out of range, repeatability).
 */
#ifndef KDA_FULL_H
#define KDA_FULL_H

#include "kda_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotation by positions. Pair j of a vector x, at position p, becomes
 *   factor * (x cos(p freqs[j]) - y sin(p freqs[j]), y cos(..) + x sin(..))
 * with angles and their functions in fp64. Scaling for long contexts is in
 * freqs and factor.
 *   freqs        [rot / 2] fp64 on the device, radians a position (8-byte aligned)
 *   rot          channels that are rotated: a multiple of 16, 16 .. 128
 *   interleaved  0: pair j is channels (j, j + rot / 2); otherwise (2j, 2j + 1)
 *   factor       finite
 */
typedef struct kda_rope {
    const double* freqs;
    int rot;
    int interleaved;
    float factor;
} kda_rope;

/*
 * Queries and keys of new tokens rotated, keys and values into their slots.
 *   q, q_out [T, Hq, d]   q_out may be exactly q; Hq may be 0
 *   k, v     [T, Hkv, d]
 *   slot_map, k_cache, v_cache   as in kda_cache_append
 *   kept_len [B], cu_new [B + 1]  int32: row cu_new[i] + t is at position
 *            max(kept_len[i], 0) + t. cu_new is meant to be non-decreasing
 *            inside [0, T]. Rows outside all requests are not written to q_out
 *            nor appended; where two requests claim a row, it has the position
 *            of one of them, or counts as outside.
 *   rope     the first rope->rot (at most d) channels are rotated, the others copied
 * Rounded once, from fp32. d in {16, 32, 64, 128}; page_size as in kda_page_plan.
 * T * (Hq + 2 Hkv) and B are at most 2^30.
 */
kda_status kda_rope_append(const void* q, const void* k, const void* v, const int* slot_map,
                           const int* kept_len, const int* cu_new, void* q_out, void* k_cache,
                           void* v_cache, int T, int B, int Hq, int Hkv, int d, int page_size,
                           int n_pool, const kda_rope* rope, kda_dtype dtype, void* stream);

/*
 * Latent rows (c, pe) of new tokens: c normalised, pe rotated, into their slots.
 *   kv       [T, dc + dr]  c: the first dc channels, pe: the last dr
 *   w        [dc] fp32 or NULL (ones)
 *   normalise  c' = w c / sqrt(mean(c^2) + eps) if not 0 (eps >= 0, finite);
 *            otherwise c' = c, and w has to be NULL
 *   cache    [n_pool, page_size, dc + dr]: slot s is row s % page_size of page
 *            s / page_size; rows (c', rotated pe). Slots as in kda_cache_append.
 *   kv_out   [T, dc + dr] or NULL: the same rows, packed; may be exactly kv
 *   q        [T, Hq, dq], q_out [T, Hq, dq_out]: the last dr channels of q_out
 *            become the last dr of q, rotated; its others are left as they are.
 *            q_out may be exactly q if dq_out = dq. Hq = 0: no queries. dq and
 *            dq_out are multiples of 8, at least dr.
 *   kept_len, cu_new  as in kda_rope_append (rows outside all requests: not
 *            written to any output)
 *   rope     rope->rot = dr; NULL: no rotation (pe and the queries' part are copied)
 * dr = 64, dc in {128, 256, 512}; page_size as in kda_page_plan. T * (Hq + 1) and
 * B are at most 2^30.
 */
kda_status kda_latent_append(const void* kv, const float* w, const int* slot_map,
                             const int* kept_len, const int* cu_new, void* cache, void* kv_out,
                             const void* q, void* q_out, int T, int B, int Hq, int dq, int dq_out,
                             int dc, int dr, int page_size, int n_pool, int normalise, float eps,
                             const kda_rope* rope, kda_dtype dtype, void* stream);

/*
 * Causal attention of new tokens over a paged latent cache that holds them
 * already. Position j's row x_j = (c_j, pe_j) is the key of every query head,
 * and c_j its value.
 *   q        [T, Hq, dc + dr]  queries, the keys' up-projection absorbed in the
 *            first dc channels; rows cu_new[i] .. cu_new[i + 1) are request i's,
 *            the t-th sees the request's positions 0 .. kept_len[i] + t
 *   cache    as in kda_latent_append
 *   block_table, kept_len, cu_new, max_new, ws  as in kda_attn_paged, with what
 *            it says of bad values and of rows outside all requests
 *   o        [T, Hq, dc]: sum_j softmax_j(scale q.x_j) c_j, before the values'
 *            up-projection. A row without any position (or with scores of
 *            -infinity alone) gives 0.
 *   lse      [T, Hq] fp32 or NULL: natural log of the sum of exp(scores)
 *   scale    above 0, at most 2^127: 1 / sqrt(width of the queries before they
 *            absorbed anything)
 * Sums over positions are fp32, of weights up to 2^8: |c| times the number of
 * positions that a row sees is meant to be at most 2^118. Scores (times log2 e) that
 * are past fp32 count as infinite.
 * What masked positions and unused cache rows hold does not reach the result. A row
 * that sees a c that is not finite, or has a score of NaN or +infinity, is not finite,
 * in part or as a whole; a position of finite c with a score of -infinity has no
 * weight. dr = 64, dc in {128, 256, 512}; T * Hq, max_pages * page_size and B are
 * at most 2^30.
 */
size_t kda_attn_latent_workspace_size(int T, int B, int Hq, int dc, int dr, int max_new,
                                      kda_dtype dtype);
kda_status kda_attn_latent(const void* q, const void* cache, const int* block_table,
                           const int* kept_len, const int* cu_new, void* o, float* lse, int T,
                           int B, int Hq, int dc, int dr, int page_size, int n_pool, int max_pages,
                           int max_new, float scale, kda_dtype dtype, void* ws, size_t ws_bytes,
                           void* stream);

/*
 * Causal attention of packed prompts over expanded keys and values. Request i
 * has query rows cu_q[i] .. cu_q[i + 1) and key rows cu_k[i] .. cu_k[i + 1), its
 * last query is at its last key: with n queries and m keys, query t sees keys
 * 0 .. m - n + t (none, if that is below 0).
 *   q        [T, H, dn + dr]
 *   kv       [N, H, dn + dv]  of head h: the first dn channels of its key, then
 *            its value
 *   k_pe     [N, dr]  the last dr channels of the keys of all heads; row stride
 *            pe_stride elements, a multiple of 8, at least dr (the rows of
 *            kda_latent_append's kv_out end in it)
 *   cu_q, cu_k  [B + 1] int32, meant to be non-decreasing inside [0, T] and
 *            [0, N]; clamped there; treated as kda_attn_paged's cu_new
 *   o        [T, H, dv], lse [T, H] fp32 or NULL; rows as in kda_attn_latent
 *   max_q    the largest number of queries of one request, 0 = unknown; selects
 *            kernels only
 *   scale    0 selects 1 / sqrt(dn + dr). Not negative, at most 2^127.
 * Masked positions do not reach the result, whatever they hold. Values are meant to
 * be at most 2^118 over the number of keys, and scores that are past fp32 count as
 * infinite, as in kda_attn_latent. dr = 64,
 * dn = dv in {64, 128}; T * H, N and B are at most 2^30, H (dn + dv) and pe_stride at
 * most 2^26.
 */
size_t kda_attn_expanded_workspace_size(int T, int B, int H, int dn, int dr, int dv, int max_q,
                                        kda_dtype dtype);
kda_status kda_attn_expanded(const void* q, const void* kv, const void* k_pe, const int* cu_q,
                             const int* cu_k, void* o, float* lse, int T, int N, int B, int H,
                             int dn, int dr, int dv, int pe_stride, int max_q, float scale,
                             kda_dtype dtype, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_FULL_H */
