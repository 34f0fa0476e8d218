/*
 * kda_serve.h — C ABI of the serving step around the recurrent layer (gfx950).
 *
 * A stack that mixes KDA layers with full-attention layers serves each step
 * with these calls next to those of kda.h:
 *   kda_page_plan      cache pages and slots of the step's new tokens
 *   kda_cache_append   their keys and values into the slots
 *   kda_attn_paged     attention of the new tokens over each request's pages
 *   kda_draft_verify   which drafted tokens stay, and the token after them
 * kda_page_plan's cu_new has the form of kda_prefill_varlen's cu_seqlens, and
 * kda_draft_verify's n_commit is that of kda_decode_multi: the tokens that
 * the recurrent state advances by, and that the next plan's kept_len grows
 * by, which gives the pages of rejected tokens back.
 *
 * The rules of kda.h hold here too: the caller owns every buffer; a call
 * allocates nothing, does not synchronise, keeps no state and runs on
 * `stream` on the current device; arguments are checked on the host before
 * anything is launched, and a rejected call has no side effect. Lengths,
 * tables and tokens are read on the device: no value in them leads to an
 * access outside the buffers. Unless a parameter says otherwise, an output
 * overlaps no input and no other output, and int32 arrays are 4-byte, every
 * other array 16-byte aligned. All calls may be captured in a graph (no
 * memset, no host-side dependence on device values). Identical calls give
 * bit-identical results. Two calls that overlap in time need workspaces of
 * their own.
 */
#ifndef KDA_SERVE_H
#define KDA_SERVE_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* *status of kda_page_plan; a positive value is the number of pages the pool
 * is short of. */
#define KDA_PLAN_OK 0
#define KDA_PLAN_INVALID (-1)   /* a length, count or ring value outside its range,
                                   or a request longer than its row of the table */
#define KDA_PLAN_NO_SLOTS (-2)  /* more new tokens than slot_map holds */

/*
 * Block tables and slot maps from request lengths.
 *
 * Request i keeps kept_len[i] tokens in the cache and adds n_new[i] (both
 * >= 0, at most INT32_MAX together; both 0 for a request that has ended or an
 * unused row). It needs
 * ceil((kept + new) / page_size) pages and holds n_pages_in[i] of them,
 * block_table[i, 0 .. n_pages_in[i]). Missing pages are taken from the pool
 * in the order of requests and positions, surplus ones go back in that order.
 *
 *   block_table [B, max_pages]  page ids; entries [0, n_pages_in[i]) are read,
 *               the entries of added pages written, all others left as they are
 *   free_ring   [n_pool]  the pool's free pages as a ring: (head, count) in
 *               ring_in, the oldest at head; pages are taken at the head and
 *               given back behind the last. Entries of taken pages stay.
 *   n_pages_out [B], ring_out [2]  the counts afterwards; each may be exactly
 *               n_pages_in / ring_in (update in place)
 *   cu_new      [B + 1]  exclusive prefix sum of n_new: request i's new tokens
 *               are rows cu_new[i] .. cu_new[i + 1) of the step's packed tensors
 *   slot_map    [n_slots]  slot (page * page_size + offset) of every new token;
 *               -1 in the rows behind cu_new[B] (a padded step), and where the
 *               page id is outside [0, n_pool)
 *   status      [1]  see above. When it is not KDA_PLAN_OK the step is empty:
 *               nothing is taken or given back (n_pages_out = n_pages_in,
 *               ring_out = ring_in), cu_new is 0 throughout and slot_map -1.
 *   page_size   a power of two, 16 .. 1024; n_pool * page_size <= INT32_MAX
 *   B           at most 2^30
 *   ws          kda_page_plan_workspace_size() bytes
 * A call that is repeated with the same inputs (and other buffers for the
 * counts afterwards) gives the same outputs: what it writes to block_table
 * and free_ring it does not read.
 */
size_t kda_page_plan_workspace_size(int B);
kda_status kda_page_plan(const int* kept_len, const int* n_new, const int* n_pages_in,
                         int* n_pages_out, int* block_table, int* free_ring,
                         const int* ring_in, int* ring_out, int* cu_new, int* slot_map,
                         int* status, int B, int max_pages, int page_size, int n_pool,
                         int n_slots, void* ws, size_t ws_bytes, void* stream);

/*
 * Keys and values of new tokens into their cache slots.
 *   k, v     [T, Hkv, d]
 *   k_cache, v_cache  [n_pool, Hkv, page_size, d]: slot s is row s % page_size
 *            of page s / page_size
 *   slot_map [T]  a slot outside [0, n_pool * page_size) is skipped. Slots are
 *            meant to be distinct: where one occurs twice, its row ends up with
 *            pieces of either token.
 * d in {16, 32, 64, 128}; page_size as above; dtype is that of k, v and cache.
 */
kda_status kda_cache_append(const void* k, const void* v, const int* slot_map,
                            void* k_cache, void* v_cache, int T, int Hkv, int d,
                            int page_size, int n_pool, kda_dtype dtype, void* stream);

/*
 * Causal attention of new tokens over a paged cache that holds them already.
 *   q        [T, Hq, d]   rows cu_new[i] .. cu_new[i + 1) are request i's new
 *            tokens; the t-th is at position kept_len[i] + t and attends to
 *            the request's positions 0 .. kept_len[i] + t
 *   k_cache, v_cache  as in kda_cache_append; query head hq reads KV head
 *            hq / (Hq / Hkv) (Hq a multiple of Hkv)
 *   block_table [B, max_pages], kept_len [B], cu_new [B + 1]  int32. Positions
 *            past max_pages * page_size or in a page outside [0, n_pool) are
 *            treated as masked. cu_new is meant to be non-decreasing inside
 *            [0, T]; it is clamped there, and where it decreases the request
 *            is empty. The values of rows that two requests claim are
 *            unspecified; requests that claim more than T rows together make
 *            the call an empty one, which writes no row.
 *   o        [T, Hq, d] in `dtype`; rows outside all requests are left as they
 *            are. A row without any position (or with scores of -infinity alone)
 *            gives 0.
 *   lse      [T, Hq] fp32 or NULL: natural log of the sum of exp(scores),
 *            -infinity for a row without any position
 *   scale    factor on q.k; 0 selects 1 / sqrt(d). Not negative, at most 2^127.
 *            T * Hq, max_pages * page_size and B are at most 2^30.
 *   max_new  the largest number of new tokens of one request, 0 = unknown. It
 *            selects kernels only: results are right whatever it says.
 *   ws       kda_attn_paged_workspace_size() bytes
 * What masked positions and unused cache rows hold (NaN and infinities
 * included) does not reach the result. d, page_size and dtype as above.
 */
size_t kda_attn_paged_workspace_size(int T, int B, int Hq, int Hkv, int d, int max_new,
                                     kda_dtype dtype);
kda_status kda_attn_paged(const void* q, const void* k_cache, const void* v_cache,
                          const int* block_table, const int* kept_len, const int* cu_new,
                          void* o, float* lse, int T, int B, int Hq, int Hkv, int d,
                          int page_size, int n_pool, int max_pages, int max_new, float scale,
                          kda_dtype dtype, void* ws, size_t ws_bytes, void* stream);

/*
 * Verification of drafted tokens by rejection sampling, so that the tokens
 * kept and sampled follow the target's distribution.
 *   target_probs p [B, T + 1, V]  row t: the target's distribution of the
 *            token that draft_tokens[b, t] proposes, row T of the one after
 *   draft_probs  q [B, T, V] in the same dtype, or NULL: the draft is certain
 *            (all of its probability on the drafted token)
 *   draft_tokens x [B, T] int32
 *   u        [B, T + 1] fp32 in [0, 1): u[b, t] decides token t, u[b, T] samples
 *   n_draft  [B] int32 or NULL (T): the request's own number of drafted tokens;
 *            above T counts as T, below 0 marks an unused row
 * Token t stays if all before it stay and u_t q_t(x_t) < p_t(x_t). With a the
 * number that stay, the next token y is drawn from max(p_a - q_a, 0) when
 * token a was rejected (from p_a when that is 0 throughout), from p_a when
 * none was: the least y with sum_{z <= y} r(z) > u_T sum r, sums in fp64.
 * Values that are negative or NaN count as 0 in r. Where no such y exists (r
 * without a positive value, infinities, u >= 1) it is the last token with
 * r > 0, 0 if there is none. A drafted token outside [0, V) is rejected.
 *   n_commit [B]  a + 1, 0 for an unused row
 *   tokens   [B, T + 1]  the tokens that stay, y, then -1
 * Only the rows a are read in full.
 *   ws       kda_draft_verify_workspace_size() bytes
 */
size_t kda_draft_verify_workspace_size(int B, int T, int V);
kda_status kda_draft_verify(const void* target_probs, const void* draft_probs,
                            const int* draft_tokens, const float* u, const int* n_draft,
                            int* n_commit, int* tokens, int B, int T, int V, kda_dtype dtype,
                            void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_SERVE_H */
