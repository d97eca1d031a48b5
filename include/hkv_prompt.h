/*
 * hkv_prompt.h -- C ABI of the prompt side of the cache: what runs before the
 * decode step of hkv.h has tiers to work on. A serving loop keeps its prompts'
 * keys and values in pages of a pool and calls, for each step of chunks,
 *   hkv_page_plan        block tables, slot map and positions from request lengths,
 *   hkv_qk_norm_rope     per-head norms and the position rotation of the
 *                        projected queries and keys, K and V rows written to
 *                        their slots,
 *   hkv_chunk_attention  the chunk's attention over the paged cache,
 * and when a prompt is complete
 *   hkv_fill_tiers       its pages become the dense and sparse tiers, as if
 *                        every token had gone through hkv_append,
 *   hkv_page_release     its pages go back to the pool.
 * From then on hkv_append and hkv_step serve the request; hkv_qk_norm_rope
 * also writes the contiguous rows that hkv_append takes.
 *
 * The conventions of hkv.h hold here: the caller owns all memory, nothing
 * allocates or synchronises, every call is asynchronous on `stream` and can be
 * captured (lengths are read on the device), host errors launch nothing,
 * device conditions set bits of the workspace's status word (hkv_get_status).
 * Calls that overlap on the GPU need separate workspaces and outputs.
 *
 * Of hkv_problem the calls use B (requests), Hq, Hkv, D, dtype and scale (the
 * rest must still validate): bf16 or fp32, D 64 or 128, Hq/Hkv 1, 2, 4 or 8.
 */
#ifndef HKV_PROMPT_H
#define HKV_PROMPT_H

#include "hkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further device status-word bit. */
#define HKV_DEV_PAGES_FULL 0x40u /* hkv_page_plan: a request was left out: no pages or rows left for it */

#define HKV_MAX_REQUESTS 8192      /* requests of one call */
#define HKV_MAX_TOKENS (1 << 22)   /* token rows of one call */

/* The page pool: K and V of page i, KV head h, row t at
 * i*stride_p + h*stride_h + t*stride_t (elements; D contiguous; 16-byte
 * aligned like a tier's rows, strides above 0 where there is more than one),
 * and the block tables: column c of row b names the page of tokens
 * c*page .. c*page + page-1 of request b. Any other entry than a page of the
 * pool means that the tokens are not there: they are masked (attention), read
 * as zeros (fill) or not written, and HKV_DEV_BAD_INDEX is set when a call
 * meets such an entry below a request's length. */
typedef struct {
    void *k, *v;                           /* device */
    int64_t stride_p, stride_h, stride_t;
    int32_t pages;                         /* pages in the pool; pages*page < 2^31 */
    int32_t page;                          /* tokens a page: 16, 32, 64, 128 or 256 */
    int32_t *table;                        /* device [B, table_cols], row stride table_stride */
    int64_t table_stride;
    int32_t table_cols;                    /* table_cols*page at most 2^30 */
} hkv_pages;

/* Allocation state beside the tables, all int32 on the device: `free` is a
 * stack of page numbers ([pages]; the top is entry free_count-1). */
typedef struct {
    int32_t *free;
    int32_t *free_count;  /* [1] */
    int32_t *held;        /* [B] pages each request holds (table columns in use) */
} hkv_page_state;

/* The rows of one step, int32 on the device: the tokens of request b are rows
 * q_start[b] .. q_start[b+1]-1 of the step's [tokens, ...] tensors; kv_len[b]
 * counts its cached tokens with the new ones, pos is a row's position in its
 * request and slot its place in the pool (page*page_size + row). Rows behind
 * q_start[B] have pos = slot = -1. */
typedef struct {
    int32_t tokens;    /* row capacity */
    int32_t *q_start;  /* [B+1] */
    int32_t *kv_len;   /* [B] */
    int32_t *pos;      /* [tokens] */
    int32_t *slot;     /* [tokens] */
} hkv_chunk;

/* Block tables and slot maps from request lengths: new_len[b] tokens join the
 * ctx_len[b] cached ones of request b. A request needs
 * max(0, ceil((ctx+new)/page) - held) pages (none when new = 0). Requests are
 * served in order of b: one that needs pages gets all of them if it and every
 * request before it (those left out included) need no more than free_count in
 * all, and likewise its new tokens need room in the `tokens` rows. One that
 * does not fit is left out whole: granted 0, no rows, no pages, kv_len = ctx,
 * and HKV_DEV_PAGES_FULL. Negative lengths, ctx above held*page, held above
 * the table's columns or more tokens than the table has room for leave a request
 * out too, with HKV_DEV_BAD_INDEX. The j-th page given out is free[free_count-1-j],
 * to the requests in order, columns ascending.
 * - in, after: the state before and after. They may be the same; `free` has to be
 *   (this call does not write it). out->kv_len may be ctx_len, so that a loop's
 *   lengths advance in place. Nothing else may overlap.
 * - pages: page, pages and the table (written at the new columns); K and V are
 *   not used and may be NULL.
 * - granted: device int32 [B] or NULL, the new tokens each request was given.
 * - ws: any workspace of at least 256 bytes. One kernel. */
hkv_status hkv_page_plan(int32_t B, const int32_t *ctx_len, const int32_t *new_len, const hkv_pages *pages,
                         const hkv_page_state *in, const hkv_page_state *after, const hkv_chunk *out,
                         int32_t *granted, void *ws, size_t ws_bytes, hkv_stream_t stream);

/* The pages of every request with done[b] != 0 go back on the stack, in
 * order of b and then of columns; its held count becomes 0 (its table row
 * keeps its entries, which then mean nothing). States as for hkv_page_plan,
 * but this call writes `free` above free_count. A state that does not fit the pool
 * (a held count below 0 or above the table's columns, more pages than the
 * stack has room for, a table entry to go back that is no page of the pool) sets
 * HKV_DEV_BAD_INDEX and releases nothing. The call knows no shared pages: one that
 * stands in several tables (a common prefix) goes back with each of them, and
 * would then be given to two requests. Of requests that share pages only one may
 * be released, after the others are done with them; the pages that the others
 * hold alone are the caller's to put on the stack. */
hkv_status hkv_page_release(int32_t B, const int32_t *done, const hkv_pages *pages, const hkv_page_state *in,
                            const hkv_page_state *after, void *ws, size_t ws_bytes, hkv_stream_t stream);

/* The position rotation: pair i < rot/2 of a head turns by pos*inv_freq[i]
 * radians (angles in 64 bits), its cosine and sine multiplied by mscale.
 * interleaved 0: pairs (i, i + rot/2); 1: (2i, 2i+1). Elements from rot on are
 * left. rot: 0 (none; inv_freq may be NULL) or a multiple of 16 up to D. */
typedef struct {
    const double *inv_freq;  /* device [rot/2] */
    int32_t rot;
    int32_t interleaved;
    float mscale;
} hkv_rope;

/* Per-head norm and rotation of the projected rows, in one pass:
 * x <- x * rsqrt(mean(x^2) + eps) * w over each query and key head (left out
 * when q_w and k_w are NULL), then the rotation; value rows pass unchanged.
 * Computed in fp32, rounded once.
 * - q, k, v: device rows of [tokens, heads, D], heads and D contiguous, row
 *   strides in elements (slices of one projection's output will do), all
 *   16-byte aligned. q_out: [tokens, Hq, D] contiguous.
 * - pos: device int32 [tokens]; a row with pos < 0 is skipped (its outputs are
 *   left as they are).
 * - K and V rows go to the pages at slot[row] (pages and slot given; -1 = not
 *   written; another slot outside the pool is not written either and sets
 *   HKV_DEV_BAD_INDEX; rows of one call that share a slot leave a mixture of
 *   their values in it), or to k_out, v_out [tokens, Hkv, D] contiguous (given
 *   instead; the layout of hkv_append's k_new, v_new).
 * - q_out may be q itself, k_out k and v_out v, where their rows are contiguous
 *   too (stride heads*D, or one token); an output that overlaps an input in any
 *   other way, or another output, is refused (HKV_ERR_INVALID_ARG; the input's
 *   span counts from its first row to its last, the gaps between rows included).
 * - q_w, k_w: device [D] of the problem's type, both or neither, 16-byte
 *   aligned; eps >= 0.
 * - ws: any workspace of at least 256 bytes. B is not used. One kernel. */
hkv_status hkv_qk_norm_rope(const hkv_problem *prob, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, int32_t tokens, const int32_t *pos, const int32_t *slot,
                            const hkv_rope *rope, const void *q_w, const void *k_w, float eps, void *q_out,
                            void *k_out, void *v_out, const hkv_pages *pages, void *ws, size_t ws_bytes,
                            hkv_stream_t stream);

/* Workspace bytes of hkv_chunk_attention for up to `tokens` rows. */
hkv_status hkv_chunk_workspace_size(const hkv_problem *prob, int32_t tokens, size_t *bytes);

/* Attention of a chunk of new tokens over the paged cache: row i of request b
 * (i < n = q_start[b+1] - q_start[b]) stands at position kv_len[b] - n + i and
 * attends, with scale q.k, to the request's tokens at positions up to its own
 * (its own K and V among them: they are in the pages already). Single new
 * tokens, whole prompts and both in one batch are the same call.
 * - q: device [tokens, Hq, D] rows of row stride q_stride (elements; heads and
 *   D contiguous; 16-byte aligned). out: [tokens, Hq, D] contiguous, of the
 *   problem's type; lse: fp32 [tokens, Hq] (natural log) or NULL. Rows behind
 *   q_start[B] are left as they are. out and lse may not overlap q (its span,
 *   gaps between rows included) or each other: HKV_ERR_INVALID_ARG.
 * - A row that attends to nothing gives out = 0, lse = -inf.
 * - Keys and values behind kv_len and in pages that are not the request's may
 *   hold anything, infinities and NaN included. Those of a request's own
 *   tokens have to be finite, or that request's rows of the call are undefined
 *   (no other request's are).
 * - q_start outside [0, tokens] or descending, or kv_len outside
 *   [0, table_cols*page], is clamped and sets HKV_DEV_LEN_CLAMPED.
 * - Sums and softmax statistics are fp32. With bf16 the weights are rounded to
 *   bf16 for the product with V, and out once at its end.
 * - ws: hkv_chunk_workspace_size bytes for at least `tokens` rows, zeroed once
 *   by hkv_workspace_init, and again after HKV_DEV_TIMEOUT. Two kernels; a wait in
 *   them ends after 2^31 ns at the latest, whatever hkv_set_wait_limit_ns allows.
 * - fp32 has a kernel for single tokens and one for chunks, chosen by the host, which
 *   does not see the lengths: the first when tokens <= B. Results are right either
 *   way, but single tokens in a step with room for more rows take up to 3.6 times
 *   as long, as does a long chunk in a step with no more rows than requests (2.4
 *   times). bf16 has one kernel for both. */
hkv_status hkv_chunk_attention(const hkv_problem *prob, const void *q, int64_t q_stride, int32_t tokens,
                               const int32_t *q_start, const int32_t *kv_len, const hkv_pages *pages, void *out,
                               float *lse, void *ws, size_t ws_bytes, hkv_stream_t stream);

/* The tiers of finished prompts, from their pages: for each request b (with
 * take[b] != 0, or all when take is NULL) and KV head, the dense window, its
 * head, the sparse tier and both lengths become what kv_len[b] calls of
 * hkv_append leave when they start from empty tiers: token t is in window slot
 * t mod dense->cap if it is among the last dense->cap tokens, else in sparse
 * slot t, or dropped when the sparse tier has no slot t. Rows are bit copies;
 * rows of the tiers that hold no token are left as they are, and so is every unit of
 * a request that is not taken.
 * - dense, dense_head, sparse: as for hkv_append (written). dropped: device
 *   int32 [B*Hkv] or NULL, the number of tokens dropped; any sets HKV_DEV_SPARSE_FULL.
 * - kv_len outside [0, table_cols*page] is clamped, with HKV_DEV_LEN_CLAMPED.
 * - ws: any workspace of at least 256 bytes. One kernel. */
hkv_status hkv_fill_tiers(const hkv_problem *prob, const hkv_pages *pages, const int32_t *kv_len,
                          const int32_t *take, const hkv_tier *dense, int32_t *dense_head, const hkv_tier *sparse,
                          int32_t *dropped, void *ws, size_t ws_bytes, hkv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* HKV_PROMPT_H */
