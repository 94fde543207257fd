/*
 * spec_attend.h - C ABI of the target pass's cache operators for GB300 (sm_103a): appending a
 * round's keys and values to a paged cache with their position rotation, and attention of the
 * round's rows over that cache (sliding window, sinks, shared prefix).
 *
 * They come directly before spec_verify on the same ragged batch: request i owns rows
 * row_off[i] .. row_off[i+1]-1 (for a verification round the pending token and its K_i drafts; for a
 * prompt, its tokens), T = row_off[B] rows in all. kv_len[i] is the number of positions of request
 * i with these rows included, and the n_i rows are its last n_i positions: row row_off[i]+j is
 * position p = kv_len[i] - n_i + j. A row with p < 0 is padding. n_i = 0 and kv_len[i] = 0 are
 * allowed.
 *
 * Offsets stay within [0, T] and do not decrease. Where they do otherwise, a request has its rows if
 * 0 <= row_off[i] <= row_off[i+1] <= T and none of the offsets within [0, T] contradicts that (no
 * earlier one is above row_off[i], no later one below row_off[i+1]), and is served like any other; the
 * rest report SPEC_REQ_BAD_SHAPE. So an offset outside [0, T] costs the two requests beside it.
 *
 * The cache is paged, with the pages spec_compact speaks of: position x lies in slot x % page_size
 * of page block_table[i][x / page_size]. In memory, element d of head h, slot s, page b of the keys
 * (and alike of the values) is
 *     cache[b * page_stride + s * slot_stride + h * head_stride + d]     (strides in elements),
 * so that both [page][slot][head][d] and [page][head][slot][d] are served.
 *
 * The conventions of spec_verify.h hold: device pointers, memory owned by the caller, no allocation
 * and no synchronisation, host-detectable argument errors returned before anything is enqueued,
 * errors in one request's data reported in req_status without disturbing the others. The pages this
 * library follows define the rows, positions and KV rows of a round ("M7.8 - Speculative Serving",
 * sections 0x03C and 0x08A); they leave the target's own arithmetic to the model.
 */
#ifndef SPEC_ATTEND_H
#define SPEC_ATTEND_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- spec_kv_append ----------------------------------------------------------------------
 * For every row at position p >= 0: the first rot_dim elements of each query and key head are
 * rotated by the angles of cos_sin row p, the rotated queries go to q_out, and the rotated keys and
 * the values go to the cache at position p. The rotation of pair c (0 <= c < rot_dim / 2) is
 *     (a, b) -> (a cos_c - b sin_c, b cos_c + a sin_c),
 * with (a, b) = elements (c, c + rot_dim/2), or (2c, 2c+1) when interleaved; it is formed in 32
 * bits and rounded once to the type. Elements from rot_dim on are copied.
 * A row whose position has no page (beyond max_blocks, or a page id outside [0, n_pages)) or no
 * cos_sin row is not written at all, and its request's status says so (SPEC_REQ_BAD_BLOCKS,
 * SPEC_REQ_BAD_SHAPE); the request's other rows are written. Padding rows are not written, nor are
 * rows of a request whose offsets are wrong or contradicted or whose kv_len is negative
 * (SPEC_REQ_BAD_SHAPE). Rows of one call must not share a cache position. */
typedef struct {
    int32_t B, total_rows;       /* requests, rows (total_rows = row_off[B])                     */
    int32_t n_q_heads, n_kv_heads, head_dim; /* head_dim <= 512; n_q_heads may be 0 (no queries)  */
    int32_t rot_dim;             /* even, 0 .. head_dim                                          */
    int32_t interleaved;         /* 0: pairs (c, c + rot_dim/2); 1: pairs (2c, 2c+1)              */
    int32_t page_size, max_blocks, n_pages;
    int32_t n_pos;               /* rows of cos_sin                                             */
    spec_dtype dtype;            /* type of q, k, v, q_out and the cache                         */
    const void *q, *k, *v;       /* [T] rows of [heads][head_dim], heads contiguous              */
    int64_t q_stride, k_stride, v_stride; /* elements from one row to the next                   */
    void *q_out;                 /* like q; may be q itself (same stride)                        */
    int64_t q_out_stride;
    const float *cos_sin;        /* [n_pos][rot_dim]: rot_dim/2 cosines, then rot_dim/2 sines    */
    void *k_cache, *v_cache;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *row_off;      /* [B+1]                                                       */
    const int32_t *kv_len;       /* [B]                                                         */
    const int32_t *block_table;  /* [B][max_blocks]                                             */
    int32_t *req_status;         /* [B] out: SPEC_REQ_* bits (may be NULL)                       */
} spec_kv_append_args;

/* Enqueues one kernel on `stream`. Any strides and alignments of the type are served; rows, heads
 * and pages on 16-byte boundaries take the vectorised kernel. */
spec_status spec_kv_append(const spec_kv_append_args *args, cudaStream_t stream);

/* ---- spec_attend -------------------------------------------------------------------------
 * Row at position p of a request sees its position x when
 *     0 <= x <= p  and  (window == 0  or  x > p - window  or  x < n_sink):
 * a sliding window of the last `window` positions (its own included) and the first n_sink
 * positions, which stay visible. For query head h, with key/value head h / (n_q_heads/n_kv_heads),
 *     out = sum_x softmax_x(scale q.k_x) v_x   over the positions it sees,
 *     lse = ln sum_x exp(scale q.k_x).
 * A row that sees nothing (padding) gets out = 0 and lse = -inf. What the cache holds at positions
 * that no row sees (other pages, slots past kv_len, positions behind the window) is never used, even
 * when it is not finite, and their block_table entries may be anything.
 *
 * shared_len > 0 says that the first shared_len positions of every request hold the same text, kept
 * in the pages of shared_table [ceil(shared_len / page_size)]: those keys and values are read once
 * for all rows of the batch and joined with each request's own part. The result is what it would be
 * if every request's block_table named these pages (block_table entries of pages wholly below
 * shared_len are not read).
 *
 * fp32: 32-bit arithmetic throughout. bf16, head_dim a multiple of 16 up to 128, and a cache whose
 * slots make the rows of a matrix (pages a whole number of slot strides apart; a slot's heads side by
 * side within its stride, or a whole number of slot strides apart): products on the tensor cores with
 * 32-bit accumulation, each softmax weight rounded to bf16 for the second product; scores, statistics
 * and the sum of the unrounded weights in 32 bits. Other bf16 calls run on the fp32 units with 32-bit
 * weights, a good deal slower. So a bf16 call's error and speed follow its head size and layout
 * (spec_attend_plan names the kernel): with rounded weights an output may be off by 2^-8 of
 * sum |weight v| beside its own rounding. Results do not depend on the order in which CTAs run.
 * A request with status bits has out = 0 and lse = -inf on its rows, if it has offsets 0 <= row_off[i]
 * <= row_off[i+1] <= T (else it has none; rows that belong to no request are not written):
 * SPEC_REQ_BAD_SHAPE for wrong or contradicted offsets or a negative kv_len, SPEC_REQ_BAD_BLOCKS for a
 * visible position without a page. SPEC_REQ_TIMEOUT on every request says that a bounded wait
 * inside the kernel gave up (an internal fault); the call's outputs then mean nothing. */
typedef struct {
    int32_t B, total_rows;
    int32_t n_q_heads, n_kv_heads, head_dim; /* n_q_heads a multiple of n_kv_heads; head_dim <= 256,
                                                a multiple of 8 (bf16) or 4 (fp32)               */
    int32_t page_size, max_blocks, n_pages;
    int32_t window, n_sink;      /* window 0: every earlier position is visible                 */
    int32_t shared_len;          /* 0: none                                                     */
    spec_dtype dtype;            /* type of q, out and the cache                                 */
    float scale;                 /* finite, > 0                                                 */
    const void *q;               /* [T] rows of [n_q_heads][head_dim]                            */
    int64_t q_stride;
    const void *k_cache, *v_cache;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *row_off, *kv_len, *block_table;
    const int32_t *shared_table; /* [ceil(shared_len / page_size)], NULL when shared_len = 0      */
    void *out;                   /* [T] rows of [n_q_heads][head_dim]; not overlapping q          */
    int64_t out_stride;
    float *lse;                  /* [T][n_q_heads] (may be NULL)                                  */
    int32_t *req_status;         /* [B] out (may be NULL)                                        */
} spec_attend_args;

/* Limits, SPEC_ERR_UNSUPPORTED beyond them: total_rows * n_q_heads and the positions a row of
 * block_table holds (max_blocks * page_size) within 2^29 and 2^30, and so many units of work as the
 * call could have by its sizes, whatever the lengths are, within 31 bits: with G = n_q_heads /
 * n_kv_heads,
 *     (total_rows * G / 16 + B + 1) * n_kv_heads * (max(max_blocks * page_size, shared_len) / 32 + 8).
 * 65536 rows of 32 / 8 heads, for instance, fit tables of 131072 positions, and not of a million: bring
 * fewer rows at a time or a narrower table. */

/* Bytes of workspace spec_attend needs for these arguments (only the sizes are read; 0 when they are
 * invalid). 256-byte aligned; its contents need no preparation. Calls that share a workspace must
 * not overlap on the GPU. */
size_t spec_attend_workspace_size(const spec_attend_args *args);

/* Enqueues the attention kernel (one more for the shared prefix) and the joining kernel on `stream`.
 * q, out and the cache must start every head's row on a 16-byte boundary (base pointers and strides),
 * else SPEC_ERR_UNSUPPORTED. */
spec_status spec_attend(const spec_attend_args *args, void *workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* The kernel that serves the requests' own positions for these arguments (a static string; a shared
 * prefix, with the rows of the whole batch, may take the one for more rows), or NULL when they are
 * invalid. A diagnostic: it enqueues nothing. */
const char *spec_attend_plan(const spec_attend_args *args);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_ATTEND_H */
