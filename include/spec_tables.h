/*
 * spec_tables.h - C ABI of the paged cache's bookkeeping for GB300 (sm_103a): block tables brought to the
 * requests' lengths on the device, and the slots of a round's rows.
 *
 * Before the target's pass a round needs pages for its rows; after the verification the length is what was
 * accepted, and pages behind it can go back. Both are one call here, on lengths that the device knows
 * (spec_compact's new_kv_len, for instance), so that a round needs no answer from the host in between. The block
 * table, the pages and the ragged rows are those of spec_compact and spec_attend.h ("M7.8 - Speculative
 * Serving", sections 0x03C and 0x08A, define KV rows by them; who hands the pages out is left to the server). The
 * conventions of spec_verify.h hold.
 */
#ifndef SPEC_TABLES_H
#define SPEC_TABLES_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- spec_block_tables -------------------------------------------------------------------
 * Request i holds n_blocks[i] pages, entries 0 .. n_blocks[i]-1 of its row of block_table, and shall hold
 * need = ceil(kv_len[i] / page_size). The pages nobody holds are a stack, free_pages[0 .. n_free-1]. The first
 * n_shared entries of every row are the pages of shared_table (a prefix that all requests share): they are
 * copied from there when a request comes to hold them, and never taken from the stack or given back.
 *
 * First, requests that hold too many give their last entries back, the last request's last entry first; then
 * those that hold too few take from the top of the stack, the first request's first new entry first. So the
 * order depends on nothing but the arguments, and giving back undoes taking: two calls, to new lengths and
 * back again, leave the stack as it was. Entries behind need keep what they hold, and mean nothing.
 *
 * Then row r of the batch, at position p = kv_len[i] - n_i + j of its request i (rows row_off[i] ..
 * row_off[i+1]-1, as for spec_attend), gets positions[r] = p and
 *     slot_map[r] = block_table[i][p / page_size] * page_size + p % page_size,
 * the physical rows that spec_compact takes as cand_kv_rows (for the drafts' rows). Padding rows (p < 0) get -1 in both,
 * and so do the rows of a request whose offsets are contradicted (row_off[i] .. row_off[i+1]-1, if 0 <= row_off[i] <=
 * row_off[i+1] <= T); rows of a request with other status bits get -1 in slot_map. Rows of no request, those beside an
 * offset outside [0, T] among them, are not written: they keep what the arrays held before.
 *
 * A request with status bits keeps its pages as they are:
 *   SPEC_REQ_BAD_SHAPE   a negative kv_len, n_blocks outside [0, max_blocks]; or offsets that are wrong or
 *                        contradicted (its pages are brought to its length all the same);
 *   SPEC_REQ_BAD_BLOCKS  need above max_blocks; the stack ran out before it (pages are handed out request after
 *                        request: from the first that does not fit on, those that need pages get none); or a stack
 *                        that cannot be right: n_free outside [0, n_pages], or more than n_pages with what comes
 *                        back (then nobody gives any back).
 * Page numbers are not looked at, except that slot_map is -1 for one outside [0, n_pages). */
typedef struct {
    int32_t B, total_rows;       /* total_rows 0: tables only                                    */
    int32_t page_size, max_blocks, n_pages;
    int32_t n_shared;            /* 0 .. max_blocks                                              */
    const int32_t *kv_len;       /* [B]                                                         */
    const int32_t *row_off;      /* [B+1]; NULL when total_rows = 0                              */
    const int32_t *shared_table; /* [n_shared]; NULL when n_shared = 0                           */
    int32_t *n_blocks;           /* [B] in and out                                               */
    int32_t *block_table;        /* [B][max_blocks] in and out                                   */
    int32_t *free_pages;         /* [n_pages] in and out                                         */
    int32_t *n_free;             /* device scalar, in and out                                    */
    int32_t *slot_map;           /* [T] out (may be NULL)                                        */
    int32_t *positions;          /* [T] out (may be NULL)                                        */
    int32_t *req_status;         /* [B] out: SPEC_REQ_* bits (may be NULL)                       */
} spec_block_tables_args;

/* Bytes of workspace for these sizes (0 when they are invalid), 256-byte aligned, no preparation. Calls that
 * share a workspace must not overlap on the GPU. */
size_t spec_block_tables_workspace_size(const spec_block_tables_args *args);

/* Enqueues one kernel on `stream`, or two (more than 512 requests, 2048 rows or 65536 entries of block_table).
 * SPEC_ERR_UNSUPPORTED when total_rows or B * max_blocks exceeds 2^31 - 2^19, or n_pages * page_size 2^31 - 1. */
spec_status spec_block_tables(const spec_block_tables_args *args, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_TABLES_H */
