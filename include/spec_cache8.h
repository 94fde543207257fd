/*
 * spec_cache8.h - C ABI of the paged cache held in 8 bits for GB300 (sm_103a): appending a round's keys
 * and values to it with their position rotation, and attention of the round's rows over it.
 *
 * The ragged batch, the pages, the block tables and all conventions are those of spec_attend.h. The cache's
 * elements are e4m3 (sign, four bits of exponent, three of mantissa; no infinity), strides of the cache
 * count elements (bytes), and each page has a scale for each key/value head, of its keys and of its values:
 * element d of head h, slot s, page b stands for
 *     cache[b * page_stride + s * slot_stride + h * head_stride + d] * scale[b * n_kv_heads + h].
 * One byte an element instead of two halves what a round reads; the scale follows each page's and head's
 * magnitude, so that e4m3's three bits of mantissa are all that is lost. The pages this library follows know no
 * such cache ("M7.8 - Speculative Serving", section 0x08A, leaves the target's cache to the model).
 */
#ifndef SPEC_CACHE8_H
#define SPEC_CACHE8_H

#include "spec_attend.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- spec_kv_append8 ---------------------------------------------------------------------
 * spec_kv_append into the 8-bit cache: the same rows are written (to q_out: rounded once to their type; to the
 * cache: x / scale rounded to the nearest e4m3, x formed in 32 bits), the same rows and requests are left out,
 * and the same status bits say so. append.k_cache and append.v_cache are the e4m3 arrays.
 *
 * Scales. Let a be the largest magnitude of the call's finite values in one page and head, and
 * need = the least power of two s with a <= 448 s, at least 2^-60. A page that holds no earlier position of the
 * request gets the scale `need`; one that does (the call's first position lies inside it) keeps its own scale if
 * that is larger, else gets `need`, and the earlier positions' elements are brought to it: each becomes the e4m3
 * nearest to element * (old scale / new scale), which is exact (a power of two) down to elements of 2^-6. A scale does
 * not shrink again: a row that is refused later (a draft) has raised it for good, and what the page's other positions lose
 * follows the loudest row appended to it, accepted or not. (Elements of 2^-14 of its largest and more lose nothing.) Slots
 * behind the call's last position mean nothing afterwards (drafts that were refused, for instance). A value that is not
 * finite becomes NaN and leaves the scale alone. (Keys above 448 * 2^60 and values above 448 * 2^30 get scales beyond what
 * spec_attend8 takes.)
 *
 * Rows of one call must not share a page unless they are one request's (a page has one scale: what two requests
 * appending to one page in the same call leave there is not defined). Prefixes are shared in whole pages, or
 * with a copy of the last one for each request. */
typedef struct {
    spec_kv_append_args append;
    float *k_scale, *v_scale;    /* [n_pages][n_kv_heads]                                        */
} spec_kv_append8_args;

/* Enqueues one kernel on `stream`. Any strides and alignments are served; rows and caches whose bases are on
 * 16-byte boundaries and whose strides, head_dim and rot_dim are multiples of 8 (bf16) or 4 (fp32) elements (without
 * interleaving rot_dim of twice that) take the vectorised kernel. SPEC_ERR_UNSUPPORTED beyond 2^20 rows, pages of
 * 2^16 slots, or (2 B + total_rows / page_size) * 2 n_kv_heads + total_rows + B of 2^30. */
spec_status spec_kv_append8(const spec_kv_append8_args *args, cudaStream_t stream);

/* ---- spec_attend8 ------------------------------------------------------------------------
 * spec_attend over the 8-bit cache: the same rows see the same positions (window, sinks, shared prefix), with
 *     k_x = k_scale * element, v_x = v_scale * element.
 * attend.dtype is the type of q and out; attend.k_cache and attend.v_cache are the e4m3 arrays. Scales are
 * finite, positive, those of keys within 2^-60 .. 2^60, those of values within 2^-60 .. 2^30 (they need not be powers of
 * two); a page whose scale is not so spoils the rows that see one of its positions, and no others. Elements that are NaN
 * give those rows what the formulas say, and no others.
 *
 * Head sizes above 128, pages that are no multiple of 8 slots, and caches whose heads lie neither side by side in a
 * slot nor a whole number of slots apart: the fp32 units, 32-bit arithmetic throughout (out is rounded once).
 * Otherwise products on the tensor cores, with 32-bit accumulation, which cuts sums off instead of rounding them; q
 * and the weights enter as sums of 8-bit parts. Scores, statistics, the weights' sum and lse are 32-bit.
 *   A query is divided by the power of two that brings its head's largest element between 224 and 448.
 *   bf16: e4m3 and e5m2, exact for elements from 2^-13 of the largest on, off by at most 2^-21 of the largest below.
 *   fp32: four e4m3, off by at most 2^-19 of the element, or 2^-25 of the largest.
 *   Weights, bf16 with up to 48 packed rows (rows times n_q_heads / n_kv_heads) a request on average: three e5m2 of the
 *   weight times its position's v_scale, off by at most 2^-11 of itself, or 2^-27 of the row's reference.
 *   bf16 with more, and the shared prefix with more rows in all: a 16-bit float of that product, off by 2^-11 of itself, or
 *   2^-32 of the row's reference; e4m3 is a 16-bit float, so values are exact.
 *   fp32: six e5m2, off by at most 2^-22 of itself, or 2^-38 of the reference; sums leave the tensor cores every
 *   256 positions. (Random batches: off from 64 bits by 7e-7 of the outputs' size; a plain 32-bit form 1.1e-6.)
 * A position adds less than 2^-32 to a row's sum of weights, relative to it, or is counted, whatever scales within the
 * range the others have. In bf16 a sum of n terms of one sign, all taken by one worker, loses about n 2^-27 of itself
 * by being cut off.
 * Results do not depend on the order in which CTAs run. */
typedef struct {
    spec_attend_args attend;
    const float *k_scale, *v_scale; /* [n_pages][n_kv_heads]                                     */
} spec_attend8_args;

/* As for spec_attend, whose limits hold too; head_dim is a multiple of 16, and every head's row of the cache starts
 * on a 16-byte boundary, else SPEC_ERR_UNSUPPORTED. */
size_t spec_attend8_workspace_size(const spec_attend8_args *args);
spec_status spec_attend8(const spec_attend8_args *args, void *workspace, size_t workspace_bytes, cudaStream_t stream);
const char *spec_attend8_plan(const spec_attend8_args *args);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_CACHE8_H */
