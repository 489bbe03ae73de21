/*
 * attn_pages.h -- C ABI of the page bookkeeping of libattn_decode.so: growing,
 * shrinking, freeing and forking the sequences of a paged cache, on the device, so
 * that a captured decode step can do it too.
 *
 * The conventions of attn_decode.h and attn_paged.h hold. One bookkeeping serves the
 * caches of all layers that use the same page numbers:
 *   refs         int32 [n_pages], 16-byte aligned: how many block-table entries
 *                hold the page; 0: free
 *   block_table  int32 [n_seq][max_pages]; a sequence of r rows holds its entries
 *                [0, ceil(r / page_size))
 * Calls on one bookkeeping are ordered by their stream; two at once are not
 * defined. Pages are given out in the order of their numbers, lowest first, so
 * that equal calls give equal tables.
 */
#ifndef ATTN_PAGES_H
#define ATTN_PAGES_H

#include "attn_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* There were fewer free pages than a call needed: the entries without one are -1. */
#define ATTN_DEVERR_NO_PAGE 0x10u
/* A sequence was cut inside a page that others hold too: an append would write to it. */
#define ATTN_DEVERR_SHARED_PAGE 0x20u

/*
 * attn_pages_resize -- from have[s] to want[s] rows for every sequence, in one
 * launch. First the entries past want[s] are released: one holder less, the entry -1;
 * then entries are filled up to want[s], by sequence and entry, with the lowest-numbered
 * free pages, those just released among them. want[s] = 0 frees a sequence.
 *   have, want  int32 [n_seq]; values outside [0, max_pages * page_size] are
 *               clamped (ATTN_DEVERR_POSITION_CLAMPED)
 *   n_seq       at most 8192, n_seq * max_pages below 2^31
 * An entry to release that is no held page of the pool sets ATTN_DEVERR_BAD_PAGE
 * (an entry of -1, of a page that was not to be had, is passed over), too few free
 * pages ATTN_DEVERR_NO_PAGE, and a sequence that is cut to a row inside a page with
 * other holders ATTN_DEVERR_SHARED_PAGE.
 */
attn_status attn_pages_resize(int32_t *refs, int n_pages, int32_t *block_table, int max_pages, int page_size,
                              const int32_t *have, const int32_t *want, int n_seq, attn_stream_t stream);

/*
 * attn_pages_fork -- sequence dst[i] becomes a copy of the first rows[i] rows of
 * sequence src[i]: it holds src's full pages too, and where rows[i] ends inside a page
 * it gets a page of its own, the lowest-numbered free one, by i, into which
 * attn_pages_copy brings the rows.
 *   src, dst, rows  int32 [n_fork], n_fork <= 4096. dst[i] holds no page before (its
 *                   entries are not looked at, and those past the rows not written)
 *   copies          int32 [n_fork][4], 16-byte aligned, written: (source page, page,
 *                   rows to copy, 0), or (-1, -1, 0, 0) where there is nothing to
 *                   copy -- the pages attn_pages_copy takes, for every layer's cache
 * A src or dst outside [0, n_seq), equal ones, or rows outside
 * [0, max_pages * page_size] set ATTN_DEVERR_BAD_REQUEST, and that fork is
 * skipped; so are, of the others, all whose dst is dst of another or src of one. An entry of src that is no page is shared as -1 (ATTN_DEVERR_BAD_PAGE); no
 * free page: the entry is -1 (ATTN_DEVERR_NO_PAGE).
 */
attn_status attn_pages_fork(int32_t *refs, int n_pages, int32_t *block_table, int max_pages, int page_size,
                            int n_seq, const int32_t *src, const int32_t *dst, const int32_t *rows, int n_fork,
                            int32_t *copies, attn_stream_t stream);

/*
 * attn_pages_copy -- rows [0, rows) of pages, K and V, with the pages' scales, from
 * one page of the pool to another.
 *   copies  int32 [n][4], 16-byte aligned: (from, to, rows, not looked at). to < 0 or
 *           rows <= 0: nothing. Rows past page_size are not there.
 * A page outside the pool sets ATTN_DEVERR_BAD_PAGE, and nothing is copied for
 * it. No page is written twice, or written and read, by one call.
 */
attn_status attn_pages_copy(const attn_paged_cache *cache, const int32_t *copies, int n, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PAGES_H */
