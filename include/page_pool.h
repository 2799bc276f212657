/* A pool of cache pages that several requests share, on gfx950: rows of a
 * block table go on from each other's context (fork), give pages up (free),
 * and the pages in use move to the front of the pool (compact). These three
 * work on the table, the free list and the counts of sharing; page contents
 * follow by rglru_page_copy, for any number of caches (keys and values, codes
 * and scales, every layer) that live under the same table.
 *
 * A pool is what rglru_page_plan keeps (block_table [N, max_pages], free_pages
 * [n_pages] with free_count [1], the tokens held_lens [N] that each row's pages
 * were taken for) and shares [n_pages] int32: the rows that hold a page beyond
 * the first, so 0 for a page of one row and for a free one, and all 0 at the
 * start. Only whole pages of tokens that will not change are shared, so
 * rglru_page_plan and the writes work on as they are, under one rule: once a
 * row has been forked, from or to, it does not go back (by the plan) to fewer
 * tokens than were shared, and it ends by rglru_page_free, not by the plan.
 *
 * All lengths are read on the device. All int32 arrays are 4-byte aligned;
 * an output (what is updated in place and the workspace too) that overlaps
 * another one or an input is RGLRU_ERR_INVALID_ARGUMENT. Lengths, table
 * entries and counts outside what is said give unspecified results, every
 * access staying in bounds. The shape's n_pages, n_seqs, max_pages and page_size
 * are read, with the limits of paged_attn.h.
 */
#ifndef RGLRU_PAGE_POOL_H_
#define RGLRU_PAGE_POOL_H_

#include "paged_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row n with fork_from[n] = s >= 0 goes on from the first lens[s] tokens of row
 * s. Its pages that are full of them are shared (named in both rows, shares
 * + 1); where the last one is not full, a fresh page is popped from the free list in
 * the order of the rows, and pairs[n] says which page to copy to which. A row
 * is served if s is another row that is not forked itself in this call, row n
 * holds nothing (lens and held_lens 0) and, where it needs a page, the
 * list still has one after all rows before it asked; any other is left as it was
 * and counted in unserved. Rows with fork_from < 0 are left as they were.
 * What belongs to a row and not to its pages, the state of a recurrent layer, is the
 * caller's to take along, for the rows whose lens_out is more than lens: with pairs
 * (fork_from[n], n) for those and -1, -1 for the others, rglru_page_copy does it over
 * the states of all layers (n_pages = N, a row a page).
 *
 *   fork_from     : [N] int32.
 *   lens          : [N] int32, tokens of every row (those that a fork takes over).
 *   held_lens     : [N] int32, or NULL for lens.
 *   block_table   : [N, max_pages] int32, in and out (the forked rows).
 *   shares        : [n_pages] int32, in and out.
 *   free_pages    : [n_pages] int32, read.       free_count : [1] int32.
 *   pairs         : [N, 2] int32 out: the page to copy and the page it goes to,
 *                   -1, -1 for a row that needs no copy.
 *   lens_out, held_lens_out : [N] int32 out: lens[s] for a row that was served,
 *                   as they were for the others.
 *   free_count_out: [1] int32 out.               unserved : [1] int32 out. */
rglru_status_t rglru_page_fork(const rglru_paged_shape_t* shape, const int32_t* fork_from, const int32_t* lens,
                               const int32_t* held_lens, int32_t* block_table, int32_t* shares, const int32_t* free_pages,
                               const int32_t* free_count, int32_t* pairs, int32_t* lens_out, int32_t* held_lens_out,
                               int32_t* free_count_out, int32_t* unserved, void* stream);

/* Row n gives up the pages behind its first keep_lens[n] tokens: columns
 * ceil(keep / page_size) .. ceil(held / page_size) - 1. A page that other
 * rows hold stays with them (shares - 1 for every row that gives it up); one that
 * nobody holds any more goes onto the free list: those of one call in descending
 * order, so that the first page of the pool among them comes off first.
 * A row that goes back to inside a page that other rows hold (fewer tokens than were
 * shared, and not a multiple of page_size) keeps it shared: it may be read and
 * forked from, but no new token of it may be written.
 *
 *   keep_lens     : [N] int32; held_lens or more keeps all, 0 ends the request.
 *   held_lens     : [N] int32.
 *   block_table   : [N, max_pages] int32, read (columns given up are left as they are).
 *   shares        : [n_pages] int32, in and out.
 *   free_pages    : [n_pages] int32, in and out.  free_count : [1] int32.
 *   held_lens_out : [N] int32 out: the smaller of keep_lens (0 for less) and held_lens.
 *   free_count_out: [1] int32 out.
 *   workspace     : rglru_page_free_workspace_bytes(shape) bytes, 16-byte aligned. */
size_t rglru_page_free_workspace_bytes(const rglru_paged_shape_t* shape);
rglru_status_t rglru_page_free(const rglru_paged_shape_t* shape, const int32_t* keep_lens, const int32_t* held_lens,
                               const int32_t* block_table, int32_t* shares, int32_t* free_pages, const int32_t* free_count,
                               int32_t* held_lens_out, int32_t* free_count_out, void* workspace, size_t workspace_bytes,
                               void* stream);

/* The pool shrinks to its first keep_pages pages (0 <= keep_pages <= n_pages):
 * of the pages from keep_pages on that rows hold, the i-th in order moves to the
 * i-th of the free ones before it, as long as there are any. Pages from
 * keep_pages on leave the free list (one that could not be moved comes back
 * to it when it is freed). With keep_pages no less than the pages in use all move,
 * and what lies behind can be given away once rglru_page_copy is done.
 *
 *   held_lens     : [N] int32; columns before ceil(held / page_size) name pages in use.
 *   block_table, shares, free_pages, free_count : as above, read.
 *   block_table_out : [N, max_pages] int32 out: the new pages; other columns as they were.
 *   shares_out    : [n_pages] int32 out: moved along, 0 for a page that was left.
 *   free_pages_out: [n_pages] int32 out: the free pages before keep_pages in descending
 *                   order, then -1.             free_count_out : [1] int32 out.
 *   pairs         : [min(keep_pages, n_pages - keep_pages), 2] int32 out: the moves in order
 *                   (from, to), then -1, -1; NULL where there is no room for one.
 *   n_pairs       : [1] int32 out, the moves.    unmoved : [1] int32 out, pages that
 *                   found no place.
 *   workspace     : rglru_page_compact_workspace_bytes(shape) bytes, 16-byte aligned. */
size_t rglru_page_compact_workspace_bytes(const rglru_paged_shape_t* shape);
rglru_status_t rglru_page_compact(const rglru_paged_shape_t* shape, int64_t keep_pages, const int32_t* held_lens,
                                  const int32_t* block_table, const int32_t* shares, const int32_t* free_pages,
                                  const int32_t* free_count, int32_t* block_table_out, int32_t* shares_out,
                                  int32_t* free_pages_out, int32_t* free_count_out, int32_t* pairs, int32_t* n_pairs,
                                  int32_t* unmoved, void* workspace, size_t workspace_bytes, void* stream);

/* Copies pages within caches: for every pair, page pairs[i][0] to page
 * pairs[i][1] of every array. Pairs with a page below 0 or past the pool are
 * skipped. No page is the target of two pairs, or the source of one and the
 * target of another; which contents it gets is unspecified otherwise.
 *
 *   n_pages    : pages of every array, 1 to 2^31 - 1.
 *   pairs      : [max_pairs, 2] int32.
 *   count      : [1] int32, the pairs to look at, or NULL for max_pairs.
 *   arrays     : n_arrays (1 to RGLRU_PAGE_COPY_ARRAYS) pointers, read on the host, to
 *                arrays of n_pages pages, each 16-byte aligned.
 *   page_bytes : [n_arrays] on the host, a multiple of 16 up to 2^31 - 16 each, those of
 *                all arrays together as well. */
#define RGLRU_PAGE_COPY_ARRAYS 64
rglru_status_t rglru_page_copy(int64_t n_pages, const int32_t* pairs, int64_t max_pairs, const int32_t* count,
                               int32_t n_arrays, void* const* arrays, const int64_t* page_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif  /* RGLRU_PAGE_POOL_H_ */
