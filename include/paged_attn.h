/* Attention over a paged key/value cache for packed serving batches, on
 * gfx950: the attention layers that stand between the recurrent ones in a
 * hybrid model, on the same packed batch (cu_seqlens) as rglru_fwd_varlen and
 * rglru_delta_rule_fwd.
 *
 * A cache is two arrays of pages, [n_pages, Hkv, page_size, D] each (keys and
 * values, D contiguous). A sequence's pages are named by its row of the block
 * table; token j of sequence n lives in page block_table[n][j / page_size] at
 * offset j % page_size, its slot being page * page_size + offset. A step:
 *
 *   rglru_page_plan        from the request lengths: pages taken from and
 *                          given back to a free list, block table, slot map
 *   rglru_paged_kv_write   the new tokens' keys and values into their slots
 *   rglru_paged_attn_fwd   the new tokens' queries over the cache
 *
 * All lengths are read on the device, so a step can be captured in a HIP graph
 * and replayed with other lengths (n_tokens and n_seqs are then capacities).
 * Conventions (streams, ownership, statuses) are those of rglru.h; none of
 * these entry points needs initial workspace contents.
 */
#ifndef RGLRU_PAGED_ATTN_H_
#define RGLRU_PAGED_ATTN_H_

#include "rglru.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits beyond which a call returns RGLRU_ERR_INVALID_ARGUMENT (an entry
 * point checks the fields it reads): 0 <= n_tokens < 2^31; 1 <= n_seqs <=
 * 2^16; page_size a power of two from 8 to 1024; n_pages >= 1 with n_pages *
 * page_size < 2^31; max_pages >= 1 with max_pages * page_size <= 2^31 -
 * 2^16; 1 <= kv_heads <= q_heads <= 2^14 with q_heads a multiple of
 * kv_heads; n_tokens * q_heads <= 2^31 - 2^16; head_dim >= 1; io_dtype an
 * rglru_io_t; max_new, window >= 0; |scale| <= 2.35e38 (times log2 e it has
 * to be finite); strides 0 or at least the dense row. Within them, a
 * head_dim other than 64, 128 or 256 is RGLRU_ERR_UNSUPPORTED, and a stride
 * that is not a multiple of 16 bytes RGLRU_ERR_MISALIGNED. An output (what
 * is updated in place and the workspace too) that overlaps another one or an
 * input is RGLRU_ERR_INVALID_ARGUMENT; strided rows count from the first
 * one's start to the last one's end. */
typedef struct {
  int64_t n_tokens;   /* T: rows of the packed batch (a capacity: rows from cu_seqlens[n_seqs] on are padding) */
  int64_t n_pages;    /* pages of the cache */
  int32_t n_seqs;     /* N */
  int32_t max_pages;  /* columns of the block table */
  int32_t page_size;  /* tokens of a page */
  int32_t q_heads;    /* Hq */
  int32_t kv_heads;   /* Hkv; query head h reads key head h / (Hq / Hkv) */
  int32_t head_dim;   /* D */
  int32_t io_dtype;   /* rglru_io_t of q, k, v, o and the cache */
  int32_t max_new;    /* most new tokens of any one sequence; 0: not known. A sequence with more gives
                         unspecified (in-bounds) results */
  int32_t window;     /* 0: a query sees every key up to its own; w > 0: the last w of them */
  float scale;        /* factor on the scores */
  int64_t q_stride;   /* elements from one token of q to the next; 0: dense (Hq * D) */
  int64_t kv_stride;  /* the same for k and v of rglru_paged_kv_write; 0: dense (Hkv * D) */
} rglru_paged_shape_t;

/* Block table and slot map of a step, from the request lengths. With have_n =
 * ceil(held_lens[n] / page_size) pages in row n, new_n = cu_seqlens[n + 1] -
 * cu_seqlens[n] and need_n = ceil((context_lens[n] + new_n) / page_size):
 *
 *   - columns need_n .. have_n - 1 of every row (a finished request, with
 *     context 0 and no new tokens, or rejected tokens) give their pages back:
 *     pushed on the free list in the order of sequences, then columns;
 *   - then columns have_n .. need_n - 1 get pages popped from the free list, in
 *     the same order (the page given back last goes first). A sequence is
 *     served if its row has need_n columns and the list still holds its pages
 *     after all sequences before it asked for theirs; one that is not served
 *     takes none and its row is left as it was. cu_seqlens still counts its
 *     tokens: they have slot -1, the write skips them, and rglru_paged_attn_fwd on
 *     this step's lengths gives their rows unspecified values (it takes them to
 *     stand at the context's end), which the caller drops wherever slot_map is -1.
 *
 *   context_lens : [N] int32, tokens in the cache before the step, at most held_lens.
 *   held_lens    : [N] int32, tokens the row's pages were taken for (the last
 *                  step's held_lens_out), or NULL for context_lens.
 *   cu_seqlens   : [N + 1] int32, 0 = cu[0] <= ... <= cu[N] <= T.
 *   block_table  : [N, max_pages] int32, in and out.
 *   free_pages   : [n_pages] int32, in and out: a stack, its first
 *                  free_count[0] entries are free pages, the last on top.
 *   free_count   : [1] int32.      free_count_out : [1] int32, the new count.
 *   slot_map     : [T] int32 out: each new token's slot; -1 for the tokens of
 *                  a sequence that was not served and for padding rows.
 *   positions    : [T] int32 out: each new token's position, -1 likewise.
 *   kv_lens      : [N] int32 out: context + new, or the context alone if not served.
 *   held_lens_out: [N] int32 out: context + new, or held_lens as it was if not served.
 *   unserved     : [1] int32 out: sequences that were not served.
 *
 * All pointers 4-byte aligned. Reads the shape's n_tokens, n_pages, n_seqs,
 * max_pages, page_size and max_new. Lengths outside what is said above give
 * unspecified results, every access staying in bounds. */
rglru_status_t rglru_page_plan(const rglru_paged_shape_t* shape, const int32_t* context_lens,
                               const int32_t* held_lens, const int32_t* cu_seqlens, int32_t* block_table,
                               int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                               int32_t* slot_map, int32_t* positions, int32_t* kv_lens, int32_t* held_lens_out,
                               int32_t* unserved, void* stream);

/* The new tokens' keys and values into the cache: row t of k and v goes to
 * slot slot_map[t], every head. A slot below 0 or past the cache is skipped;
 * slots are distinct otherwise (of two rows with one slot, which one stays is
 * unspecified, piece by piece). No other row of the cache is touched.
 *
 *   k, v             : [T, Hkv, D] io, rows kv_stride apart, 16-byte aligned.
 *   k_cache, v_cache : [n_pages, Hkv, page_size, D] io, 16-byte aligned.
 *   slot_map         : [T] int32.
 * At most 2^36 - 2^12 bytes of keys a call. Reads the shape's n_tokens, n_pages,
 * page_size, kv_heads, head_dim (any multiple of 16 bytes here), io_dtype and
 * kv_stride. */
rglru_status_t rglru_paged_kv_write(const rglru_paged_shape_t* shape, const void* k, const void* v, void* k_cache,
                                    void* v_cache, const int32_t* slot_map, void* stream);

/* Attention of the new tokens. Row i of sequence n (i < new_n) stands at
 * position p = kv_lens[n] - new_n + i and sees the keys j of its sequence with
 * max(0, p - window + 1) <= j <= p (from 0 without a window); the new tokens'
 * own keys are in the cache already:
 *
 *   o   = sum_j softmax_j(scale q . k_j) v_j        lse = ln sum_j exp(scale q . k_j)
 *
 * with q . k, scores, softmax and sums in float32, the scale applied to q . k.
 * A row that sees no key (p < 0, or all its scores -inf) gets o = 0 and lse =
 * -inf; one with a score of +inf or NaN gets NaN in both. What a row does not
 * see has no influence on it, infinities and NaN included (at given lengths
 * not on a bit of it); padding rows of o and lse are left as they were.
 * Weights of 2^-118 of a row's largest and less, the 0 of a score of -inf
 * among them, may count as nothing: a finite value adds nothing there, an
 * infinite one gives infinity or NaN. Sums are formed with weights up to 2^8
 * and divided at the end, so of n visible values none should pass 3.4e38 /
 * (2^8 n), or they may overflow. For bf16 the softmax weights are rounded to
 * bf16 where they enter the product with the values (2^-8 relative at most).
 * The same call gives the same bits each time.
 *
 *   cu_seqlens       : [N + 1] int32 as above.       kv_lens : [N] int32, new tokens included.
 *   block_table      : [N, max_pages] int32; pages outside the cache give
 *                      unspecified (in-bounds) results.
 *   q                : [T, Hq, D] io, rows q_stride apart, 16-byte aligned.
 *   k_cache, v_cache : [n_pages, Hkv, page_size, D] io, 16-byte aligned.
 *   o                : [T, Hq, D] io, dense, 16-byte aligned.
 *   lse              : NULL or [T, Hq] float32.
 *   workspace        : rglru_paged_attn_workspace_bytes(shape) bytes, 256-byte
 *                      aligned: up to 153 MB (D = 256 in bf16, prompt chunks among
 *                      more than 16 sequences) whatever the lengths, 40 bytes for
 *                      every 128 rows of n_tokens * q_heads / kv_heads (256 in
 *                      bf16) and 48 for every sequence. Calls that share one must
 *                      not overlap in time. */
size_t rglru_paged_attn_workspace_bytes(const rglru_paged_shape_t* shape);
rglru_status_t rglru_paged_attn_fwd(const rglru_paged_shape_t* shape, const int32_t* cu_seqlens,
                                    const int32_t* kv_lens, const int32_t* block_table, const void* q,
                                    const void* k_cache, const void* v_cache, void* o, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif  /* RGLRU_PAGED_ATTN_H_ */
