/* A paged key/value cache held in 4 bits, and attention over it, on gfx950:
 * the cache of paged_attn.h in 0.27 of the bytes, on the same block table,
 * slots and lengths (rglru_page_plan serves both).
 *
 * A head's row of D elements is D / 32 blocks of 32. A block is a power of two
 * and 32 codes of 4 bits (the FP4 blocks of the OCP microscaling formats):
 *
 *   codes  [n_pages, Hkv, page_size, D / 2] bytes: element 2i of a row in the
 *          low half of byte i, element 2i + 1 in the high half; a code is a sign
 *          (bit 3) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (bits 0 to 2, in order);
 *   scales [n_pages, Hkv, page_size, D / 32] bytes: b stands for 2^(b - 127),
 *          255 for a block that holds an infinity or a NaN and reads as NaN.
 *
 * An element's value is its code times its block's power: exact in bf16 and
 * in float32. The write takes the smallest power, from 2^-126 to 2^125, that
 * takes the block's largest magnitude to 6 or less, divides (exactly) and
 * rounds to the nearest code, a half to the even one, magnitudes past 6 times
 * 2^125 to that; a block that is not finite gets codes 0. It writes bytes 1 to
 * 252 and 255; what 253 and 254 give is unspecified where a value passes bf16.
 *
 * Conventions (streams, ownership, statuses) and limits are those of rglru.h
 * and paged_attn.h; io_dtype is that of k, v, q and o.
 */
#ifndef RGLRU_PAGED_Q4_H_
#define RGLRU_PAGED_Q4_H_

#include "paged_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The new tokens' keys and values into the cache, as rglru_paged_kv_write: row t
 * to slot slot_map[t], every head; a slot below 0 or past the cache is skipped,
 * slots are distinct otherwise, no other row of the cache is touched.
 *
 *   k, v                 : [T, Hkv, D] io, rows kv_stride apart, 16-byte aligned.
 *   k_codes, v_codes, k_scales, v_scales : as above, each 16-byte aligned.
 *   slot_map             : [T] int32.
 * At most 2^36 - 2^12 bytes of keys a call. Reads the shape's n_tokens, n_pages,
 * page_size, kv_heads, head_dim (any multiple of 32 here; others are
 * RGLRU_ERR_UNSUPPORTED), io_dtype and kv_stride. */
rglru_status_t rglru_paged_kv_write_q4(const rglru_paged_shape_t* shape, const void* k, const void* v, uint8_t* k_codes,
                                       uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, const int32_t* slot_map,
                                       void* stream);

/* The values of rows of the cache: row t of k and v (io, dense, kv_stride is
 * not read) gets those of slot slot_map[t], 0 for a slot below 0 or past the
 * cache. Slots may repeat. Arguments and limits otherwise as above. */
rglru_status_t rglru_paged_kv_read_q4(const rglru_paged_shape_t* shape, const uint8_t* k_codes, const uint8_t* k_scales,
                                      const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* slot_map, void* k,
                                      void* v, void* stream);

/* Attention of the new tokens over a 4-bit cache: the formula, the masks and
 * all that is said of rglru_paged_attn_fwd, with k_j and v_j the values of the
 * cache (so a key or value that is not finite is NaN). q . k is formed with
 * the values as they are and q as it is (float32 queries in three bf16 parts,
 * which hold all of their bits), in float32. For bf16 the softmax weights are
 * rounded to bf16 where they enter the product with the values; for float32
 * they enter in three bf16 parts. Weights of 2^-80 of a row's largest and less
 * may count as nothing, beside a NaN too.
 *
 *   k_codes, k_scales, v_codes, v_scales : as above, each 16-byte aligned.
 *   workspace : rglru_paged_attn_q4_workspace_bytes(shape) bytes, 256-byte aligned:
 *               up to 203 MB whatever the lengths (what is used of it is a few MB in
 *               a decode step), 40 bytes for every 128 rows of n_tokens * q_heads /
 *               kv_heads (256 in bf16), 48 for every sequence and 8 for every key
 *               head of one. Calls that share one must not overlap in time.
 * Everything else as for rglru_paged_attn_fwd. */
size_t rglru_paged_attn_q4_workspace_bytes(const rglru_paged_shape_t* shape);
rglru_status_t rglru_paged_attn_q4_fwd(const rglru_paged_shape_t* shape, const int32_t* cu_seqlens, const int32_t* kv_lens,
                                       const int32_t* block_table, const void* q, const uint8_t* k_codes,
                                       const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales, void* o,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif  /* RGLRU_PAGED_Q4_H_ */
