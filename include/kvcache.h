/*
 * kvcache.h - C ABI of the paged MXFP4 key-value cache of the MI355X (gfx950)
 * library: block tables and slots of new tokens, writing and reading of the
 * cache, and the attention of queries over it.
 *
 * The conventions of mxfp8.h hold here too: device pointers, a hipStream_t
 * passed as void*, validation on the host before anything is launched, no
 * allocation, no synchronisation, no fallback, and the same status codes.
 * Results do not depend on the order in which workgroups run.
 *
 * The cache holds `pages` pages of `page_size` tokens for each of kv_heads heads
 * of head_dim values.  Token t of page p has slot p * page_size + t.  A value is
 * MXFP4 (mxfp4.h) with blocks of 32 along the head.  A page and head is a record
 * of page_size * (head_dim + head_dim / 16) bytes, records [pages][kv_heads]:
 *   keys' codes    [page_size][head_dim / 2]
 *   values' codes  [page_size / 4][head_dim / 8][4 tokens][4 bytes]
 *   keys' scales   [page_size][head_dim / 32]
 *   values' scales [head_dim / 32][page_size]
 * page_size: 16, 32, 64, 128 or 256; head_dim: 64, 128 or 256; cache 16-byte
 * aligned; pages >= 1, pages * page_size < 2^31.
 */
#ifndef MXFP8_KVCACHE_H
#define MXFP8_KVCACHE_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Room for counts[b] new tokens behind the lengths[b] that request b has in the
 * cache, for b < requests (negative numbers count as 0):
 *   offsets[b]     the row of b's first new token (offsets[requests]: all rows,
 *                  at most `tokens`);
 *   lengths_out[b] lengths[b] + counts[b];
 *   table[b][j]    for the pages that this takes beyond those b has: page
 *                  numbers from the end of the stack free[0 .. free_count - 1],
 *                  request by request; other entries are not written;
 *   slots[i], positions[i]  of row i: its place in the cache and in its request
 *                  (rows from offsets[requests] on: -1 and 0);
 *   free_count_out the number left on the stack, which is not written.
 * A request whose pages are more than table_width, whose rows end behind
 * `tokens`, or whose pages the stack does not cover any more (with those of the
 * requests before it, also the ones that got nothing for that reason) gets
 * nothing: lengths_out[b] = lengths[b], and its rows have slot -1 (and positions
 * that end at 2^31 - 1).  A page
 * number outside [0, pages) gives slot -1.
 *
 * table [requests][ld_table] int32, ld_table >= table_width >= 0; lengths,
 * counts, lengths_out int32 [requests]; offsets int32 [requests + 1]; free int32
 * [pages]; free_count, free_count_out int32 [1]; slots, positions int32 [tokens].
 * The outputs may not overlap the inputs.
 * requests < 2^24, tokens < 2^31.
 * Errors: NULL, SHAPE, MISALIGNED, LIMIT, HIP.
 */
mxfp8_status kv_extend(int32_t *table, int64_t ld_table, int64_t table_width, const int32_t *lengths,
                       const int32_t *counts, int64_t requests, const int32_t *free, const int32_t *free_count,
                       int64_t pages, int32_t page_size, int64_t tokens, int32_t *offsets, int32_t *lengths_out,
                       int32_t *slots, int32_t *positions, int32_t *free_count_out, void *stream);

/*
 * Gives the pages of every request with finished[b] != 0 back to the stack, in
 * order: free[free_count ..] = table[b][0 .. pages of lengths[b] - 1], those
 * entries of the table become -1, lengths_out[b] = 0 (other requests:
 * lengths[b]).  Entries that are no page number are not put on the stack, nor are
 * pages beyond its `pages` places.  finished uint8 [requests]; the other
 * arguments as for kv_extend.
 */
mxfp8_status kv_release(int32_t *table, int64_t ld_table, int64_t table_width, const int32_t *lengths,
                        const uint8_t *finished, int64_t requests, int32_t *free, const int32_t *free_count,
                        int64_t pages, int32_t page_size, int32_t *lengths_out, int32_t *free_count_out, void *stream);

/*
 * Writes the MXFP4 copy of k and v, BF16 [tokens][kv_heads][head_dim] with the
 * strides (in elements, multiples of 8) k_token, k_head, v_token, v_head, to
 * slots[i] of the cache; a slot outside it is skipped.  The slots of a call are
 * different (of equal ones any may win, byte by byte).  Codes and scales are
 * those of mxfp4_quantize; NaN and infinities give unspecified finite values.
 * k and v 16-byte aligned.  Errors: NULL, SHAPE, MISALIGNED, LIMIT, HIP.
 */
mxfp8_status kv_append(uint8_t *cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                       const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token,
                       int64_t v_head, const int32_t *slots, int64_t tokens, void *stream);

/*
 * The BF16 values at slots[i], k and v [tokens][kv_heads][head_dim] dense,
 * 16-byte aligned; zeros for a slot outside the cache.
 */
mxfp8_status kv_read(const uint8_t *cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                     const int32_t *slots, int64_t tokens, void *k, void *v, void *stream);

/*
 * out[i][h] = sum_j p_j v_j,  p = softmax_j(scale <q[i][h], k_j>),
 * for query row i of sequence b, the n queries of which stand at the end of its
 * lengths[b] keys: query x (0 .. n - 1) is at position lengths[b] - n + x and sees
 * the keys j at and before it, with window > 0 only the last `window` of them.
 * Key j of b is token j % page_size of page table[b][j / page_size]; keys of a
 * page number outside [0, pages) and beyond table_width pages are not there: a
 * length past the table moves no query, and a query whose keys all lie behind the
 * table sees none.  A query that sees no key gets zeros.
 * Head h of q uses head h / (heads / kv_heads) of the cache.
 *
 * q        BF16 [tokens][heads][head_dim] with strides q_token, q_head in
 *          elements (multiples of 8), 16-byte aligned.
 * lengths  int32 [sequences], negative ones count as 0.
 * offsets  int32 [sequences + 1], rows offsets[b] .. offsets[b + 1] - 1 of q
 *          belong to b (clamped into [0, tokens] and raised to the running
 *          maximum); NULL: one query a sequence, tokens == sequences.  Rows of no
 *          sequence are not written.
 * max_queries  the longest run of queries as far as the caller knows it, >= 1:
 *          it decides which kernel runs, not what comes out.
 * scale    > 0, finite.   window >= 0 (0: none).
 * out      BF16 [tokens][heads][head_dim] dense, 16-byte aligned; no output
 *          overlaps an input.
 * lse      fp32 [tokens][heads] or NULL: log sum_j exp(scale <q, k_j>), -inf for
 *          a query that sees no key.
 * workspace  kv_attention_workspace_bytes(...) of the same sizes, at most 80 MiB,
 *          16-byte aligned (NULL where that is 0); not kept.
 *
 * Keys meet the queries in 32 bits: a query is taken apart into two E4M3 parts
 * that hold all of its bits down to 2^-21 of its largest value.  The softmax's
 * statistics and sums are fp32; a weight p_j is rounded to BF16 for the sum of the
 * values, which holds values of up to 2^88.  What a place holds that no query of a
 * sequence sees does not matter.  A value that is not finite, which kv_append does
 * not write, at a place that some queries see may reach others of the sequence,
 * through 0 * inf.
 * kv_heads >= 1, heads a multiple of it, heads / kv_heads <= 65536; tokens *
 * heads < 2^31.
 * Errors: NULL, SHAPE, MISALIGNED, WORKSPACE, LIMIT, HIP.
 */
size_t kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                    int64_t sequences, int64_t table_width, int32_t page_size, int32_t ragged,
                                    int64_t max_queries, int64_t window);
mxfp8_status kv_attention(const void *q, int64_t q_token, int64_t q_head, int64_t tokens, int32_t heads,
                          const uint8_t *cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                          const int32_t *table, int64_t ld_table, int64_t table_width, const int32_t *lengths,
                          const int32_t *offsets, int64_t sequences, int64_t max_queries, float scale,
                          int64_t window, void *out, float *lse, void *workspace, size_t workspace_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_KVCACHE_H */
