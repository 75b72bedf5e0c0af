/*
 * nf4_kv_mask.h -- C ABI of the masked attention to the 4-bit key/value cache of libnf4
 * (MI355X, gfx950): a sliding window that leaves a few first positions visible, and a
 * call's rows as a tree of drafted tokens. It stands beside nf4_kv.h and shares its
 * cache, rows, status codes and conventions.
 */
#ifndef NF4_KV_MASK_H
#define NF4_KV_MASK_H

#include "nf4_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace nf4_kv_attention_masked takes for these sizes, as
 * nf4_kv_attention_workspace_bytes. */
int64_t nf4_kv_attention_masked_workspace_bytes(int32_t batch, int32_t max_rows, int32_t max_len,
                                                int32_t num_heads, int32_t num_kv_heads,
                                                int32_t head_dim, int32_t dtype, int32_t window,
                                                int32_t sinks);

/* nf4_kv_attention with causal = 1 and other masks; arguments, rounding and errors are its.
 *
 * sinks: with window > 0, row i of the n_b rows of sequence b, whose place is P = kv_lens[b] -
 * n_b + i, sees the positions p <= P of which p > P - window or p < sinks. (Without a window
 * all p <= P, whatever sinks is.) Where the window begins behind the table's last column the first
 * positions are still in sight.
 *
 * tree: NULL, or the rows that each row sees of its sequence's in the call: row t of the row
 * tensors has tree_words words of 32 bits at tree + t tree_stride (device memory, 4-byte
 * aligned; tree_stride >= tree_words), and bit j % 32 of word j / 32 says whether it sees row j
 * of its sequence's (its own bit among them: a row that is not to see itself does not). Rows
 * past the last word, and bits past the sequence's last row, are not seen. Of the positions
 * before the call's, p < kv_lens[b] - n_b, a row sees all; with window > 0 those with p > P -
 * window or p < sinks, where its place P = kv_lens[b] - n_b + d - 1 goes by the number d of rows
 * that it sees (its depth in the tree, the root's 1). The window does not hide rows of the call.
 * Any set of bits is a valid mask; a row that sees nothing is zeros. */
nf4_status nf4_kv_attention_masked(const nf4_kv_cache *cache, const nf4_kv_rows *rows,
                                   const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                   int32_t num_heads, int32_t dtype, float scale, int32_t window,
                                   int32_t sinks, const uint32_t *tree, int64_t tree_stride,
                                   int32_t tree_words, int32_t max_rows, int32_t max_len, void *out,
                                   int64_t out_row_stride, int64_t out_head_stride,
                                   void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_KV_MASK_H */
