/*
 * nf4_kv.h -- C ABI of the 4-bit key/value cache of libnf4 (MI355X, gfx950):
 * keys and values quantized as they are written, read back, and attended to in
 * their 4 bits. It stands beside nf4.h and shares its codebooks, block scales,
 * status codes, dtypes and conventions (device pointers, validation before any
 * launch, asynchronous on `stream`, no allocation, no pointer kept).
 *
 * Quantization is nf4_quantize's: per block of `blocksize` consecutive elements
 * of one head vector a = max|x|, s = RN(x / a), the nearest code value with an
 * exact tie going to the smaller one (s = 0 where a = 0). A code stands for
 * RN(c[code] a), as in nf4_dequantize. Inputs must be finite: the codes and scales
 * of a head vector that is not are unspecified, all others are not affected.
 *
 * The cache is paged. A page holds `page_size` positions of every key/value
 * head; position p of sequence b lies in page block_table[b][p / page_size].
 *
 *   packed  uint8 [num_pages][num_kv_heads][page_size][head_dim / 2]
 *   absmax  float [num_pages][num_kv_heads][page_size][head_dim / blocksize]
 *
 * for keys and for values. Pages may lie further apart than that (the page
 * strides), so the layers of a model can share one allocation. Within a head of
 * a page the codes are laid out for the matrix cores. Byte 16 k + m (0 <= m <
 * 16) of a head vector holds elements 32 k + 2 m (bits 7..4) and 32 k + 2 m + 1
 * (bits 3..0). With P = head_dim / 32 it is stored
 *   keys:    position p at byte  p (16 P) + m P + k
 *   values:  position p at byte  (p / 4) (64 P) + m (4 P) + (p % 4) P + k
 * so four neighbouring positions' values share one run. nf4_kv_write and
 * nf4_kv_read convert; scales are in plain order.
 *
 * Rows. A call deals with the last n_b positions of each sequence b: with
 * row_offsets, n_b = row_offsets[b+1] - row_offsets[b] and these are rows
 * row_offsets[b] ... of the row tensors (keys, values, queries, outputs);
 * without, n_b = total_rows / batch. Row i of the n_b is position kv_lens[b] -
 * n_b + i. kv_lens counts the positions written in the same call. So one set of
 * lengths serves the write of a step and the attention after it.
 *
 * Device data out of range never becomes an access out of range: offsets are
 * clamped to [0, total_rows], lengths to [0, 2^31 - 2^20], and a page index
 * outside [0, num_pages) (-1 behind a sequence's last page, say) means that its
 * positions are not there: not written, read as zeros, not attended to. The same
 * holds for negative positions and for those past the table's last column, so a
 * step on a sequence whose table is full leaves what is cached as it is. Rows behind the last offset are left as they
 * are in every output. The positions of one nf4_kv_write must be distinct
 * (sequences may share pages that a call does not write to).
 */
#ifndef NF4_KV_H
#define NF4_KV_H

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache: four caller-owned device buffers. Limits (NF4_ERR_UNSUPPORTED
 * otherwise): head_dim 64, 96, 128, 192 or 256; blocksize 32, 64 or 128
 * dividing head_dim; page_size a multiple of 16 with page_size head_dim / 2 <
 * 2^31; at most 65535 key/value heads and sequences; packed_page_stride < 2^36
 * and absmax_page_stride < 2^32. A sequence has at most 2^31 - 2^20 positions
 * (what the table can hold beyond that is not used). Strides are between pages, of
 * keys and values alike: packed_page_stride in bytes (a multiple of 16, at
 * least num_kv_heads page_size head_dim / 2), absmax_page_stride in floats (at
 * least num_kv_heads page_size head_dim / blocksize). */
typedef struct nf4_kv_cache {
  uint8_t *k_packed;
  float *k_absmax;
  uint8_t *v_packed;
  float *v_absmax;
  int64_t num_pages;
  int64_t packed_page_stride;
  int64_t absmax_page_stride;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t blocksize;
  int32_t quant_type; /* nf4_quant_type */
} nf4_kv_cache;

/* The sequences of a call (device pointers). block_table: int32 [batch] rows of
 * table_cols page indices, table_stride elements apart. kv_lens: int32 [batch].
 * row_offsets: int32 [batch + 1], ascending, or NULL where every sequence has
 * total_rows / batch rows (total_rows must then be a multiple of batch). The
 * three need 4-byte alignment only. */
typedef struct nf4_kv_rows {
  const int32_t *block_table;
  const int32_t *kv_lens;
  const int32_t *row_offsets;
  int64_t table_stride;
  int32_t table_cols;
  int32_t batch;
  int32_t total_rows;
} nf4_kv_rows;

/* Quantizes rows of keys and values into the cache. k, v: [total_rows][
 * num_kv_heads][head_dim] of `dtype`, row_stride and head_stride elements apart
 * (the same for both; multiples of 16 bytes). k_values, v_values: what the codes
 * stand for, rounded to dtype, contiguous [total_rows][num_kv_heads][head_dim];
 * both or neither may be NULL. They are written for every row of a sequence,
 * also for one that has no place in the cache. */
nf4_status nf4_kv_write(const nf4_kv_cache *cache, const nf4_kv_rows *rows, const void *k,
                        const void *v, int64_t row_stride, int64_t head_stride, int32_t dtype,
                        void *k_values, void *v_values, void *stream);

/* Reads rows of the cache back: k, v [total_rows][num_kv_heads][head_dim] of
 * `dtype` with strides as in nf4_kv_write, each element RN(c[code] a) rounded to
 * dtype (nf4_dequantize's value); rows that are not there are zeros. */
nf4_status nf4_kv_read(const nf4_kv_cache *cache, const nf4_kv_rows *rows, int32_t dtype, void *k,
                       void *v, int64_t row_stride, int64_t head_stride, void *stream);

/* Bytes of device workspace nf4_kv_attention takes for these sizes on the
 * current device (0 where one pass over the positions suffices, -1 for sizes
 * that nf4_kv_attention rejects). max_rows and max_len are the values in effect
 * there: total_rows / batch without row_offsets, the table's capacity for 0. */
int64_t nf4_kv_attention_workspace_bytes(int32_t batch, int32_t max_rows, int32_t max_len,
                                         int32_t num_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t dtype, int32_t window);

/* Attention of query rows to the cache. q, out: [total_rows][num_heads][
 * head_dim] of `dtype` with strides as in nf4_kv_write; num_heads is a multiple
 * of num_kv_heads (at most 65535 times as many), and head h attends to
 * key/value head h / (num_heads / num_kv_heads). Row i of the n_b rows of sequence b sees positions
 *   lo <= p < hi,  hi = causal ? kv_lens[b] - n_b + i + 1 : kv_lens[b],
 *                  lo = window > 0 ? max(0, hi - window) : 0,
 *   out = sum_p e_p v_p / sum_p e_p,  e_p = exp(scale q . k_p - max)
 * and a row that sees nothing is zeros. Keys and values enter as c[code] a with
 * no rounding to dtype in between; sums and softmax statistics are fp32.
 *   fp32 rows: as in fp32 arithmetic (relative error about 1e-6);
 *   fp16 rows: likewise, but for the output's rounding;
 *   bf16 rows: the keys' code values (6e-5 relative in the norm) and the softmax
 *   weights carry 11 significant bits;
 *   all: a position's share e_p a / sum e is resolved to 2^-32 of the largest value
 *   scale a that the row sees, which only shows where scales differ by as much. (Of
 *   2^-150 of the largest one that any row sees, if that is more.)
 * A query that is not finite spoils its own row only, and a scale in the cache that
 * is not the rows that see its position. (Key scales of 2^96 and more overflow in up to
 * 32 neighbouring rows of which one has a query of 2^89 or more; else in none.)
 * Sums e_p v_p are formed before they are divided: a value scale times 16 times the
 * positions seen has to stay below 2^128.
 * max_rows: the most rows of any sequence (rows past it are left as they are; 0
 * stands for total_rows, which plans that many for every sequence and takes several
 * times as long where there are many); ignored without row_offsets. max_len: about the longest
 * kv_lens, which sizes the split of the positions over the device (any value gives
 * a right result; 0 stands for the table's capacity). workspace: at least
 * nf4_kv_attention_workspace_bytes of these sizes (16-byte aligned; NF4_ERR_SCRATCH
 * where it is smaller); it holds no state between calls, and calls that may run at
 * once need one each. Results do not depend on anything but the arguments and the
 * device's CU count, bit for bit. */
nf4_status nf4_kv_attention(const nf4_kv_cache *cache, const nf4_kv_rows *rows, const void *q,
                            int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads,
                            int32_t dtype, float scale, int32_t causal, int32_t window,
                            int32_t max_rows, int32_t max_len, void *out, int64_t out_row_stride,
                            int64_t out_head_stride, void *workspace, int64_t workspace_bytes,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_KV_H */
