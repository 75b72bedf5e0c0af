// kv_api.hip -- the extern "C" boundary of the 4-bit key/value cache (declared in
// include/nf4_kv.h and nf4_kv_mask.h): argument validation and dispatch to the launchers.
// Every check runs before the first launch, so a rejected call writes nothing.
#include <math.h>

#include <initializer_list>

#include "kv_internal.h"

using namespace nf4;

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool valid_dtype(int32_t d) {
  return d == NF4_DTYPE_BF16 || d == NF4_DTYPE_FP32 || d == NF4_DTYPE_FP16;
}

int64_t dtype_bytes(int32_t d) { return d == NF4_DTYPE_FP32 ? 4 : 2; }

bool valid_head_dim(int32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

nf4_status from_hip(hipError_t e) {
  if (e == hipSuccess) return NF4_OK;
  return e == hipErrorNotSupported ? NF4_ERR_UNSUPPORTED : NF4_ERR_DEVICE;
}

// Cache and rows of a call, as the kernels take them. `any` is false where
// there is nothing to do.
nf4_status check_call(const nf4_kv_cache *c, const nf4_kv_rows *r, int32_t dtype, KvArgs *kv,
                      KvShape *sh, bool *any) {
  if (c == nullptr || r == nullptr || !valid_dtype(dtype)) return NF4_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 0 || c->page_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return NF4_ERR_INVALID_ARGUMENT;
  if (c->quant_type != NF4_QUANT_NF4 && c->quant_type != NF4_QUANT_FP4)
    return NF4_ERR_INVALID_ARGUMENT;
  if (c->blocksize < 32 || c->blocksize > 4096 || (c->blocksize & (c->blocksize - 1)) != 0)
    return NF4_ERR_INVALID_ARGUMENT;
  if (r->batch < 0 || r->total_rows < 0 || r->table_cols < 0 || r->table_stride < r->table_cols)
    return NF4_ERR_INVALID_ARGUMENT;
  if (!valid_head_dim(c->head_dim) || c->blocksize > 128 || c->head_dim % c->blocksize != 0)
    return NF4_ERR_UNSUPPORTED;
  // a head's part of a page is addressed with 31-bit byte offsets, and pages with
  // 32-bit strides in 16 bytes and in floats
  if (c->page_size % 16 != 0 || (int64_t)c->page_size * (c->head_dim / 2) >= ((int64_t)1 << 31))
    return NF4_ERR_UNSUPPORTED;
  if (c->num_pages > INT32_MAX || c->num_kv_heads > 65535 || r->batch > 65535)
    return NF4_ERR_UNSUPPORTED;
  if (c->packed_page_stride >= ((int64_t)1 << 36) || c->absmax_page_stride >= ((int64_t)1 << 32))
    return NF4_ERR_UNSUPPORTED;
  const int64_t positions = (int64_t)c->num_kv_heads * c->page_size;
  if (c->num_pages > 0) {
    if (c->k_packed == nullptr || c->k_absmax == nullptr || c->v_packed == nullptr ||
        c->v_absmax == nullptr)
      return NF4_ERR_INVALID_ARGUMENT;
    if (c->packed_page_stride < positions * (c->head_dim / 2) ||
        c->absmax_page_stride < positions * (c->head_dim / c->blocksize))
      return NF4_ERR_INVALID_ARGUMENT;
    if (c->packed_page_stride > (INT64_MAX >> 1) / c->num_pages ||
        c->absmax_page_stride > (INT64_MAX >> 3) / c->num_pages)
      return NF4_ERR_INVALID_ARGUMENT;
    if (!aligned(c->k_packed, 16) || !aligned(c->v_packed, 16) || !aligned(c->k_absmax, 16) ||
        !aligned(c->v_absmax, 16) || c->packed_page_stride % 16 != 0)
      return NF4_ERR_MISALIGNED;
  }
  *any = r->batch > 0 && r->total_rows > 0;
  if (r->row_offsets == nullptr) {
    if (r->batch == 0 ? r->total_rows != 0 : r->total_rows % r->batch != 0)
      return NF4_ERR_INVALID_ARGUMENT;
  }
  if (*any) {
    if (r->kv_lens == nullptr || (r->table_cols > 0 && r->block_table == nullptr))
      return NF4_ERR_INVALID_ARGUMENT;
    if (!aligned(r->kv_lens, 4) || !aligned(r->block_table, 4) || !aligned(r->row_offsets, 4))
      return NF4_ERR_MISALIGNED;
  }
  int64_t capacity = (int64_t)r->table_cols * c->page_size;
  // a range of positions may be rounded up past it, and stays below 2^31
  if (capacity > kMaxPositions) capacity = kMaxPositions;
  if (c->num_pages == 0) capacity = 0;
  kv->packed[0] = c->k_packed;
  kv->packed[1] = c->v_packed;
  kv->absmax[0] = c->k_absmax;
  kv->absmax[1] = c->v_absmax;
  kv->packed_stride = c->packed_page_stride;
  kv->absmax_stride = c->absmax_page_stride;
  kv->num_pages = (int32_t)c->num_pages;
  kv->page_size = c->page_size;
  kv->kv_heads = c->num_kv_heads;
  kv->table = r->block_table;
  kv->lens = r->kv_lens;
  kv->offsets = r->row_offsets;
  kv->table_stride = r->table_stride;
  kv->table_cols = r->table_cols;
  kv->batch = r->batch;
  kv->total_rows = r->total_rows;
  kv->uniform = r->row_offsets == nullptr && r->batch > 0 ? r->total_rows / r->batch : 0;
  kv->capacity = (int32_t)capacity;
  *sh = KvShape{c->head_dim, c->blocksize, c->quant_type, dtype};
  return NF4_OK;
}

// A [total_rows][heads][head_dim] tensor that is read or written in pieces of
// up to 16 bytes.
nf4_status check_rows(const void *p, int64_t row_stride, int64_t head_stride, int32_t heads,
                      int32_t head_dim, int32_t dtype, const KvArgs &kv, bool any) {
  if (!any) return NF4_OK;
  if (p == nullptr) return NF4_ERR_INVALID_ARGUMENT;
  // rows may have their heads apart (token-major) or the heads their rows
  if (row_stride < head_dim || head_stride < head_dim) return NF4_ERR_INVALID_ARGUMENT;
  const int64_t most = (INT64_MAX >> 3) / ((int64_t)kv.total_rows + heads);
  if (row_stride > most || head_stride > most) return NF4_ERR_INVALID_ARGUMENT;
  const int64_t e = dtype_bytes(dtype);
  if (!aligned(p, 16) || (row_stride * e) % 16 != 0 || (head_stride * e) % 16 != 0)
    return NF4_ERR_MISALIGNED;
  return NF4_OK;
}

int64_t attention_bytes(const KvAttentionSizes &z) {
  if (z.batch < 0 || z.max_rows < 0 || z.max_len < 0 || z.heads <= 0 || z.kv_heads <= 0 ||
      z.heads % z.kv_heads != 0 || !valid_head_dim(z.head_dim) || !valid_dtype(z.dtype) ||
      z.window < 0)
    return -1;
  if (z.batch == 0 || z.max_rows == 0) return 0;
  return kv_attention_fits(z) ? kv_attention_bytes(z) : -1;
}

nf4_status attention(const nf4_kv_cache *cache, const nf4_kv_rows *rows, const KvAttentionCall &c,
                     int32_t num_heads, int32_t dtype, int32_t window, int32_t sinks,
                     int32_t max_rows, int32_t max_len, int64_t workspace_bytes, void *stream) {
  KvArgs kv;
  KvShape sh;
  bool any = false;
  nf4_status st = check_call(cache, rows, dtype, &kv, &sh, &any);
  if (st != NF4_OK) return st;
  if (num_heads <= 0 || num_heads % kv.kv_heads != 0) return NF4_ERR_INVALID_ARGUMENT;
  if (window < 0 || max_rows < 0 || max_len < 0 || workspace_bytes < 0 || !isfinite(c.scale))
    return NF4_ERR_INVALID_ARGUMENT;
  if (workspace_bytes > 0 && c.workspace == nullptr) return NF4_ERR_INVALID_ARGUMENT;
  st = check_rows(c.q, c.q_row, c.q_head, num_heads, sh.head_dim, dtype, kv, any);
  if (st != NF4_OK) return st;
  st = check_rows(c.out, c.out_row, c.out_head, num_heads, sh.head_dim, dtype, kv, any);
  if (st != NF4_OK) return st;
  if (!aligned(c.workspace, 16) || !aligned(c.tree, 4)) return NF4_ERR_MISALIGNED;
  if (!any) return NF4_OK;
  const KvAttentionSizes z{
      kv.batch, kv.offsets == nullptr ? kv.uniform : (max_rows > 0 ? max_rows : kv.total_rows),
      max_len > 0 ? max_len : kv.capacity, num_heads, kv.kv_heads, sh.head_dim, dtype, window,
      sinks, c.masked};
  if (!kv_attention_fits(z)) return NF4_ERR_UNSUPPORTED;
  st = nf4_device_check();
  if (st != NF4_OK) return st;
  const int64_t need = kv_attention_bytes(z);
  if (workspace_bytes < need) return NF4_ERR_SCRATCH;
  if (log_on())
    log_msg("kv_attention%s rows=%d batch=%d heads=%d/%d head_dim=%d bs=%d dtype=%d max_rows=%d "
            "max_len=%d: kv_attention_kernel%s", c.masked ? "_masked" : "", kv.total_rows, kv.batch,
            num_heads, kv.kv_heads, sh.head_dim, sh.blocksize, dtype, z.max_rows, z.max_len,
            need > 0 ? ", positions split, joined by kv_attention_join_kernel" : "");
  return from_hip(launch_kv_attention(kv, sh, z, c, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

nf4_status nf4_kv_write(const nf4_kv_cache *cache, const nf4_kv_rows *rows, const void *k,
                        const void *v, int64_t row_stride, int64_t head_stride, int32_t dtype,
                        void *k_values, void *v_values, void *stream) {
  KvArgs kv;
  KvShape sh;
  bool any = false;
  nf4_status st = check_call(cache, rows, dtype, &kv, &sh, &any);
  if (st != NF4_OK) return st;
  for (const void *p : {k, v}) {
    st = check_rows(p, row_stride, head_stride, kv.kv_heads, sh.head_dim, dtype, kv, any);
    if (st != NF4_OK) return st;
  }
  if ((k_values == nullptr) != (v_values == nullptr)) return NF4_ERR_INVALID_ARGUMENT;
  if (!aligned(k_values, 16) || !aligned(v_values, 16)) return NF4_ERR_MISALIGNED;
  if (!any) return NF4_OK;
  st = nf4_device_check();
  if (st != NF4_OK) return st;
  if (log_on())
    log_msg("kv_write rows=%d batch=%d heads=%d head_dim=%d bs=%d dtype=%d values=%d: "
            "kv_write_kernel", kv.total_rows, kv.batch, kv.kv_heads, sh.head_dim, sh.blocksize,
            dtype, k_values != nullptr);
  return from_hip(launch_kv_write(kv, sh, k, v, row_stride, head_stride, k_values, v_values,
                                  reinterpret_cast<hipStream_t>(stream)));
}

nf4_status nf4_kv_read(const nf4_kv_cache *cache, const nf4_kv_rows *rows, int32_t dtype, void *k,
                       void *v, int64_t row_stride, int64_t head_stride, void *stream) {
  KvArgs kv;
  KvShape sh;
  bool any = false;
  nf4_status st = check_call(cache, rows, dtype, &kv, &sh, &any);
  if (st != NF4_OK) return st;
  for (const void *p : {k, v}) {
    st = check_rows(p, row_stride, head_stride, kv.kv_heads, sh.head_dim, dtype, kv, any);
    if (st != NF4_OK) return st;
  }
  if (!any) return NF4_OK;
  st = nf4_device_check();
  if (st != NF4_OK) return st;
  if (log_on())
    log_msg("kv_read rows=%d batch=%d heads=%d head_dim=%d bs=%d dtype=%d: kv_read_kernel",
            kv.total_rows, kv.batch, kv.kv_heads, sh.head_dim, sh.blocksize, dtype);
  return from_hip(launch_kv_read(kv, sh, k, v, row_stride, head_stride,
                                 reinterpret_cast<hipStream_t>(stream)));
}

int64_t nf4_kv_attention_workspace_bytes(int32_t batch, int32_t max_rows, int32_t max_len,
                                         int32_t num_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t dtype, int32_t window) {
  return attention_bytes(
      {batch, max_rows, max_len, num_heads, num_kv_heads, head_dim, dtype, window});
}

int64_t nf4_kv_attention_masked_workspace_bytes(int32_t batch, int32_t max_rows, int32_t max_len,
                                                int32_t num_heads, int32_t num_kv_heads,
                                                int32_t head_dim, int32_t dtype, int32_t window,
                                                int32_t sinks) {
  if (sinks < 0) return -1;
  KvAttentionSizes z{batch, max_rows, max_len, num_heads, num_kv_heads, head_dim, dtype, window, sinks,
                     true};
  const int64_t bytes = attention_bytes(z);
  if (bytes < 0 || (window > 0 && sinks > 0)) return bytes;
  // (without a tree these are nf4_kv_attention's)
  z.masked = false;
  z.sinks = 0;
  const int64_t plain = attention_bytes(z);
  return bytes > plain ? bytes : plain;
}

nf4_status nf4_kv_attention(const nf4_kv_cache *cache, const nf4_kv_rows *rows, const void *q,
                            int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads,
                            int32_t dtype, float scale, int32_t causal, int32_t window,
                            int32_t max_rows, int32_t max_len, void *out, int64_t out_row_stride,
                            int64_t out_head_stride, void *workspace, int64_t workspace_bytes,
                            void *stream) {
  KvAttentionCall c;
  c.q = q;
  c.out = out;
  c.q_row = q_row_stride;
  c.q_head = q_head_stride;
  c.out_row = out_row_stride;
  c.out_head = out_head_stride;
  c.scale = scale;
  c.causal = causal != 0;
  c.workspace = workspace;
  return attention(cache, rows, c, num_heads, dtype, window, 0, max_rows, max_len, workspace_bytes,
                   stream);
}

nf4_status nf4_kv_attention_masked(const nf4_kv_cache *cache, const nf4_kv_rows *rows,
                                   const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                   int32_t num_heads, int32_t dtype, float scale, int32_t window,
                                   int32_t sinks, const uint32_t *tree, int64_t tree_stride,
                                   int32_t tree_words, int32_t max_rows, int32_t max_len, void *out,
                                   int64_t out_row_stride, int64_t out_head_stride,
                                   void *workspace, int64_t workspace_bytes, void *stream) {
  if (sinks < 0) return NF4_ERR_INVALID_ARGUMENT;
  if (tree != nullptr && (tree_words < 0 || tree_stride < tree_words ||
                          (rows != nullptr && rows->total_rows > 0 &&
                           tree_stride > (INT64_MAX >> 3) / rows->total_rows)))
    return NF4_ERR_INVALID_ARGUMENT;
  KvAttentionCall c;
  c.q = q;
  c.out = out;
  c.q_row = q_row_stride;
  c.q_head = q_head_stride;
  c.out_row = out_row_stride;
  c.out_head = out_head_stride;
  c.scale = scale;
  c.causal = 1;
  c.workspace = workspace;
  // first positions are in sight anyway where there is no window
  if (window == 0) sinks = 0;
  c.masked = tree != nullptr || sinks > 0;
  c.tree = tree;
  c.tree_stride = tree_stride;
  c.tree_words = tree_words;
  return attention(cache, rows, c, num_heads, dtype, window, sinks, max_rows, max_len,
                   workspace_bytes, stream);
}

}  // extern "C"
