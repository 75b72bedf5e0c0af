// kv_internal.h -- host-side interface between the C ABI of the 4-bit
// key/value cache (kv_api.hip) and its kernel launchers, and the device code
// they share. Launchers assume validated arguments.
#pragma once

#include "nf4_internal.h"
#include "nf4_kv.h"
#include "nf4_kv_mask.h"

namespace nf4 {

// The cache and the rows of a call as the kernels take them (by value).
struct KvArgs {
  uint8_t *packed[2];  // keys, values
  float *absmax[2];
  int64_t packed_stride, absmax_stride;  // bytes / floats between pages
  int32_t num_pages, page_size, kv_heads;
  const int32_t *table, *lens, *offsets;
  int64_t table_stride;
  int32_t table_cols, batch, total_rows;
  int32_t uniform;   // rows of every sequence where offsets is null
  int32_t capacity;  // positions that the table can hold
};

// Most positions of a sequence: lengths are clamped to it.
constexpr int32_t kMaxPositions = 0x7ff00000;

struct KvShape {
  int head_dim, blocksize, quant_type, dtype;
};

hipError_t launch_kv_write(const KvArgs &kv, const KvShape &sh, const void *k, const void *v,
                           int64_t row_stride, int64_t head_stride, void *k_values, void *v_values,
                           hipStream_t stream);

hipError_t launch_kv_read(const KvArgs &kv, const KvShape &sh, void *k, void *v,
                          int64_t row_stride, int64_t head_stride, hipStream_t stream);

// What a call's split goes by.
struct KvAttentionSizes {
  int32_t batch, max_rows, max_len, heads, kv_heads, head_dim, dtype, window;
  int32_t sinks = 0;  // of the masked form
  bool masked = false;
};

struct KvAttentionCall {
  const void *q;
  void *out;
  int64_t q_row, q_head, out_row, out_head;  // strides in elements
  float scale;
  int32_t causal;
  void *workspace;
  // the masked form (nf4_kv_mask.h)
  bool masked = false;
  const uint32_t *tree = nullptr;
  int64_t tree_stride = 0;
  int32_t tree_words = 0;
};

// Workspace bytes of a call, and whether its launches stay within the device's grid
// limits.
int64_t kv_attention_bytes(const KvAttentionSizes &z);
bool kv_attention_fits(const KvAttentionSizes &z);
hipError_t launch_kv_attention(const KvArgs &kv, const KvShape &sh, const KvAttentionSizes &z,
                               const KvAttentionCall &c, hipStream_t stream);

// ------------------------------------------------------------ device code

typedef const __attribute__((address_space(4))) int32_t *ConstI32;

// Loads of the call's int32 arrays at wave-uniform indices, through the
// constant cache (the kernels never write them).
__device__ __forceinline__ int32_t scalar_load(const int32_t *p, int64_t i) {
  return ((ConstI32)(uintptr_t)p)[i];
}

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// 4-lane-row maximum of 16 lanes by DPP, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  auto step = [](float x, int ctrl_result) {
    return fmaxf(x, __uint_as_float((uint32_t)ctrl_result));
  };
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0xb1, 0xf, 0xf, false));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x4e, 0xf, 0xf, false));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x141, 0xf, 0xf, false));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x140, 0xf, 0xf, false));
  return v;
}

}  // namespace nf4
