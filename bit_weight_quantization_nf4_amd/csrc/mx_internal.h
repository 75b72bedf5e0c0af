// mx_internal.h -- host-side interface between the C ABI of the microscaled 4-bit
// matrices (mx_api.hip) and its kernel launchers, and the device code they share.
// Launchers assume validated arguments.
#pragma once

#include "nf4_internal.h"
#include "nf4_mx.h"

namespace nf4 {

constexpr int kMxStep = 128;   // elements of a matrix-core step, a row's padding
constexpr int kMxBlock = 32;   // elements that share a scale

// Elements of rows of `cols` with their padding.
inline int64_t mx_padded(int64_t cols) { return (cols + kMxStep - 1) / kMxStep * kMxStep; }

struct MxMatrix {
  const uint8_t *codes;   // [rows][padded / 2]
  const uint8_t *scales;  // [padded / 128][rows][4]
  int64_t rows;
  int32_t cols, padded;
};

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t rows, int32_t cols, int64_t ld,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx_dequantize(const MxMatrix &m, int dtype, void *out, int64_t ld,
                                hipStream_t stream);
// Whether a matrix' quantisation or restoring stays within the device's grid limits.
bool mx_elementwise_fits(int64_t rows, int64_t cols);

// A product's right side and result.
struct MxProduct {
  MxMatrix w;
  const void *bias;  // of out_dtype, or null
  int out_dtype;
  void *y;
  int64_t ldy;
};

// Products of few rows (mx_gemv.hip), where mx_gemv_takes() says so; launch_mx_gemv_quantizing
// takes x as it is, where mx_gemv_quantizes() says so.
bool mx_gemv_takes(int64_t M, int64_t N, int64_t K);
bool mx_gemv_quantizes(int64_t M, int64_t K);
hipError_t launch_mx_gemv(const MxMatrix &x, const MxProduct &p, hipStream_t stream);
hipError_t launch_mx_gemv_quantizing(const void *x, int x_dtype, int64_t ldx, int M,
                                     const MxProduct &p, hipStream_t stream);

// Products of many rows (mx_gemm.hip).
int64_t mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
bool mx_gemm_fits(int64_t M, int64_t N);
// Side of its tiles, ranges of K and their 128-wide steps.
struct MxGemmShape {
  int tile, splits, split_steps;
};
MxGemmShape mx_gemm_shape(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_gemm(const MxMatrix &x, const MxProduct &p, void *workspace,
                          hipStream_t stream);

// ------------------------------------------------------------ device code

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t mx_u32x4 __attribute__((ext_vector_type(4)));

// 16x16x128 step on E2M1 operands: acc += A(16x128) B(128x16). Lane (n = lane & 15, g = lane >> 4)
// gives elements 32 g .. 32 g + 31 of row n of A and of column n of B, 16 bytes each, and these
// blocks' scales as the low bytes of sa and sb; it holds rows 4 g .. 4 g + 3 of column n of acc.
// (Within a block the order of the elements does not matter as long as it is the same in both.)
__device__ __forceinline__ f32x4 mfma_mx(mx_u32x4 a, mx_u32x4 b, f32x4 acc, uint32_t sa,
                                         uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 4, 0, (int)sa, 0,
                                                          (int)sb);
}

// Eight consecutive elements of a row as a lane holds them.
template <int DT>
struct MxEight {
  uint32_t w[DT == kFP32 ? 8 : 4];
};

// (of any alignment: the memory instructions take it, 16 bytes at once)
typedef mx_u32x4 mx_any_u32x4 __attribute__((aligned(2)));

template <int DT, bool ONCE = false>  // ONCE: not kept in the caches
__device__ __forceinline__ MxEight<DT> mx_load_eight(const void *row, int64_t col) {
  MxEight<DT> e;
  const auto *p = reinterpret_cast<const mx_any_u32x4 *>(static_cast<const char *>(row) +
                                                         col * (DT == kFP32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (DT == kFP32 ? 2 : 1); ++i) {
    const mx_u32x4 v = ONCE ? __builtin_nontemporal_load(p + i) : p[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) e.w[4 * i + j] = v[j];
  }
  return e;
}

// The same element by element: zeros from `cols` on.
template <int DT>
__device__ __forceinline__ MxEight<DT> mx_load_ragged(const void *row, int64_t col, int64_t cols) {
  MxEight<DT> e;
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e.w[i] = col + i < cols ? static_cast<const uint32_t *>(row)[col + i] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto *p = static_cast<const uint16_t *>(row) + col + 2 * i;
      const uint32_t lo = col + 2 * i < cols ? p[0] : 0u;
      const uint32_t hi = col + 2 * i + 1 < cols ? p[1] : 0u;
      e.w[i] = lo | hi << 16;
    }
  }
  return e;
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true);
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true);
  return v > b ? v : b;
}

// Quantizes a block that four neighbouring lanes (4 q .. 4 q + 3) hold: the lane's eight codes,
// element 0 in the topmost nibble of the lowest byte, and the block's scale in every lane.
// Magnitudes compare as integers, so a NaN counts as the largest. The conversion instruction
// divides by a power of two given as a float, of which it reads the exponent (0: 2^-127), rounds
// to the nearest even and clamps to 6.
template <int DT>
__device__ __forceinline__ uint32_t mx_encode(const MxEight<DT> &e, uint32_t &scale) {
  uint32_t top = 0;  // fp32 bits of the largest magnitude
  if constexpr (DT == kFP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = e.w[i] & 0x7fffffffu;
      top = top > m ? top : m;
    }
    top = quad_max(top);
  } else {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, e.w[i] & 0x7fff7fffu));
    const uint32_t most = quad_max(m[0] > m[1] ? m[0] : m[1]);
    top = __float_as_uint(widen16<DT>(most));
  }
  const uint32_t ex = top >> 23;
  const bool fine = ex < 255;
  scale = ex > 2 ? ex - 2 : 0;
  scale = top == 0 ? 127 : scale;
  const float s = __uint_as_float(scale << 23);
  scale = fine ? scale : 255;
  uint32_t c = 0;
  if constexpr (DT == kFP32) {
    auto f = [&](int i) { return __uint_as_float(e.w[i]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(1), f(0), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(3), f(2), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(5), f(4), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(7), f(6), s, 3);
  } else if constexpr (DT == kBF16) {
    auto f = [&](int i) { return __builtin_bit_cast(bf16x2, e.w[i]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, f(0), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, f(1), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, f(2), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, f(3), s, 3);
  } else {
    auto f = [&](int i) { return __builtin_bit_cast(f16x2, e.w[i]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f(0), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f(1), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f(2), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, f(3), s, 3);
  }
  if constexpr (DT != kFP32) c = (c & 0x0f0f0f0fu) << 4 | (c >> 4 & 0x0f0f0f0fu);
  return fine ? c : 0;
}

}  // namespace nf4
