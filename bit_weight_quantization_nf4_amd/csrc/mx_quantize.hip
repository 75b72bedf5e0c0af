// mx_quantize.hip -- microscaled 4-bit quantisation of a matrix, and its reverse.
//
// A workgroup takes 32 rows of 512 columns, a wave 8 of the rows; a lane holds 8 neighbouring
// elements (16 bytes of 16-bit ones), so a block of 32 is four lanes, and its largest
// magnitude two lane exchanges. Codes leave as a dword a lane, scales through LDS as whole
// 128-byte lines of 32 rows.
#include "mx_internal.h"

namespace nf4 {

namespace {

constexpr int kRows = 32, kCols = 512, kThreads = 256, kWaves = 4, kWaveRows = kRows / kWaves;

template <int DT, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void *x, int64_t rows,
                                                               int32_t cols, int32_t padded,
                                                               int64_t ld, int32_t col_tiles,
                                                               uint8_t *codes, uint8_t *scales) {
  __shared__ uint8_t s_lds[kCols / kMxStep][kRows][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)(blockIdx.x / (unsigned)col_tiles) * kRows;
  const int32_t col0 = (int32_t)(blockIdx.x % (unsigned)col_tiles) * kCols;
  const int32_t col = col0 + 8 * lane;
  const int here = (int)(rows - row0 < kRows ? rows - row0 : kRows);
  MxEight<DT> e[kWaveRows];
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
    const char *row = static_cast<const char *>(x) + (row0 + r) * ld * (DT == kFP32 ? 4 : 2);
    if (ALIGNED && col + 8 <= cols) e[i] = mx_load_eight<DT>(row, col);
    else e[i] = mx_load_ragged<DT>(row, col, cols);
  }
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
    uint32_t scale;
    const uint32_t c = mx_encode<DT>(e[i], scale);
    if (col < padded)
      *reinterpret_cast<uint32_t *>(codes + (row0 + r) * (padded / 2) + col / 2) = c;
    if ((lane & 3) == 0) s_lds[lane >> 4][r][lane >> 2 & 3] = (uint8_t)scale;
  }
  __syncthreads();
  const int t = threadIdx.x / kRows, r = threadIdx.x % kRows;
  if (t < kCols / kMxStep && r < here && col0 + t * kMxStep < padded)
    reinterpret_cast<uint32_t *>(scales)[(col0 / kMxStep + t) * rows + row0 + r] =
        *reinterpret_cast<const uint32_t *>(s_lds[t][r]);
}

template <int DT, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(MxMatrix m, int32_t col_tiles,
                                                                 void *out, int64_t ld) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)(blockIdx.x / (unsigned)col_tiles) * kRows;
  const int32_t col = (int32_t)(blockIdx.x % (unsigned)col_tiles) * kCols + 8 * lane;
  const int here = (int)(m.rows - row0 < kRows ? m.rows - row0 : kRows);
  if (col >= m.cols) return;
  uint32_t c[kWaveRows], s[kWaveRows];
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
    c[i] = *reinterpret_cast<const uint32_t *>(m.codes + (row0 + r) * (m.padded / 2) + col / 2);
    s[i] = m.scales[4 * ((int64_t)(col / kMxStep) * m.rows + row0 + r) + (col / kMxBlock & 3)];
  }
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
    // elements in order from the low nibble on
    const uint32_t v = (c[i] & 0x0f0f0f0fu) << 4 | (c[i] >> 4 & 0x0f0f0f0fu);
    const float scale = __uint_as_float(s[i] << 23);
    const bool nan = s[i] == 255;
    f32x2 f[4];
    f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 0);
    f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 1);
    f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 2);
    f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 3);
    if (nan) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = f32x2{__builtin_nanf(""), __builtin_nanf("")};
    }
    const int64_t at = (row0 + r) * ld + col;
    if constexpr (DT == kFP32) {
      float *p = static_cast<float *>(out) + at;
      if (ALIGNED && col + 8 <= m.cols) {
        reinterpret_cast<f32x4 *>(p)[0] = f32x4{f[0].x, f[0].y, f[1].x, f[1].y};
        reinterpret_cast<f32x4 *>(p)[1] = f32x4{f[2].x, f[2].y, f[3].x, f[3].y};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < m.cols) p[j] = f[j / 2][j % 2];
      }
    } else {
      uint16_t *p = static_cast<uint16_t *>(out) + at;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2<DT>(f[j].x, f[j].y);
      if (ALIGNED && col + 8 <= m.cols) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j < m.cols) p[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
      }
    }
  }
}

bool rows_aligned(const void *p, int64_t rows, int64_t ld, int dtype) {
  const int64_t bytes = ld * (dtype == kFP32 ? 4 : 2);
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || bytes % 16 == 0);
}

int64_t tiles_of(int64_t rows, int64_t cols) {
  return (rows + kRows - 1) / kRows * ((mx_padded(cols) + kCols - 1) / kCols);
}

template <int DT>
void quantize_as(bool aligned, unsigned grid, const void *x, int64_t rows, int32_t cols, int64_t ld,
                 int32_t col_tiles, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int32_t padded = (int32_t)mx_padded(cols);
  if (aligned)
    hipLaunchKernelGGL((mx_quantize_kernel<DT, true>), dim3(grid), dim3(kThreads), 0, stream, x,
                       rows, cols, padded, ld, col_tiles, codes, scales);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<DT, false>), dim3(grid), dim3(kThreads), 0, stream, x,
                       rows, cols, padded, ld, col_tiles, codes, scales);
}

template <int DT>
void dequantize_as(bool aligned, unsigned grid, const MxMatrix &m, int32_t col_tiles, void *out,
                   int64_t ld, hipStream_t stream) {
  if (aligned)
    hipLaunchKernelGGL((mx_dequantize_kernel<DT, true>), dim3(grid), dim3(kThreads), 0, stream, m,
                       col_tiles, out, ld);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<DT, false>), dim3(grid), dim3(kThreads), 0, stream, m,
                       col_tiles, out, ld);
}

}  // namespace

bool mx_elementwise_fits(int64_t rows, int64_t cols) {
  return tiles_of(rows, cols) * kThreads <= 0xffffffffll;
}

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t rows, int32_t cols, int64_t ld,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const unsigned grid = (unsigned)tiles_of(rows, cols);
  const int32_t col_tiles = (int32_t)((mx_padded(cols) + kCols - 1) / kCols);
  const bool al = rows_aligned(x, rows, ld, dtype);
  if (dtype == kFP32) quantize_as<kFP32>(al, grid, x, rows, cols, ld, col_tiles, codes, scales, stream);
  else if (dtype == kFP16) quantize_as<kFP16>(al, grid, x, rows, cols, ld, col_tiles, codes, scales, stream);
  else quantize_as<kBF16>(al, grid, x, rows, cols, ld, col_tiles, codes, scales, stream);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxMatrix &m, int dtype, void *out, int64_t ld,
                                hipStream_t stream) {
  const unsigned grid = (unsigned)tiles_of(m.rows, m.cols);
  const int32_t col_tiles = (int32_t)((m.padded + kCols - 1) / kCols);
  const bool al = rows_aligned(out, m.rows, ld, dtype);
  if (dtype == kFP32) dequantize_as<kFP32>(al, grid, m, col_tiles, out, ld, stream);
  else if (dtype == kFP16) dequantize_as<kFP16>(al, grid, m, col_tiles, out, ld, stream);
  else dequantize_as<kBF16>(al, grid, m, col_tiles, out, ld, stream);
  return hipGetLastError();
}

}  // namespace nf4
