// mx_quantize.hip -- microscaled 4-bit quantisation of a matrix, and its reverse.
//
// With a = max |x| of a block of 32, its scale is 2^(floor(log2 a) - 2): a's exponent bits less 2,
// so x / scale is exact, lies below 8, and is rounded once, to the nearest of E2M1's values.
//
// A workgroup takes 32 rows of 512 columns, a wave 8 of the rows (1 where that leaves fewer than four
// workgroups a CU); a lane holds 8 neighbouring elements (16 bytes of 16-bit ones), so a block of 32
// is four lanes, and its largest magnitude two lane exchanges. Codes leave as a dword a lane,
// scales through LDS as whole 128-byte lines of 32 rows.
//
// What bounds it, on one MI355X: HBM. 11008 x 4096 in bf16 (114 MB): quantized in 22 to 23 us, 5.0
// TB/s, restored in 17, 6.7 TB/s (four fifths of it writes); a copy moves 5.2. In fp32 (203 MB): 44 us,
// 4.6 TB/s, and 35, 5.9 TB/s. One row of 4096: 2.2 us each, a launch.
#include <type_traits>

#include "mx_internal.h"

namespace nf4 {

namespace {

constexpr int kCols = 512, kThreads = 256, kWaves = 4;

template <int DT, int kWaveRows, bool ONCE>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void *x, int64_t rows,
                                                               int32_t cols, int32_t padded,
                                                               int64_t ld, int32_t col_tiles,
                                                               uint8_t *codes, uint8_t *scales) {
  constexpr int kRows = kWaves * kWaveRows;
  __shared__ __attribute__((aligned(4))) uint8_t s_lds[kCols / kMxStep][kRows][4];
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
    if (col + 8 <= cols) e[i] = mx_load_eight<DT, ONCE>(row, col);
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

template <bool ONCE>
__device__ __forceinline__ void put(mx_u32x4 v, mx_any_u32x4 *p) {
  if constexpr (ONCE) __builtin_nontemporal_store(v, p);
  else *p = v;
}

template <int DT, int kWaveRows, bool ONCE>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(MxMatrix m, int32_t col_tiles,
                                                                 void *out, int64_t ld) {
  constexpr int kRows = kWaves * kWaveRows;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)(blockIdx.x / (unsigned)col_tiles) * kRows;
  // Eight elements of a row a lane, 16 bytes of 16-bit values; of fp32 values four and four that
  // are half a tile on, so that each store's 16 bytes of the lanes are neighbours. (11008 x 4096:
  // 38 us, with eight neighbouring ones 83.)
  constexpr int kEach = DT == kFP32 ? 4 : 8, kPieces = 8 / kEach;
  const int32_t col0 = (int32_t)(blockIdx.x % (unsigned)col_tiles) * kCols + kEach * lane;
  const int here = (int)(m.rows - row0 < kRows ? m.rows - row0 : kRows);
  uint32_t c[kWaveRows][kPieces], s[kWaveRows][kPieces];
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
#pragma unroll
    for (int h = 0; h < kPieces; ++h) {
      const int32_t col = col0 + h * (kCols / kPieces);
      if (col >= m.cols) continue;
      const uint8_t *at = m.codes + (row0 + r) * (m.padded / 2) + col / 2;
      if constexpr (kEach == 4) c[i][h] = *reinterpret_cast<const uint16_t *>(at);
      else c[i][h] = *reinterpret_cast<const uint32_t *>(at);
      s[i][h] = m.scales[4 * ((int64_t)(col / kMxStep) * m.rows + row0 + r) + (col / kMxBlock & 3)];
    }
  }
#pragma unroll
  for (int i = 0; i < kWaveRows; ++i) {
    const int r = wave + kWaves * i;
    if (r >= here) continue;
#pragma unroll
    for (int h = 0; h < kPieces; ++h) {
      const int32_t col = col0 + h * (kCols / kPieces);
      if (col >= m.cols) continue;
      // elements in order from the low nibble on
      const uint32_t v = (c[i][h] & 0x0f0f0f0fu) << 4 | (c[i][h] >> 4 & 0x0f0f0f0fu);
      const float scale = __uint_as_float(s[i][h] << 23);
      f32x2 f[4];
      f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 0);
      f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 1);
      if constexpr (kEach == 8) {
        f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 2);
        f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, 3);
      }
      if (s[i][h] == 255) {
#pragma unroll
        for (int j = 0; j < kEach / 2; ++j) f[j] = f32x2{__builtin_nanf(""), __builtin_nanf("")};
      }
      const int64_t at = (row0 + r) * ld + col;
      if constexpr (DT == kFP32) {
        float *p = static_cast<float *>(out) + at;
        if (col + 4 <= m.cols) {
          put<ONCE>(mx_u32x4{__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                             __float_as_uint(f[1].x), __float_as_uint(f[1].y)},
                    reinterpret_cast<mx_any_u32x4 *>(p));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < m.cols) p[j] = f[j / 2][j % 2];
        }
      } else {
        uint16_t *p = static_cast<uint16_t *>(out) + at;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2<DT>(f[j].x, f[j].y);
        if (col + 8 <= m.cols) {
          put<ONCE>(mx_u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<mx_any_u32x4 *>(p));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < m.cols) p[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
        }
      }
    }
  }
}

int64_t col_tiles_of(int64_t cols) { return (mx_padded(cols) + kCols - 1) / kCols; }
int64_t tiles_of(int64_t rows, int64_t cols, int tile_rows) {
  return (rows + tile_rows - 1) / tile_rows * col_tiles_of(cols);
}

// Rows of a wave: 8, or 1 where four workgroups a CU of 32 rows are not reached. (Quantized: 16 x
// 11008 4.4 us and 2.2, 2048 x 4096 4.9 and 4.4, 1024 x 14336 7.1 and 6.7.) From kOnceBytes of values
// on these go past the caches, which the codes then have to themselves. (In bf16, quantized and
// restored, other inputs each time: 11008 x 4096 42.5 us, 49.5 through the caches, 8192 x 4096 33,
// 39; 2048 x 4096 quantized in 7.0 and 6.6.)
constexpr int kWideFrom = 4;  // workgroups a CU
constexpr int64_t kOnceBytes = (int64_t)64 << 20;

template <typename F>
void by_size(int64_t rows, int64_t cols, int64_t bytes_each, F &&run) {
  using std::integral_constant;
  if (tiles_of(rows, cols, 8 * kWaves) < kWideFrom * device_cu_count())
    run(integral_constant<int, 1>{}, std::false_type{});
  else if (rows * cols * bytes_each < kOnceBytes)
    run(integral_constant<int, 8>{}, std::false_type{});
  else
    run(integral_constant<int, 8>{}, std::true_type{});
}

template <int DT>
void quantize_as(const void *x, int64_t rows, int32_t cols, int64_t ld, uint8_t *codes,
                 uint8_t *scales, hipStream_t stream) {
  by_size(rows, cols, DT == kFP32 ? 4 : 2, [&](auto wave_rows, auto once) {
    constexpr int R = decltype(wave_rows)::value;
    hipLaunchKernelGGL((mx_quantize_kernel<DT, R, decltype(once)::value>),
                       dim3((unsigned)tiles_of(rows, cols, R * kWaves)), dim3(kThreads), 0, stream,
                       x, rows, cols, (int32_t)mx_padded(cols), ld, (int32_t)col_tiles_of(cols),
                       codes, scales);
  });
}

template <int DT>
void dequantize_as(const MxMatrix &m, void *out, int64_t ld, hipStream_t stream) {
  by_size(m.rows, m.cols, DT == kFP32 ? 4 : 2, [&](auto wave_rows, auto once) {
    constexpr int R = decltype(wave_rows)::value;
    hipLaunchKernelGGL((mx_dequantize_kernel<DT, R, decltype(once)::value>),
                       dim3((unsigned)tiles_of(m.rows, m.cols, R * kWaves)), dim3(kThreads), 0,
                       stream, m, (int32_t)col_tiles_of(m.cols), out, ld);
  });
}

}  // namespace

// (where waves have one row, there are fewer than 8 kWideFrom workgroups a CU)
bool mx_elementwise_fits(int64_t rows, int64_t cols) {
  return tiles_of(rows, cols, 8 * kWaves) * kThreads <= 0xffffffffll;
}

hipError_t launch_mx_quantize(const void *x, int dtype, int64_t rows, int32_t cols, int64_t ld,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  if (dtype == kFP32) quantize_as<kFP32>(x, rows, cols, ld, codes, scales, stream);
  else if (dtype == kFP16) quantize_as<kFP16>(x, rows, cols, ld, codes, scales, stream);
  else quantize_as<kBF16>(x, rows, cols, ld, codes, scales, stream);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxMatrix &m, int dtype, void *out, int64_t ld,
                                hipStream_t stream) {
  if (dtype == kFP32) dequantize_as<kFP32>(m, out, ld, stream);
  else if (dtype == kFP16) dequantize_as<kFP16>(m, out, ld, stream);
  else dequantize_as<kBF16>(m, out, ld, stream);
  return hipGetLastError();
}

}  // namespace nf4
