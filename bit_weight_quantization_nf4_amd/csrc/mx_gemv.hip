// mx_gemv.hip -- products of few rows with a microscaled 4-bit weight.
//
// y[m][f] = sum_k x[m][k] w[f][k], both in 4 bits, 16x16x128 matrix-core steps with the weight
// as the first operand: a lane's 16 bytes of codes go to the instruction as they come from
// memory. A workgroup has 16 FT features and all of K; its waves take the 128-wide steps in
// turn, batches of kBatch steps' loads in flight at once, and add their sums up in wave order.
// With few rows of x the workgroup quantizes them itself into LDS while the weight's first
// batch is on its way; else x is quantized before and its codes are read beside the weight's.
#include "mx_internal.h"

namespace nf4 {

namespace {

struct GemvArgs {
  MxMatrix w;
  const void *bias;
  void *y;
  int64_t ldy;
  int32_t M;
  // x quantized ...
  MxMatrix x;
  // ... or as it is
  const void *raw;
  int64_t ldx;
  int32_t raw_aligned;
};

constexpr int kWaves = 8, kThreads = 64 * kWaves, kBatch = 4;
// LDS for rows that a workgroup quantizes itself.
constexpr int kRawBytes = 32 * 1024;

// bytes of a quantized row in LDS: its codes, padded against bank conflicts, and scales
__host__ __device__ constexpr int64_t raw_row_bytes(int64_t padded) {
  return padded / 2 + 16 + padded / kMxBlock;
}

template <int OUT>
__device__ __forceinline__ float load_as_float(const void *p, int64_t i) {
  if constexpr (OUT == kFP32) return static_cast<const float *>(p)[i];
  else return widen16<OUT>(static_cast<const uint16_t *>(p)[i]);
}

template <int OUT>
__device__ __forceinline__ void store_from_float(void *p, int64_t i, float v) {
  if constexpr (OUT == kFP32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = (uint16_t)out_bits<OUT>(v);
}

// RAW: dtype of x that the workgroup quantizes, -1 where x is quantized. TT: 16-row tiles of
// x. FT: 16-feature tiles of the workgroup.
template <int RAW, int OUT, int TT, int FT>
__global__ __launch_bounds__(kThreads) void mx_gemv_kernel(GemvArgs a) {
  __shared__ __attribute__((aligned(16))) char x_lds[RAW >= 0 ? kRawBytes : 16];
  __shared__ f32x4 part[kWaves][FT * TT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t f0 = (int64_t)blockIdx.x * (16 * FT);
  const int64_t half = a.w.padded / 2;
  const int steps = a.w.padded / kMxStep;

  // the lane's rows of the weight (past the last one: the last one, which is not stored)
  const uint8_t *wc[FT], *ws[FT];
#pragma unroll
  for (int i = 0; i < FT; ++i) {
    int64_t f = f0 + 16 * i + n;
    f = f < a.w.rows ? f : a.w.rows - 1;
    wc[i] = a.w.codes + f * half + 16 * g;
    ws[i] = a.w.scales + 4 * f + g;
  }
  struct Batch {
    mx_u32x4 c[kBatch][FT];
    uint32_t s[kBatch][FT];
  };
  // steps past the last one load it again
  auto load = [&](Batch &b, int t0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      int t = t0 + u * kWaves;
      t = t < steps ? t : steps - 1;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        b.c[u][i] = *reinterpret_cast<const mx_u32x4 *>(wc[i] + 64 * (int64_t)t);
        b.s[u][i] = ws[i][4 * t * a.w.rows];
      }
    }
  };
  Batch b;
  load(b, wave);

  const int64_t row_bytes = raw_row_bytes(a.w.padded);
  if constexpr (RAW >= 0) {
    for (int m = 0; m < a.M; ++m) {
      const char *row = static_cast<const char *>(a.raw) + m * a.ldx * (RAW == kFP32 ? 4 : 2);
      char *dst = x_lds + m * row_bytes;
      // (whole quads of lanes stay together: padded is a multiple of 32)
      for (int col = 8 * (int)threadIdx.x; col < a.w.padded; col += 8 * kThreads) {
        MxEight<RAW> e;
        if (a.raw_aligned && col + 8 <= a.w.cols) e = mx_load_eight<RAW>(row, col);
        else e = mx_load_ragged<RAW>(row, col, a.w.cols);
        uint32_t scale;
        *reinterpret_cast<uint32_t *>(dst + col / 2) = mx_encode<RAW>(e, scale);
        if ((lane & 3) == 0) dst[half + 16 + col / kMxBlock] = (char)scale;
      }
    }
    __syncthreads();
  }

  f32x4 acc[FT][TT];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int token[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) token[j] = 16 * j + n < a.M ? 16 * j + n : a.M - 1;

  for (int t0 = wave; t0 < steps; t0 += kWaves * kBatch) {
    const Batch now = b;
    if (t0 + kWaves * kBatch < steps) load(b, t0 + kWaves * kBatch);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int t = t0 + u * kWaves;
      if (t < steps) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          mx_u32x4 xc;
          uint32_t xs;
          if constexpr (RAW >= 0) {
            const char *src = x_lds + token[j] * row_bytes;
            xc = *reinterpret_cast<const mx_u32x4 *>(src + 64 * t + 16 * g);
            xs = (uint8_t)src[half + 16 + 4 * t + g];
          } else {
            xc = *reinterpret_cast<const mx_u32x4 *>(a.x.codes + token[j] * half + 64 * t + 16 * g);
            xs = a.x.scales[4 * (t * a.x.rows + token[j]) + g];
          }
#pragma unroll
          for (int i = 0; i < FT; ++i) acc[i][j] = mfma_mx(now.c[u][i], xc, acc[i][j], now.s[u][i], xs);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[wave][i * TT + j][lane] = acc[i][j];
  __syncthreads();
  // tile (i, j), row m of it, feature 4 q + r
  for (int at = threadIdx.x; at < FT * TT * 256; at += kThreads) {
    const int ij = at >> 8, f = at & 15, m = at >> 4 & 15;
    const int i = ij / TT, j = ij - i * TT;
    const int64_t feature = f0 + 16 * i + f;
    const int row = 16 * j + m;
    if (row >= a.M || feature >= a.w.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][ij][16 * (f >> 2) + m][f & 3];
    if (a.bias != nullptr) v += load_as_float<OUT>(a.bias, feature);
    store_from_float<OUT>(a.y, row * a.ldy + feature, v);
  }
}

template <int RAW, int OUT, int TT, int FT>
hipError_t launch(const GemvArgs &a, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.w.rows + 16 * FT - 1) / (16 * FT));
  hipLaunchKernelGGL((mx_gemv_kernel<RAW, OUT, TT, FT>), dim3(grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int RAW>
hipError_t launch_raw(const GemvArgs &a, int out_dtype, hipStream_t stream) {
  if (out_dtype == kFP32) return launch<RAW, kFP32, 1, 1>(a, stream);
  if (out_dtype == kFP16) return launch<RAW, kFP16, 1, 1>(a, stream);
  return launch<RAW, kBF16, 1, 1>(a, stream);
}

template <int OUT>
hipError_t launch_tiles(const GemvArgs &a, hipStream_t stream) {
  if (a.M <= 16) return launch<-1, OUT, 1, 1>(a, stream);
  if (a.M <= 32) return launch<-1, OUT, 2, 1>(a, stream);
  return launch<-1, OUT, 4, 1>(a, stream);
}

GemvArgs args_of(const MxProduct &p, int M) {
  GemvArgs a{};
  a.w = p.w;
  a.bias = p.bias;
  a.y = p.y;
  a.ldy = p.ldy;
  a.M = M;
  return a;
}

}  // namespace

int mx_gemv_max_rows() { return 64; }

bool mx_gemv_quantizes(int64_t M, int64_t K) {
  return M <= 16 && M * raw_row_bytes(mx_padded(K)) <= kRawBytes;
}

hipError_t launch_mx_gemv(const MxMatrix &x, const MxProduct &p, hipStream_t stream) {
  GemvArgs a = args_of(p, (int)x.rows);
  a.x = x;
  if (p.out_dtype == kFP32) return launch_tiles<kFP32>(a, stream);
  if (p.out_dtype == kFP16) return launch_tiles<kFP16>(a, stream);
  return launch_tiles<kBF16>(a, stream);
}

hipError_t launch_mx_gemv_quantizing(const void *x, int x_dtype, int64_t ldx, int M,
                                     const MxProduct &p, hipStream_t stream) {
  GemvArgs a = args_of(p, M);
  a.raw = x;
  a.ldx = ldx;
  a.raw_aligned = (reinterpret_cast<uintptr_t>(x) & 15) == 0 &&
                  (M <= 1 || ldx * (x_dtype == kFP32 ? 4 : 2) % 16 == 0);
  if (x_dtype == kFP32) return launch_raw<kFP32>(a, p.out_dtype, stream);
  if (x_dtype == kFP16) return launch_raw<kFP16>(a, p.out_dtype, stream);
  return launch_raw<kBF16>(a, p.out_dtype, stream);
}

}  // namespace nf4
