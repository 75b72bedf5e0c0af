// mx_gemv.hip -- products of few rows, and small ones, with a microscaled 4-bit weight.
//
// y[m][f] = sum_k x[m][k] w[f][k], both in 4 bits, 16x16x128 matrix-core steps with the weight
// as the first operand: a lane's 16 bytes of codes go to the instruction as they come from
// memory. A workgroup has 16 FT features, 16 TT rows of x and all of K; its waves take the
// 128-wide steps in turn, batches of kBatch steps' loads in flight at once, and add their sums up
// in wave order.
// With few rows of x the workgroup quantizes them itself into LDS while the weight's first
// batch is on its way; else x is quantized before and its codes are read beside the weight's.
//
// What bounds it, on one MI355X: the weight's bytes, each of which comes once, and a launch's own
// 2 us. One row, 11008 x 4096 (23.9 MB): 6.7 us, 3.6 TB/s; a kernel that hardly does a thing takes
// 2.2 there, and what is left moves at 5.3 TB/s (a copy: 5.2). 16 rows, 4096 x 11008: 8.1 us, and
// 2.2 to 3.0 for the launch that quantizes x. 64 rows, 11008 x 4096: 12 us and 2.5.
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
};

// Elements of x that a workgroup quantizes itself at most, and LDS for them (of a row, a gap of 16
// bytes and up to 12 of rounding).
constexpr int kRawElements = 20480, kRawBytes = kRawElements / 32 * 17 + 16 * (16 + 12);

// bytes of a quantized row in LDS: its codes, padded against bank conflicts, and scales, up to a
// multiple of 16, for rows are read in pieces of 16
__host__ __device__ constexpr int64_t raw_row_bytes(int64_t padded) {
  return (padded / 2 + 16 + padded / kMxBlock + 15) / 16 * 16;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *p, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  void *q = reinterpret_cast<void *>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 |
                                     (uint32_t)uniform((int)v));
  return __builtin_amdgcn_make_buffer_rsrc(q, (short)0, uniform((int)bytes), 0x00020000);
}

// From a register whose lane (n, g) holds row n's four scales of step g: those of step U in every
// lane.
struct FourSteps {
  uint32_t of[4];
};
__device__ __forceinline__ FourSteps spread(uint32_t v) {
  const auto odd = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // rows 0, 0, 2, 2 and 1, 1, 3, 3
  const auto a = __builtin_amdgcn_permlane32_swap(odd[0], odd[0], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(odd[1], odd[1], false, false);
  return FourSteps{{a[0], b[0], a[1], b[1]}};
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
// x. FT: 16-feature tiles of the workgroup. kBatch: steps of a wave whose loads are in flight at
// once. kEights: loads of x of a lane that are, where it is quantized here.
template <int RAW, int OUT, int TT, int FT, int kWaves, int kBatch, int kEights>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_kernel(GemvArgs a) {
  constexpr int kThreads = 64 * kWaves;
  __shared__ __attribute__((aligned(16))) char x_lds[RAW >= 0 ? kRawBytes : 16];
  __shared__ f32x4 part[kWaves][FT * TT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int64_t f0 = (int64_t)blockIdx.x * (16 * FT);
  const int m0 = RAW < 0 ? (int)blockIdx.y * (16 * TT) : 0;
  const int m_rows = a.M - m0 < 16 * TT ? a.M - m0 : 16 * TT;
  const int64_t half = a.w.padded / 2;
  const int steps = a.w.padded / kMxStep;

  // Loads go by buffers: rows past the last one, and steps, read zeros and cost nothing.
  const int f_rows = uniform((int)(a.w.rows - f0 < 16 * FT ? a.w.rows - f0 : 16 * FT));
  const __amdgpu_buffer_rsrc_t wr = buffer_of(a.w.codes + f0 * half, (uint32_t)f_rows * (uint32_t)half);
  const __amdgpu_buffer_rsrc_t xr = RAW < 0
      ? buffer_of(a.x.codes + m0 * half, (uint32_t)m_rows * (uint32_t)half) : buffer_of(nullptr, 0);
  constexpr int XB = RAW < 0 ? TT : 1;
  // Scales go by four steps a load, one for each lane of the four that share a row: a byte a lane
  // and step cost 1 us of 9 at 16 rows.
  static_assert(kBatch % 4 == 0, "scales by four steps");
  struct Batch {
    mx_u32x4 c[kBatch][FT], xc[kBatch][XB];
    uint32_t s[kBatch / 4][FT], xs[kBatch / 4][XB];
  };
  auto load_scales = [&](const MxMatrix &m, int64_t row, int t0, int u4) {
    int t = t0 + (4 * u4 + g) * kWaves;
    t = t < steps ? t : steps - 1;
    return reinterpret_cast<const uint32_t *>(m.scales)[t * m.rows + (row < m.rows ? row : m.rows - 1)];
  };
  auto load = [&](Batch &b, int t0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool there = t0 + u * kWaves < steps;
      const uint32_t none = there ? 0u : 0x80000000u, at = there ? 64u * (uint32_t)(t0 + u * kWaves) : 0u;
      auto codes_of = [&](__amdgpu_buffer_rsrc_t r, uint32_t row) {
        return __builtin_bit_cast(mx_u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                r, (int)((row * (uint32_t)half + 16 * g) | none), (int)at, 0));
      };
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        b.c[u][i] = codes_of(wr, 16 * i + n);
        if (u % 4 == 0) b.s[u / 4][i] = load_scales(a.w, f0 + 16 * i + n, t0, u / 4);
      }
      if constexpr (RAW < 0) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          b.xc[u][j] = codes_of(xr, 16 * j + n);
          if (u % 4 == 0) b.xs[u / 4][j] = load_scales(a.x, m0 + 16 * j + n, t0, u / 4);
        }
      }
    }
  };
  Batch b;
  load(b, wave);

  const int64_t row_bytes = raw_row_bytes(a.w.padded);
  if constexpr (RAW >= 0) {
    // eight neighbouring elements at a time (whole quads of lanes stay together: rows are
    // multiples of 128)
    const uint32_t eights = (uint32_t)a.w.padded / 8, total = (uint32_t)a.M * eights;
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kEights * kThreads) {
      MxEight<RAW> e[kEights];
#pragma unroll
      for (int k = 0; k < kEights; ++k) {
        const uint32_t i = i0 + k * kThreads;
        if (i >= total) continue;
        const uint32_t m = i / eights;
        const int col = 8 * (int)(i - m * eights);
        const char *row = static_cast<const char *>(a.raw) + m * a.ldx * (RAW == kFP32 ? 4 : 2);
        if (col + 8 <= a.w.cols) e[k] = mx_load_eight<RAW>(row, col);
        else e[k] = mx_load_ragged<RAW>(row, col, a.w.cols);
      }
#pragma unroll
      for (int k = 0; k < kEights; ++k) {
        const uint32_t i = i0 + k * kThreads;
        if (i >= total) continue;
        const uint32_t m = i / eights;
        const int col = 8 * (int)(i - m * eights);
        char *dst = x_lds + m * row_bytes;
        uint32_t scale;
        *reinterpret_cast<uint32_t *>(dst + col / 2) = mx_encode<RAW>(e[k], scale);
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
  for (int t0 = wave; t0 < steps; t0 += kWaves * kBatch) {
    if (t0 != wave) load(b, t0);
#pragma unroll
    for (int u4 = 0; u4 < kBatch / 4; ++u4) {
      if (t0 + 4 * u4 * kWaves >= steps) break;
      FourSteps sw[FT], sx[XB];
#pragma unroll
      for (int i = 0; i < FT; ++i) sw[i] = spread(b.s[u4][i]);
      if constexpr (RAW < 0) {
#pragma unroll
        for (int j = 0; j < TT; ++j) sx[j] = spread(b.xs[u4][j]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + (4 * u4 + u) * kWaves;
        if (t >= steps) continue;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          mx_u32x4 c;
          uint32_t sc;
          if constexpr (RAW >= 0) {
            const int row = 16 * j + n < a.M ? 16 * j + n : 0;  // (not stored past the last)
            const char *src = x_lds + row * row_bytes;
            c = *reinterpret_cast<const mx_u32x4 *>(src + 64 * t + 16 * g);
            sc = (uint8_t)src[half + 16 + 4 * t + g];
          } else {
            c = b.xc[4 * u4 + u][j];
            sc = sx[j].of[u] >> (8 * g);
          }
#pragma unroll
          for (int i = 0; i < FT; ++i)
            acc[i][j] = mfma_mx(b.c[4 * u4 + u][i], c, acc[i][j], sw[i].of[u] >> (8 * g), sc);
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
    const int row = m0 + 16 * j + m;
    if (row >= a.M || feature >= a.w.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][ij][16 * (f >> 2) + m][f & 3];
    if (a.bias != nullptr) v += load_as_float<OUT>(a.bias, feature);
    store_from_float<OUT>(a.y, row * a.ldy + feature, v);
  }
}

constexpr int kWaves = 8;

template <int RAW, int OUT, int TT, int FT, int kBatch, int kEights = 1>
hipError_t launch(const GemvArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.w.rows + 16 * FT - 1) / (16 * FT)),
                  (unsigned)(((int64_t)a.M + 16 * TT - 1) / (16 * TT)));
  hipLaunchKernelGGL((mx_gemv_kernel<RAW, OUT, TT, FT, kWaves, kBatch, kEights>), grid,
                     dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

// All of a wave's loads are in flight at once up to 96 steps (K = 12288); short rows keep to few
// registers, so that several workgroups share a CU. (One weight after another, 11008 x 4096 at one
// row: 6.6 us with 4 steps, 12 with 11; 4096 x 11008: 8.1 and 7.4, at 16 rows 9.5 and 8.9.)
constexpr int kShortSteps = 32;

template <int RAW, int OUT>
hipError_t launch_one_tile(const GemvArgs &a, hipStream_t stream) {
  const bool few = (int64_t)a.M * a.w.padded <= 8 * 64 * kWaves;  // a load of x a lane
  if (a.w.padded / kMxStep <= kShortSteps) {
    if (RAW >= 0 && !few) return launch<RAW, OUT, 1, 1, 4, 4>(a, stream);
    return launch<RAW, OUT, 1, 1, 4>(a, stream);
  }
  return launch<RAW, OUT, 1, 1, 12, RAW >= 0 ? 4 : 1>(a, stream);
}

template <int RAW>
hipError_t launch_raw(const GemvArgs &a, int out_dtype, hipStream_t stream) {
  if (out_dtype == kFP32) return launch_one_tile<RAW, kFP32>(a, stream);
  if (out_dtype == kFP16) return launch_one_tile<RAW, kFP16>(a, stream);
  return launch_one_tile<RAW, kBF16>(a, stream);
}

// Tiles of 16 features and 16 TT rows.
int64_t tiles_of(int64_t N, int64_t M, int TT) {
  return (N + 15) / 16 * ((M + 16 * TT - 1) / (16 * TT));
}

// More rows of x are read again by every workgroup: these take as many features as leave one for
// each CU. (64 rows, 11008 x 4096: 17.1 us with 16 features, 16.6 with 32, 11.9 with 64; 4096 x
// 4096: 7.5, 8.9, 11.7. 32 rows: 11.1, 10.3, 9.0; 5.5, 6.5, 8.8.)
int features_of(int64_t N, int64_t M) {  // 16-feature tiles of a workgroup
  if (M <= 16) return 1;
  const int64_t tiles = tiles_of(N, M, M <= 32 ? 2 : 4), cus = device_cu_count();
  return tiles <= cus ? 1 : tiles <= 2 * cus ? 2 : 4;
}

template <int OUT, int TT>
hipError_t launch_features(const GemvArgs &a, hipStream_t stream) {
  const int features = features_of(a.w.rows, a.M);
  if (features == 1) return launch<-1, OUT, TT, 1, 4>(a, stream);
  if (features == 2) return launch<-1, OUT, TT, 2, 4>(a, stream);
  return launch<-1, OUT, TT, 4, 4>(a, stream);
}

template <int OUT>
hipError_t launch_tiles(const GemvArgs &a, hipStream_t stream) {
  if (a.M <= 16) return launch_one_tile<-1, OUT>(a, stream);
  if (a.M <= 32) return launch_features<OUT, 2>(a, stream);
  return launch_features<OUT, 4>(a, stream);
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

// Products of more rows than 64 come here where the device has a CU for each two of their tiles and
// rows are not long. (Here and in mx_gemm.hip's kernel, us: 128 x 1024 x 1024 4.2 and 5.8, 256 x
// 1024 x 4096 7.2 and 10.9, 512 x 1024 x 8192 14.6 and 16.3, 128 x 4096 x 4096 9.0 and 13.6; longer
// rows, 256 x 1024 x 14336, 19.8 and 16.3; more tiles, 256 x 4096 x 1024, 7.2 and 6.1.)
constexpr int64_t kGemvMaxK = 8192;

bool mx_gemv_takes(int64_t M, int64_t N, int64_t K) {
  // (what passes the device's grid has few enough tiles of the other kernel)
  const int64_t wide = 16 * features_of(N, M);
  if ((N + wide - 1) / wide * (64 * kWaves) > 0xffffffffll) return false;
  return M <= 64 || (tiles_of(N, M, 4) <= 2 * device_cu_count() && K <= kGemvMaxK);
}

// Every workgroup quantizes all of x, which has to cost less than a launch before: about 2.2 us.
// (One weight after another: 4 rows, 11008 x 4096 8.4 us and 9.0, 8 rows, 4096 x 4096 5.7 and 5.7,
// 11 rows 6.9 and 5.9; 2 rows, 4096 x 11008 10.2 and 9.4.)
bool mx_gemv_quantizes(int64_t M, int64_t K) {
  return M <= 16 && M * mx_padded(K) <= kRawElements;
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
  if (x_dtype == kFP32) return launch_raw<kFP32>(a, p.out_dtype, stream);
  if (x_dtype == kFP16) return launch_raw<kFP16>(a, p.out_dtype, stream);
  return launch_raw<kBF16>(a, p.out_dtype, stream);
}

}  // namespace nf4
