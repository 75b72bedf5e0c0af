// mx_gemm.hip -- products of many rows with a microscaled 4-bit weight.
//
// y[m][f] = sum_k x[m][k] w[f][k] on 16x16x128 matrix-core steps, the weight as the first
// operand. A workgroup computes a tile of features x rows of x, its waves parts of it: FT x TT
// tiles of 16 x 16. K goes by 256: both operands' codes (128 bytes a row) and scales are
// brought straight to LDS, into one of two buffers while the other is multiplied.
//
// Which rows of the operands make up a matrix-core tile is free: tile i of a wave takes rows FT m
// + i (m < 16), so a lane finds the scales of its FT rows side by side in LDS, and holds FT
// neighbouring features of a result. A row's eight 16-byte pieces lie at places xor'ed with a
// number of the row that differs between the rows which are read together.
#include "mx_internal.h"

namespace nf4 {

namespace {

struct GemmArgs {
  MxMatrix w, x;
  const void *bias;
  void *y;
  int64_t ldy;
  int32_t f_tiles, m_tiles;
};

constexpr int kPieces = 8;               // 16-byte pieces of a row in LDS: 256 elements
constexpr int kRowBytes = 16 * kPieces;

typedef const __attribute__((address_space(1))) uint32_t *GlobalWords;
typedef __attribute__((address_space(3))) uint32_t *LdsWords;

template <int BYTES>
__device__ __forceinline__ void to_lds(const void *src, void *dst) {
  static_assert(BYTES == 16 || BYTES == 4, "a lane's piece");
  if constexpr (BYTES == 16)
    __builtin_amdgcn_global_load_lds((GlobalWords)(uintptr_t)src, (LdsWords)dst, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds((GlobalWords)(uintptr_t)src, (LdsWords)dst, 4, 0, 0);
}

// WF x WT waves, each with FT x TT tiles (features x rows of x).
template <int OUT, int FT, int TT, int WF, int WT>
__global__ __launch_bounds__(64 * WF * WT) void mx_gemm_kernel(GemmArgs a) {
  constexpr int kWaves = WF * WT;
  constexpr int BF = 16 * FT * WF, BT = 16 * TT * WT;
  constexpr int kRows = BF + BT;  // of both operands, the weight's first
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][kRows][kRowBytes];
  __shared__ __attribute__((aligned(16))) uint32_t scales[2][2][kRows];  // [buffer][half][row]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int wf = wave % WF, wt = wave / WF;
  const int fb = (int)blockIdx.x % a.f_tiles, mb = (int)blockIdx.x / a.f_tiles;
  const int64_t f0 = (int64_t)fb * BF, m0 = (int64_t)mb * BT;
  const int f_last = (int)(a.w.rows - f0 < BF ? a.w.rows - f0 : BF) - 1;
  const int m_last = (int)(a.x.rows - m0 < BT ? a.x.rows - m0 : BT) - 1;
  const int64_t half = a.w.padded / 2;
  const int steps = a.w.padded / kMxStep;  // of 128
  const int pairs = (steps + 1) / 2;

  // a row's number that its pieces' places are xor'ed with
  auto turn_f = [](int row) { return row / FT & 7; };
  auto turn_m = [](int row) { return row / TT & 7; };

  // rows of both operands past their last repeat it; nothing of theirs is stored
  constexpr int kLoads = kRows / 8 / kWaves;
  static_assert(kRows % (8 * kWaves) == 0 && BF % 8 == 0, "whole loads");
  const uint8_t *src[kLoads];
  int piece[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * (wave * kLoads + i) + (lane >> 3);
    const bool of_w = r < BF;
    int row = of_w ? r : r - BF;
    piece[i] = (lane & 7) ^ (of_w ? turn_f(row) : turn_m(row));
    const int last = of_w ? f_last : m_last;
    row = row < last ? row : last;
    src[i] = (of_w ? a.w.codes + (f0 + row) * half : a.x.codes + (m0 + row) * half);
  }
  // scales: 64 rows of one half a load
  constexpr int kScaleLoads = 2 * kRows / 64;
  static_assert(kRows % 64 == 0 && BF % 64 == 0, "whole loads");
  auto load = [&](int buf, int p) {
    const bool whole = 2 * p + 1 < steps;  // both halves are there
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = whole ? piece[i] : piece[i] & 3;
      to_lds<16>(src[i] + (int64_t)p * kRowBytes + 16 * c, codes[buf][8 * (wave * kLoads + i)]);
    }
#pragma unroll
    for (int i = 0; i < (kScaleLoads + kWaves - 1) / kWaves; ++i) {
      const int s = wave + kWaves * i;
      if (s < kScaleLoads) {
        const int h = s / (kRows / 64), r0 = 64 * (s % (kRows / 64));
        const bool of_w = r0 < BF;
        int row = (of_w ? r0 : r0 - BF) + lane;
        const int last = of_w ? f_last : m_last;
        row = row < last ? row : last;
        const int64_t t = whole ? 2 * p + h : 2 * p;
        const uint8_t *from = of_w ? a.w.scales + 4 * (t * a.w.rows + f0 + row)
                                   : a.x.scales + 4 * (t * a.x.rows + m0 + row);
        to_lds<4>(from, &scales[buf][h][r0]);
      }
    }
  };

  f32x4 acc[FT][TT];
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int row_f = wf * 16 * FT + FT * n, row_m = wt * 16 * TT + TT * n;
  const int at_f = turn_f(row_f), at_m = turn_m(row_m);  // the same for the lane's FT (TT) rows
  load(0, 0);
  for (int p = 0; p < pairs; ++p) {
    const int buf = p & 1;
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    __syncthreads();
    if (p + 1 < pairs) load(buf ^ 1, p + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * p + h < steps) {
        mx_u32x4 fa[FT], fm[TT];
        uint32_t sa[FT], sm[TT];
#pragma unroll
        for (int i = 0; i < FT; ++i) {
          fa[i] = *reinterpret_cast<const mx_u32x4 *>(
              &codes[buf][row_f + i][16 * ((4 * h + g) ^ at_f)]);
          sa[i] = scales[buf][h][row_f + i] >> (8 * g);
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          fm[j] = *reinterpret_cast<const mx_u32x4 *>(
              &codes[buf][BF + row_m + j][16 * ((4 * h + g) ^ at_m)]);
          sm[j] = scales[buf][h][BF + row_m + j] >> (8 * g);
        }
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
          for (int j = 0; j < TT; ++j) acc[i][j] = mfma_mx(fa[i], fm[j], acc[i][j], sa[i], sm[j]);
      }
    }
  }

  // lane (n, g): rows TT n + j of x, features FT (4 g + r) + i
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = row_m + j;
    if (m > m_last) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int f = wf * 16 * FT + FT * (4 * g + r);
      const int64_t at = (m0 + m) * a.ldy + f0 + f;
#pragma unroll
      for (int i = 0; i < FT; ++i) {
        if (f + i > f_last) continue;
        float v = acc[i][j][r];
        if (a.bias != nullptr) {
          if constexpr (OUT == kFP32) v += static_cast<const float *>(a.bias)[f0 + f + i];
          else v += widen16<OUT>(static_cast<const uint16_t *>(a.bias)[f0 + f + i]);
        }
        if constexpr (OUT == kFP32) static_cast<float *>(a.y)[at + i] = v;
        else static_cast<uint16_t *>(a.y)[at + i] = (uint16_t)out_bits<OUT>(v);
      }
    }
  }
}

template <int OUT, int FT, int TT, int WF, int WT>
hipError_t launch(GemmArgs a, hipStream_t stream) {
  a.f_tiles = (int32_t)((a.w.rows + 16 * FT * WF - 1) / (16 * FT * WF));
  a.m_tiles = (int32_t)((a.x.rows + 16 * TT * WT - 1) / (16 * TT * WT));
  hipLaunchKernelGGL((mx_gemm_kernel<OUT, FT, TT, WF, WT>),
                     dim3((unsigned)((int64_t)a.f_tiles * a.m_tiles)), dim3(64 * WF * WT), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace

int64_t mx_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

bool mx_gemm_fits(int64_t M, int64_t N) {
  return ((M + 127) / 128) * ((N + 127) / 128) * 512 <= 0xffffffffll;
}

hipError_t launch_mx_gemm(const MxMatrix &x, const MxProduct &p, void *, hipStream_t stream) {
  GemmArgs a{};
  a.w = p.w;
  a.x = x;
  a.bias = p.bias;
  a.y = p.y;
  a.ldy = p.ldy;
  if (p.out_dtype == kFP32) return launch<kFP32, 4, 4, 2, 2>(a, stream);
  if (p.out_dtype == kFP16) return launch<kFP16, 4, 4, 2, 2>(a, stream);
  return launch<kBF16, 4, 4, 2, 2>(a, stream);
}

}  // namespace nf4
