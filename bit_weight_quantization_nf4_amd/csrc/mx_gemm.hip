// mx_gemm.hip -- products of many rows with a microscaled 4-bit weight.
//
// y[m][f] = sum_k x[m][k] w[f][k] on 32x32x64 matrix-core steps, the weight as the first
// operand. A workgroup computes a tile of features x rows of x, its waves parts of it: FT x TT
// tiles of 32 x 32 each. K goes by 256: both operands' codes, 128 bytes a row, and scales
// are brought straight to LDS, into one of two stages, and multiplied in two steps of 128. A wave
// reads a step's operands into registers while the step before is multiplied, so a stage is free
// for new loads from its second step on, and these have that step and the next to come.
// (Whole cache lines: with steps of 64 bytes a row each line came twice; 2048 x 14336 x 4096, with
// four waves of 128 x 128 each, 98 us and 89.)
//
// Which rows of the operands make up a matrix-core tile is free. Tile i of a wave takes rows FT p
// + i, p < 32: a lane finds the scales of its FT rows side by side in LDS and holds runs of 4 FT
// neighbouring features of a result.
//
// LDS: the sixteen 16-byte pieces of two neighbouring rows lie at places xor'ed with p, which
// differs between the sixteen lanes that are read together (no conflicts; 8192 cubed 318 -> 276 us).
//
// What bounds it, on one MI355X: 8192 cubed takes 250 to 280 us, 3.9 to 4.4 PFLOP/s; without its
// loads and stores 209 us, 5.3 PFLOP/s, where a single workgroup's steps take half the time that
// they do with all CUs at work: the matrix cores' clock under that load. 2048 x 14336 x 4096, 448
// tiles in two rounds of 256: 64 to 75 us, 3.2 to 3.7 PFLOP/s; the second round leaves a quarter of
// the CUs idle, and each round's results, 33 MB, are written while nothing is multiplied.
#include <type_traits>

#include "mx_internal.h"

namespace nf4 {

namespace {

struct GemmArgs {
  MxMatrix w, x;
  const void *bias;
  void *y;
  int64_t ldy;
  int32_t f_tiles, m_tiles;
  // ranges of K: 128-wide steps of each (even), and how far their results lie apart
  int32_t split_steps;
  int64_t split_stride;
};

constexpr int kStages = 2;
constexpr int kBufferFlags = 0x00020000;
// s_waitcnt: all LDS reads, and all but n of the loads.
constexpr int waitcnt(int n) { return 0x0070 | (n & 15) | (n >> 4) << 14; }

typedef __attribute__((address_space(3))) void *LdsPtr;

// A place in LDS that loads write to, as one that the compiler knows nothing of: it would have
// every read of what may be the same array wait for them. The kernel's own waits and barriers
// order the two.
__device__ __forceinline__ LdsPtr lds_place(void *p) {
  uint32_t at = (uint32_t)(uintptr_t)(LdsPtr)p;
  asm("" : "+s"(at));
  return (LdsPtr)(uintptr_t)at;
}

// A wave-uniform value that 64-bit arithmetic left in vector registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint8_t *uniform(const uint8_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<uint8_t *>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 |
                                     (uint32_t)uniform((int)v));
}

// 32x32x64 step on E2M1 operands: acc += A(32x64) B(64x32). Lane (p = lane & 31, h = lane >> 5) gives
// elements 32 h .. 32 h + 31 of row p of A and of column p of B, and these blocks' scales as byte S
// of sa and sb; it holds rows 8 q + 4 h + r of column p at acc[4 q + r].
template <int S>
__device__ __forceinline__ f32x16 mfma_mx32(mx_u32x4 a, mx_u32x4 b, f32x16 acc, uint32_t sa,
                                            uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, S, (int)sa, S, (int)sb);
}

// The order of a step's instructions: the loads first, LA behind each product, then the LDS reads,
// one behind each product, then the other products.
template <int PRODUCTS, int READS, int LOADS, int LA = 1>
__device__ __forceinline__ void interleave() {
  if constexpr (PRODUCTS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (LOADS > 0) {
      __builtin_amdgcn_sched_group_barrier(0x020, LOADS < LA ? LOADS : LA, 0);
      interleave<PRODUCTS - 1, READS, (LOADS < LA ? 0 : LOADS - LA), LA>();
    } else if constexpr (READS > 0) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      interleave<PRODUCTS - 1, READS - 1, 0, LA>();
    } else {
      interleave<PRODUCTS - 1, 0, 0, LA>();
    }
  }
}

// WF x WT waves, each with FT x TT tiles (features x rows of x).
template <int OUT, int FT, int TT, int WF, int WT, int WAVES_PER_EU>
__global__ __launch_bounds__(64 * WF * WT) __attribute__((amdgpu_waves_per_eu(WAVES_PER_EU, WAVES_PER_EU)))
void mx_gemm_kernel(GemmArgs a) {
  constexpr int kWaves = WF * WT;
  constexpr int BF = 32 * FT * WF, BT = 32 * TT * WT;
  constexpr int kRows = BF + BT;  // of both operands, the weight's first
  constexpr int kLoads = kRows / 8 / kWaves, kLoadsF = BF / 8 / kWaves;
  static_assert(BF % (8 * kWaves) == 0 && BT % (8 * kWaves) == 0, "a wave's loads of each operand");
  constexpr int kScaleLoads = 2 * kRows / 64 / kWaves;  // 64 rows of a half each
  static_assert(2 * kRows % (64 * kWaves) == 0 && BF % 64 == 0, "whole loads");
  static_assert(FT > 1 && TT > 1 && (FT & (FT - 1)) == 0 && (TT & (TT - 1)) == 0, "two rows of one p");
  __shared__ __attribute__((aligned(128))) uint8_t codes[kStages][128 * kRows];
  __shared__ __attribute__((aligned(16))) uint32_t scales[kStages][2][kRows];
  __shared__ __attribute__((aligned(16))) float bias[BF];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pl = lane & 31, h = lane >> 5;
  const int wf = wave % WF, wt = wave / WF;
  const int tiles = a.f_tiles * a.m_tiles;
  const int split = uniform((int)blockIdx.x / tiles), tile = (int)blockIdx.x - split * tiles;
  const int mb = uniform(tile / a.f_tiles), fb = tile - mb * a.f_tiles;
  const int64_t f0 = (int64_t)fb * BF, m0 = (int64_t)mb * BT;
  const int f_rows = uniform((int)(a.w.rows - f0 < BF ? a.w.rows - f0 : BF));
  const int m_rows = uniform((int)(a.x.rows - m0 < BT ? a.x.rows - m0 : BT));
  const uint32_t half = (uint32_t)a.w.padded / 2;
  const int step0 = split * a.split_steps, left = a.w.padded / kMxStep - step0;
  const int steps = left < a.split_steps ? left : a.split_steps;

  // a load brings 8 rows' codes, or 64 rows' scales; rows past the last read zeros
  const __amdgpu_buffer_rsrc_t fc = __builtin_amdgcn_make_buffer_rsrc(
      uniform(a.w.codes + f0 * half), (short)0, (int)((uint32_t)f_rows * half), kBufferFlags);
  const __amdgpu_buffer_rsrc_t mc = __builtin_amdgcn_make_buffer_rsrc(
      uniform(a.x.codes + m0 * half), (short)0, (int)((uint32_t)m_rows * half), kBufferFlags);
  uint32_t code_at[kLoads];
  uint32_t late = 0;  // loads (by bit) of which the lane's piece is of the stage's second half
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const bool of_w = i < kLoadsF;
    const int two = 8 * (wave + kWaves * (of_w ? i : i - kLoadsF)) + 2 * (lane >> 4);  // rows two, two + 1
    const int piece = (lane & 15) ^ (two / (of_w ? FT : TT) & 15);
    code_at[i] = (uint32_t)(two + (piece >> 3)) * half + 16 * (piece & 7) + 64 * (uint32_t)step0;
    late |= (uint32_t)(piece >> 2 & 1) << i;
  }
  // the wave's scales: loads wave, wave + kWaves, ... of the halves' rows
  const int64_t stride_f = 4 * a.w.rows, stride_m = 4 * a.x.rows;
  const uint8_t *base_f = uniform(a.w.scales + step0 * stride_f + 4 * f0);
  const uint8_t *base_m = uniform(a.x.scales + step0 * stride_m + 4 * m0);
  // stage b, of the stages in order. (What is past the last step, a stage or its second half, is
  // loaded as zeros, so that each stage issues as many loads and none leaves the matrix.)
  auto fill = [&](int b) {
    const int stage = b % kStages;
    const bool there = 2 * b < steps;
    const uint32_t at = there ? 128u * (uint32_t)b : 0u;
    const uint32_t out = !there ? 0xffffffffu : 2 * b + 1 < steps ? 0u : late;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const LdsPtr dst = lds_place(&codes[stage][1024 * (wave + kWaves * i)]);
      const uint32_t none = out << (31 - i) & 0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(i < kLoadsF ? fc : mc, dst, 16,
                                               (int)(code_at[i] | none), (int)at, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int l = wave + kWaves * i, s = l / (kRows / 64), r0 = 64 * (l % (kRows / 64));
      const bool of_w = r0 < BF, here = 2 * b + s < steps;
      const uint8_t *base = (of_w ? base_f : base_m) + (s ? (of_w ? stride_f : stride_m) : 0);
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          uniform(base), (short)0, here ? 4 * (of_w ? f_rows : m_rows) : 0, kBufferFlags);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, lds_place(&scales[stage][s][r0]), 4,
                                               4 * ((of_w ? r0 : r0 - BF) + lane), 0, 0, 0);
    }
    base_f += there ? 2 * stride_f : 0;
    base_m += there ? 2 * stride_m : 0;
  };

  const int row_f = FT * (32 * wf + pl), row_m = TT * (32 * wt + pl);
  struct Operands {
    mx_u32x4 f[FT][2], m[TT][2];  // both halves of the step
    uint32_t sf[FT], sm[TT];
  };
  auto place = [&](int row, int piece) {
    return 128 * (row & ~1) + 16 * ((8 * (row & 1) + piece) ^ (pl & 15));
  };
  // step t's operands
  auto read = [&](int t, Operands &o) {
    const int stage = t / 2 % kStages, c = 4 * (t & 1);
#pragma unroll
    for (int i = 0; i < FT; ++i) o.sf[i] = scales[stage][t & 1][row_f + i];
#pragma unroll
    for (int j = 0; j < TT; ++j) o.sm[j] = scales[stage][t & 1][BF + row_m + j];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < FT; ++i)
        o.f[i][s] = *reinterpret_cast<const mx_u32x4 *>(&codes[stage][place(row_f + i, c + 2 * s + h)]);
#pragma unroll
      for (int j = 0; j < TT; ++j)
        o.m[j][s] = *reinterpret_cast<const mx_u32x4 *>(&codes[stage][128 * BF + place(row_m + j, c + 2 * s + h)]);
    }
  };
  f32x16 acc[FT][TT];
  auto multiply = [&](const Operands &o) {
    // a lane's scales of the step's halves: bytes 0 and 2
    uint32_t sf[FT], sm[TT];
#pragma unroll
    for (int i = 0; i < FT; ++i) sf[i] = o.sf[i] >> (8 * h);
#pragma unroll
    for (int j = 0; j < TT; ++j) sm[j] = o.sm[j] >> (8 * h);
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = mfma_mx32<0>(o.f[i][0], o.m[j][0], acc[i][j], sf[i], sm[j]);
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = mfma_mx32<2>(o.f[i][1], o.m[j][1], acc[i][j], sf[i], sm[j]);
  };
  constexpr int kMem = kLoads + kScaleLoads;
  constexpr int kLds = 2 * (FT + TT) + (FT + 3) / 4 + (TT + 3) / 4, kProducts = 2 * FT * TT;
  // Step t: the operands of step t + 1 on their way while it is multiplied; in a stage's second
  // step, from which on nobody reads it, the loads of the stage after the next too. (The reads are
  // done at each barrier.) Then the loads of the next stage have come, before its first operands are
  // read. Bare barriers: a fence would wait for all loads.
  auto first = [&](int t, const Operands &now, Operands &next) {
    read(t + 1, next);
    multiply(now);
    interleave<kProducts, kLds, 0>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt(0));
    __builtin_amdgcn_s_barrier();
  };
  auto second = [&](int t, const Operands &now, Operands &next) {
    fill(t / 2 + 2);
    read(t + 1, next);
    multiply(now);
    interleave<kProducts, kLds, kMem>();
    __builtin_amdgcn_sched_barrier(0);
  };

  fill(0);
  fill(1);
  for (int i = threadIdx.x; i < BF; i += 64 * kWaves) {
    float v = 0.0f;
    if (a.bias != nullptr && i < f_rows) {
      if constexpr (OUT == kFP32) v = static_cast<const float *>(a.bias)[f0 + i];
      else v = widen16<OUT>(static_cast<const uint16_t *>(a.bias)[f0 + i]);
    }
    bias[i] = v;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0));
  __syncthreads();
  // the sums begin with the bias
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[i][j][e] = bias[FT * (32 * wf + 8 * (e / 4) + 4 * h + e % 4) + i];
  Operands o0, o1;
  read(0, o0);
  int t = 0;
  for (; t + 1 < steps; t += 2) {
    first(t, o0, o1);
    second(t + 1, o1, o0);
  }
  if (t < steps) multiply(o0);
  // Loads past the last step may still be on their way to LDS, and other waves at its operands.
  __builtin_amdgcn_s_waitcnt(waitcnt(0));
  __syncthreads();

  // Results leave through the wave's own part of LDS, 32 rows of x at a time, as whole lines. Of
  // row TT p + j of x a lane has features FT (8 q + 4 h + r) + i: a run of 4 FT for each q.
  using Out = std::conditional_t<OUT == kFP32, float, uint16_t>;
  constexpr int kRun = 4 * FT, kWide = 32 * FT;     // features of a run, of the wave
  constexpr int kPitch = kWide * sizeof(Out) + 16;  // (apart by a piece: no bank conflicts)
  constexpr int kEach = 16 / sizeof(Out), kPerRow = kWide / kEach;  // a lane's piece
  static_assert(32 * kPitch * kWaves <= sizeof(codes), "room");
  Out *out = static_cast<Out *>(a.y) + split * a.split_stride;
  uint8_t *mine = codes[0] + wave * (32 * kPitch);
  const int f_first = 32 * FT * wf;  // of the tile
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    __builtin_amdgcn_sched_barrier(0);  // (rows ahead of their turn would spill)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[e] = acc[e % FT][j][4 * q + e / FT];
      uint4 *dst = reinterpret_cast<uint4 *>(mine + pl * kPitch + kRun * (2 * q + h) * sizeof(Out));
#pragma unroll
      for (int e = 0; e < kRun; e += kEach) {
        if constexpr (OUT == kFP32)
          dst[e / kEach] = make_uint4(__float_as_uint(v[e]), __float_as_uint(v[e + 1]),
                                      __float_as_uint(v[e + 2]), __float_as_uint(v[e + 3]));
        else
          dst[e / kEach] = make_uint4(pack2<OUT>(v[e], v[e + 1]), pack2<OUT>(v[e + 2], v[e + 3]),
                                      pack2<OUT>(v[e + 4], v[e + 5]), pack2<OUT>(v[e + 6], v[e + 7]));
      }
    }
#pragma unroll 2
    for (int k = 0; k < 32 * kPerRow / 64; ++k) {
      const int at = 64 * k + lane, row = at / kPerRow, f = f_first + at % kPerRow * kEach;
      const uint4 piece = *reinterpret_cast<const uint4 *>(mine + row * kPitch + at % kPerRow * 16);
      const int m = TT * (32 * wt + row) + j;
      if (m >= m_rows) continue;
      Out *dst = out + (m0 + m) * a.ldy + f0 + f;
      if (f + kEach <= f_rows) {  // (of any alignment: the memory instructions take it)
        *reinterpret_cast<mx_any_u32x4 *>(dst) = mx_u32x4{piece.x, piece.y, piece.z, piece.w};
      } else {
        const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (f + e >= f_rows) continue;
          if constexpr (OUT == kFP32) dst[e] = __uint_as_float(w[e]);
          else dst[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
        }
      }
    }
  }
}

// Joins the ranges of K: y = sum over the ranges, in order, and the bias. Four features a thread.
template <int OUT>
__global__ __launch_bounds__(256) void mx_gemm_join_kernel(const float *part, int splits,
                                                           int64_t split_stride, int64_t pitch,
                                                           const void *bias, int64_t M, int64_t N,
                                                           void *y, int64_t ldy) {
  const int64_t quads = pitch / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= M * quads) return;
  const int64_t m = i / quads, f = 4 * (i - m * quads);
  const float *p = part + m * pitch + f;
  f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * split_stride);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (f + e >= N) continue;
    float r = v[e];
    if constexpr (OUT == kFP32) {
      if (bias != nullptr) r += static_cast<const float *>(bias)[f + e];
      static_cast<float *>(y)[m * ldy + f + e] = r;
    } else {
      if (bias != nullptr) r += widen16<OUT>(static_cast<const uint16_t *>(bias)[f + e]);
      static_cast<uint16_t *>(y)[m * ldy + f + e] = (uint16_t)out_bits<OUT>(r);
    }
  }
}

// ------------------------------------------------------------------- host

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  bool large;       // tiles of 256 x 256, else of 128 x 128
  int splits;       // ranges of K
  int split_steps;  // 128-wide steps of each
};

int64_t tiles_of(int64_t M, int64_t N, bool large) {
  const int side = large ? 256 : 128;
  return ceil_div(M, side) * ceil_div(N, side);
}

int64_t pitch_of(int64_t N) { return ceil_div(N, 4) * 4; }  // of a range's results

// Tiles and ranges by about the time that they take. In us, of 256-wide stages: a workgroup of
// large tiles has a CU to itself and takes 1.9 a stage where all CUs work, down to 1.3 with few, and
// 6 to begin and end; of small tiles 0.6 and 3, but 1.25 and 4 where two share a CU; a second launch 4
// and its traffic. (2048 x 14336 x 4096: large 75, small 80; 8192 cubed 280, 337; 4096 x 4096 x 4096:
// 40, 46; 2048 x 11008 x 4096: 60, 66, x 4096: 30, 25; 512 x 4096 x 4096: 25, 13; 1024 x 4096 x 14336:
// 58, 43. 128 x 4096 x 14336 in 1, 2, 4, 6, 8 ranges: 38, 26, 19, 18, 19; x 4096: 12.1, 13.6, 14.1,
// 16.1, 18.8.)
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  const int64_t cus = device_cu_count(), steps = mx_padded(K) / kMxStep, stages = ceil_div(steps, 2);
  const int64_t large = tiles_of(M, N, true), small = tiles_of(M, N, false);
  Plan best{true, 1, (int)steps};
  const int64_t rest = large % cus;  // of the last round of workgroups
  double least = (double)(large / cus) * (1.9 * (double)stages + 6);
  if (rest > 0) least += (1.3 + 0.6 * (double)rest / (double)cus) * (double)stages + 6;
  for (int64_t s = 1; s <= stages && s <= 32 && (s == 1 || s * small <= 2 * cus); ++s) {
    const int64_t each = ceil_div(stages, s);
    if (ceil_div(stages, each) != s) continue;  // the same ranges as of fewer
    double t = s * small <= cus ? 0.6 * (double)each + 3
                                : ((double)(s * small) / (double)(2 * cus) + 0.25) * (1.25 * (double)each + 4);
    if (s > 1) t += 4 + (double)(s * M) * (double)N * 8 / 4.5e6;
    if (t >= least) continue;
    least = t;
    best = Plan{false, (int)s, (int)(s > 1 ? 2 * each : steps)};
  }
  return best;
}

template <int OUT, int FT, int TT, int WF, int WT, int WAVES_PER_EU>
hipError_t launch(GemmArgs a, int splits, hipStream_t stream) {
  a.f_tiles = (int32_t)ceil_div(a.w.rows, 32 * FT * WF);
  a.m_tiles = (int32_t)ceil_div(a.x.rows, 32 * TT * WT);
  hipLaunchKernelGGL((mx_gemm_kernel<OUT, FT, TT, WF, WT, WAVES_PER_EU>),
                     dim3((unsigned)((int64_t)a.f_tiles * a.m_tiles * splits)), dim3(64 * WF * WT),
                     0, stream, a);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_plan(const GemmArgs &a, const Plan &plan, hipStream_t stream) {
  if (plan.large) return launch<OUT, 2, 4, 4, 2, 2>(a, plan.splits, stream);
  return launch<OUT, 2, 2, 2, 2, 2>(a, plan.splits, stream);
}

template <int OUT>
hipError_t launch_as(GemmArgs a, const Plan &plan, void *workspace, hipStream_t stream) {
  if (plan.splits == 1) return launch_plan<OUT>(a, plan, stream);
  GemmArgs b = a;
  b.bias = nullptr;
  b.y = workspace;
  b.ldy = pitch_of(a.w.rows);
  b.split_stride = a.x.rows * b.ldy;
  const hipError_t e = launch_plan<kFP32>(b, plan, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mx_gemm_join_kernel<OUT>),
                     dim3((unsigned)ceil_div(a.x.rows * (b.ldy / 4), 256)), dim3(256), 0, stream,
                     static_cast<const float *>(workspace), plan.splits, b.split_stride, b.ldy,
                     a.bias, a.x.rows, a.w.rows, a.y, a.ldy);
  return hipGetLastError();
}

}  // namespace

int64_t mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_of(M, N, K);
  return p.splits == 1 ? 0 : 4 * p.splits * M * pitch_of(N);
}

bool mx_gemm_fits(int64_t M, int64_t N) {
  // (products with several ranges are far smaller)
  return tiles_of(M, N, false) * 256 <= 0xffffffffll && tiles_of(M, N, true) * 512 <= 0xffffffffll;
}

MxGemmShape mx_gemm_shape(int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_of(M, N, K);
  return MxGemmShape{p.large ? 256 : 128, p.splits, p.split_steps};
}

hipError_t launch_mx_gemm(const MxMatrix &x, const MxProduct &p, void *workspace,
                          hipStream_t stream) {
  const Plan plan = plan_of(x.rows, p.w.rows, p.w.cols);
  GemmArgs a{};
  a.w = p.w;
  a.x = x;
  a.bias = p.bias;
  a.y = p.y;
  a.ldy = p.ldy;
  a.split_steps = plan.split_steps;
  if (p.out_dtype == kFP32) return launch_as<kFP32>(a, plan, workspace, stream);
  if (p.out_dtype == kFP16) return launch_as<kFP16>(a, plan, workspace, stream);
  return launch_as<kBF16>(a, plan, workspace, stream);
}

}  // namespace nf4
