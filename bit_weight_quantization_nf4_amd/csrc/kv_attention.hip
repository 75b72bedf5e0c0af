// kv_attention.hip -- host side of the attention to a 4-bit cache: how a call is
// split, and the kernel that joins the splits of a row.
#include "kv_attention_kernel.h"

namespace nf4 {

using namespace kvattn;

namespace {

// Joins the ranges of a row: out = sum_i O_i 2^(m_i - m) / sum_i l_i 2^(m_i - m), in
// range order within a wave. ROWS_APART: each of the workgroup's waves has a row of
// its own, else they share one and add up in wave order. Rows that see nothing
// become zeros.
constexpr int kJoinWaves = 4;

template <int D, int DT, bool ROWS_APART>
__global__ __launch_bounds__(64 * kJoinWaves) void kv_attention_join_kernel(AttnArgs, int align) {
  constexpr int C = (D + 127) / 128;  // element pairs of a lane, at 2 lane + 128 c
  constexpr int SW = ROWS_APART ? 1 : kJoinWaves;  // waves of a row
  __shared__ float acc[SW][D];
  __shared__ float sums[SW];
  fetch_args();
  KernelArgs &args = *kernel_args();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sw = ROWS_APART ? 0 : wave;
  const int pair = ROWS_APART ? (int)blockIdx.x * kJoinWaves + wave : (int)blockIdx.x;
  const int h = (int)blockIdx.y, seq = (int)blockIdx.z;
  const int wb = args.wg_blocks == 1 ? 0 : pair / args.wg_rows, row = pair - wb * args.wg_rows;
  const Block blk = block_of(args, sequence_of(args, seq), wb * args.wg_rows, args.wg_rows);
  if (pair >= blk.pairs) return;
  const int range = range_of(blk, args.splits, align);
  const int pieces = range > 0 ? (blk.hi - blk.lo - 1) / range + 1 : 0;  // (no sum past 2^31)
  const int64_t base = item_of(args, seq, h, wb) * args.splits * args.part_rows + row;
  auto part_row = [&](int i) { return base + (int64_t)i * args.part_rows; };

  float top = -__builtin_inff();
  for (int i = lane; i < pieces; i += 64) top = fmaxf(top, args.stats[part_row(i)].x);
  top = max_over_groups(row16_max(top));
  const float use = top == -__builtin_inff() ? 0.0f : top;

  float sum = 0.0f;
  f32x2 o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = f32x2{0.0f, 0.0f};
#pragma unroll 4
  for (int i = sw; i < pieces; i += SW) {
    const int64_t at = part_row(i);
    const float2 st = args.stats[at];
    const float f = __builtin_amdgcn_exp2f(st.x - use);
    sum = __builtin_fmaf(st.y, f, sum);
    const float *p = args.part + at * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 2 * lane + 128 * c;
      if (e < D) {
        const f32x2 v = *reinterpret_cast<const f32x2 *>(p + e);
        o[c].x = __builtin_fmaf(v.x, f, o[c].x);
        o[c].y = __builtin_fmaf(v.y, f, o[c].y);
      }
    }
  }
  if constexpr (!ROWS_APART) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 2 * lane + 128 * c;
      if (e < D) *reinterpret_cast<f32x2 *>(&acc[sw][e]) = o[c];
    }
    if (lane == 0) sums[sw] = sum;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int i = 1; i < SW; ++i) {
      sum += sums[i];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = 2 * lane + 128 * c;
        if (e < D) o[c] += *reinterpret_cast<const f32x2 *>(&acc[i][e]);
      }
    }
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  const int token = pair / args.group;
  const int64_t at = (int64_t)(blk.first + token) * args.out_row +
                     (int64_t)(h * args.group + pair - token * args.group) * args.out_head;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 2 * lane + 128 * c;
    if (e >= D) continue;
    if constexpr (DT == kFP32)
      *reinterpret_cast<f32x2 *>(static_cast<float *>(args.out) + at + e) = o[c] * inv;
    else
      *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(args.out) + at + e) =
          pack2<DT>(o[c].x * inv, o[c].y * inv);
  }
}

// ------------------------------------------------------------------- host

// Waves have rows of their own where that gives a workgroup for every CU: they then
// merge nothing (1024 and 512 rows at 5000 and 2500 positions, 32 query heads of 8: 213
// us, 247 merged; 4 sequences of 256 rows at 1000: 54, 65). With fewer the waves that
// share a block finish sooner (512 rows at 4096: 87 merged, 109 apart; 32 rows at 2048:
// 17, 93). Sequences of fewer rows than a workgroup's leave its waves without any (64 of
// one row at 4000: 63 merged, 165).
constexpr int kApartMinRows = 128;

// From how many positions on an item is split, and the fewest that a range has. The
// second launch takes about as long as 1500 positions of a workgroup: 1536 positions,
// one row, 15.0 us whole and 17.8 split, 2048 18.0 either way, 4096 29.6 and 18.0.
// Ranges of 256, 512 and 1024 differ by less than 1 us. A range of waves with rows of
// their own costs more to join (1024 rows at 2048 positions: 94.7 whole, 99.0 in two; at
// 4096 176.7 whole, 162.9 in two).
constexpr int64_t kSplitFrom = 2048, kMinRange = 512;
constexpr int64_t kSplitFromApart = 4096, kMinRangeApart = 2048;
// What a range costs besides its positions, in positions.
constexpr int64_t kRangeCost = 700;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The split of a call: blocks of rows, and ranges of positions.
Plan plan_of(const KvAttentionSizes &z) {
  Plan p;
  const int64_t pairs = (int64_t)z.max_rows * (z.heads / z.kv_heads);
  const int64_t apart_blocks = ceil_div(pairs, 16 * max_tiles(z.head_dim) * kApartWaves);
  p.merge = pairs < kApartMinRows ||
            (int64_t)z.batch * z.kv_heads * apart_blocks < device_cu_count();
  // More rows than a tile's: blocks of two tiles look a position's codes up once for both.
  // (8 kv heads of 128 in bf16, 16 sequences at 6000 positions: 20 rows a kv head 43 us, in
  // one-tile blocks 53; 48 rows 63, 70; 96 rows 118, 114. Short calls lose by the second
  // tile's merge: one sequence at 1000, 20 rows 16.6, 15.9.)
  p.tiles = p.merge && pairs <= 16 ? 1 : max_tiles(z.head_dim);
  p.wg_rows = 16 * p.tiles * (p.merge ? 1 : kApartWaves);
  p.wg_blocks = (int)ceil_div(pairs, p.wg_rows);
  p.align = kStep * (p.merge ? kMergeWaves : 1);
  const int64_t items = (int64_t)z.batch * z.kv_heads * p.wg_blocks;
  // positions that a row sees at most, in units of the time that one takes at 16 bits
  // and head_dim 128
  int64_t span = z.max_len;
  if (z.window > 0 && span > (int64_t)z.window + z.max_rows) span = (int64_t)z.window + z.max_rows;
  const int64_t weight = z.head_dim * (z.dtype == kFP32 ? 3 : 1);
  int64_t s = 1;
  if (span * weight >= (p.merge ? kSplitFrom : kSplitFromApart) * 128) {
    // as many ranges as fill the device once, or twice where workgroups of uneven
    // sequences share a CU, whichever is done first: every round of workgroups takes a
    // range's time. (Sequences up to 8000, 8 kv heads, one row: 40 of them 64.6 us with
    // two rounds allowed, 79.0 with one; of equal length 4000, 53.2 and 49.1. Where a
    // workgroup has a CU to itself, 10 sequences of 16 rows at 4000, 44.4 with one
    // round, 54.7 with two.)
    // (as many workgroups of a CU as the kernel's kWavesPerSimd allows)
    const bool two = !p.merge || (p.tiles == 1 && z.head_dim <= 128 && z.dtype != kFP32);
    const int64_t slots = (two ? 2 : 1) * (int64_t)device_cu_count();
    int64_t best = ceil_div(items, slots) * (span + kRangeCost);
    for (int rounds = 1; items > 0 && rounds <= (p.merge && two ? 2 : 1); ++rounds) {
      const int64_t c = rounds * slots / items;
      if (c <= 1) continue;
      const int64_t cost = ceil_div(items * c, slots) * (span / c + kRangeCost);
      if (cost >= best) continue;
      best = cost;
      s = c;
    }
    const int64_t least = p.merge ? kMinRange * 128 / weight : kMinRangeApart;
    const int64_t most = ceil_div(span, least > 0 ? least : 1);
    if (s > most) s = most;
  }
  if (s < 1) s = 1;
  p.splits = (int)s;
  p.part_rows = (int)(pairs < p.wg_rows ? pairs : p.wg_rows);
  p.stats = s > 1 ? items * s * p.part_rows : 0;
  p.part_floats = p.stats * z.head_dim;
  return p;
}

// c' = c mu of the 16 codes as two fp16 values.
constexpr double kMuNF4 = 128 * 1.6776896, kMuFP4 = 128 * 6.0;

uint32_t f16_bits(double v, double *rest) {
  const _Float16 h = (_Float16)v;
  if (rest != nullptr) *rest = v - (double)h;
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}

template <int D, int DT>
hipError_t launch_join(const AttnArgs &a, const Plan &p, hipStream_t stream) {
  const int rows = a.max_rows * a.group;
  dim3 grid((unsigned)rows, (unsigned)a.kv.kv_heads, (unsigned)a.kv.batch);
  if (p.merge) {
    hipLaunchKernelGGL((kv_attention_join_kernel<D, DT, false>), grid, dim3(64 * kJoinWaves), 0,
                       stream, a, p.align);
  } else {
    grid.x = (unsigned)ceil_div(rows, kJoinWaves);
    hipLaunchKernelGGL((kv_attention_join_kernel<D, DT, true>), grid, dim3(64 * kJoinWaves), 0,
                       stream, a, p.align);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const AttnArgs &a, const Plan &p, const KvShape &sh, hipStream_t stream) {
  const hipError_t e = launch_shape<DT>(a, p, sh.head_dim, sh.blocksize, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  switch (sh.head_dim) {
    case 64: return launch_join<64, DT>(a, p, stream);
    case 96: return launch_join<96, DT>(a, p, stream);
    case 128: return launch_join<128, DT>(a, p, stream);
    case 192: return launch_join<192, DT>(a, p, stream);
    case 256: return launch_join<256, DT>(a, p, stream);
  }
  return hipErrorNotSupported;
}

}  // namespace

int64_t kv_attention_bytes(const KvAttentionSizes &z) {
  const Plan p = plan_of(z);
  const int64_t bytes = p.part_floats * 4 + p.stats * 8;
  return (bytes + 255) / 256 * 256;
}

bool kv_attention_fits(const KvAttentionSizes &z) {
  const int64_t pairs = (int64_t)z.max_rows * (z.heads / z.kv_heads);
  if (pairs * (64 * kJoinWaves) > 0xffffffffll || z.batch > 65535 || z.kv_heads > 65535)
    return false;
  if (z.heads / z.kv_heads > 65535) return false;  // a head's number is exact in row_at
  const Plan p = plan_of(z);
  return (int64_t)p.wg_blocks * p.splits * (64 * kMergeWaves) <= 0xffffffffll;
}

hipError_t launch_kv_attention(const KvArgs &kv, const KvShape &sh, const KvAttentionSizes &z,
                               const KvAttentionCall &c, hipStream_t stream) {
  const Plan p = plan_of(z);
  AttnArgs a;
  a.kv = kv;
  a.q = c.q;
  a.out = c.out;
  a.q_row = c.q_row;
  a.q_head = c.q_head;
  a.out_row = c.out_row;
  a.out_head = c.out_head;
  a.group = z.heads / z.kv_heads;
  a.max_rows = z.max_rows;
  a.causal = c.causal;
  a.window = z.window;
  a.wg_rows = p.wg_rows;
  a.wg_blocks = p.wg_blocks;
  a.splits = p.splits;
  a.part_rows = p.part_rows;
  a.part = static_cast<float *>(c.workspace);
  a.stats = reinterpret_cast<float2 *>(a.part + p.part_floats);
  const double mu = sh.quant_type == kQuantFP4 ? kMuFP4 : kMuNF4;
  a.f = (float)((double)c.scale * 1.4426950408889634 / mu);
  a.inv_mu = (float)(1.0 / mu);
  const CodeTables &t = code_tables(sh.quant_type);
  for (int i = 0; i < 16; ++i) {
    double rest;
    const uint32_t c1 = f16_bits((double)t.value[i] * mu, &rest);
    a.codes[i] = c1 | f16_bits(rest, nullptr) << 16;
  }
  if (sh.dtype == kFP32) return launch_dt<kFP32>(a, p, sh, stream);
  if (sh.dtype == kFP16) return launch_dt<kFP16>(a, p, sh, stream);
  return launch_dt<kBF16>(a, p, sh, stream);
}

}  // namespace nf4
