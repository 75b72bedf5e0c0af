// kv_attention.hip -- host side of the attention to a 4-bit cache: how a call is
// split, and the kernel that joins the splits of a row.
#include "kv_attention_kernel.h"

namespace nf4 {

using namespace kvattn;

namespace {

// Joins the splits of a row: out = sum_s O_s 2^(m_s - m) / sum_s l_s 2^(m_s - m),
// in split order within each of the workgroup's waves, then in wave order.
constexpr int kJoinWaves = 4;

template <int D, int DT>
__global__ __launch_bounds__(64 * kJoinWaves) void kv_attention_join_kernel(AttnArgs args, int rows) {
  constexpr int C = D / 64 > 0 ? D / 64 : 1;  // elements of a lane, at lane + 64 c
  __shared__ float acc[kJoinWaves][D];
  __shared__ float sums[kJoinWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = (int)blockIdx.x, h = (int)blockIdx.y, seq = (int)blockIdx.z;
  const int rb = pair / rows, row = pair - rb * rows;
  const Block blk = block_of(args, seq, rb, rows);
  if (pair >= blk.pairs) return;
  const int chunk = chunk_of(blk, args.splits);
  const int used = chunk > 0 ? (blk.hi - blk.lo + chunk - 1) / chunk : 0;
  const int64_t item = ((int64_t)seq * args.kv.kv_heads + h) * args.row_blocks + rb;
  const int64_t base = item * args.splits * args.part_rows + row;

  float top = -__builtin_inff();
  for (int s = lane; s < used; s += 64)
    top = fmaxf(top, args.stats[base + (int64_t)s * args.part_rows].x);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  const float use = top == -__builtin_inff() ? 0.0f : top;

  float sum = 0.0f, o[C + 1];
#pragma unroll
  for (int c = 0; c <= C; ++c) o[c] = 0.0f;
  for (int s = wave; s < used; s += kJoinWaves) {
    const int64_t at = base + (int64_t)s * args.part_rows;
    const float2 st = args.stats[at];
    const float f = __builtin_amdgcn_exp2f(st.x - use);
    sum = __builtin_fmaf(st.y, f, sum);
    const float *p = args.part + at * D;
#pragma unroll
    for (int c = 0; c < (D + 63) / 64; ++c)
      if (lane + 64 * c < D) o[c] = __builtin_fmaf(p[lane + 64 * c], f, o[c]);
  }
#pragma unroll
  for (int c = 0; c < (D + 63) / 64; ++c)
    if (lane + 64 * c < D) acc[wave][lane + 64 * c] = o[c];
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  const int token = pair / args.group;
  const int64_t at = (int64_t)(blk.first + token) * args.out_row +
                     (int64_t)(h * args.group + pair - token * args.group) * args.out_head;
  float l = sums[0];
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) l += sums[i];
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  for (int e = threadIdx.x; e < D; e += 64 * kJoinWaves) {
    float v = acc[0][e];
#pragma unroll
    for (int i = 1; i < kJoinWaves; ++i) v += acc[i][e];
    v *= inv;
    if constexpr (DT == kFP32) static_cast<float *>(args.out)[at + e] = v;
    else static_cast<uint16_t *>(args.out)[at + e] = (uint16_t)out_bits<DT>(v);
  }
}

// ------------------------------------------------------------------- host

// The split of a call: 16-row tiles of a workgroup, and ranges of positions so
// that the launch has about two workgroups for each CU.
Plan plan_of(int64_t batch, int64_t max_rows, int64_t max_len, int64_t heads, int64_t kv_heads,
             int head_dim) {
  Plan p;
  const int64_t pairs = max_rows * (heads / kv_heads);
  p.tiles = pairs <= 16 ? 1 : max_tiles(head_dim);
  const int64_t rows = 16 * p.tiles;
  const int64_t rb = (pairs + rows - 1) / rows;
  const int64_t items = batch * kv_heads * rb;
  const int64_t want = 2 * (int64_t)device_cu_count();
  int64_t s = items > 0 ? (want + items - 1) / items : 1;
  const int64_t most = (max_len + kChunkAlign - 1) / kChunkAlign;
  if (s > most) s = most;
  if (s < 1) s = 1;
  p.row_blocks = (int)rb;
  p.splits = (int)s;
  p.part_rows = (int)(pairs < rows ? pairs : rows);
  p.part_floats = s > 1 ? items * s * p.part_rows * head_dim : 0;
  p.stats = s > 1 ? items * s * p.part_rows : 0;
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
  const dim3 grid((unsigned)(a.max_rows * a.group), (unsigned)a.kv.kv_heads,
                  (unsigned)a.kv.batch);
  hipLaunchKernelGGL((kv_attention_join_kernel<D, DT>), grid, dim3(64 * kJoinWaves), 0, stream, a,
                     16 * p.tiles);
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

int64_t kv_attention_bytes(int batch, int max_rows, int max_len, int heads, int kv_heads,
                           int head_dim) {
  const Plan p = plan_of(batch, max_rows, max_len, heads, kv_heads, head_dim);
  const int64_t bytes = p.part_floats * 4 + p.stats * 8;
  return (bytes + 255) / 256 * 256;
}

bool kv_attention_fits(int batch, int max_rows, int max_len, int heads, int kv_heads,
                       int head_dim) {
  const int64_t pairs = (int64_t)max_rows * (heads / kv_heads);
  if (pairs * (64 * kJoinWaves) > 0xffffffffll || batch > 65535 || kv_heads > 65535) return false;
  const Plan p = plan_of(batch, max_rows, max_len, heads, kv_heads, head_dim);
  return (int64_t)p.row_blocks * p.splits * kThreads <= 0xffffffffll;
}

hipError_t launch_kv_attention(const KvArgs &kv, const KvShape &sh, const KvAttentionCall &c,
                               hipStream_t stream) {
  const int heads = c.group * kv.kv_heads;
  const Plan p = plan_of(kv.batch, c.max_rows, c.max_len, heads, kv.kv_heads, sh.head_dim);
  AttnArgs a;
  a.kv = kv;
  a.q = c.q;
  a.out = c.out;
  a.q_row = c.q_row;
  a.q_head = c.q_head;
  a.out_row = c.out_row;
  a.out_head = c.out_head;
  a.group = c.group;
  a.max_rows = c.max_rows;
  a.causal = c.causal;
  a.window = c.window;
  a.row_blocks = p.row_blocks;
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
    a.hi[i] = f16_bits((double)t.value[i] * mu, &rest);
    a.lo[i] = f16_bits(rest, nullptr);
  }
  if (sh.dtype == kFP32) return launch_dt<kFP32>(a, p, sh, stream);
  if (sh.dtype == kFP16) return launch_dt<kFP16>(a, p, sh, stream);
  return launch_dt<kBF16>(a, p, sh, stream);
}

}  // namespace nf4
