// kv_attention_kernel.h -- attention of query rows to a key/value cache held in
// 4 bits.
//
// Mathematics. With code values c scaled by mu to c' = c mu, K = c'k ak / mu
// and V = c'v av / mu (ak, av the block scales), in log2 units
//   t_ij = f sum_b ak_jb (q_i . c'k_j)_b,   f = scale log2(e) / mu,
//   out_i = sum_j 2^(t_ij - m_i) av_j c'v_j / (mu sum_j 2^(t_ij - m_i)),
// one pass over the positions with a running reference m_i. m_i follows the
// maximum only when a score passes it by 4 (2^4 still fits everything below),
// so the accumulators are rarely rescaled; V's scales have such a reference A_i,
// a power of two that follows the maximum over the positions that the row sees when it
// is passed 8-fold. The weights w = 2^(t - m_i) av / A_i 2^8 <= 2^15 go to the matrix
// cores in fp16: a position that a row does not see has no part in its rounding.
//
// Both products run transposed on 16x16x32 fp16 MFMA tiles: S^T = K Q^T leaves
// lane (n = lane & 15, g = lane >> 4) with query row n and positions 16 t + 4 g +
// r (t < 2, r < 4) of a 32-position step, which is the layout of the second
// operand of O^T = V^T W^T. So the softmax, its reference and the rescaling are
// all within a lane, and scores never move through LDS.
//   - K tile: position n's bytes of group g, 8 elements of each 32-wide piece.
//   - V tile k: lane m's bytes k of positions 4 g .. 4 g + 3, elements 32 k + 2 m
//     (high nibbles) and + 1 (low), as rows of two tiles; two positions' nibbles
//     are merged into one byte.
//   - A block scale is needed by the 16 lanes of a DPP row at a compile-time
//     place: each lane loads one or a few of the step's scales and the products
//     read them through row_newbcast.
// Codes become fp16 pairs through a 256-entry table in LDS indexed by the byte,
// in 32 copies (64 KB; entry e at 256 e + 4 (lane & 31), its second parts 128
// bytes on), so that lookups never meet in a bank and an address is one byte
// permute.
//
// Rounding. c' = c mu is held as two fp16 values c1 + c2 (mu carries 2^7, which
// keeps c2 normal). Values take both: the error of c1 alone is the same at every
// position of a code, so its mean over the codes stays while the sum of many
// positions averages out (5e-3 of the result at 70000 positions). Keys of bf16
// rows take c1: there such a mean shifts all scores alike. mu = 1.6776896 2^7 makes
// the 2-norm of NF4's c1 errors 6.2e-5 of the values' (1.6e-4 at mu = 2^7; a search
// over 2^20 factors); E2M1 values are exact (mu = 6 2^7). 16-bit queries enter as fp16
// after a power of two of the row's own, so no row depends on another's size: fp16 rows
// exactly, elements of bf16 rows to 2^-39 of the row's largest at least (fp16's least step
// is 2^-24, the largest is brought to 2^14 ..).
// w: one fp16 for bf16 rows (2^-12), two for fp16 rows, whose output resolves 2^-11; so
// do their keys (one part would cost 3e-4 of the result at scores of size 3). fp32 rows:
// q, c' and w in two parts each, the three leading products. Accumulators and
// statistics are fp32.
//
// Work. An item is a workgroup's block of rows of one sequence and kv head; where
// items are few its positions are split into equal ranges, whose partial sums a second
// kernel joins (plan_of in kv_attention.hip has the rules and both sides of each).
//
// What bounds it, on one MI355X (256 CUs; a copy moves 4.99 TB/s, a library matrix
// product of 16-bit numbers reaches 1260 TFLOP/s):
//   - one row of a long cache (131071 positions, 8 kv heads, 142.6 MB): 31.9 us, 4.5
//     TB/s, and 5 us of joining; a batch of 32 uneven sequences up to 8000 (152.6 MB):
//     42 us, 3.6 TB/s. Half of the SIMDs' cycles issue (VALU 37 %, MFMA 12 %): a position
//     costs a fixed number of lookups, exponentials and products per 16 rows, of which
//     4 are used. The rest waits for HBM and the uneven ends.
//   - many rows (1024 and 512, 32 heads, 5000 and 2500 positions, 94 GFLOP): 212 us, 444
//     TFLOP/s of the definition's, 660 of those issued (V's two parts). A wave's step is
//     some 370 VALU instructions (107 us of every SIMD: addresses and merging of codes,
//     scales of scores and weights, softmax) and 48 MFMA (56 us); these do not overlap
//     well within a SIMD. Each wave decodes the same codes for rows of its own.
//   - short calls: 9 us, of which the arguments' way, the table and the merge of the
//     waves are 6.
#pragma once

#include <type_traits>

#include "kv_internal.h"

namespace nf4 {
namespace kvattn {

constexpr int kStep = 32;   // positions of a wave's step
constexpr int kTableBytes = 256 * 256;
// Two shapes of workgroup. Few rows: its 8 waves share one block of rows and take
// the steps of its positions in turn, then merge. Many rows: each of its 4 waves
// has a block of rows of its own and takes every step, so nothing is merged.
constexpr int kMergeWaves = 8;
constexpr int kApartWaves = 4;

struct AttnArgs {
  KvArgs kv;
  const void *q;
  void *out;
  int64_t q_row, q_head, out_row, out_head;
  int32_t group, max_rows;
  float f;       // scale log2(e) / mu
  float inv_mu;
  int32_t causal, window;
  int32_t wg_rows;    // (row, head) pairs of a workgroup's block
  int32_t wg_blocks;  // such blocks of a sequence and kv head
  int32_t splits;     // ranges of positions of an item
  int32_t part_rows;  // rows of a partial result
  float *part;        // [item][split][part_rows][D]
  float2 *stats;      // [item][split][part_rows]: reference, sum
  uint32_t codes[16];  // by nibble: c1 in the low half, c2 in the high one (fp16)
};

// The kernels read their arguments through this type, from the argument segment
// and through a pointer that is renewed where a kernel's phases meet: held in
// scalar registers from end to end they would not leave enough of these.
typedef const __attribute__((address_space(4))) AttnArgs KernelArgs;

__device__ __forceinline__ KernelArgs *kernel_args() {
  auto *p = (KernelArgs *)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// Has every 64-byte line of the arguments on its way to the scalar cache at once:
// they lie in host memory, and a line takes about a microsecond.
__device__ __forceinline__ void fetch_args() {
  const auto *p = (const __attribute__((address_space(4))) uint32_t *)kernel_args();
  constexpr int kLines = (sizeof(AttnArgs) + 63) / 64;
  uint32_t v[kLines];
#pragma unroll
  for (int i = 0; i < kLines; ++i) v[i] = p[16 * i];
#pragma unroll
  for (int i = 0; i < kLines; ++i) asm volatile("" ::"s"(v[i]));
}

// A block of rows of one sequence, and the positions that they see.
struct Block {
  int n;         // rows of the sequence in the call
  int first;     // their first row in the tensors
  int len;
  int row0;      // first (row, head) pair of the block, row-major by token
  int pairs;     // such pairs of the sequence (up to max_rows tokens)
  int lo, hi;    // positions [lo, hi) that any row of the block sees
  int all_lo, all_hi;  // positions that every row sees
};

// Positions of a range: equal multiples of `align`.
__device__ __forceinline__ int range_of(const Block &b, int splits, int align) {
  const int total = b.hi - b.lo;
  const int range = splits == 1 ? total : (total + splits - 1) / splits;
  return (range + align - 1) / align * align;
}

__device__ __forceinline__ int64_t item_of(KernelArgs &a, int seq, int h, int wb) {
  return ((int64_t)seq * a.kv.kv_heads + h) * a.wg_blocks + wb;
}

__device__ __forceinline__ int seen_end(KernelArgs &a, const Block &b, int token) {
  return a.causal ? b.len - b.n + token + 1 : b.len;
}

__device__ __forceinline__ int seen_begin(KernelArgs &a, int end) {
  return a.window > 0 && end > a.window ? end - a.window : 0;
}

// A row's end as far as the table goes: a length may pass it.
__device__ __forceinline__ int within(KernelArgs &a, int end) {
  return end < a.kv.capacity ? end : a.kv.capacity;
}

// A sequence of the call.
struct Sequence {
  int first;  // its first row in the tensors
  int n;      // its rows in the call
  int len;
};

__device__ __forceinline__ Sequence sequence_of(KernelArgs &a, int seq) {
  Sequence s;
  const int len = scalar_load(a.kv.lens, seq);
  int end;
  if (a.kv.offsets == nullptr) {
    s.first = seq * a.kv.uniform;
    end = s.first + a.kv.uniform;
  } else {
    const int b0 = scalar_load(a.kv.offsets, seq), b1 = scalar_load(a.kv.offsets, seq + 1);
    s.first = clamp_to(b0, 0, a.kv.total_rows);
    end = clamp_to(b1, 0, a.kv.total_rows);
  }
  s.n = end > s.first ? end - s.first : 0;
  s.len = clamp_to(len, 0, kMaxPositions);
  return s;
}

__device__ __forceinline__ Block block_of(KernelArgs &a, const Sequence &s, int row0, int rows) {
  Block b;
  b.n = s.n;
  b.first = s.first;
  b.len = s.len;
  const int tokens = b.n < a.max_rows ? b.n : a.max_rows;
  b.pairs = tokens * a.group;
  b.row0 = row0;
  b.lo = b.hi = b.all_lo = b.all_hi = 0;
  if (b.row0 < b.pairs) {
    // divisions only where a sequence has several blocks
    const int token0 = row0 == 0 ? 0 : row0 / a.group;
    const int token1 = row0 + rows >= b.pairs ? tokens - 1 : (row0 + rows - 1) / a.group;
    const int end0 = seen_end(a, b, token0), end1 = seen_end(a, b, token1);
    b.hi = within(a, end1);
    b.lo = seen_begin(a, end0);
    b.all_hi = within(a, end0);
    b.all_lo = seen_begin(a, end1);
    if (b.hi <= b.lo) b.lo = b.hi = 0;
    b.lo &= ~(kStep - 1);
  }
  return b;
}

// Byte SRC of w as the second byte of a table address, lane_off as its first.
template <int SRC>
__device__ __forceinline__ uint32_t table_address(uint32_t w, uint32_t lane_off) {
  return __builtin_amdgcn_perm(w, lane_off, 0x0c0c0000u | ((4 + SRC) << 8));
}

// The scale of index V (of those a DPP row shares) from the lane that holds it.
template <int V>
__device__ __forceinline__ float row_scale(const float *s) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(s[V / 16]), 0x150 + V % 16, 0xf, 0xf, true));
}

// Maximum of numbers: fmaxf would first quiet NaNs, one instruction an operand.
__device__ __forceinline__ float max2(float a, float b) {
  return __builtin_amdgcn_fmed3f(a, b, __builtin_inff());
}
__device__ __forceinline__ float max3(float a, float b, float c) { return max2(max2(a, b), c); }

// The nearest number.
__device__ __forceinline__ float finite(float v) {
  return __builtin_amdgcn_fmed3f(v, -3.402823466e38f, 3.402823466e38f);
}

// A barrier for what the workgroup shares in LDS. (__syncthreads would also wait
// for every load from memory.)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A lane's value that is not known before this point: what a loop derives from it is
// not computed ahead of the loop and held in registers throughout.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A value that is computed at this point and not moved into a later block, away from the
// lane exchanges that it takes as operands.
__device__ __forceinline__ float here(float v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A wave-uniform value to be held in scalar registers from here on.
template <typename T>
__device__ __forceinline__ T pin(T v) {
  asm volatile("" : "+s"(v));
  return v;
}

// Maximum over the lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ float max_over_groups(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = max2(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max2(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float sum_over_groups(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<I + 1, N>(static_cast<F &&>(f));
  }
}

// Which parts of the table's entries a lookup takes.
constexpr std::integral_constant<int, 0> kFirst;
constexpr std::integral_constant<int, 1> kSecond;

// What an fp16 pair leaves of two fp32, as another.
__device__ __forceinline__ uint32_t rest_f16x2(float a, float b, uint32_t h) {
  return pack_f16x2(a - widen16<kFP16>(h & 0xffffu), b - widen16<kFP16>(h >> 16));
}

// Pointers to global memory that stay so (not generic) through pin().
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(1))) uint8_t *GlobalU8;
typedef const __attribute__((address_space(1))) float *GlobalF32;

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&d)[N], GlobalU8 p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = ((const __attribute__((address_space(1))) u32x4 *)p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[4 * i + j] = v[j];
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const u32x2 v = ((const __attribute__((address_space(1))) u32x2 *)p)[i];
      d[2 * i] = v[0];
      d[2 * i + 1] = v[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = ((const __attribute__((address_space(1))) uint32_t *)p)[i];
  }
}

// 4 bytes of a lane's run starting at byte O (compile-time); bytes past the
// run's end are don't-cares.
template <int O, int N>
__device__ __forceinline__ uint32_t word_at(const uint32_t (&d)[N]) {
  if constexpr (O % 4 == 0) return d[O / 4];
  else if constexpr (O / 4 + 1 < N) return __builtin_amdgcn_alignbyte(d[O / 4 + 1], d[O / 4], O % 4);
  else return d[O / 4] >> (8 * (O % 4));
}

// DT: element type of q and out. NR: 16-row tiles of a wave's block of rows. MERGE:
// the workgroup's waves share the block (the first shape).
template <int D, int BS, int DT, int NR, bool MERGE>
struct Attn {
  static constexpr int kWaves = MERGE ? kMergeWaves : kApartWaves;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int P = D / 32;          // 32-wide pieces
  static constexpr int NB = D / BS;         // blocks of a head vector
  static constexpr int PB = BS / 32;        // pieces of a block
  static constexpr int NS = (8 * NB + 15) / 16;  // scales a lane holds of a step
  static constexpr bool kSplitW = DT != kBF16;   // two-part weights
  static constexpr bool kSplitK = DT != kBF16;   // two-part code values of keys
  static constexpr bool kSplitQ = DT == kFP32;   // two-part queries
  static constexpr int kRows = 16 * NR;
  // waves for which registers are shared out: two workgroups of a CU where they
  // suffice (128 registers), else one of 8 waves or two of 4 (256)
  static constexpr int kWavesPerSimd = MERGE && NR == 1 && D <= 128 && DT != kFP32 ? 4 : 2;
  // with two waves on a SIMD, lookups are kept ahead of the products that they feed;
  // with four the others fill the wait, and the registers are needed. So they are for wide
  // heads in two parts, which would spill (fp16, heads of 256 in blocks of 64: 16 uneven
  // sequences up to 8000 positions 70 us, 96 with lookups ahead; 227, 300 at 512 and 256
  // rows of 3000 and 1500)
  static constexpr bool kAhead =
      kWavesPerSimd < 4 && !(kSplitQ && D > 128) && !(kSplitK && D > 192);
  // the merge of the waves' results handles this many rows and columns at once, so
  // that its buffer and the table leave room for a second workgroup where there is one.
  // It goes by whole 32-wide pieces: half of 96 columns would end inside one
  static constexpr int kMergeRows = kWavesPerSimd == 4 ? 4 : 16;
  static constexpr int kMergeCols = (kWavesPerSimd == 4 || D > 128) && P % 2 == 0 ? D / 2 : D;
  static_assert(kMergeCols % 32 == 0 && D % kMergeCols == 0, "whole pieces");
  static constexpr int kMergeStride = kMergeCols + 4;
  static constexpr int kMergeFloats = MERGE ? kWaves * kMergeRows * kMergeStride : 1;
};

// Raw inputs of a step.
template <int D, int BS>
struct StepIn {
  uint32_t k[2][D / 32];
  uint32_t v[2][D / 32];
  float ks[(8 * (D / BS) + 15) / 16], vs[(8 * (D / BS) + 15) / 16];
};

template <int D, int BS, int DT, int NR, bool MERGE>
__global__ __launch_bounds__((Attn<D, BS, DT, NR, MERGE>::kThreads)) __attribute__((
    amdgpu_waves_per_eu(Attn<D, BS, DT, NR, MERGE>::kWavesPerSimd))) void kv_attention_kernel(
    AttnArgs) {
  using A = Attn<D, BS, DT, NR, MERGE>;
  constexpr int P = A::P, NB = A::NB, PB = A::PB, NS = A::NS;
  constexpr int kWaves = A::kWaves, kThreads = A::kThreads;
  constexpr int TW = MERGE ? kWaves : 1;  // waves that share a block's steps
  __shared__ __attribute__((aligned(16))) char lds[kTableBytes];
  // the waves' results where they merge; before, the queries they share
  __shared__ __attribute__((aligned(16))) float merge_buf[A::kMergeFloats];
  __shared__ float wave_m[MERGE ? kWaves : 1][A::kRows];
  __shared__ float wave_l[MERGE ? kWaves : 1][A::kRows];
  __shared__ float total_l[A::kRows];
  __shared__ float wave_top[kWaves][16];
  // as many workgroups of a CU's 160 KB as the registers allow
  static_assert(A::kWavesPerSimd * 4 / kWaves *
                        (sizeof(lds) + sizeof(merge_buf) + sizeof(wave_m) + sizeof(wave_l) +
                         sizeof(total_l) + sizeof(wave_top)) <= 160 * 1024, "LDS");

  fetch_args();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tw = MERGE ? wave : 0;
  const uint32_t my_code = kernel_args()->codes[threadIdx.x & 15];

  // the table, in pieces of 128 bytes: first and second parts of an entry. Lane l
  // holds code l & 15. A barrier follows before it is read.
  auto write_table = [&] {
    for (int i = threadIdx.x; i < 512; i += kThreads) {
      const int e = i >> 1;
      const uint32_t a = (uint32_t)__shfl((int)my_code, e >> 4, 64);
      const uint32_t b = (uint32_t)__shfl((int)my_code, e & 15, 64);
      const uint32_t w = i & 1 ? a >> 16 | (b & 0xffff0000u) : (a & 0xffffu) | b << 16;
      uint4 *dst = reinterpret_cast<uint4 *>(lds + 128 * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[(j + i) & 7] = make_uint4(w, w, w, w);
    }
  };

  // ---- the positions [begin, end) of an item
  const int lane = (int)threadIdx.x & 63;
  const int n = lane & 15, g = lane >> 4;
  const uint32_t lane_off = 4u * (lane & 31);
  KernelArgs &args = *kernel_args();
  const auto &kv = args.kv;
  const int h = (int)blockIdx.y, seq = (int)blockIdx.z;
  int wb = (int)blockIdx.x, split = 0;
  if (args.splits > 1) {
    wb = (int)blockIdx.x / args.splits;
    split = (int)blockIdx.x - wb * args.splits;
  }
  // blocks of later rows see more positions: they come first
  wb = args.wg_blocks - 1 - wb;
  const Sequence of = sequence_of(args, seq);
  const Block item = block_of(args, of, wb * args.wg_rows, args.wg_rows);
  const int range = range_of(item, args.splits, kStep * TW);
  int begin = item.lo + split * range;
  int end = range < item.hi - begin ? begin + range : item.hi;
  // a workgroup without rows, or with a range past the positions, leaves nothing
  // behind; with one range the rows that see nothing are still written
  if (item.row0 >= item.pairs || (begin >= item.hi && args.splits > 1)) return;
  const bool whole_item = args.splits == 1;
  const int64_t part_row0 = (item_of(args, seq, h, wb) * args.splits + split) * args.part_rows;
  // a wave's own rows may see less, and there may be none
  const Block blk = MERGE ? item : block_of(args, of, item.row0 + wave * A::kRows, A::kRows);
  const bool have_rows = blk.row0 < blk.pairs;
  if (!MERGE) {
    begin = begin > blk.lo ? begin : blk.lo;
    end = end < blk.hi ? end : blk.hi;
  }

  // ---- where its steps lie, and the first one's inputs on their way
  const int steps_all = end > begin ? (end - begin + kStep - 1) / kStep : 0;
  const int nsteps = steps_all > tw ? (steps_all - tw + TW - 1) / TW : 0;
  // scalars of the loop, kept in registers
  const int64_t head_packed = (int64_t)h * kv.page_size * (16 * P);
  const int64_t head_absmax = (int64_t)h * kv.page_size * NB;
  const GlobalU8 k_base = pin((GlobalU8)(uintptr_t)kv.packed[0] + head_packed);
  const GlobalU8 v_base = pin((GlobalU8)(uintptr_t)kv.packed[1] + head_packed);
  const GlobalF32 ks_base = pin((GlobalF32)(uintptr_t)kv.absmax[0] + head_absmax);
  const GlobalF32 vs_base = pin((GlobalF32)(uintptr_t)kv.absmax[1] + head_absmax);
  const uint32_t packed_units = pin((uint32_t)(kv.packed_stride >> 4));
  const uint32_t absmax_units = pin((uint32_t)kv.absmax_stride);
  const ConstI32 table = pin((ConstI32)(uintptr_t)kv.table + (int64_t)seq * kv.table_stride);
  const int last_col = pin(kv.table_cols - 1);
  const uint32_t num_pages = pin((uint32_t)kv.num_pages);
  const int tiles_per_page = pin(kv.page_size / 16);
  // both tiles of a step in one page, which holds an even number of them
  const bool paired = (tiles_per_page & 1) == 0;
  const int tile0 = (begin >> 4) + 2 * tw;
  const int first_col = nsteps > 0 ? tile0 / tiles_per_page : 0;
  int col = first_col, in_page = tile0 - first_col * tiles_per_page;
  const int step_cols = pin(2 * TW / tiles_per_page);
  const int step_in_page = pin(2 * TW - step_cols * tiles_per_page);
  auto advance = [&] {
    col += step_cols;
    in_page += step_in_page;
    if (in_page >= tiles_per_page) {
      in_page -= tiles_per_page;
      ++col;
    }
  };
  // pages (and tiles within them) of a step's two 16-position tiles
  struct Where { uint32_t page[2]; int at[2]; };
  // (both loaded always: a page id copied here would have to be waited for here)
  auto locate = [&] {
    const bool turn = in_page + 1 == tiles_per_page;
    const int col1 = turn ? col + 1 : col;
    Where w;
    w.page[0] = (uint32_t)table[col];
    w.page[1] = (uint32_t)table[col1 < last_col ? col1 : last_col];
    w.at[0] = in_page;
    w.at[1] = turn ? 0 : in_page + 1;
    return w;
  };
  // where the tiles' codes and scales lie; a page that is not there is read as the
  // first one and masked
  struct Places {
    GlobalU8 k[2], v[2];
    GlobalF32 ks[2], vs[2];
    bool ok[2];
  };
  auto places_of = [&](const Where &w) {
    Places p;
    uint64_t codes = 0, scales = 0;
    // both pages are looked at here, so that neither load sinks into the branch below
    p.ok[0] = w.page[0] < num_pages;
    p.ok[1] = w.page[1] < num_pages;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t == 0 || !paired) {
        const uint32_t page = p.ok[t] ? w.page[t] : 0;
        codes = ((uint64_t)page * packed_units + (uint32_t)(w.at[t] * (16 * P))) << 4;
        scales = (uint64_t)page * absmax_units + (uint32_t)(w.at[t] * (16 * NB));
      } else {
        codes += 256 * P;
        scales += 16 * NB;
      }
      p.k[t] = k_base + codes;
      p.v[t] = v_base + codes;
      p.ks[t] = ks_base + scales;
      p.vs[t] = vs_base + scales;
    }
    return p;
  };
  // where a window leaves no position of the wave's first step to all rows, that step comes
  // last: their common A is then known (52 rows of 16 sequences in a window of 1024: 14.2
  // us, 15.2 in order)
  int step = nsteps > 1 && blk.all_lo >= begin + kStep * (tw + 1) ? 1 : 0;
  if (step > 0) advance();
  StepIn<D, BS> in;
  // the scales that the lane holds: values 16 u + n of the DPP row's 8 positions
  auto scale_index = [&](int u) {
    const int v = 16 * u + n;
    return v < 8 * NB ? v : v % (8 * NB);
  };
  // and their positions in the step
  auto position_of = [&](int u) {
    const int tk = scale_index(u) / NB;
    return 16 * (tk >> 2) + 4 * g + (tk & 3);
  };
  auto load_scales = [&](float (&s)[NS], const GlobalF32 (&base)[2]) {
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      const int v = scale_index(u), tk = v / NB;
      s[u] = (tk < 4 ? base[0] : base[1])[(uint32_t)((4 * g + (tk & 3)) * NB + (v - tk * NB))];
    }
  };
  auto load_k = [&](const Places &p) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      load_words(in.k[t], p.k[t] + (uint32_t)(n * (16 * P) + g * (4 * P)));
    load_scales(in.ks, p.ks);
  };
  auto load_v = [&](const Places &p) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      load_words(in.v[t], p.v[t] + (uint32_t)(g * (64 * P) + n * (4 * P)));
    load_scales(in.vs, p.vs);
  };
  bool ok0 = false, ok1 = false;
  if (nsteps > 0) {
    const Places p = places_of(locate());
    load_k(p);
    load_v(p);
    ok0 = p.ok[0];
    ok1 = p.ok[1];
  }

  // token and head (of the group) of a row of the block: small numbers, so a
  // product with the reciprocal and half a step is the quotient
  struct RowAt { int token, head; };
  const int token0 = blk.row0 == 0 ? 0 : blk.row0 / args.group, head0 = blk.row0 - token0 * args.group;
  const float per_group = 1.0f / (float)args.group;
  auto row_at = [&](int i) {
    const int q = (int)(((float)(head0 + i) + 0.5f) * per_group);
    return RowAt{token0 + q, head0 + i - q * args.group};
  };

  // ---- queries: lane (n, g) holds elements 32 c + 8 g .. + 7 of row n of each tile,
  // as fp16 after a power of two of the row's own that brings its largest below 2^15.
  // Rows past the last repeat the first one; nothing of theirs is stored. Waves that
  // share a block convert a fragment each.
  uint4 qh[NR][P];
  uint4 ql[A::kSplitQ && !MERGE ? NR : 1][A::kSplitQ && !MERGE ? P : 1];
  int row_lo[NR], row_hi[NR];  // positions the row sees
  // a row's scores are its products times this. The products, below 2^31 times a key scale,
  // are kept in range by 2^-31 with the key scales, unless a query of the wave's reaches
  // 2^90: small key scales have to be exact there, and large ones have no finite scores.
  float qscale[NR];
  float key_factor = 1.0f;
  uint4 *const q_shared = reinterpret_cast<uint4 *>(merge_buf);  // [first, second parts][fragment][lane]
  {
    struct Raw { uint4 v[DT == kFP32 ? 2 : 1]; };
    auto load_raw = [&](int nr, int c) {
      Raw r;
      const RowAt ra = row_at(blk.row0 + 16 * nr + n < blk.pairs ? 16 * nr + n : 0);
      const int64_t at = (int64_t)(blk.first + ra.token) * args.q_row +
                         (int64_t)(h * args.group + ra.head) * args.q_head + 8 * g + 32 * c;
      const uint4 *p = reinterpret_cast<const uint4 *>(
          static_cast<const char *>(args.q) + at * (DT == kFP32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < (DT == kFP32 ? 2 : 1); ++i) r.v[i] = p[i];
      return r;
    };
    auto element = [](const Raw &r, int i) {
      if constexpr (DT == kFP32) {
        const uint32_t w[4] = {r.v[i >> 2].x, r.v[i >> 2].y, r.v[i >> 2].z, r.v[i >> 2].w};
        return __uint_as_float(w[i & 3]);
      } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
        return widen16<DT>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu);
      }
    };
    auto largest = [&](const Raw &r) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) top = max3(top, fabsf(element(r, i)), fabsf(element(r, i + 1)));
      return top;
    };
    auto exponent = [](float top) {
      return top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;
    };
    // qscale and key_factor from the rows' exponents
    auto set_scales = [&](const int (&ex)[NR]) {
      bool large = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) large = large || ex[nr] > 90;
      const int down = __builtin_amdgcn_ballot_w64(large) != 0 ? 0 : 31;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) qscale[nr] = __builtin_amdgcn_ldexpf(args.f, ex[nr] - 15 + down);
      key_factor = __uint_as_float(pin(down == 0 ? 0x3f800000u : 0x30000000u));  // 1, 2^-31
    };
    auto convert = [&](const Raw &r, int ex, uint4 &hi, uint4 &lo) {
      uint32_t h16[4], l16[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = __builtin_amdgcn_ldexpf(element(r, 2 * i), 15 - ex);
        const float x1 = __builtin_amdgcn_ldexpf(element(r, 2 * i + 1), 15 - ex);
        h16[i] = pack_f16x2(x0, x1);
        if constexpr (A::kSplitQ) l16[i] = rest_f16x2(x0, x1, h16[i]);
      }
      hi = make_uint4(h16[0], h16[1], h16[2], h16[3]);
      if constexpr (A::kSplitQ) lo = make_uint4(l16[0], l16[1], l16[2], l16[3]);
    };
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const bool have = blk.row0 + 16 * nr + n < blk.pairs;
      const int end_of_row = have ? seen_end(args, blk, row_at(16 * nr + n).token) : 0;
      row_hi[nr] = within(args, end_of_row);
      row_lo[nr] = seen_begin(args, end_of_row);
    }
    if constexpr (MERGE) {
      static_assert(NR * P <= kWaves, "a fragment for each wave");
      Raw raw;
      const int nr = wave / P, c = wave - nr * P;
      if (wave < NR * P) raw = load_raw(nr, c);
      write_table();
      if (wave < NR * P) {
        const float top = max_over_groups(largest(raw));
        if (g == 0) wave_top[wave][n] = top;
      }
      lds_barrier();
      int ex[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float top = wave_top[i * P][n];
#pragma unroll
        for (int j = 1; j < P; ++j) top = max2(top, wave_top[i * P + j][n]);
        ex[i] = exponent(top);
        if (wave < NR * P && nr == i) {
          uint4 hi, lo;
          convert(raw, ex[i], hi, lo);
          q_shared[64 * wave + lane] = hi;
          if constexpr (A::kSplitQ) q_shared[64 * (NR * P + wave) + lane] = lo;
        }
      }
      set_scales(ex);
      lds_barrier();
#pragma unroll
      for (int f = 0; f < NR * P; ++f) qh[f / P][f % P] = q_shared[64 * f + lane];
    } else {
      Raw raw[NR][P];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int c = 0; c < P; ++c)
          if (have_rows) raw[nr][c] = load_raw(nr, c);
      write_table();
      lds_barrier();
      int ex[NR];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < P; ++c) top = max2(top, largest(raw[nr][c]));
        ex[nr] = exponent(max_over_groups(top));
#pragma unroll
        for (int c = 0; c < P; ++c)
          convert(raw[nr][c], ex[nr], qh[nr][c], ql[A::kSplitQ ? nr : 0][A::kSplitQ ? c : 0]);
      }
      set_scales(ex);
    }
  }
  // the second parts of a fragment
  auto q_low = [&](auto nrc, auto cc) {
    if constexpr (MERGE) return q_shared[64 * (NR * P + nrc * P + cc) + lane];
    else return ql[nrc][cc];
  };

  // ---- state. A row's A is 2^(a_exp - e): the scales, which the wave's rows share, are
  // multiplied by 2^(8 - a_exp), and a row's part 2^e of 2^8 / A goes to its exponentials
  // (l_sum carries it too). e is 0 but where rows have seen scales of different size (`even`
  // is false). It is kept in m_limit, as e + 128 of the last steps past 4: no register of its
  // own. There 0 stands for a row that has seen scales of 0 only (its A is still open, e = 0).
  constexpr float kNothing = -__builtin_inff();  // no position seen
  auto limit_of = [](int e) { return __uint_as_float(0x40800000u + (uint32_t)(e + 128)); };
  constexpr float kZeros = 4.0f;
  auto e_of = [](float limit) {
    return limit == kNothing || limit == kZeros ? 0 : (int)(__float_as_uint(limit) & 255u) - 128;
  };
  f32x4 o[NR][2 * P];
  float m_use[NR], m_limit[NR], l_sum[NR];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) o[nr][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    m_use[nr] = 0.0f;
    m_limit[nr] = kNothing;  // a score past m_use by more moves the reference
    l_sum[nr] = 0.0f;
  }
  constexpr int kStart = -1000;  // before any row has seen a scale that is not 0
  // from -119 to 127: 2^(8 - a_exp) is finite, and smaller scales are exact in fp16 steps
  // finer than the result's
  constexpr int kLeast = -119, kMost = 127;
  int a_exp = kStart;
  float a_inv = 1.0f;    // 2^(8 - a_exp)
  float a_limit = 0.0f;  // 8 A, where it is the same for all rows
  bool even = true;      // one A for all rows, e = 0

  const int all_lo = pin(blk.all_lo), all_hi = pin(blk.all_hi);
  const int any_hi = pin(blk.hi);
  for (int s = 0; s < nsteps; ++s) {
    // (steps begin at a multiple of 32 bytes: where the compiler happens to put them, many
    // rows take up to 2 % longer)
    asm volatile(".p2align 5");
    const int pos0 = begin + kStep * (tw + TW * step);
    if (s + 1 < nsteps) {  // the last one loads its own inputs again
      advance();
      if (++step == nsteps) {
        step = 0;
        col = first_col;
        in_page = tile0 - first_col * tiles_per_page;
      }
    }
    const Where next_at = locate();
    const bool ok[2] = {ok0, ok1};
    // every row sees the whole step (uniform)
    const bool whole = ok0 && ok1 && pos0 >= all_lo && pos0 + kStep <= all_hi;

    // ---- S^T = K Q^T, combined over blocks into log2 units past m_use
    f32x4 t[NR][2];
    float ks[NS];
#pragma unroll
    for (int u = 0; u < NS; ++u) ks[u] = in.ks[u] * key_factor;
    // An entry's second parts. (volatile: fetched in one instruction with the first, they
    // would come beside them and be copied; 32.8 us instead of 30.8 at 8 sequences up to
    // 4000 positions, fp16, 32 of 32 heads.)
    auto second_part = [&](uint32_t address) -> uint32_t {
      return *(const volatile __attribute__((address_space(3))) uint32_t *)(
          (const __attribute__((address_space(3))) char *)lds + address + 128);
    };
    // four code pairs of piece c: the byte of elements 32 c + 8 g + 2 i is i P + c of
    // the lane's run
    auto look_up_k = [&](auto tc, auto cc, auto x) {
      uint32_t e[4];
      unroll<0, 4>([&](auto ic) {
        constexpr int O = ic * P + cc;
        const uint32_t ad = table_address<O % 4>(in.k[tc][O / 4], lane_off);
        if constexpr (x == 0) e[ic] = *reinterpret_cast<const uint32_t *>(lds + ad);
        else e[ic] = second_part(ad);
      });
      return make_uint4(e[0], e[1], e[2], e[3]);
    };
    uint4 ahead[A::kAhead ? 2 : 1][A::kAhead ? P : 1];
    auto look_up_tile = [&](auto tc) {
      unroll<0, P>([&](auto cc) { ahead[tc][cc] = look_up_k(tc, cc, kFirst); });
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (A::kAhead) look_up_tile(std::integral_constant<int, 0>{});
    unroll<0, 2>([&](auto tc) {
      constexpr int T = tc;
      if constexpr (A::kAhead && T == 0) look_up_tile(std::integral_constant<int, 1>{});
      unroll<0, NB>([&](auto bc) {
        constexpr int B = bc;
        f32x4 acc[NR];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) acc[nr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        unroll<0, PB>([&](auto pc) {
          constexpr int C = B * PB + pc;  // 32-wide piece
          const std::integral_constant<int, C> cc;
          uint4 k1;
          if constexpr (A::kAhead) k1 = ahead[T][C];
          else k1 = look_up_k(tc, cc, kFirst);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) acc[nr] = mfma16x16x32<kFP16>(k1, qh[nr][C], acc[nr]);
          if constexpr (A::kSplitK) {
            const uint4 k2 = look_up_k(tc, cc, kSecond);
            unroll<0, NR>([&](auto nrc) {
              constexpr int nr = nrc;
              if constexpr (A::kSplitQ) acc[nr] = mfma16x16x32<kFP16>(k1, q_low(nrc, cc), acc[nr]);
              acc[nr] = mfma16x16x32<kFP16>(k2, qh[nr][C], acc[nr]);
            });
          }
        });
        unroll<0, 4>([&](auto rc) {
          constexpr int R = rc;
          const float a = row_scale<(4 * T + R) * NB + B>(ks);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            t[nr][T][R] = B == 0    ? acc[nr][R] * a
                          : NR == 1 ? t[nr][T][R] + acc[nr][R] * a
                                    : __builtin_fmaf(acc[nr][R], a, t[nr][T][R]);
        });
      });
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = t[nr][T][r];
          t[nr][T][r] = here(__builtin_fmaf(v, qscale[nr], -m_use[nr]));
        }
    });
    const Places next = places_of(next_at);
    load_k(next);

    // ---- masks
    float vs[NS];
#pragma unroll
    for (int u = 0; u < NS; ++u) vs[u] = in.vs[u];
    if (!whole) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int T = 0; T < 2; ++T)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int p = pos0 + 16 * T + 4 * g + r;
            const bool see = ok[T] && p >= row_lo[nr] && p < row_hi[nr];
            t[nr][T][r] = see ? t[nr][T][r] : -__builtin_inff();
          }
      // scales of positions that no row sees may be anything
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int p = position_of(u);
        vs[u] = pos0 + p < any_hi && (p < 16 ? ok[0] : ok[1]) ? vs[u] : 0.0f;
      }
    }

    // ---- references
    float top[NR];
    bool far = false, far_scale = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const f32x4 u = t[nr][0], v = t[nr][1];
      top[nr] = max3(max3(u[0], u[1], u[2]), max3(u[3], v[0], v[1]), max2(v[2], v[3]));
      far = far || top[nr] > m_limit[nr];
    }
#pragma unroll
    for (int u = 0; u < NS; ++u) far_scale = far_scale || fabsf(vs[u]) > a_limit;
    if (__builtin_amdgcn_ballot_w64(far || far_scale) != 0) {
      // the scales, of the finite ones: an infinity is its own rows' matter
      auto size = [&](int u) {
        return fabsf(vs[u]) < __builtin_inff() ? fabsf(vs[u]) : 0.0f;
      };
      int ex = a_exp;
      bool common = even;
      if (__builtin_amdgcn_ballot_w64(far_scale) != 0) {
        // one A for all rows, by the positions that all of them see, serves where no other
        // scale is 8 times as large. (A of each row's own, which is longer, only where some
        // position that not all rows see has a larger one.)
        float av = 0.0f, any = 0.0f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          any = max2(any, size(u));
          const int p = pos0 + position_of(u);
          av = max2(av, whole || (p >= all_lo && p < all_hi) ? size(u) : 0.0f);
        }
        av = max_over_groups(row16_max(av));
        ex = __builtin_amdgcn_readfirstlane(
            av > 0.0f ? clamp_to(__builtin_amdgcn_frexp_expf(av), kLeast, kMost) : kStart);
        ex = ex > a_exp ? ex : a_exp;
        common = even && __builtin_amdgcn_ballot_w64(any > __builtin_amdgcn_ldexpf(8.0f, ex)) == 0;
      }
      if (common) {
        const int fall = a_exp - ex;
        a_exp = ex;
        a_limit = __builtin_amdgcn_ldexpf(8.0f, ex);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          const float mx = max_over_groups(top[nr]);
          const bool first = m_limit[nr] == kNothing;
          const bool some = mx != -__builtin_inff();
          // how far the reference moves: to the maximum, never back
          const float move = !some ? 0.0f : (first ? mx : fmaxf(mx, 0.0f));
          const float alpha = first ? 0.0f : __builtin_amdgcn_exp2f(-move);
          const float beta = __builtin_amdgcn_ldexpf(alpha, fall);
          m_use[nr] += move;
          m_limit[nr] = some ? limit_of(0) : m_limit[nr];
          l_sum[nr] *= alpha;
#pragma unroll
          for (int T = 0; T < 2; ++T) t[nr][T] -= move;
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) o[nr][j] *= beta;
        }
      } else {
        // ---- A by row: the largest scale that a row sees
        float sizes[NS], seen[NR];
#pragma unroll
        for (int u = 0; u < NS; ++u) sizes[u] = size(u);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) seen[nr] = 0.0f;
        unroll<0, 8>([&](auto ic) {
          constexpr int T = ic / 4, R = ic % 4;
          float scale = row_scale<ic * NB>(sizes);
          unroll<1, NB>([&](auto bc) { scale = max2(scale, row_scale<ic * NB + bc>(sizes)); });
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            seen[nr] = max2(seen[nr], t[nr][T][R] == -__builtin_inff() ? 0.0f : scale);
          __builtin_amdgcn_sched_barrier(0);
        });
        // exponents of the rows' A before and after this step, and their range over the rows
        constexpr int kNone = -1000;
        int was[NR], now[NR];
        float lo = -kNone, hi = kNone;
        bool without = false;  // a row that may come to see a scale, but has not
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          seen[nr] = max_over_groups(seen[nr]);
          was[nr] = m_limit[nr] == kNothing || m_limit[nr] == kZeros || a_exp == kStart
                        ? kNone
                        : a_exp - e_of(m_limit[nr]);
          const int e_seen = seen[nr] > 0.0f ? __builtin_amdgcn_frexp_expf(seen[nr]) : kNone;
          now[nr] = e_seen > was[nr] ? e_seen : was[nr];
          lo = now[nr] != kNone ? fminf(lo, (float)now[nr]) : lo;
          hi = fmaxf(hi, (float)now[nr]);
          without = without || (now[nr] == kNone && row_hi[nr] > 0);
        }
        const int low = __builtin_amdgcn_readfirstlane((int)-row16_max(-lo));
        const int high = __builtin_amdgcn_readfirstlane((int)row16_max(hi));
        // e = a_exp - (exponent of A) is 0 for the rows of the least A, unless a row's is
        // more than 2^64 times that: then -64 for the greatest. It is 89 at most (the sum of
        // 2^31 weights up to 2^(4 + 89) is in fp32's range), so A is more than a row's own
        // scales ask for where another row's are 2^153 times as large.
        if (high != kNone) ex = clamp_to(low > high - 64 ? low : high - 64, kLeast, kMost);
        else ex = a_exp;
        // rows whose A are within the 8-fold of the least all take that one
        even = __builtin_amdgcn_ballot_w64(without) == 0 && high <= ex + 3;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          const float mx = max_over_groups(top[nr]);
          const bool first = m_limit[nr] == kNothing;
          const bool some = mx != -__builtin_inff();
          const bool scaled = now[nr] != kNone;
          const int e = scaled && !even ? (ex - now[nr] < 89 ? ex - now[nr] : 89) : 0;
          const float move = !some ? 0.0f : (first ? mx : fmaxf(mx, 0.0f));
          const float alpha = first ? 0.0f : __builtin_amdgcn_exp2f(-move);
          const float beta = __builtin_amdgcn_ldexpf(alpha, was[nr] - (ex - e));
          m_use[nr] += move;
          l_sum[nr] *= __builtin_amdgcn_ldexpf(alpha, e - e_of(m_limit[nr]));
          m_limit[nr] = first && !some ? kNothing : (scaled ? limit_of(e) : kZeros);
#pragma unroll
          for (int T = 0; T < 2; ++T) t[nr][T] = (t[nr][T] - move) + (float)e;
#pragma unroll
          for (int j = 0; j < 2 * P; ++j) o[nr][j] *= beta;
        }
        a_exp = ex;
        // else every step comes here: e is added to its scores
        a_limit = even ? __builtin_amdgcn_ldexpf(8.0f, ex) : -1.0f;
      }
      a_inv = __builtin_amdgcn_ldexpf(1.0f, 8 - (a_exp > kLeast ? a_exp : kLeast));
    }

    // ---- weights. A scale of infinity or NaN stands as the largest number: times the
    // weight 0 of a row that does not see its position it is 0, and for the others it
    // passes fp16's range.
    uint4 wh[NR][NB];
    uint4 wl[A::kSplitW ? NR : 1][A::kSplitW ? NB : 1];
#pragma unroll
    for (int u = 0; u < NS; ++u) vs[u] = finite(vs[u] * a_inv);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(t[nr][i >> 2][i & 3]);
      l_sum[nr] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      unroll<0, NB>([&](auto bc) {
        constexpr int B = bc;
        uint32_t hi[4], lo[4];
        unroll<0, 4>([&](auto ic) {
          const float w0 = p[2 * ic] * row_scale<(2 * ic) * NB + B>(vs);
          const float w1 = p[2 * ic + 1] * row_scale<(2 * ic + 1) * NB + B>(vs);
          hi[ic] = pack_f16x2(w0, w1);
          if constexpr (A::kSplitW) lo[ic] = rest_f16x2(w0, w1, hi[ic]);
        });
        wh[nr][B] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (A::kSplitW) wl[nr][B] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      });
    }

    // ---- O^T += V^T W^T. Waves that share a block go first here, so that others'
    // softmax fills the wait (32 uneven sequences 46.2 -> 45.3 us, one row of 131071
    // positions 39.3 -> 38.8); waves with rows of their own lose by it (204 -> 207).
    if constexpr (MERGE) __builtin_amdgcn_s_setprio(1);
    // word wd of the positions' runs: merged nibbles of [tile][pair of positions]
    uint32_t even[2][2], odd[2][2];
    auto merge_nibbles = [&](auto wc) {
      unroll<0, 2>([&](auto tc) {
        constexpr int T = tc;
        unroll<0, 2>([&](auto pc) {
          constexpr int R = 2 * pc;
          const uint32_t a = word_at<R * P + 4 * wc>(in.v[T]);
          const uint32_t b = word_at<(R + 1) * P + 4 * wc>(in.v[T]);
          even[T][pc] = (a & 0xf0f0f0f0u) | ((b >> 4) & 0x0f0f0f0fu);
          odd[T][pc] = ((a << 4) & 0xf0f0f0f0u) | (b & 0x0f0f0f0fu);
        });
      });
    };
    // the first parts of the positions' pairs (x = 0) or the second ones
    auto look_up_v = [&](auto kk, auto jc, auto x) {
      uint32_t e[4];
      unroll<0, 4>([&](auto ic) {
        constexpr int T = ic / 2, I = ic % 2;
        const uint32_t ad =
            table_address<kk % 4>(jc == 0 ? even[T][I] : odd[T][I], lane_off);
        if constexpr (x == 0) e[ic] = *reinterpret_cast<const uint32_t *>(lds + ad);
        else e[ic] = second_part(ad);
      });
      return make_uint4(e[0], e[1], e[2], e[3]);
    };
    // [tile of elements][part], of this piece and the next
    uint4 vc[A::kAhead ? 2 : 1][2][2];
    auto look_up_piece = [&](auto kk) {
      if constexpr (kk % 4 == 0) merge_nibbles(std::integral_constant<int, kk / 4>{});
      unroll<0, 2>([&](auto xc) {
        unroll<0, 2>([&](auto jc) { vc[kk & 1][jc][xc] = look_up_v(kk, jc, xc); });
      });
      __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (A::kAhead) look_up_piece(std::integral_constant<int, 0>{});
    unroll<0, P>([&](auto kk) {
      constexpr int K = kk;
      constexpr int B = K / PB;
      if constexpr (!A::kAhead && K % 4 == 0) merge_nibbles(std::integral_constant<int, K / 4>{});
      if constexpr (A::kAhead && K + 1 < P) look_up_piece(std::integral_constant<int, K + 1>{});
      unroll<0, 2>([&](auto xc) {
        unroll<0, 2>([&](auto jc) {
          uint4 v;
          if constexpr (A::kAhead) v = vc[K & 1][jc][xc];
          else v = look_up_v(kk, jc, xc);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            f32x4 &acc = o[nr][2 * K + jc];
            acc = mfma16x16x32<kFP16>(v, wh[nr][B], acc);
            // (the second parts' product, 2^-22 of a term at most, is left out)
            if constexpr (xc == 0 && A::kSplitW) acc = mfma16x16x32<kFP16>(v, wl[nr][B], acc);
          }
        });
      });
    });
    if constexpr (MERGE) __builtin_amdgcn_s_setprio(0);
    load_v(next);
    ok0 = next.ok[0];
    ok1 = next.ok[1];
  }

  // ---- results: a row's output, or its partial sums
  float l_row[NR], m_ref[NR];
  int a_row[NR];  // exponents of 2^8 / A, undone apart from other factors: their product
                  // may be subnormal
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    l_row[nr] = __builtin_amdgcn_ldexpf(sum_over_groups(l_sum[nr]), -e_of(m_limit[nr]));
    m_ref[nr] = m_limit[nr] == kNothing ? kNothing : m_use[nr];
    a_row[nr] = a_exp - e_of(m_limit[nr]) - 8;
  }
  KernelArgs &end_args = *kernel_args();
  const int tid = fresh((int)threadIdx.x);
  auto out_at = [&](int i) {
    const RowAt ra = row_at(i);
    return (int64_t)(blk.first + ra.token) * end_args.out_row +
           (int64_t)(h * end_args.group + ra.head) * end_args.out_head;
  };

  if constexpr (!MERGE) {
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int pair = blk.row0 + 16 * nr + n;
      if (pair >= blk.pairs) continue;
      const int64_t part_row = part_row0 + wave * A::kRows + 16 * nr + n;
      const float f = !whole_item ? end_args.inv_mu
                                  : (l_row[nr] > 0.0f ? end_args.inv_mu / l_row[nr] : 0.0f);
      auto undo = [&](float v) { return __builtin_amdgcn_ldexpf(v * f, a_row[nr]); };
      if (!whole_item && g == 0) end_args.stats[part_row] = make_float2(m_ref[nr], l_row[nr]);
      float *part = end_args.part + part_row * D + 8 * g;
      const int64_t at = out_at(16 * nr + n) + 8 * g;
      // the lane holds elements 32 k + 8 g + 2 r + {0, 1}
      unroll<0, P>([&](auto kc) {
        constexpr int K = kc;
        const f32x4 e = o[nr][2 * K], d = o[nr][2 * K + 1];
        const f32x4 v0 = {undo(e[0]), undo(d[0]), undo(e[1]), undo(d[1])};
        const f32x4 v1 = {undo(e[2]), undo(d[2]), undo(e[3]), undo(d[3])};
        if (!whole_item || DT == kFP32) {
          f32x4 *dst = reinterpret_cast<f32x4 *>(
              whole_item ? static_cast<float *>(end_args.out) + at + 32 * K : part + 32 * K);
          dst[0] = v0;
          dst[1] = v1;
        } else {
          constexpr int T = DT == kFP32 ? kBF16 : DT;
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(end_args.out) + at + 32 * K) =
              make_uint4(pack2<T>(v0[0], v0[1]), pack2<T>(v0[2], v0[3]), pack2<T>(v1[0], v1[1]),
                         pack2<T>(v1[2], v1[3]));
        }
      });
    }
  } else {
    // merge the waves: one reference per row, then the sums in wave order
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      if (g == 0) {
        wave_m[wave][16 * nr + n] = m_ref[nr];
        wave_l[wave][16 * nr + n] = l_row[nr];
      }
    }
    lds_barrier();
    float factor[NR];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float mx = wave_m[0][16 * nr + n];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) mx = fmaxf(mx, wave_m[i][16 * nr + n]);
      const float use = mx == -__builtin_inff() ? 0.0f : mx;
      factor[nr] = end_args.inv_mu * __builtin_amdgcn_exp2f(m_ref[nr] - use);
      if (wave == 0 && g == 0) {
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
          l += wave_l[i][16 * nr + n] * __builtin_amdgcn_exp2f(wave_m[i][16 * nr + n] - use);
        total_l[16 * nr + n] = l;
        if (!whole_item && 16 * nr + n < end_args.part_rows)
          end_args.stats[part_row0 + 16 * nr + n] = make_float2(mx, l);
      }
    }
    constexpr int MR = A::kMergeRows, MC = A::kMergeCols, ML = A::kMergeStride;
    const int rows = blk.pairs - blk.row0;  // of the block, where fewer than its tiles
    unroll<0, NR>([&](auto nrc) {
      constexpr int nr = nrc;
      for (int r0 = 0; r0 < 16 && 16 * nr + r0 < rows; r0 += MR) {
        unroll<0, D / MC>([&](auto cc) {
          constexpr int K0 = cc * (MC / 32);
          lds_barrier();
          if (n >= r0 && n < r0 + MR) {
            unroll<0, MC / 32>([&](auto kc) {
              constexpr int K = K0 + kc;
              float *dst = merge_buf + (wave * MR + n - r0) * ML + 32 * kc + 8 * g;
              auto undo = [&](float v) {
                return __builtin_amdgcn_ldexpf(v * factor[nr], a_row[nr]);
              };
              const f32x4 e = o[nr][2 * K], d = o[nr][2 * K + 1];
              reinterpret_cast<f32x4 *>(dst)[0] =
                  f32x4{undo(e[0]), undo(d[0]), undo(e[1]), undo(d[1])};
              reinterpret_cast<f32x4 *>(dst)[1] =
                  f32x4{undo(e[2]), undo(d[2]), undo(e[3]), undo(d[3])};
            });
          }
          lds_barrier();
          for (int idx = tid; idx < MR * (MC / 4); idx += kThreads) {
            const int row = idx / (MC / 4), cl = 4 * (idx - row * (MC / 4));
            const int in_block = 16 * nr + r0 + row;
            if (in_block >= rows) continue;
            f32x4 sum = *reinterpret_cast<const f32x4 *>(merge_buf + row * ML + cl);
#pragma unroll
            for (int i = 1; i < kWaves; ++i)
              sum += *reinterpret_cast<const f32x4 *>(merge_buf + (i * MR + row) * ML + cl);
            const int ccol = cc * MC + cl;
            if (!whole_item) {
              *reinterpret_cast<f32x4 *>(end_args.part + (part_row0 + in_block) * D + ccol) = sum;
            } else {
              const float l = total_l[in_block];
              const float inv = l > 0.0f ? 1.0f / l : 0.0f;
              const int64_t at = out_at(in_block) + ccol;
              if constexpr (DT == kFP32) {
                *reinterpret_cast<f32x4 *>(static_cast<float *>(end_args.out) + at) = sum * inv;
              } else {
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(end_args.out) + at) = make_uint2(
                    pack2<DT>(sum[0] * inv, sum[1] * inv), pack2<DT>(sum[2] * inv, sum[3] * inv));
              }
            }
          }
        });
      }
    });
  }
}

// ------------------------------------------------------------------- host

struct Plan {
  bool merge;             // shape of the workgroups
  int tiles;              // 16-row tiles of a wave's block of rows
  int wg_rows, wg_blocks;
  int splits, align;      // ranges of positions, their granularity
  int part_rows;
  int64_t part_floats, stats;  // totals
};

// Largest number of 16-row tiles of a wave's block: what its registers hold.
constexpr int max_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }

template <int D, int BS, int DT, int NR, bool MERGE>
hipError_t launch_one(const AttnArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.wg_blocks * a.splits), (unsigned)a.kv.kv_heads,
                  (unsigned)a.kv.batch);
  hipLaunchKernelGGL((kv_attention_kernel<D, BS, DT, NR, MERGE>), grid,
                     dim3(Attn<D, BS, DT, NR, MERGE>::kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int D, int BS, int DT>
hipError_t launch_main(const AttnArgs &a, const Plan &p, hipStream_t stream) {
  constexpr int T = max_tiles(D);
  if (!p.merge) return launch_one<D, BS, DT, T, false>(a, stream);
  if constexpr (T > 1) {
    if (p.tiles > 1) return launch_one<D, BS, DT, T, true>(a, stream);
  }
  return launch_one<D, BS, DT, 1, true>(a, stream);
}

// Instantiated for each element type in a file of its own.
template <int DT>
hipError_t launch_shape(const AttnArgs &a, const Plan &p, int head_dim, int blocksize,
                        hipStream_t stream) {
  switch (head_dim * 1000 + blocksize) {
#define NF4_KV_CASE(DV, BSV) \
  case DV * 1000 + BSV: return launch_main<DV, BSV, DT>(a, p, stream);
    NF4_KV_CASE(64, 32)
    NF4_KV_CASE(64, 64)
    NF4_KV_CASE(96, 32)
    NF4_KV_CASE(128, 32)
    NF4_KV_CASE(128, 64)
    NF4_KV_CASE(128, 128)
    NF4_KV_CASE(192, 32)
    NF4_KV_CASE(192, 64)
    NF4_KV_CASE(256, 32)
    NF4_KV_CASE(256, 64)
    NF4_KV_CASE(256, 128)
#undef NF4_KV_CASE
  }
  return hipErrorNotSupported;
}

extern template hipError_t launch_shape<kBF16>(const AttnArgs &, const Plan &, int, int, hipStream_t);
extern template hipError_t launch_shape<kFP16>(const AttnArgs &, const Plan &, int, int, hipStream_t);
extern template hipError_t launch_shape<kFP32>(const AttnArgs &, const Plan &, int, int, hipStream_t);

}  // namespace kvattn
}  // namespace nf4
