// kv_attention_kernel.h -- attention of query rows to a key/value cache held in
// 4 bits.
//
// Mathematics. With code values c scaled by mu to c' = c mu, K = c'k ak / mu
// and V = c'v av / mu (ak, av the block scales), in log2 units
//   t_ij = f sum_b ak_jb (q_i . c'k_j)_b,   f = scale log2(e) / mu,
//   out_i = sum_j 2^(t_ij - m_i) av_j c'v_j / (mu sum_j 2^(t_ij - m_i)),
// one pass over the positions with a running reference m_i. m_i follows the
// maximum only when a score passes it by 4 (2^4 still fits everything below),
// so the accumulators are rarely rescaled; V's scales have such a reference A,
// a power of two that follows their maximum when it is passed 8-fold. The
// weights w = 2^(t - m) av / A 2^8 <= 2^15 go to the matrix cores in fp16.
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
// positions averages out (5e-3 of the result at 70000 positions). Keys of 16-bit
// rows take c1: there such a mean shifts all scores alike. mu = 1.6776896 2^7 makes
// the 2-norm of NF4's c1 errors 6.2e-5 of the values' (1.6e-4 at mu = 2^7; a search
// over 2^20 factors); E2M1 values are exact (mu = 6 2^7). 16-bit queries are exact
// in fp16 after a power of two. w: one fp16 for bf16 rows (2^-12), two for fp16
// rows, whose output resolves 2^-11. fp32 rows: q, c' and w in two parts each, the
// three leading products. Accumulators and statistics are fp32.
#pragma once

#include <type_traits>

#include "kv_internal.h"

namespace nf4 {
namespace kvattn {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;                  // positions of a wave's step
constexpr int kTableBytes = 256 * 256;
constexpr int kChunkAlign = kStep * kWaves;  // a workgroup's range is a multiple

struct AttnArgs {
  KvArgs kv;
  const void *q;
  void *out;
  int64_t q_row, q_head, out_row, out_head;
  int32_t group, max_rows;
  float f;       // scale log2(e) / mu
  float inv_mu;
  int32_t causal, window;
  int32_t row_blocks;  // per sequence and kv head
  int32_t splits;
  int32_t part_rows;   // rows of a partial result
  float *part;         // [item][split][part_rows][D]
  float2 *stats;       // [item][split][part_rows]: reference, sum
  uint32_t hi[16], lo[16];  // fp16 code values c' by nibble, and what they leave
};

// A row block of one sequence: its rows and the positions that they see.
struct Block {
  int n;         // rows of the sequence in the call
  int first;     // their first row in the tensors
  int len;
  int row0;      // first (row, head) pair of the block, row-major by token
  int pairs;     // such pairs of the sequence (up to max_rows tokens)
  int lo, hi;    // positions [lo, hi) that any row of the block sees
};

__device__ __forceinline__ int seen_end(const AttnArgs &a, const Block &b, int token) {
  return a.causal ? b.len - b.n + token + 1 : b.len;
}

__device__ __forceinline__ int seen_begin(const AttnArgs &a, int end) {
  return a.window > 0 && end > a.window ? end - a.window : 0;
}

__device__ __forceinline__ Block block_of(const AttnArgs &a, int seq, int rb, int rows) {
  Block b;
  b.first = row_begin(a.kv, seq);
  const int end = row_begin(a.kv, seq + 1);
  b.n = end > b.first ? end - b.first : 0;
  b.len = clamp_to(scalar_load(a.kv.lens, seq), 0, a.kv.capacity);
  const int tokens = b.n < a.max_rows ? b.n : a.max_rows;
  b.pairs = tokens * a.group;
  b.row0 = rb * rows;
  b.lo = b.hi = 0;
  if (b.row0 < b.pairs) {
    const int last = (b.row0 + rows < b.pairs ? b.row0 + rows : b.pairs) - 1;
    b.hi = seen_end(a, b, last / a.group);
    b.lo = seen_begin(a, seen_end(a, b, b.row0 / a.group));
    if (b.hi <= b.lo) b.lo = b.hi = 0;
    b.lo &= ~(kStep - 1);
  }
  return b;
}

// Positions of a split: equal multiples of kChunkAlign.
__device__ __forceinline__ int chunk_of(const Block &b, int splits) {
  const int total = b.hi - b.lo;
  const int chunk = (total + splits - 1) / splits;
  return (chunk + kChunkAlign - 1) / kChunkAlign * kChunkAlign;
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

__device__ __forceinline__ float max4(f32x4 v) {
  return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
}

template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<I + 1, N>(static_cast<F &&>(f));
  }
}

// Two fp32 as an fp16 pair, and what that leaves as another.
__device__ __forceinline__ uint32_t rest_f16x2(float a, float b, uint32_t h) {
  return pack_f16x2(a - widen16<kFP16>(h & 0xffffu), b - widen16<kFP16>(h >> 16));
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&d)[N], const uint8_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
      d[4 * i] = v.x; d[4 * i + 1] = v.y; d[4 * i + 2] = v.z; d[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2 *>(p)[i];
      d[2 * i] = v.x; d[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = reinterpret_cast<const uint32_t *>(p)[i];
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

// DT: element type of q and out. NR: 16-row tiles of query rows.
template <int D, int BS, int DT, int NR>
struct Attn {
  static constexpr int P = D / 32;          // 32-wide pieces
  static constexpr int NB = D / BS;         // blocks of a head vector
  static constexpr int PB = BS / 32;        // pieces of a block
  static constexpr int RW = D / 32;         // words a lane holds of a 16-position tile
  static constexpr int NS = (8 * NB + 15) / 16;  // scales a lane holds of a step
  static constexpr bool kSplitW = DT != kBF16;   // two-part weights
  static constexpr bool kSplitQ = DT == kFP32;   // two-part queries and keys' code values
  static constexpr int kRows = 16 * NR;
  static constexpr int kPad = D + 4;
  // the merge of the waves' results handles this many 16-row tiles and columns at once
  static constexpr int kMergeCols = D > 128 ? D / 2 : D;
  static constexpr int kMergeBytes = kWaves * 16 * (kMergeCols + 4) * 4;
  static constexpr int kLds = kTableBytes > kMergeBytes ? kTableBytes : kMergeBytes;
};

// Raw inputs of a step.
template <int D, int BS>
struct StepIn {
  uint32_t k[2][D / 32];
  uint32_t v[2][D / 32];
  float ks[(8 * (D / BS) + 15) / 16], vs[(8 * (D / BS) + 15) / 16];
};

template <int D, int BS, int DT, int NR>
__global__ __launch_bounds__(kThreads) void kv_attention_kernel(AttnArgs args) {
  using A = Attn<D, BS, DT, NR>;
  constexpr int P = A::P, NB = A::NB, PB = A::PB, NS = A::NS;
  __shared__ __attribute__((aligned(16))) char lds[A::kLds];
  __shared__ float wave_m[kWaves][A::kRows];
  __shared__ float wave_l[kWaves][A::kRows];
  __shared__ float total_l[A::kRows];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const KvArgs &kv = args.kv;
  const int split = (int)blockIdx.x % args.splits;
  const int rb = (int)blockIdx.x / args.splits;
  const int h = (int)blockIdx.y, seq = (int)blockIdx.z;

  const Block blk = block_of(args, seq, rb, A::kRows);
  if (blk.row0 >= blk.pairs) return;
  const int chunk = chunk_of(blk, args.splits);
  const int begin = blk.lo + split * chunk;
  const int end = begin + chunk < blk.hi ? begin + chunk : blk.hi;
  // a split past the positions leaves nothing behind; with one split the rows
  // that see nothing are still written
  if (begin >= blk.hi && args.splits > 1) return;

  // the table: thread t fills the half t & 1 of entry t >> 1
  {
    const int e = tid >> 1;
    const uint32_t w = tid & 1 ? args.lo[e >> 4] | args.lo[e & 15] << 16
                               : args.hi[e >> 4] | args.hi[e & 15] << 16;
    uint4 *dst = reinterpret_cast<uint4 *>(lds + 256 * e + 128 * (tid & 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[(i + tid) & 7] = make_uint4(w, w, w, w);
  }
  const uint32_t lane_off = 4u * (lane & 31);

  // queries: lane (n, g) holds elements 32 c + 8 g .. + 7 of row n of each tile
  const void *qbase = args.q;
  uint4 qh[NR][P];
  uint4 ql[A::kSplitQ ? NR : 1][A::kSplitQ ? P : 1];
  int row_lo[NR], row_hi[NR];  // positions the row sees
  int min_hi = 0x7fffffff, max_lo = 0;
  float qscale_f;
  {
    float qf[NR][P][8];
    float top = 0.0f;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int pair = blk.row0 + 16 * nr + n;
      const bool have = pair < blk.pairs;
      const int token = have ? pair / args.group : 0;
      const int64_t at = (int64_t)(blk.first + token) * args.q_row +
                         (int64_t)(h * args.group + (have ? pair - token * args.group : 0)) *
                             args.q_head + 8 * g;
      row_hi[nr] = have ? seen_end(args, blk, token) : 0;
      row_lo[nr] = have ? seen_begin(args, row_hi[nr]) : 0;
#pragma unroll
      for (int c = 0; c < P; ++c) {
        float (&x)[8] = qf[nr][c];
        if constexpr (DT == kFP32) {
          const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(qbase) + at + 32 * c);
          const float4 u = p[0], v = p[1];
          x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
          x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
        } else {
          const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(qbase) + at + 32 * c);
          const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[2 * i] = widen16<DT>(d[i] & 0xffffu);
            x[2 * i + 1] = widen16<DT>(d[i] >> 16);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = have ? x[i] : 0.0f;
          top = fmaxf(top, fabsf(x[i]));
        }
      }
      if (have) {
        min_hi = row_hi[nr] < min_hi ? row_hi[nr] : min_hi;
        max_lo = row_lo[nr] > max_lo ? row_lo[nr] : max_lo;
      }
    }
    // one power of two for all rows brings the largest element below 2^15
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      top = fmaxf(top, __shfl_xor(top, off, 64));
      const int oh = __shfl_xor(min_hi, off, 64), ol = __shfl_xor(max_lo, off, 64);
      min_hi = oh < min_hi ? oh : min_hi;
      max_lo = ol > max_lo ? ol : max_lo;
    }
    min_hi = __builtin_amdgcn_readfirstlane(min_hi);
    max_lo = __builtin_amdgcn_readfirstlane(max_lo);
    const int ex = __builtin_amdgcn_readfirstlane(top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int c = 0; c < P; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = __builtin_amdgcn_ldexpf(qf[nr][c][2 * i], 15 - ex);
          const float x1 = __builtin_amdgcn_ldexpf(qf[nr][c][2 * i + 1], 15 - ex);
          hi[i] = pack_f16x2(x0, x1);
          if constexpr (A::kSplitQ) lo[i] = rest_f16x2(x0, x1, hi[i]);
        }
        qh[nr][c] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (A::kSplitQ) ql[nr][c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    qscale_f = __builtin_amdgcn_ldexpf(args.f, ex - 15);
  }

  f32x4 o[NR][2 * P];
  float m_ref[NR], m_use[NR], l_sum[NR];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
    for (int j = 0; j < 2 * P; ++j) o[nr][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    m_ref[nr] = -__builtin_inff();
    m_use[nr] = 0.0f;
    l_sum[nr] = 0.0f;
  }
  int a_exp = -1000;       // A = 2^a_exp
  float a_inv = 0.0f;      // 2^8 / A
  float a_limit = -1.0f;   // 8 A

  // ---- the wave's steps: 32-position steps wave, wave + 8, ... of the range
  const int steps_all = (end - begin + kStep - 1) / kStep;
  const int nsteps = steps_all > wave ? (steps_all - wave + kWaves - 1) / kWaves : 0;
  const int tiles_per_page = kv.page_size / 16;
  const int64_t head_packed = (int64_t)h * kv.page_size * (16 * P);
  const int64_t head_absmax = (int64_t)h * kv.page_size * NB;
  const int64_t table_row = (int64_t)seq * kv.table_stride;

  // page and tile within it of a 16-position tile
  struct Where { int32_t page; int at; };
  auto where = [&](int tile) {
    int col = tile / tiles_per_page;
    const int at = tile - col * tiles_per_page;
    col = col < kv.table_cols ? col : kv.table_cols - 1;
    return Where{scalar_load(kv.table, table_row + col), at};
  };
  auto valid_page = [&](int32_t page) { return page >= 0 && page < kv.num_pages; };

  StepIn<D, BS> in;
  bool ok[2];
  auto load_k = [&](const Where (&w)[2]) {
    const uint8_t *base[2];
    const float *sbase[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t page = valid_page(w[t].page) ? w[t].page : 0;
      base[t] = kv.packed[0] + page * kv.packed_stride + head_packed + w[t].at * (256 * P);
      sbase[t] = kv.absmax[0] + page * kv.absmax_stride + head_absmax + w[t].at * (16 * NB);
      load_words(in.k[t], base[t] + (uint32_t)(n * (16 * P) + g * (4 * P)));
    }
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      int v = 16 * u + n;
      v = v < 8 * NB ? v : v % (8 * NB);
      const int tk = v / NB;
      const uint32_t off = (uint32_t)((4 * g + (tk & 3)) * NB + (v - tk * NB));
      in.ks[u] = (tk < 4 ? sbase[0] : sbase[1])[off];
    }
  };
  auto load_v = [&](const Where (&w)[2]) {
    const float *sbase[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t page = valid_page(w[t].page) ? w[t].page : 0;
      const uint8_t *base = kv.packed[1] + page * kv.packed_stride + head_packed + w[t].at * (256 * P);
      sbase[t] = kv.absmax[1] + page * kv.absmax_stride + head_absmax + w[t].at * (16 * NB);
      load_words(in.v[t], base + (uint32_t)(g * (64 * P) + n * (4 * P)));
    }
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      int v = 16 * u + n;
      v = v < 8 * NB ? v : v % (8 * NB);
      const int tk = v / NB;
      const uint32_t off = (uint32_t)((4 * g + (tk & 3)) * NB + (v - tk * NB));
      in.vs[u] = (tk < 4 ? sbase[0] : sbase[1])[off];
    }
  };

  Where w[2], wn[2];
  const int tile0 = (begin >> 4) + 2 * wave;
  if (nsteps > 0) {
    w[0] = where(tile0);
    w[1] = where(tile0 + 1);
    load_k(w);
    load_v(w);
  }
  __syncthreads();  // the table

  for (int s = 0; s < nsteps; ++s) {
    const int pos0 = begin + kStep * (wave + kWaves * s);
    const int next = s + 1 < nsteps ? s + 1 : s;
    wn[0] = where(tile0 + 2 * kWaves * next);
    wn[1] = where(tile0 + 2 * kWaves * next + 1);
    ok[0] = valid_page(w[0].page);
    ok[1] = valid_page(w[1].page);
    // every row sees the whole step (uniform)
    const bool whole = ok[0] && ok[1] && pos0 >= max_lo && pos0 + kStep <= min_hi;

    // ---- S^T = K Q^T, combined over blocks into log2 units
    float ks[NS];
#pragma unroll
    for (int u = 0; u < NS; ++u) ks[u] = in.ks[u] * qscale_f;
    f32x4 t[NR][2];
    unroll<0, 2>([&](auto tc) {
      constexpr int T = tc;
      unroll<0, NB>([&](auto bc) {
        constexpr int B = bc;
        f32x4 acc[NR];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) acc[nr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        unroll<0, PB>([&](auto pc) {
          constexpr int C = B * PB + pc;  // 32-wide piece
          uint32_t kh[4], kl[4];
          unroll<0, 4>([&](auto ic) {
            constexpr int O = ic * P + C;  // the byte of elements 32 C + 8 g + 2 i
            const uint32_t ad = table_address<O % 4>(in.k[T][O / 4], lane_off);
            kh[ic] = *reinterpret_cast<const uint32_t *>(lds + ad);
            if constexpr (A::kSplitQ) kl[ic] = *reinterpret_cast<const uint32_t *>(lds + ad + 128);
          });
          const uint4 a = make_uint4(kh[0], kh[1], kh[2], kh[3]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            acc[nr] = mfma16x16x32<kFP16>(a, qh[nr][C], acc[nr]);
            if constexpr (A::kSplitQ) {
              acc[nr] = mfma16x16x32<kFP16>(a, ql[nr][C], acc[nr]);
              acc[nr] = mfma16x16x32<kFP16>(make_uint4(kl[0], kl[1], kl[2], kl[3]), qh[nr][C],
                                            acc[nr]);
            }
          }
        });
        unroll<0, 4>([&](auto rc) {
          constexpr int R = rc;
          const float a = row_scale<(4 * T + R) * NB + B>(ks);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            t[nr][T][R] = B == 0 ? acc[nr][R] * a : __builtin_fmaf(acc[nr][R], a, t[nr][T][R]);
        });
      });
    });
    load_k(wn);

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
      // scales of positions that are not there may be anything
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        int v = 16 * u + n;
        v = v < 8 * NB ? v : v % (8 * NB);
        const int tk = v / NB;
        const int p = pos0 + 16 * (tk >> 2) + 4 * g + (tk & 3);
        vs[u] = p < blk.len && (tk < 4 ? ok[0] : ok[1]) ? vs[u] : 0.0f;
      }
    }

    // ---- references
    float top[NR];
    bool far = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      top[nr] = fmaxf(max4(t[nr][0]), max4(t[nr][1]));
      far = far || top[nr] > m_ref[nr] + 4.0f;
    }
#pragma unroll
    for (int u = 0; u < NS; ++u) far = far || vs[u] > a_limit;
    if (__builtin_amdgcn_ballot_w64(far) != 0) {
      float av = vs[0];
#pragma unroll
      for (int u = 1; u < NS; ++u) av = fmaxf(av, vs[u]);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) av = fmaxf(av, __shfl_xor(av, off, 64));
      // 2^8 / A stays finite: from 2^127 on, smaller scales are exact in fp16 steps
      // finer than the result's
      int ex = __builtin_amdgcn_readfirstlane(av > 0.0f ? __builtin_amdgcn_frexp_expf(av) : -119);
      ex = clamp_to(ex, -119, 127);
      ex = ex > a_exp ? ex : a_exp;
      const int shift = a_exp - ex;
      a_exp = ex;
      a_inv = __builtin_amdgcn_ldexpf(1.0f, 8 - ex);
      a_limit = __builtin_amdgcn_ldexpf(8.0f, ex);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float mx = top[nr];
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float m_new = fmaxf(m_ref[nr], mx);
        const float use = m_new == -__builtin_inff() ? 0.0f : m_new;
        // a row that has seen nothing has nothing to rescale
        const float alpha = __builtin_amdgcn_exp2f(m_ref[nr] - use);
        const float beta = __builtin_amdgcn_ldexpf(alpha, shift);
        m_ref[nr] = m_new;
        m_use[nr] = use;
        l_sum[nr] *= alpha;
#pragma unroll
        for (int j = 0; j < 2 * P; ++j) o[nr][j] *= beta;
      }
    }

    // ---- weights
    uint4 wh[NR][NB];
    uint4 wl[A::kSplitW ? NR : 1][A::kSplitW ? NB : 1];
#pragma unroll
    for (int u = 0; u < NS; ++u) vs[u] *= a_inv;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(t[nr][i >> 2][i & 3] - m_use[nr]);
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

    // ---- O^T += V^T W^T
    unroll<0, (P + 3) / 4>([&](auto wc) {
      constexpr int WD = wc;                              // word of a position's run
      constexpr int KN = P - 4 * WD < 4 ? P - 4 * WD : 4;  // its bytes
      uint32_t even[2][2], odd[2][2];  // [tile][pair of positions]: merged nibbles
      unroll<0, 2>([&](auto tc) {
        constexpr int T = tc;
        unroll<0, 2>([&](auto pc) {
          constexpr int R = 2 * pc;
          const uint32_t a = word_at<R * P + 4 * WD>(in.v[T]);
          const uint32_t b = word_at<(R + 1) * P + 4 * WD>(in.v[T]);
          even[T][pc] = (a & 0xf0f0f0f0u) | ((b >> 4) & 0x0f0f0f0fu);
          odd[T][pc] = ((a << 4) & 0xf0f0f0f0u) | (b & 0x0f0f0f0fu);
        });
      });
      unroll<0, KN>([&](auto kc) {
        constexpr int K = 4 * WD + kc;
        constexpr int B = K / PB;
        unroll<0, 2>([&](auto jc) {
          uint32_t vh[4], vl[4];
          unroll<0, 4>([&](auto ic) {
            const uint32_t src = jc == 0 ? even[ic >> 1][ic & 1] : odd[ic >> 1][ic & 1];
            const uint32_t ad = table_address<kc>(src, lane_off);
            vh[ic] = *reinterpret_cast<const uint32_t *>(lds + ad);
            vl[ic] = *reinterpret_cast<const uint32_t *>(lds + ad + 128);
          });
          const uint4 a = make_uint4(vh[0], vh[1], vh[2], vh[3]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            f32x4 &acc = o[nr][2 * K + jc];
            acc = mfma16x16x32<kFP16>(a, wh[nr][B], acc);
            if constexpr (A::kSplitW) acc = mfma16x16x32<kFP16>(a, wl[nr][B], acc);
            acc = mfma16x16x32<kFP16>(make_uint4(vl[0], vl[1], vl[2], vl[3]), wh[nr][B], acc);
          }
        });
      });
    });
    load_v(wn);
    w[0] = wn[0];
    w[1] = wn[1];
  }

  // ---- merge the waves: one reference per row, then the sums in wave order
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    float l = l_sum[nr];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
      wave_m[wave][16 * nr + n] = m_ref[nr];
      wave_l[wave][16 * nr + n] = l;
    }
  }
  __syncthreads();
  float factor[NR];
  const int64_t item = ((int64_t)seq * kv.kv_heads + h) * args.row_blocks + rb;
  const int64_t part_row0 = (item * args.splits + split) * args.part_rows;
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    float mx = wave_m[0][16 * nr + n];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) mx = fmaxf(mx, wave_m[i][16 * nr + n]);
    const float use = mx == -__builtin_inff() ? 0.0f : mx;
    factor[nr] = args.inv_mu * __builtin_amdgcn_exp2f(m_ref[nr] - use);
    if (wave == 0 && g == 0) {
      float l = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i)
        l += wave_l[i][16 * nr + n] * __builtin_amdgcn_exp2f(wave_m[i][16 * nr + n] - use);
      total_l[16 * nr + n] = l;
      if (args.splits > 1 && 16 * nr + n < args.part_rows)
        args.stats[part_row0 + 16 * nr + n] = make_float2(mx, l);
    }
  }
  constexpr int MC = A::kMergeCols, ML = MC + 4;
  float *buf = reinterpret_cast<float *>(lds);
  unroll<0, NR>([&](auto nrc) {
    constexpr int nr = nrc;
    unroll<0, D / MC>([&](auto cc) {
      constexpr int K0 = cc * (MC / 32);
      __syncthreads();
      // lane (n, g) holds row n's elements 32 k + 8 g + 2 r + {0, 1}
      unroll<0, MC / 32>([&](auto kc) {
        constexpr int K = K0 + kc;
        float *dst = buf + (wave * 16 + n) * ML + 32 * kc + 8 * g;
        // undo A apart from the factor: their product may be subnormal
        auto undo = [&](float v) { return __builtin_amdgcn_ldexpf(v * factor[nr], a_exp - 8); };
        const f32x4 e = o[nr][2 * K], d = o[nr][2 * K + 1];
        reinterpret_cast<f32x4 *>(dst)[0] = f32x4{undo(e[0]), undo(d[0]), undo(e[1]), undo(d[1])};
        reinterpret_cast<f32x4 *>(dst)[1] = f32x4{undo(e[2]), undo(d[2]), undo(e[3]), undo(d[3])};
      });
      __syncthreads();
      for (int idx = tid; idx < 16 * (MC / 4); idx += kThreads) {
        const int row = idx / (MC / 4), col = 4 * (idx - row * (MC / 4));
        f32x4 sum = *reinterpret_cast<const f32x4 *>(buf + row * ML + col);
#pragma unroll
        for (int i = 1; i < kWaves; ++i)
          sum += *reinterpret_cast<const f32x4 *>(buf + (i * 16 + row) * ML + col);
        const int pair = blk.row0 + 16 * nr + row;
        const int ccol = cc * MC + col;
        if (pair >= blk.pairs) continue;
        if (args.splits > 1) {
          *reinterpret_cast<f32x4 *>(args.part + (part_row0 + 16 * nr + row) * D + ccol) = sum;
        } else {
          const float l = total_l[16 * nr + row];
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          const int token = pair / args.group;
          const int64_t at = (int64_t)(blk.first + token) * args.out_row +
                             (int64_t)(h * args.group + pair - token * args.group) * args.out_head +
                             ccol;
          if constexpr (DT == kFP32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(args.out) + at) = sum * inv;
          } else {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(args.out) + at) =
                make_uint2(pack2<DT>(sum[0] * inv, sum[1] * inv), pack2<DT>(sum[2] * inv, sum[3] * inv));
          }
        }
      }
    });
  });
}

// ------------------------------------------------------------------- host

struct Plan {
  int tiles, row_blocks, splits, part_rows;
  int64_t part_floats, stats;  // totals
};

// Largest number of 16-row tiles of a workgroup: what its registers hold.
constexpr int max_tiles(int head_dim) { return head_dim <= 128 ? 2 : 1; }

template <int D, int BS, int DT>
hipError_t launch_main(const AttnArgs &a, const Plan &p, hipStream_t stream) {
  const dim3 grid((unsigned)(p.row_blocks * p.splits), (unsigned)a.kv.kv_heads,
                  (unsigned)a.kv.batch);
  if constexpr (max_tiles(D) >= 2) {
    if (p.tiles == 2) {
      hipLaunchKernelGGL((kv_attention_kernel<D, BS, DT, 2>), grid, dim3(kThreads), 0, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((kv_attention_kernel<D, BS, DT, 1>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
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
