// kv_cache.hip -- the 4-bit key/value cache: rows of keys and values quantized
// into their pages (kv_write_kernel) and read back (kv_read_kernel).
//
// Mathematics: nf4_quantize's and nf4_dequantize's on every head vector. Per
// block of BS elements a = max|x|, s = RN(x / a), the code nearest to s (a tie
// to the smaller value); a code stands for RN(c[code] a).
//
// Layout of the work. A wave takes the same heads of four neighbouring rows, a DPP
// row of 16 lanes (j = lane / 4 & 3, i = lane & 3) a head vector. Its 32-element
// pieces are taken in parts of W = 4, 2 or 1; a lane owns 2 W consecutive elements of
// a part, so rows move in 16-byte accesses that cover whole lines, and holds their W
// code bytes. The cache keeps together what lane m = 4 j + i of another arrangement
// owns, byte m of every piece: the bytes change hands within quads of lanes, by DPP and
// byte permutes. Four neighbouring positions' values share a run of 64 P bytes.
//   W = 4: elements 32 (k0 + i) + 8 j ..         W = 1: 32 k0 + 2 m ..
//   W = 2: elements 32 (k0 + i % 2) + 8 j + 4 (i / 2) ..
// Both kernels are bound by HBM. A row's place costs a chain of dependent loads, so a
// wave takes as many heads of it as leave the launch enough waves (kJobsWanted).
// Measured on one MI355X, 8 heads of 128 in bf16: prompts of 16396 rows in all written,
// 153 MB, 32 us, 4.8 TB/s (a copy: 4.99); 73728 rows read, 387 MB, 60-72 us, 5.4-6.4
// TB/s (three quarters are writes). A single token: 3.6 us of GPU time, launch and
// arguments.
#include <type_traits>

#include "kv_internal.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct KvRowsArgs {
  KvArgs kv;
  const void *in[2];   // write: keys, values
  void *out[2];        // read: keys, values; write: their stored values or null
  int64_t row_stride, head_stride;  // elements
  int64_t jobs;        // waves' worth of work: row groups x head groups x 2
  int32_t job_heads, head_groups;
  float value[16];
  float cell_thr[kCells];
  uint32_t cell_codes[kCells];
};

// A row's sequence, by bisection of the offsets (or division), and its place.
struct RowPlace {
  bool in_call;   // the row belongs to a sequence
  bool in_cache;  // and its position to a page
  int32_t page, at;
};

__device__ __forceinline__ RowPlace place_of(const KvArgs &kv, int row) {
  int b, begin, end;
  if (kv.offsets == nullptr) {
    b = kv.uniform > 0 ? row / kv.uniform : 0;
    begin = b * kv.uniform;
    end = begin + kv.uniform;
  } else {
    int lo = 0, hi = kv.batch;  // offsets[lo] <= row < offsets[hi], where they ascend
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (kv.offsets[mid] <= row) lo = mid;
      else hi = mid;
    }
    b = lo;
    begin = clamp_to(kv.offsets[b], 0, kv.total_rows);
    end = clamp_to(kv.offsets[b + 1], 0, kv.total_rows);
  }
  RowPlace r{false, false, 0, 0};
  r.in_call = row >= begin && row < end;
  if (!r.in_call) return r;
  const int pos = clamp_to(kv.lens[b], 0, kMaxPositions) - (end - row);
  if (pos < 0 || pos >= kv.capacity) return r;
  const int col = pos / kv.page_size;
  r.page = kv.table[(int64_t)b * kv.table_stride + col];
  r.at = pos - col * kv.page_size;
  r.in_cache = r.page >= 0 && r.page < kv.num_pages;
  return r;
}

// Where lane m's P bytes of head h at a place live (which: 0 keys, 1 values).
template <int P>
__device__ __forceinline__ int64_t run_offset(const KvArgs &kv, const RowPlace &r, int h,
                                              int which, int m) {
  const int64_t head = (int64_t)r.page * kv.packed_stride +
                       (int64_t)h * kv.page_size * (16 * P);
  if (which == 0) return head + (int64_t)r.at * (16 * P) + m * P;
  return head + (int64_t)(r.at >> 2) * (64 * P) + m * (4 * P) + (r.at & 3) * P;
}

// P bytes, aligned to the largest power of two that divides P.
template <int P>
__device__ __forceinline__ void store_run(uint8_t *p, const uint32_t (&w)[2]) {
  if constexpr (P == 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else if constexpr (P == 4) {
    *reinterpret_cast<uint32_t *>(p) = w[0];
  } else if constexpr (P == 3) {
    for (int i = 0; i < 3; ++i) p[i] = (uint8_t)(w[0] >> (8 * i));
  } else {
    for (int i = 0; i < P / 2; ++i)
      reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

template <int P>
__device__ __forceinline__ void load_run(const uint8_t *p, uint32_t (&w)[2]) {
  w[0] = w[1] = 0;
  if constexpr (P == 8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else if constexpr (P == 4) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (P == 3) {
    for (int i = 0; i < 3; ++i) w[0] |= (uint32_t)p[i] << (8 * i);
  } else {
    for (int i = 0; i < P / 2; ++i)
      w[i >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << (16 * (i & 1));
  }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Part X of P pieces: its first piece and how many.
template <int P, int X>
struct Part {
  static constexpr int K0 = 4 * X;
  static constexpr int W = P - K0 >= 4 ? 4 : (P - K0 >= 2 ? 2 : 1);
};
// P = 3 is 2 + 1, P = 6 is 4 + 2.
template <>
struct Part<3, 0> {
  static constexpr int K0 = 0, W = 2;
};
template <>
struct Part<3, 1> {
  static constexpr int K0 = 2, W = 1;
};
template <int P>
constexpr int kParts = P == 3 ? 2 : (P + 3) / 4;

// First element of a lane's in a part, and its piece.
template <int P, int X>
__device__ __forceinline__ int part_element(int m) {
  constexpr int K0 = Part<P, X>::K0, W = Part<P, X>::W;
  const int i = m & 3, j = m >> 2;
  if (W == 4) return 32 * (K0 + i) + 8 * j;
  if (W == 2) return 32 * (K0 + (i & 1)) + 8 * j + 4 * (i >> 1);
  return 32 * K0 + 2 * m;
}
template <int P, int X>
__device__ __forceinline__ int part_piece(int m) {
  constexpr int K0 = Part<P, X>::K0, W = Part<P, X>::W;
  return K0 + (W == 4 ? m & 3 : (W == 2 ? m & 1 : 0));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// W bytes of a lane, one for each m it covers, to W bytes, one for each piece (or
// back): the exchange is its own inverse. m: lane & 15.
template <int W>
__device__ __forceinline__ uint32_t exchange(uint32_t v, int m) {
  if constexpr (W == 4) {
    const uint32_t i = (uint32_t)m & 3u;
    const uint32_t sel = 0x0c0c0400u + 0x0101u * i;
    const uint32_t q01 = __builtin_amdgcn_perm(dpp<0x55>(v), dpp<0x00>(v), sel);
    const uint32_t q23 = __builtin_amdgcn_perm(dpp<0xff>(v), dpp<0xaa>(v), sel);
    return q01 | q23 << 16;
  } else if constexpr (W == 2) {
    const uint32_t sel = 0x0c0c0400u + 0x0101u * ((uint32_t)m & 1u);
    return __builtin_amdgcn_perm(dpp<0xf5>(v), dpp<0xa0>(v), sel);  // lanes 1 1 3 3, 0 0 2 2
  } else {
    return v;
  }
}

// Maximum over the lanes that own a block (PB pieces) of a part with W pieces.
template <int W, int PB>
__device__ __forceinline__ float block_max(float v) {
  auto with = [](float x, uint32_t o) { return fmaxf(x, __uint_as_float(o)); };
  v = with(v, dpp<0x124>(__float_as_uint(v)));  // row_ror 4, 8: the lanes of equal i
  v = with(v, dpp<0x128>(__float_as_uint(v)));
  if (W < 4 || PB == 4) v = with(v, dpp<0x4e>(__float_as_uint(v)));  // quad 2 3 0 1
  if (W < 2 || PB >= 2) v = with(v, dpp<0xb1>(__float_as_uint(v)));  // quad 1 0 3 2
  return v;
}

// The 2 W elements of a lane's in a part as they are stored.
template <int DT, int W>
struct Raw {
  static constexpr int kWords = (DT == kFP32 ? 2 : 1) * W;
  uint32_t w[kWords];
};

template <int DT, int W>
__device__ __forceinline__ void load_raw(Raw<DT, W> &r, const void *base, int64_t e) {
  const char *p = static_cast<const char *>(base) + e * (DT == kFP32 ? 4 : 2);
  constexpr int N = Raw<DT, W>::kWords;
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[4 * i + k] = v[k];
    }
  } else if constexpr (N == 2) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// Written once and not read back here: past the caches' reuse.
template <int DT, int W>
__device__ __forceinline__ void store_raw(const Raw<DT, W> &r, void *base, int64_t e) {
  char *p = static_cast<char *>(base) + e * (DT == kFP32 ? 4 : 2);
  constexpr int N = Raw<DT, W>::kWords;
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = {r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p) + i);
    }
  } else if constexpr (N == 2) {
    const u32x2 v = {r.w[0], r.w[1]};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2 *>(p));
  } else {
    __builtin_nontemporal_store(r.w[0], reinterpret_cast<uint32_t *>(p));
  }
}

template <int DT, int W>
__device__ __forceinline__ float element(const Raw<DT, W> &r, int i) {
  if constexpr (DT == kFP32) return __uint_as_float(r.w[i]);
  else return widen16<DT>(i & 1 ? r.w[i >> 1] >> 16 : r.w[i >> 1] & 0xffffu);
}

// Elements 2 i and 2 i + 1.
template <int DT, int W>
__device__ __forceinline__ void set_pair(Raw<DT, W> &r, int i, float v0, float v1) {
  if constexpr (DT == kFP32) {
    r.w[2 * i] = __float_as_uint(v0);
    r.w[2 * i + 1] = __float_as_uint(v1);
  } else {
    r.w[i] = pack2<DT>(v0, v1);
  }
}

// Largest magnitude of a lane's elements; those of 16-bit types order like integers.
template <int DT, int W>
__device__ __forceinline__ float largest(const Raw<DT, W> &r) {
  if constexpr (DT == kFP32) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) v = fmaxf(v, fabsf(element(r, i)));
    return v;
  } else {
    u16x2 m = __builtin_bit_cast(u16x2, r.w[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < W; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.w[i] & 0x7fff7fffu));
    return widen16<DT>(m.x > m.y ? m.x : m.y);
  }
}

template <int I, int N, typename F>
__device__ __forceinline__ void unroll(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<I + 1, N>(static_cast<F &&>(f));
  }
}

// All parts of a head vector.
template <int DT, int P>
struct Row {
  Raw<DT, Part<P, 0>::W> a;
  Raw<DT, Part<P, kParts<P> - 1>::W> b;  // the second part, where there is one
  template <int X>
  __device__ __forceinline__ auto &part() {
    if constexpr (X == 0) return a;
    else return b;
  }
};

template <int DT, int P>
__device__ __forceinline__ void load_row(Row<DT, P> &r, const void *base, int64_t e, int m) {
  unroll<0, kParts<P>>([&](auto x) {
    load_raw(r.template part<x>(), base, e + part_element<P, x>(m));
  });
}

// The rows and heads of a job; consecutive jobs take keys and values of the same.
struct Job {
  int which, head0, head1;
  int64_t row_group;
};

__device__ __forceinline__ Job job_of(const KvRowsArgs &args, int64_t job) {
  Job j;
  j.which = (int)(job & 1);
  j.row_group = (job >> 1) / args.head_groups;
  j.head0 = (int)((job >> 1) - j.row_group * args.head_groups) * args.job_heads;
  j.head1 = j.head0 + args.job_heads < args.kv.kv_heads ? j.head0 + args.job_heads
                                                        : args.kv.kv_heads;
  return j;
}

// Heads whose codes a reading wave has in flight: 73728 rows of 8 heads take 71.7 us, 85
// with 4.
constexpr int kInFlight = 8;

// RN(x / a) given r = RN(1 / a): one product and one residual step (Markstein),
// correctly rounded while a, r and the residual stay normal (a in [2^-100,
// 2^120); a quotient so small that it does not lies in zero's cell anyway). For
// bf16 x and a the product alone gives the same NF4 code, shown for every pair
// (quantize.hip).
template <bool PRODUCT>
__device__ __forceinline__ float quotient(float x, float a, float r) {
  const float q = x * r;
  if (PRODUCT) return q;
  return __builtin_fmaf(__builtin_fmaf(-q, a, x), r, q);
}

// Entries of the lookup: cell floor(RN(128 s + 128) / 8) of s. Any bit pattern of s, a
// NaN included, has one of the 64.
constexpr int kLutSize = 64;

// Lookup of s: its cell's entry (a threshold; the codes below and above it in the bytes
// 0 and 1, shifted to the high nibble in 2 and 3) and, 64 entries on, the values of
// these codes. t = 2^23 + RN(128 s + 128) in one fma: its low bits masked to a multiple
// of 8 are the entry's byte offset. Byte J of `codes` becomes the code in the nibble
// that SRC selects (2: high, 0: low), `value` its value; J = 0 clears the other bytes.
// (The select of `value` stands between the byte write and its first reader.)
template <int J, int SRC>
__device__ __forceinline__ void encode(uint32_t &codes, float &value, float s, const uint2 *lut) {
  const float t = __builtin_fmaf(s, 128.0f, 8388736.0f);  // 2^23 + 128
  const uint2 *entry = reinterpret_cast<const uint2 *>(reinterpret_cast<const char *>(lut) +
                                                       (__float_as_uint(t) & 0x1f8u));
  const uint2 e = entry[0], v = entry[kLutSize];
  if constexpr (J == 0) {
    asm("v_cmp_gt_f32 vcc, %2, %3\n\t"
        "s_nop 1\n\t"
        "v_cndmask_b32_sdwa %0, %4, %4, vcc dst_sel:BYTE_0 dst_unused:UNUSED_PAD "
        "src0_sel:BYTE_%7 src1_sel:BYTE_%8\n\t"
        "v_cndmask_b32 %1, %5, %6, vcc"
        : "=&v"(codes), "=v"(value)
        : "v"(s), "v"(e.x), "v"(e.y), "v"(v.x), "v"(v.y), "n"(SRC), "n"(SRC + 1)
        : "vcc");
  } else {
    asm("v_cmp_gt_f32 vcc, %2, %3\n\t"
        "s_nop 1\n\t"
        "v_cndmask_b32_sdwa %0, %4, %4, vcc dst_sel:BYTE_%9 dst_unused:UNUSED_PRESERVE "
        "src0_sel:BYTE_%7 src1_sel:BYTE_%8\n\t"
        "v_cndmask_b32 %1, %5, %6, vcc"
        : "+&v"(codes), "=v"(value)
        : "v"(s), "v"(e.x), "v"(e.y), "v"(v.x), "v"(v.y), "n"(SRC), "n"(SRC + 1), "n"(J)
        : "vcc");
  }
}

template <int D, int BS, int DT, bool PRODUCT>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvRowsArgs args) {
  constexpr int P = D / 32, NB = D / BS, PB = BS / 32;  // pieces of a row, blocks, pieces a block
  __shared__ uint2 lut[2 * kLutSize];
  if (threadIdx.x < kLutSize) {
    const int c = threadIdx.x < kCells ? threadIdx.x : kCells - 1;
    const uint32_t codes = args.cell_codes[c];
    lut[threadIdx.x] = make_uint2(__float_as_uint(args.cell_thr[c]), codes);
    lut[kLutSize + threadIdx.x] = make_uint2(__float_as_uint(args.value[codes & 15]),
                                             __float_as_uint(args.value[codes >> 8 & 15]));
  }
  __syncthreads();
  const KvArgs &kv = args.kv;
  const int lane = threadIdx.x & 63, m = lane & 15;
  const int64_t wave = (int64_t)blockIdx.x * kWaves +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nwaves = (int64_t)gridDim.x * kWaves;
  for (int64_t job = wave; job < args.jobs; job += nwaves) {
    const Job j = job_of(args, job);
    const int64_t row = j.row_group * 4 + (lane >> 4);
    // rows past the last take its elements and have no place
    const int64_t from = row < kv.total_rows ? row : kv.total_rows - 1;
    const void *in = args.in[j.which];
    Row<DT, P> next;
    load_row<DT, P>(next, in, from * args.row_stride + j.head0 * args.head_stride, m);
    const RowPlace place =
        row < kv.total_rows ? place_of(kv, (int)row) : RowPlace{false, false, 0, 0};
    const bool values = args.out[0] != nullptr && place.in_call;
    for (int h = j.head0; h < j.head1; ++h) {
      Row<DT, P> x = next;
      // the next head's elements are on their way while this one's are encoded
      const int hn = h + 1 < j.head1 ? h + 1 : h;
      load_row<DT, P>(next, in, from * args.row_stride + hn * args.head_stride, m);

      uint32_t run[2] = {0, 0};
      unroll<0, kParts<P>>([&](auto xc) {
        constexpr int X = xc, K0 = Part<P, X>::K0, W = Part<P, X>::W;
        auto &raw = x.template part<X>();
        const float a = block_max<W, PB>(largest(raw));
        // outside [2^-100, 2^120) x and a are first scaled by the power of two that
        // brings a into [1, 2): the quotient is the same. One branch for the wave.
        float as = a;
        int sh = 0;
        const bool scaled = __builtin_amdgcn_ballot_w64(!(a >= 0x1p-100f && a < 0x1p120f)) != 0;
        if (scaled && a > 0.0f) {
          sh = 1 - __builtin_amdgcn_frexp_expf(a);
          as = __builtin_amdgcn_ldexpf(a, sh);
        }
        const float r = as == 0.0f ? 0.0f : 1.0f / as;
        uint32_t high, low;  // the codes of the even and of the odd elements
        Raw<DT, W> out;
        unroll<0, W>([&](auto ic) {
          constexpr int I = ic;
          float x0 = element(raw, 2 * I), x1 = element(raw, 2 * I + 1);
          if (scaled) {
            x0 = __builtin_amdgcn_ldexpf(x0, sh);
            x1 = __builtin_amdgcn_ldexpf(x1, sh);
          }
          float v0, v1;
          encode<I, 2>(high, v0, quotient<PRODUCT>(x0, as, r), lut);
          encode<I, 0>(low, v1, quotient<PRODUCT>(x1, as, r), lut);
          set_pair(out, I, v0 * a, v1 * a);
        });
        if (values)
          store_raw(out, args.out[j.which], (row * kv.kv_heads + h) * D + part_element<P, X>(m));
        const uint32_t bytes = exchange<W>(high | low, m);
        run[K0 >> 2] |= bytes << (8 * (K0 & 3));
        // a block's scale from the first of its lanes
        const int piece = part_piece<P, X>(m);
        const bool first = W == 1 ? m == 0 : (W == 2 ? m < 2 : m < 4);
        if (place.in_cache && first && piece % PB == 0)
          kv.absmax[j.which][place.page * kv.absmax_stride +
                             ((int64_t)h * kv.page_size + place.at) * NB + piece / PB] = a;
      });
      if (place.in_cache)
        store_run<P>(kv.packed[j.which] + run_offset<P>(kv, place, h, j.which, m), run);
    }
  }
}

template <int D, int BS, int DT>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvRowsArgs args) {
  constexpr int P = D / 32, NB = D / BS, PB = BS / 32;
  __shared__ float value[16];
  if (threadIdx.x < 16) value[threadIdx.x] = args.value[threadIdx.x];
  __syncthreads();
  const KvArgs &kv = args.kv;
  const int lane = threadIdx.x & 63, m = lane & 15;
  const int64_t wave = (int64_t)blockIdx.x * kWaves +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nwaves = (int64_t)gridDim.x * kWaves;
  for (int64_t job = wave; job < args.jobs; job += nwaves) {
    const Job j = job_of(args, job);
    const int64_t row = j.row_group * 4 + (lane >> 4);
    const RowPlace place =
        row < kv.total_rows ? place_of(kv, (int)row) : RowPlace{false, false, 0, 0};
    void *out = args.out[j.which];
    // kInFlight heads' codes and scales a time; lanes without a place hold zeros
    for (int h0 = j.head0; h0 < j.head1; h0 += kInFlight) {
      uint32_t run[kInFlight][2];
      float a[kInFlight][kParts<P>];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int h = h0 + u < j.head1 ? h0 + u : j.head1 - 1;
        run[u][0] = run[u][1] = 0;
#pragma unroll
        for (int x = 0; x < kParts<P>; ++x) a[u][x] = 0.0f;
        if (place.in_cache) {
          load_run<P>(kv.packed[j.which] + run_offset<P>(kv, place, h, j.which, m), run[u]);
          const float *s = kv.absmax[j.which] + place.page * kv.absmax_stride +
                           ((int64_t)h * kv.page_size + place.at) * NB;
          unroll<0, kParts<P>>([&](auto x) { a[u][x] = s[part_piece<P, x>(m) / PB]; });
        }
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (h0 + u >= j.head1) break;
        unroll<0, kParts<P>>([&](auto xc) {
          constexpr int X = xc, K0 = Part<P, X>::K0, W = Part<P, X>::W;
          const uint32_t bytes = exchange<W>(run[u][K0 >> 2] >> (8 * (K0 & 3)), m);
          Raw<DT, W> r;
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const uint32_t byte = bytes >> (8 * i) & 0xffu;
            const float v0 = value[byte >> 4] * a[u][X], v1 = value[byte & 15] * a[u][X];
            // code 0 is not the value 0
            set_pair(r, i, place.in_cache ? v0 : 0.0f, place.in_cache ? v1 : 0.0f);
          }
          if (place.in_call)
            store_raw(r, out, row * args.row_stride + (h0 + u) * args.head_stride +
                                  part_element<P, X>(m));
        });
      }
    }
  }
}

// Waves' worth of work wanted before a wave takes more heads: prompts written in 32.9 us
// with 1024 and with 4096, 35.8 with 16384; a few hundred rows are bound by the launch.
constexpr int64_t kJobsWanted = 4096;

KvRowsArgs make_args(const KvArgs &kv, const KvShape &sh) {
  KvRowsArgs a;
  a.kv = kv;
  const CodeTables &t = code_tables(sh.quant_type);
  for (int i = 0; i < 16; ++i) a.value[i] = t.value[i];
  for (int i = 0; i < kCells; ++i) {
    a.cell_thr[i] = t.cell_thr[i];
    a.cell_codes[i] = t.cell_codes[i];
  }
  a.in[0] = a.in[1] = nullptr;
  a.out[0] = a.out[1] = nullptr;
  const int64_t row_groups = ((int64_t)kv.total_rows + 3) / 4;
  int heads = 1;
  while (heads < kv.kv_heads &&
         row_groups * 2 * ((kv.kv_heads + 2 * heads - 1) / (2 * heads)) >= kJobsWanted)
    heads *= 2;
  a.job_heads = heads < kv.kv_heads ? heads : kv.kv_heads;
  a.head_groups = (kv.kv_heads + a.job_heads - 1) / a.job_heads;
  a.jobs = row_groups * a.head_groups * 2;
  return a;
}

template <bool WRITE, int D, int BS, int DT>
void launch_cfg(const KvRowsArgs &a, bool nf4, hipStream_t stream) {
  int64_t blocks = (a.jobs + kWaves - 1) / kWaves;
  if (blocks > 16384) blocks = 16384;
  const dim3 grid((unsigned)blocks), block(kThreads);
  if constexpr (!WRITE) {
    hipLaunchKernelGGL((kv_read_kernel<D, BS, DT>), grid, block, 0, stream, a);
  } else if constexpr (DT == kBF16) {
    if (nf4) hipLaunchKernelGGL((kv_write_kernel<D, BS, DT, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((kv_write_kernel<D, BS, DT, false>), grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((kv_write_kernel<D, BS, DT, false>), grid, block, 0, stream, a);
  }
}

template <bool WRITE, int D, int BS>
hipError_t launch_dt(const KvRowsArgs &a, const KvShape &sh, hipStream_t stream) {
  const bool nf4 = sh.quant_type == kQuantNF4;
  const int dtype = sh.dtype;
  if (dtype == kFP32) launch_cfg<WRITE, D, BS, kFP32>(a, nf4, stream);
  else if (dtype == kFP16) launch_cfg<WRITE, D, BS, kFP16>(a, nf4, stream);
  else launch_cfg<WRITE, D, BS, kBF16>(a, nf4, stream);
  return hipGetLastError();
}

template <bool WRITE>
hipError_t launch_shape(const KvRowsArgs &a, const KvShape &sh, hipStream_t stream) {
  switch (sh.head_dim * 1000 + sh.blocksize) {
#define NF4_KV_CASE(DV, BSV) \
  case DV * 1000 + BSV: return launch_dt<WRITE, DV, BSV>(a, sh, stream);
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

}  // namespace

hipError_t launch_kv_write(const KvArgs &kv, const KvShape &sh, const void *k, const void *v,
                           int64_t row_stride, int64_t head_stride, void *k_values, void *v_values,
                           hipStream_t stream) {
  KvRowsArgs a = make_args(kv, sh);
  a.in[0] = k;
  a.in[1] = v;
  a.out[0] = k_values;
  a.out[1] = v_values;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  return launch_shape<true>(a, sh, stream);
}

hipError_t launch_kv_read(const KvArgs &kv, const KvShape &sh, void *k, void *v,
                          int64_t row_stride, int64_t head_stride, hipStream_t stream) {
  KvRowsArgs a = make_args(kv, sh);
  a.out[0] = k;
  a.out[1] = v;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  return launch_shape<false>(a, sh, stream);
}

}  // namespace nf4
