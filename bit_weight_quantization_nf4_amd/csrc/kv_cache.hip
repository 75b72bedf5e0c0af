// kv_cache.hip -- the 4-bit key/value cache: rows of keys and values quantized
// into their pages (kv_write_kernel) and read back (kv_read_kernel).
//
// Mathematics: nf4_quantize's and nf4_dequantize's on every head vector. Per
// block of BS elements a = max|x|, s = RN(x / a), the code nearest to s (a tie
// to the smaller value); a code stands for RN(c[code] a).
//
// Layout of the work. A head vector belongs to the 16 lanes of a DPP row: lane
// m owns elements 32 k + 2 m and + 1 for every k < P = D / 32, which are the P
// bytes that the cache keeps together for it (nf4_kv.h), so a lane stores (or
// loads) its codes in one piece and nothing moves between lanes but the block
// maxima. A wave takes the same head of four neighbouring rows: of one
// sequence these share the run of 64 P bytes that holds four positions' values.
// Both kernels are bound by HBM; a lane's 4-byte accesses to the 16-bit rows
// cover 64 contiguous bytes per head vector and k.
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
  const int pos = clamp_to(kv.lens[b], 0, kv.capacity) - (end - row);
  if (pos < 0) return r;
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

// A pair of neighbouring elements at element offset e (even).
template <int DT>
__device__ __forceinline__ void store_pair(void *base, int64_t e, float v0, float v1) {
  if constexpr (DT == kFP32) {
    *reinterpret_cast<f32x2 *>(static_cast<float *>(base) + e) = f32x2{v0, v1};
  } else {
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + e) = pack2<DT>(v0, v1);
  }
}

// A lane's elements of a head vector as they are stored, and widened.
template <int DT, int P>
struct Pieces {
  typename std::conditional<DT == kFP32, f32x2, uint32_t>::type v[P];
};

template <int DT, int P>
__device__ __forceinline__ void load_row(Pieces<DT, P> &p, const void *base, int64_t e) {
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if constexpr (DT == kFP32)
      p.v[k] = *reinterpret_cast<const f32x2 *>(static_cast<const float *>(base) + e + 32 * k);
    else
      p.v[k] =
          *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + e + 32 * k);
  }
}

template <int DT, int P>
__device__ __forceinline__ void widen(f32x2 (&x)[P], const Pieces<DT, P> &p) {
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if constexpr (DT == kFP32) x[k] = p.v[k];
    else x[k] = f32x2{widen16<DT>(p.v[k] & 0xffffu), widen16<DT>(p.v[k] >> 16)};
  }
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

// Heads whose codes a reading wave has in flight.
constexpr int kInFlight = 4;

// RN(x / a) given r = RN(1 / a): one product and one residual step (Markstein),
// correctly rounded while a, r and the residual stay normal (a in [2^-100,
// 2^120); a quotient so small that it does not lies in zero's cell anyway).
__device__ __forceinline__ float quotient(float x, float a, float r) {
  const float q = x * r;
  return __builtin_fmaf(__builtin_fmaf(-q, a, x), r, q);
}

template <int D, int BS, int DT>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvRowsArgs args) {
  constexpr int P = D / 32, NB = D / BS, PB = BS / 32;  // pieces of a row, blocks, pieces a block
  __shared__ uint2 lut[kLutSize];
  __shared__ float value[16];
  if (threadIdx.x < kLutSize) {
    const int c = threadIdx.x < kCells ? threadIdx.x : kCells - 1;
    lut[threadIdx.x] = make_uint2(__float_as_uint(args.cell_thr[c]), args.cell_codes[c]);
  } else if (threadIdx.x < kLutSize + 16) {
    value[threadIdx.x - kLutSize] = args.value[threadIdx.x - kLutSize];
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
    // rows past the last take its values and have no place
    const int64_t from = row < kv.total_rows ? row : kv.total_rows - 1;
    const void *in = args.in[j.which];
    Pieces<DT, P> next;
    load_row(next, in, from * args.row_stride + j.head0 * args.head_stride + 2 * m);
    const RowPlace place =
        row < kv.total_rows ? place_of(kv, (int)row) : RowPlace{false, false, 0, 0};
    const bool values = args.out[0] != nullptr && place.in_call;
    for (int h = j.head0; h < j.head1; ++h) {
      f32x2 x[P];
      widen(x, next);
      // the next head's elements are on their way while this one's are encoded
      const int hn = h + 1 < j.head1 ? h + 1 : h;
      load_row(next, in, from * args.row_stride + hn * args.head_stride + 2 * m);

      float a[NB], as[NB], r[NB];
      int sh[NB];
      bool normal = true;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float v = 0.0f;
#pragma unroll
        for (int k = b * PB; k < (b + 1) * PB; ++k)
          v = fmaxf(v, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
        a[b] = row16_max(v);
        normal = normal && a[b] >= 0x1p-100f && a[b] < 0x1p120f;
      }
      // outside that range x and a are first scaled by the power of two that
      // brings a into [1, 2): the quotient is the same. One branch for the wave.
      const bool scaled = __builtin_amdgcn_ballot_w64(!normal) != 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        as[b] = a[b];
        sh[b] = 0;
        if (scaled && a[b] > 0.0f) {
          sh[b] = 1 - __builtin_amdgcn_frexp_expf(a[b]);
          as[b] = __builtin_amdgcn_ldexpf(a[b], sh[b]);
        }
        r[b] = as[b] == 0.0f ? 0.0f : 1.0f / as[b];
      }
      uint32_t w[2] = {0, 0};
      const int64_t ve = (row * kv.kv_heads + h) * D + 2 * m;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int b = k / PB;
        float x0 = x[k].x, x1 = x[k].y;
        if (scaled) {
          x0 = __builtin_amdgcn_ldexpf(x0, sh[b]);
          x1 = __builtin_amdgcn_ldexpf(x1, sh[b]);
        }
        const uint32_t c0 = code_of(quotient(x0, as[b], r[b]), lut);
        const uint32_t c1 = code_of(quotient(x1, as[b], r[b]), lut);
        w[k >> 2] |= (c0 << 4 | c1) << (8 * (k & 3));
        if (values) store_pair<DT>(args.out[j.which], ve + 32 * k, value[c0] * a[b], value[c1] * a[b]);
      }
      if (place.in_cache) {
        store_run<P>(kv.packed[j.which] + run_offset<P>(kv, place, h, j.which, m), w);
        float mine = a[0];
#pragma unroll
        for (int b = 1; b < NB; ++b) mine = m == b ? a[b] : mine;
        if (m < NB)
          kv.absmax[j.which][place.page * kv.absmax_stride +
                           ((int64_t)h * kv.page_size + place.at) * NB + m] = mine;
      }
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
    if (row >= kv.total_rows) continue;
    const RowPlace place = place_of(kv, (int)row);
    if (!place.in_call) continue;
    void *out = args.out[j.which];
    if (!place.in_cache) {
      for (int h = j.head0; h < j.head1; ++h)
#pragma unroll
        for (int k = 0; k < P; ++k)
          store_pair<DT>(out, row * args.row_stride + h * args.head_stride + 2 * m + 32 * k, 0.0f,
                         0.0f);
      continue;
    }
    // kInFlight heads' codes and scales a time
    for (int h0 = j.head0; h0 < j.head1; h0 += kInFlight) {
      uint32_t w[kInFlight][2];
      float a[kInFlight][NB];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int h = h0 + u < j.head1 ? h0 + u : j.head1 - 1;
        load_run<P>(kv.packed[j.which] + run_offset<P>(kv, place, h, j.which, m), w[u]);
        const float *s = kv.absmax[j.which] + place.page * kv.absmax_stride +
                         ((int64_t)h * kv.page_size + place.at) * NB;
#pragma unroll
        for (int b = 0; b < NB; ++b) a[u][b] = s[b];
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        if (h0 + u >= j.head1) break;
        const int64_t e = row * args.row_stride + (h0 + u) * args.head_stride + 2 * m;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const uint32_t byte = w[u][k >> 2] >> (8 * (k & 3)) & 0xffu;
          store_pair<DT>(out, e + 32 * k, value[byte >> 4] * a[u][k / PB],
                         value[byte & 15] * a[u][k / PB]);
        }
      }
    }
  }
}

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
  // A row's place costs a chain of dependent loads, so a wave takes as many heads
  // of it as leave the launch kJobsWanted waves.
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
void launch_cfg(const KvRowsArgs &a, hipStream_t stream) {
  int64_t blocks = (a.jobs + kWaves - 1) / kWaves;
  if (blocks > 16384) blocks = 16384;
  if constexpr (WRITE)
    hipLaunchKernelGGL((kv_write_kernel<D, BS, DT>), dim3((unsigned)blocks), dim3(kThreads), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((kv_read_kernel<D, BS, DT>), dim3((unsigned)blocks), dim3(kThreads), 0,
                       stream, a);
}

template <bool WRITE, int D, int BS>
hipError_t launch_dt(const KvRowsArgs &a, int dtype, hipStream_t stream) {
  if (dtype == kFP32) launch_cfg<WRITE, D, BS, kFP32>(a, stream);
  else if (dtype == kFP16) launch_cfg<WRITE, D, BS, kFP16>(a, stream);
  else launch_cfg<WRITE, D, BS, kBF16>(a, stream);
  return hipGetLastError();
}

template <bool WRITE>
hipError_t launch_shape(const KvRowsArgs &a, const KvShape &sh, hipStream_t stream) {
  switch (sh.head_dim * 1000 + sh.blocksize) {
#define NF4_KV_CASE(DV, BSV) \
  case DV * 1000 + BSV: return launch_dt<WRITE, DV, BSV>(a, sh.dtype, stream);
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
