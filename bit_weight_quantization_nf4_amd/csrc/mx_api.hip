// mx_api.hip -- the extern "C" boundary of the microscaled 4-bit matrices (declared in
// include/nf4_mx.h): argument validation and dispatch to the launchers. Every check runs
// before the first launch, so a rejected call writes nothing.
#include "mx_internal.h"

using namespace nf4;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 23;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool valid_dtype(int32_t d) {
  return d == NF4_DTYPE_BF16 || d == NF4_DTYPE_FP32 || d == NF4_DTYPE_FP16;
}

int64_t dtype_bytes(int32_t d) { return d == NF4_DTYPE_FP32 ? 4 : 2; }

nf4_status from_hip(hipError_t e) { return e == hipSuccess ? NF4_OK : NF4_ERR_DEVICE; }

nf4_status check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return NF4_ERR_INVALID_ARGUMENT;
  if (rows > INT32_MAX || cols > kMaxCols) return NF4_ERR_UNSUPPORTED;
  return NF4_OK;
}

nf4_status check_matrix(const nf4_mx_matrix *m, MxMatrix *to) {
  if (m == nullptr) return NF4_ERR_INVALID_ARGUMENT;
  const nf4_status st = check_sizes(m->rows, m->cols);
  if (st != NF4_OK) return st;
  if (m->rows > 0 && m->cols > 0) {
    if (m->codes == nullptr || m->scales == nullptr) return NF4_ERR_INVALID_ARGUMENT;
    if (!aligned(m->codes, 16) || !aligned(m->scales, 4)) return NF4_ERR_MISALIGNED;
  }
  *to = MxMatrix{m->codes, m->scales, m->rows, (int32_t)m->cols, (int32_t)mx_padded(m->cols)};
  return NF4_OK;
}

// A [rows][cols] tensor of `dtype` whose rows are `stride` elements apart.
nf4_status check_rows(const void *p, int32_t dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (!valid_dtype(dtype) || stride < cols) return NF4_ERR_INVALID_ARGUMENT;
  if (rows > 0 && stride > (INT64_MAX >> 3) / rows) return NF4_ERR_INVALID_ARGUMENT;
  if (rows > 0 && cols > 0 && p == nullptr) return NF4_ERR_INVALID_ARGUMENT;
  return aligned(p, (uintptr_t)dtype_bytes(dtype)) ? NF4_OK : NF4_ERR_MISALIGNED;
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Which kernel a product takes, and what it needs of the workspace.
struct Plan {
  enum Kind { kGemvQuantizing, kGemv, kGemm } kind;
  int64_t codes, scales, product;  // bytes: x quantized, the kernel's own
};

Plan plan_of(int64_t M, int64_t N, int64_t K, bool raw) {
  Plan p{Plan::kGemm, 0, 0, 0};
  if (mx_gemv_takes(M, N, K)) p.kind = Plan::kGemv;
  if (raw && p.kind == Plan::kGemv && mx_gemv_quantizes(M, K)) p.kind = Plan::kGemvQuantizing;
  if (raw && p.kind != Plan::kGemvQuantizing) {
    const int64_t padded = mx_padded(K);
    p.codes = align256(M * (padded / 2));
    p.scales = align256(M * (padded / kMxBlock));
  }
  if (p.kind == Plan::kGemm) p.product = align256(mx_gemm_workspace_bytes(M, N, K));
  return p;
}

int64_t workspace_bytes(int64_t M, int64_t N, int64_t K, bool raw) {
  if (check_sizes(M, K) != NF4_OK || check_sizes(N, K) != NF4_OK) return -1;
  if (M > 0 && N > 0 && (!mx_elementwise_fits(M, K) || !mx_gemm_fits(M, N))) return -1;
  if (M == 0 || N == 0) return 0;
  const Plan p = plan_of(M, N, K, raw);
  return p.codes + p.scales + p.product;
}

// Checks that both products share, after x's own.
nf4_status check_product(int64_t M, int64_t K, const nf4_mx_matrix *w, const void *bias,
                         int32_t out_dtype, void *y, int64_t ldy, void *workspace,
                         int64_t workspace_size, MxProduct *p) {
  nf4_status st = check_matrix(w, &p->w);
  if (st != NF4_OK) return st;
  if (w->cols != K || workspace_size < 0 || (workspace_size > 0 && workspace == nullptr))
    return NF4_ERR_INVALID_ARGUMENT;
  st = check_rows(y, out_dtype, M, w->rows, ldy);
  if (st != NF4_OK) return st;
  if (!aligned(bias, (uintptr_t)dtype_bytes(out_dtype)) || !aligned(workspace, 16))
    return NF4_ERR_MISALIGNED;
  p->bias = bias;
  p->out_dtype = out_dtype;
  p->y = y;
  p->ldy = ldy;
  return NF4_OK;
}

// x: raw (of x_dtype, rows ldx apart) where not null, else the matrix.
nf4_status run_product(const MxMatrix *x, const void *raw, int32_t x_dtype, int64_t ldx, int64_t M,
                       const MxProduct &p, void *workspace, int64_t workspace_size,
                       hipStream_t stream) {
  const int64_t N = p.w.rows, K = p.w.cols;
  if (M == 0 || N == 0) return NF4_OK;
  // (a sum of no products would still be the bias: there is no such matrix)
  if (K == 0) return NF4_ERR_UNSUPPORTED;
  if (!mx_elementwise_fits(M, K) || !mx_gemm_fits(M, N)) return NF4_ERR_UNSUPPORTED;
  const nf4_status st = nf4_device_check();
  if (st != NF4_OK) return st;
  const Plan plan = plan_of(M, N, K, x == nullptr);
  if (workspace_size < plan.codes + plan.scales + plan.product) return NF4_ERR_SCRATCH;
  if (log_on()) {
    const char *how = x != nullptr ? ""
                      : plan.kind == Plan::kGemvQuantizing ? ", x quantized in it"
                                                           : " after mx_quantize_kernel";
    if (plan.kind == Plan::kGemm) {
      const MxGemmShape shape = mx_gemm_shape(M, N, K);
      log_msg("mx product M=%lld N=%lld K=%lld: mx_gemm_kernel%s, tiles of %d, %d range(s) of %d steps",
              (long long)M, (long long)N, (long long)K, how, shape.tile, shape.splits,
              shape.split_steps);
    } else {
      log_msg("mx product M=%lld N=%lld K=%lld: mx_gemv_kernel%s", (long long)M, (long long)N,
              (long long)K, how);
    }
  }
  if (plan.kind == Plan::kGemvQuantizing)
    return from_hip(launch_mx_gemv_quantizing(raw, x_dtype, ldx, (int)M, p, stream));
  MxMatrix own;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  if (x == nullptr) {
    const hipError_t e =
        launch_mx_quantize(raw, x_dtype, M, (int32_t)K, ldx, at, at + plan.codes, stream);
    if (e != hipSuccess) return from_hip(e);
    own = MxMatrix{at, at + plan.codes, M, (int32_t)K, (int32_t)mx_padded(K)};
    x = &own;
  }
  at += plan.codes + plan.scales;
  return from_hip(plan.kind == Plan::kGemv ? launch_mx_gemv(*x, p, stream)
                                           : launch_mx_gemm(*x, p, at, stream));
}

}  // namespace

extern "C" {

int64_t nf4_mx_padded(int64_t cols) {
  return check_sizes(0, cols) == NF4_OK ? mx_padded(cols) : -1;
}

nf4_status nf4_mx_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols,
                           int64_t row_stride, uint8_t *codes, uint8_t *scales, void *stream) {
  nf4_status st = check_sizes(rows, cols);
  if (st != NF4_OK) return st;
  st = check_rows(x, dtype, rows, cols, row_stride);
  if (st != NF4_OK) return st;
  const nf4_mx_matrix to{codes, scales, rows, cols};
  MxMatrix m;
  st = check_matrix(&to, &m);
  if (st != NF4_OK) return st;
  if (rows == 0 || cols == 0) return NF4_OK;
  if (!mx_elementwise_fits(rows, cols)) return NF4_ERR_UNSUPPORTED;
  st = nf4_device_check();
  if (st != NF4_OK) return st;
  if (log_on())
    log_msg("mx_quantize rows=%lld cols=%lld ld=%lld dtype=%d: mx_quantize_kernel", (long long)rows,
            (long long)cols, (long long)row_stride, dtype);
  return from_hip(launch_mx_quantize(x, dtype, rows, (int32_t)cols, row_stride, codes, scales,
                                     reinterpret_cast<hipStream_t>(stream)));
}

nf4_status nf4_mx_dequantize(const nf4_mx_matrix *m, int32_t dtype, void *out, int64_t row_stride,
                             void *stream) {
  MxMatrix from;
  nf4_status st = check_matrix(m, &from);
  if (st != NF4_OK) return st;
  st = check_rows(out, dtype, from.rows, from.cols, row_stride);
  if (st != NF4_OK) return st;
  if (from.rows == 0 || from.cols == 0) return NF4_OK;
  if (!mx_elementwise_fits(from.rows, from.cols)) return NF4_ERR_UNSUPPORTED;
  st = nf4_device_check();
  if (st != NF4_OK) return st;
  if (log_on())
    log_msg("mx_dequantize rows=%lld cols=%d dtype=%d: mx_dequantize_kernel", (long long)from.rows,
            from.cols, dtype);
  return from_hip(launch_mx_dequantize(from, dtype, out, row_stride,
                                       reinterpret_cast<hipStream_t>(stream)));
}

int64_t nf4_mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return workspace_bytes(M, N, K, false);
}

int64_t nf4_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return workspace_bytes(M, N, K, true);
}

nf4_status nf4_mx_matmul(const nf4_mx_matrix *x, const nf4_mx_matrix *w, const void *bias,
                         int32_t out_dtype, void *y, int64_t ldy, void *workspace,
                         int64_t workspace_bytes, void *stream) {
  MxMatrix xm;
  MxProduct p;
  nf4_status st = check_matrix(x, &xm);
  if (st != NF4_OK) return st;
  st = check_product(xm.rows, xm.cols, w, bias, out_dtype, y, ldy, workspace, workspace_bytes, &p);
  if (st != NF4_OK) return st;
  return run_product(&xm, nullptr, 0, 0, xm.rows, p, workspace, workspace_bytes,
                     reinterpret_cast<hipStream_t>(stream));
}

nf4_status nf4_mx_linear(const void *x, int32_t x_dtype, int64_t ldx, int64_t M,
                         const nf4_mx_matrix *w, const void *bias, int32_t out_dtype, void *y,
                         int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream) {
  if (w == nullptr) return NF4_ERR_INVALID_ARGUMENT;
  MxProduct p;
  nf4_status st = check_sizes(M, w->cols);
  if (st != NF4_OK) return st;
  st = check_rows(x, x_dtype, M, w->cols, ldx);
  if (st != NF4_OK) return st;
  st = check_product(M, w->cols, w, bias, out_dtype, y, ldy, workspace, workspace_bytes, &p);
  if (st != NF4_OK) return st;
  return run_product(nullptr, x, x_dtype, ldx, M, p, workspace, workspace_bytes,
                     reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
