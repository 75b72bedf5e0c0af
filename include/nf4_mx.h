/*
 * nf4_mx.h -- C ABI of the microscaled 4-bit matrices of libnf4 (MI355X, gfx950):
 * quantisation, restoring, and the product of two of them on the matrix cores.
 * It stands beside nf4.h and shares its status codes, dtypes and conventions
 * (device pointers, validation before any launch, asynchronous on `stream`, no
 * allocation, no pointer kept).
 *
 * Format. Elements are E2M1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives), and
 * each block of 32 consecutive elements of a row shares a scale 2^(s - 127), one
 * byte s of 0 .. 254; s = 255 stands for NaN. Quantisation of a block: with a its
 * largest magnitude,
 *   2^(s - 127) = 2^(floor(log2 a) - 2), s at least 0;  1 (s = 127) where a = 0,
 *   element = x / 2^(s - 127) rounded to the nearest E2M1 value, a tie to the even
 *   code, magnitudes above 6 to 6; the sign is x's, of zeros too.
 * A block that holds an infinity or a NaN has s = 255 and codes 0: every element
 * of it stands for NaN.
 *
 * Storage of a matrix of `rows` rows of `cols` elements: rows are padded with zeros
 * to Kp = nf4_mx_padded(cols), a multiple of 128.
 *   codes   uint8 [rows][Kp / 2]: element 2i of a row in bits 7..4 of byte i, element
 *           2i + 1 in bits 3..0; sign in bit 3 of a code, as in nf4.h's FP4
 *   scales  uint8 [Kp / 128][rows][4]: the scales of the blocks 4t .. 4t + 3 of row
 *           r at [t][r], so that a step of the product finds neighbouring rows' side
 *           by side
 * What the padding holds takes part in products: nf4_mx_quantize writes zeros of
 * scale 1 there, and matrices from elsewhere have to.
 */
#ifndef NF4_MX_H
#define NF4_MX_H

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A microscaled matrix: device pointers (codes 16-byte aligned, scales 4-byte),
 * contiguous as above. Limits (NF4_ERR_UNSUPPORTED otherwise): cols <= 2^23, rows <
 * 2^31. */
typedef struct nf4_mx_matrix {
  const uint8_t *codes;
  const uint8_t *scales;
  int64_t rows;
  int64_t cols;
} nf4_mx_matrix;

/* cols rounded up to a multiple of 128 (-1 where cols is negative or past the limit). */
int64_t nf4_mx_padded(int64_t cols);

/* Quantizes x [rows][cols] of `dtype`, rows row_stride elements apart (at least cols;
 * any alignment of the type's own). */
nf4_status nf4_mx_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols,
                           int64_t row_stride, uint8_t *codes, uint8_t *scales, void *stream);

/* Restores a matrix: out [rows][cols] of `dtype`, rows row_stride elements apart, each
 * element's value rounded to dtype (an infinity where it is past the type's range; fp32 holds all
 * that nf4_mx_quantize makes). */
nf4_status nf4_mx_dequantize(const nf4_mx_matrix *m, int32_t dtype, void *out, int64_t row_stride,
                             void *stream);

/* Workspace bytes of nf4_mx_matmul and of nf4_mx_linear on the current device (-1 for sizes
 * they reject). */
int64_t nf4_mx_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);
int64_t nf4_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* y[M][N] = x w^T (+ bias[N]) of microscaled x [M][K] and w [N][K] of equal cols, summed in
 * fp32 (where the absolute products' sum passes its range the result may be an infinity or NaN)
 * and rounded to out_dtype once; bias is of out_dtype and may be NULL. y's rows are ldy
 * elements apart (at least N; any alignment of the type's own). A NaN block makes its row of
 * x's results, or its column of w's, NaN. workspace: at least
 * nf4_mx_matmul_workspace_bytes(M, N, K), 16-byte aligned (NF4_ERR_SCRATCH where it is smaller);
 * it holds no state between calls, and calls that may run at once need one each. Results depend
 * on the arguments and the device's CU count only, bit for bit. */
nf4_status nf4_mx_matmul(const nf4_mx_matrix *x, const nf4_mx_matrix *w, const void *bias,
                         int32_t out_dtype, void *y, int64_t ldy, void *workspace,
                         int64_t workspace_bytes, void *stream);

/* The same with x [M][K] of x_dtype, rows ldx elements apart, which the call quantizes as
 * nf4_mx_quantize does: bitwise nf4_mx_matmul's result on that. Workspace:
 * nf4_mx_linear_workspace_bytes(M, N, K). (Products of matrices without columns are not
 * supported.) */
nf4_status nf4_mx_linear(const void *x, int32_t x_dtype, int64_t ldx, int64_t M,
                         const nf4_mx_matrix *w, const void *bias, int32_t out_dtype, void *y,
                         int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NF4_MX_H */
