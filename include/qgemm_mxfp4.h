/*
 * qgemm_mxfp4.h -- microscaled 4-bit floating point (MXFP4): rows quantised and
 * read back, and the product of two MXFP4 matrices.  Conventions, status codes
 * and dtype codes are those of qgemm.h.
 *
 * Storage of a matrix [rows][k], k % 32 == 0: blocks of 32 consecutive elements of
 * a row share one power-of-two scale.
 *   codes   uint8 [rows][ld], ld >= k / 2: element 2i of a row in the low nibble of
 *           byte i, element 2i + 1 in the high one.  A code is e2m1: bit 3 the
 *           sign, bits 2..0 one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  16-byte aligned,
 *           ld % 16 == 0, ld <= 2^22.
 *   scales  uint8 [rows][ld], ld >= k / 32: byte b of a row stands for 2^(byte - 127)
 *           (0 .. 254); 255 is NaN, and makes its whole block NaN.  ld <= 2^22, any alignment;
 *           rows that start on 16 bytes (4 bytes) are read fastest (faster).
 * An element's value is code * scale.
 */
#ifndef QGEMM_MXFP4_H
#define QGEMM_MXFP4_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mxfp4_quantize -- codes and scales of x [rows][ldx] (dtype QG_BF16, QG_FP16 or
 * QG_FP32).  With a the block's largest magnitude, its scale is 2^e,
 * e = floor(log2 a) - 2 held to -127 .. 127 (-127 when a is 0), so that a / 2^e lies
 * in [4, 8); every element divided by 2^e is rounded to the nearest code value,
 * ties to the even code, magnitudes above 6 to 6.  A block that holds an infinity
 * or a NaN gets the scale 255 and codes of zero.
 *
 * mxfp4_dequantize -- the values, rounded to dtype (nearest even): exact in bf16 and
 * fp32 but for values past their range (6 x 2^127 becomes infinite).
 *
 * rows >= 0, k >= 0, rows * k < 2^35; ldx / ldy >= k, pointers aligned to the
 * element's size (16-byte loads and stores where rows start on 16 bytes).
 * Errors: QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_DTYPE, QG_ERR_HIP.
 */
int32_t mxfp4_quantize(int32_t dtype, int64_t rows, int64_t k, const void* x, int64_t ldx, uint8_t* codes,
                       int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream);
int32_t mxfp4_dequantize(int32_t dtype, int64_t rows, int64_t k, const uint8_t* codes, int64_t ld_codes,
                         const uint8_t* scales, int64_t ld_scales, void* y, int64_t ldy, void* stream);

/*
 * gemm_mxfp4 -- C = A . B^T of two MXFP4 matrices A [M][K] and B [N][K] (a linear
 * layer's activations and weight), the products exact, summed in fp32 and rounded
 * once to dtype (C [M][ldc], ldc >= N, aligned to its element):
 *
 *   C[i][j] = sum_b 2^(sa[i][b] - 127) 2^(sb[j][b] - 127) sum_{t in block b} A[i][t] B[j][t]
 *
 * A block of NaN scale makes its row of C (A's) or column of C (B's) NaN.  Any M
 * and N; K % 32 == 0; K == 0 writes zeros; sizes below 2^31 - 1024.  C must not
 * overlap A or B.
 * Errors: QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_DTYPE, QG_ERR_HIP.
 */
int32_t gemm_mxfp4(int32_t dtype, int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                   const uint8_t* a_scales, int64_t lda_scales, const uint8_t* b, int64_t ldb,
                   const uint8_t* b_scales, int64_t ldb_scales, void* c, int64_t ldc, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_MXFP4_H */
