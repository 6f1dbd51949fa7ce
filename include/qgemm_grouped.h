/*
 * qgemm_grouped.h -- products grouped by expert: the linear layers of a model
 * whose tokens are routed to experts.  Conventions, status codes, dtype and
 * layout codes are those of qgemm.h.
 *
 * The rows of the grouped dimension are sorted by expert ("group"); a device
 * vector of groups + 1 non-decreasing int32 offsets gives group e the rows
 * offsets[e] .. offsets[e + 1] - 1 (none when the two are equal).  The counts
 * stay on the device: the host neither reads them nor waits for them, so a call
 * can be captured in a HIP graph and replayed with other counts.
 *
 *   - Rows before offsets[0] and from offsets[groups] on belong to no group:
 *     they are not read, and their outputs are left as they were.
 *   - Offsets are taken as data: each is held to 0 .. rows, and a group whose end
 *     lies before its start is empty.  If they decrease somewhere, or overlap
 *     in consequence, the rows concerned hold unspecified values; nothing
 *     outside the operands is read or written.
 */
#ifndef QGEMM_GROUPED_H
#define QGEMM_GROUPED_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QG_MAX_GROUPS 4096 /* groups of one call */

/*
 * gemm_grouped -- the three products of a linear layer whose weight depends on
 * the row's group, bf16 / fp16 with fp32 accumulation or fp32 throughout:
 *
 *   QG_NT  forward:          C[r] = A[r] . B_e^T      rows r of group e
 *                            A[M][K], B_e[N][K], C[M][N]
 *   QG_NN  input gradient:   C[r] = A[r] . B_e        rows r of group e
 *                            A[M][K], B_e[K][N], C[M][N]
 *   QG_TN  weight gradient:  C_e = A[rows of e]^T . B[rows of e]
 *                            A[K][M], B[K][N], C_e[M][N]; zeros for an empty group
 *
 * with B_e = B + e * stride_b (NT, NN; 0 gives every group the same matrix) and
 * C_e = C + e * stride_c (TN; stride_c >= (M - 1) * ldc + N).  The grouped rows are
 * the M rows of NT and NN and the K rows of TN.  Results are rounded once from
 * the fp32 sums and do not depend on the other groups' sizes beyond the choice
 * of kernel (the order of summation).
 *
 * Any sizes, leading dimensions (>= the row length) and alignments of the
 * element's size are accepted (sizes below 2^31 - 1024, groups <= QG_MAX_GROUPS,
 * and at most 2^32 threads over all tiles); bf16 / fp16 take 16-byte loads when
 * A and B are 16-byte aligned and their contiguous extents, leading dimensions
 * and stride_b are multiples of 8 elements (leading dimensions up to 2^21, C's too).  M, N or groups of zero enqueue
 * nothing; K of zero (NT, NN) writes zeros to the groups' rows.  C must not
 * overlap A, B or offsets.
 * Errors: QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_DTYPE, QG_ERR_LAYOUT,
 * QG_ERR_HIP.
 */
int32_t gemm_grouped(int32_t layout, int32_t dtype, int64_t groups, const int32_t* offsets, int64_t M, int64_t N,
                     int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b, void* C,
                     int64_t ldc, int64_t stride_c, void* stream);

/*
 * qgemm_int4_grouped -- qgemm_int4 with a weight per expert:
 *
 *   Y[r] = X[r] . dequant(W_e)^T for the rows r of expert e,
 *
 * the storage of qgemm_int4 once per expert, back to back: qweight
 * [experts][k/8][n], scales [experts][k/128][n], qzeros [experts][k/128][n/8] or
 * NULL; x bf16 [m][ldx], y bf16 [m][ldy].  offsets [experts + 1] as above (the
 * grouped rows are the m rows).  Limits, alignments, rounding and errors of x, y
 * and the weights as qgemm_int4; k == 0 writes zeros to the experts' rows.
 *
 *   workspace, workspace_bytes
 *            optional device scratch (16-byte aligned) of
 *            qgemm_int4_grouped_workspace_size bytes, which holds the activations in
 *            the decode's order and their sums during the call (its contents need no
 *            initialisation and are not kept).  With NULL or fewer bytes the
 *            product does both itself, slower.  Calls that share a workspace must
 *            not overlap.
 */
int32_t qgemm_int4_grouped(const void* x, int64_t ldx, const uint32_t* qweight, const uint16_t* scales,
                           const uint32_t* qzeros, int64_t experts, const int32_t* offsets, void* y, int64_t ldy,
                           int64_t m, int64_t n, int64_t k, int32_t group_size, void* workspace,
                           int64_t workspace_bytes, void* stream);

/* Workspace bytes qgemm_int4_grouped can use (0: none); < 0: -error. */
int64_t qgemm_int4_grouped_workspace_size(int64_t experts, int64_t m, int64_t n, int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_GROUPED_H */
