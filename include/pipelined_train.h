/*
 * pipelined_train.h -- operators around a projection that is being trained,
 * beside the GEMM of pipelined_gemm.h and in its library: layer norm, its
 * gradient, and the Newton-Schulz orthogonalisation of a weight's update.
 *
 * The conventions are those of pipelined_gemm.h: row-major matrices with
 * leading dimensions in elements; device pointers owned by the caller, of
 * which the library keeps none after the call; no memory allocated by the
 * library; work enqueued on `stream` (a cudaStream_t, NULL: the legacy
 * default stream) without synchronising; a gemm_status returned, with nothing
 * enqueued unless it is GEMM_OK.  Bounded waits that expire are recorded in
 * the status word gemm_device_status() reads.
 */
#ifndef PIPELINED_TRAIN_H
#define PIPELINED_TRAIN_H

#include <stddef.h>

#include "pipelined_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators below. */
enum gemm_dtype {
    GEMM_DTYPE_F32 = 0,
    GEMM_DTYPE_BF16 = 1
};

/*
 * layer_norm: for each row i of x,
 *
 *   mean_i = (1/cols) sum_j x_ij
 *   rstd_i = 1 / sqrt((1/cols) sum_j (x_ij - mean_i)^2 + eps)
 *   y_ij   = (x_ij - mean_i) * rstd_i * weight_j + bias_j
 *
 * computed in float32 and rounded once to y's type.  The variance is taken
 * from differences to a mean, never as a difference of two large sums.
 *
 *   rows, cols   rows >= 0 (0: nothing is done), cols 1 .. 2^28 (beyond:
 *                GEMM_ERR_UNSUPPORTED).
 *   x, ldx       rows x cols of `dtype`, ldx >= cols (any ldx when rows is 0
 *                or 1).  A pitch of any alignment works; rows whose base and
 *                pitch are 16-byte aligned move in 16-byte pieces.
 *   dtype        GEMM_DTYPE_F32 or GEMM_DTYPE_BF16, of x and y.
 *   weight, bias cols elements of `weight_dtype` each; either may be NULL
 *                (1 and 0).
 *   y, ldy       output of `dtype`; may be x itself (same pointer and pitch),
 *                otherwise shares no byte with x.
 *   mean, rstd   rows floats each, or both NULL when no gradient is wanted.
 *   eps          >= 0 and finite.
 *
 * A row that holds a NaN or an infinity gives NaN in that row alone.  Squared
 * differences are float32: where they overflow (differences of about 1e19 and
 * more) rstd is 0 and y the bias.
 */
int layer_norm(int rows, int cols,
               const void *x, long long ldx, int dtype,
               const void *weight, const void *bias, int weight_dtype,
               void *y, long long ldy,
               float *mean, float *rstd, float eps,
               void *stream);

/*
 * layer_norm_backward: with xhat_ij = (x_ij - mean_i) * rstd_i and
 * t_ij = dy_ij * weight_j,
 *
 *   dx_ij     = rstd_i * (t_ij - (1/cols) sum_k t_ik
 *                              - xhat_ij * (1/cols) sum_k t_ik xhat_ik)
 *   dweight_j = sum_i dy_ij xhat_ij
 *   dbias_j   = sum_i dy_ij
 *
 * Sums are float32, in an order fixed by the sizes (the same inputs give the
 * same bits), each result rounded once to its type.
 *
 *   dy, x, dx    rows x cols of `dtype`, pitches >= cols.  dx may be dy or x
 *                itself (same pointer and pitch), otherwise shares no byte
 *                with either.
 *   mean, rstd   what layer_norm returned for x.
 *   weight       cols elements of `weight_dtype`, or NULL (1).
 *   dweight,     cols elements of `weight_dtype` each; either may be NULL
 *   dbias        when it is not wanted.  With rows 0 they are set to zero.
 *   workspace    device memory of at least layer_norm_backward_workspace()
 *                bytes, 16-byte aligned; needs no initialisation, holds
 *                nothing between calls, serves one call at a time.  May be
 *                NULL when neither dweight nor dbias is wanted.
 */
int layer_norm_backward(int rows, int cols,
                        const void *dy, long long lddy,
                        const void *x, long long ldx, int dtype,
                        const float *mean, const float *rstd,
                        const void *weight, int weight_dtype,
                        void *dx, long long lddx,
                        void *dweight, void *dbias,
                        void *workspace, size_t workspace_bytes,
                        void *stream);

/* Bytes layer_norm_backward needs for these sizes on the current device
 * (a 152-SM part where no device can be asked). */
int layer_norm_backward_workspace(int rows, int cols, size_t *bytes);

/*
 * orthogonalize: the orthogonalised form of a weight's update, by
 * Newton-Schulz products.  For each m x n matrix G of a batch, with X seen
 * on its shorter side (X^T is iterated where m > n, which gives the same):
 *
 *   X <- G / (|G|_F + eps)
 *   steps times:  A = X X^T;   X <- a X + (b A + c A A) X
 *   out = X
 *
 * With (a, b, c) = (3.4445, -4.7750, 2.0315) five steps take every singular
 * value that is not tiny beside |G|_F to somewhere in 0.68 .. 1.2 and keep the
 * singular vectors.
 *
 *   batch, m, n   matrices and their sizes, each >= 0 (any of them 0: nothing
 *                 is done); sides to 2^20, m n below 2^31, batch to 65535.
 *   G             matrix b, element (i, j) at G[b*g_batch + i*ldg + j], of
 *                 `dtype`; ldg >= n, any alignment.
 *   out           likewise with ldo, o_batch, of `out_dtype`, its matrices one
 *                 after the other or row by row in turn; may be G itself
 *                 (pointer, pitches and type), otherwise shares no byte with
 *                 it.  The products run in the precision this type
 *                 asks for, on float16 planes with float32 sums: what they
 *                 add to bfloat16's rounding stays below it for
 *                 GEMM_DTYPE_BF16, and is that of float32 arithmetic for
 *                 GEMM_DTYPE_F32 (at about four times the time).
 *   steps         1 .. 32.
 *   coefficients  3 * steps floats in host memory: a, b, c of each step.
 *                 c = 0 or |b| <= 8 |c|, and from singular values x in
 *                 [0, 1] no step may leave [-2.8, 2.8], or pass 15.5 in
 *                 a + b x^2 + c x^4 or 7.98 in x^2 + b / 2c; else
 *                 GEMM_ERR_UNSUPPORTED.
 *   eps           >= 0, finite.  A zero G gives zeros (NaN with eps 0).
 *   workspace     device memory of at least orthogonalize_workspace() bytes,
 *                 256-byte aligned; needs no initialisation, holds nothing
 *                 between calls, serves one call at a time.
 *
 * A matrix that holds a NaN or an infinity comes out as NaN throughout; the
 * others of the batch are not touched by it.
 */
int orthogonalize(int batch, int m, int n,
                  const void *G, long long ldg, long long g_batch, int dtype,
                  void *out, long long ldo, long long o_batch, int out_dtype,
                  int steps, const float *coefficients, float eps,
                  void *workspace, size_t workspace_bytes,
                  void *stream);

/* Bytes orthogonalize needs for these sizes on the current device (a 152-SM
 * part where no device can be asked).  None for a bfloat16 result of small
 * matrices (a side of at most 128 and the other at most 2048), which stay on
 * chip; workspace may then be NULL. */
int orthogonalize_workspace(int batch, int m, int n, int out_dtype, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* PIPELINED_TRAIN_H */
