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
 *   rows, cols   rows >= 0 (0: nothing is done), cols >= 1.
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
 * A row that holds a NaN or an infinity gives NaN in that row alone.
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

#ifdef __cplusplus
}
#endif

#endif /* PIPELINED_TRAIN_H */
