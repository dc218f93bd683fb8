// Layer norm over rows, and its gradient.
//
//   y    = (x - mean) rstd weight + bias
//   dx   = rstd (t - mean_k(t) - xhat mean_k(t xhat)),  t = dy weight
//   dw_j = sum_i dy_ij xhat_ij,  db_j = sum_i dy_ij
//
// A few operations per element: the bytes of x and y (dy, x and dx) bound
// every size that fills the GPU, and the launch bounds a row or two.
#include <cmath>
#include <cstdint>

#include "gemm_internal.h"
#include "pipelined_train.h"
#include "vector_io.cuh"

namespace pg {

namespace ln {

struct Forward {
    int rows, cols;
    const void *x;
    long long ldx;
    const void *weight, *bias; // either may be null
    int weight_bf16;
    void *y;
    long long ldy;
    float *mean, *rstd; // both or neither
    float eps;
};

struct Backward {
    int rows, cols;
    const void *dy, *x;
    long long lddy, ldx;
    const float *mean, *rstd;
    const void *weight; // may be null
    int weight_bf16;
    void *dx;
    long long lddx;
    void *dweight, *dbias; // either may be null
    float *partial;        // [parts][2][cols]: dweight's and dbias's partial sums
    int parts;
};

// Sum over the CTA, the same value in every thread.  `scratch` holds 32
// floats; the caller's next use of it comes after another barrier.
__device__ __forceinline__ float cta_sum(float v, float *scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x / 32;
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w)
        s += scratch[w];
    __syncthreads();
    return s;
}

// ------------------------------------------------------------ rows of any length
// One CTA per row at a time, three passes over the row (mean, squared
// differences, output): the second and third find it in the caches.
constexpr int kAnyThreads = 512;

template <class T>
__global__ void __launch_bounds__(kAnyThreads) forward_any_kernel(const Forward p)
{
    __shared__ float scratch[32];
    const float n = static_cast<float>(p.cols);
    for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        T *y = static_cast<T *>(p.y) + row * p.ldy;
        float s = 0.0f;
        for (int j = threadIdx.x; j < p.cols; j += kAnyThreads)
            s += to_f32(x[j]);
        const float mean = cta_sum(s, scratch) / n;
        float q = 0.0f;
        for (int j = threadIdx.x; j < p.cols; j += kAnyThreads) {
            const float d = to_f32(x[j]) - mean;
            q = fmaf(d, d, q);
        }
        const float rstd = 1.0f / sqrtf(cta_sum(q, scratch) / n + p.eps);
        for (int j = threadIdx.x; j < p.cols; j += kAnyThreads) {
            const float w = p.weight ? load_f32(p.weight, p.weight_bf16, j) : 1.0f;
            const float b = p.bias ? load_f32(p.bias, p.weight_bf16, j) : 0.0f;
            y[j] = from_f32<T>(fmaf((to_f32(x[j]) - mean) * rstd, w, b));
        }
        if (p.mean && threadIdx.x == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kAnyThreads) backward_any_kernel(const Backward p)
{
    __shared__ float scratch[32];
    const float n = static_cast<float>(p.cols);
    for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int j = threadIdx.x; j < p.cols; j += kAnyThreads) {
            const float w = p.weight ? load_f32(p.weight, p.weight_bf16, j) : 1.0f;
            const float t = to_f32(dy[j]) * w;
            s1 += t;
            s2 = fmaf(t, (to_f32(x[j]) - mean) * rstd, s2);
        }
        const float c1 = cta_sum(s1, scratch) / n;
        const float c2 = cta_sum(s2, scratch) / n;
        for (int j = threadIdx.x; j < p.cols; j += kAnyThreads) {
            const float w = p.weight ? load_f32(p.weight, p.weight_bf16, j) : 1.0f;
            const float xhat = (to_f32(x[j]) - mean) * rstd;
            dx[j] = from_f32<T>(rstd * (to_f32(dy[j]) * w - c1 - xhat * c2));
        }
    }
}

// Partial column sums over one run of rows per blockIdx.y: 32 columns by 8
// rows of threads.  Runs before dx is written, which may be dy or x.
constexpr int kColumnRows = 8;

template <class T>
__global__ void __launch_bounds__(32 * kColumnRows) columns_kernel(const Backward p)
{
    __shared__ float sw[kColumnRows][32], sb[kColumnRows][32];
    const int j = blockIdx.x * 32 + threadIdx.x;
    const int per = (p.rows + p.parts - 1) / p.parts;
    const int r0 = blockIdx.y * per, r1 = min(p.rows, r0 + per);
    float dw = 0.0f, db = 0.0f;
    if (j < p.cols) {
        for (int row = r0 + threadIdx.y; row < r1; row += kColumnRows) {
            const float g = to_f32(static_cast<const T *>(p.dy)[row * p.lddy + j]);
            const float xhat = (to_f32(static_cast<const T *>(p.x)[row * p.ldx + j]) - p.mean[row]) * p.rstd[row];
            dw = fmaf(g, xhat, dw);
            db += g;
        }
    }
    sw[threadIdx.y][threadIdx.x] = dw;
    sb[threadIdx.y][threadIdx.x] = db;
    __syncthreads();
    if (threadIdx.y == 0 && j < p.cols) {
        for (int k = 1; k < kColumnRows; ++k) {
            dw += sw[k][threadIdx.x];
            db += sb[k][threadIdx.x];
        }
        float *out = p.partial + static_cast<long long>(blockIdx.y) * 2 * p.cols;
        out[j] = dw;
        out[p.cols + j] = db;
    }
}

// dweight and dbias from the partial sums, in part order: 32 columns by 8
// parts of threads, blockIdx.y choosing which of the two.
__global__ void __launch_bounds__(256) finish_kernel(const Backward p)
{
    __shared__ float s[8][32];
    const int j = blockIdx.x * 32 + threadIdx.x;
    const int which = blockIdx.y;
    void *out = which == 0 ? p.dweight : p.dbias;
    if (!out)
        return;
    float v = 0.0f;
    if (j < p.cols)
        for (int k = threadIdx.y; k < p.parts; k += 8)
            v += p.partial[(static_cast<long long>(k) * 2 + which) * p.cols + j];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && j < p.cols) {
        for (int k = 1; k < 8; ++k)
            v += s[k][threadIdx.x];
        store_f32(out, p.weight_bf16, j, v);
    }
}

// Runs of rows the column sums are cut into.
int backward_parts(int rows, int sms)
{
    const int most = 2 * sms;
    return rows < most ? (rows < 1 ? 1 : rows) : most;
}

template <class T>
int launch_forward(const Forward &p, cudaStream_t s)
{
    const int grid = p.rows < 65536 ? p.rows : 65536;
    forward_any_kernel<T><<<grid, kAnyThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <class T>
int launch_backward(const Backward &p, cudaStream_t s)
{
    const unsigned column_blocks = static_cast<unsigned>((p.cols + 31) / 32);
    if (p.dweight || p.dbias) {
        columns_kernel<T><<<dim3(column_blocks, p.parts), dim3(32, kColumnRows), 0, s>>>(p);
        finish_kernel<<<dim3(column_blocks, 2), dim3(32, 8), 0, s>>>(p);
    }
    const int grid = p.rows < 65536 ? p.rows : 65536;
    if (grid > 0)
        backward_any_kernel<T><<<grid, kAnyThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

bool valid_dtype(int d) { return d == GEMM_DTYPE_F32 || d == GEMM_DTYPE_BF16; }

bool aligned_to(const void *p, int dtype)
{
    return (reinterpret_cast<uintptr_t>(p) & (dtype == GEMM_DTYPE_F32 ? 3u : 1u)) == 0;
}

} // namespace ln

} // namespace pg

using namespace pg;

extern "C" {

int layer_norm(int rows, int cols, const void *x, long long ldx, int dtype, const void *weight, const void *bias,
               int weight_dtype, void *y, long long ldy, float *mean, float *rstd, float eps, void *stream)
{
    if (rows < 0 || cols < 1 || !ln::valid_dtype(dtype) || !ln::valid_dtype(weight_dtype))
        return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || (mean == nullptr) != (rstd == nullptr))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 1 && (ldx < cols || ldy < cols))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y))
        return GEMM_ERR_INVALID_ARG;
    if (!ln::aligned_to(x, dtype) || !ln::aligned_to(y, dtype) || !ln::aligned_to(weight, weight_dtype) ||
        !ln::aligned_to(bias, weight_dtype) || !ln::aligned_to(mean, GEMM_DTYPE_F32) ||
        !ln::aligned_to(rstd, GEMM_DTYPE_F32))
        return GEMM_ERR_MISALIGNED;
    int dev;
    const int st = device_checked(&dev);
    if (st != GEMM_OK)
        return st;
    if (rows == 0)
        return GEMM_OK;
    const ln::Forward p{rows, cols, x, ldx, weight, bias, weight_dtype == GEMM_DTYPE_BF16, y, ldy, mean, rstd, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == GEMM_DTYPE_F32 ? ln::launch_forward<float>(p, s) : ln::launch_forward<__nv_bfloat16>(p, s);
}

int layer_norm_backward_workspace(int rows, int cols, size_t *bytes)
{
    if (rows < 0 || cols < 1 || !bytes)
        return GEMM_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(ln::backward_parts(rows, device_sms())) * 2u * static_cast<size_t>(cols) * 4u;
    return GEMM_OK;
}

int layer_norm_backward(int rows, int cols, const void *dy, long long lddy, const void *x, long long ldx, int dtype,
                        const float *mean, const float *rstd, const void *weight, int weight_dtype, void *dx,
                        long long lddx, void *dweight, void *dbias, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    if (rows < 0 || cols < 1 || !ln::valid_dtype(dtype) || !ln::valid_dtype(weight_dtype))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 1 && (ldx < cols || lddy < cols || lddx < cols))
        return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !dx || !mean || !rstd))
        return GEMM_ERR_INVALID_ARG;
    if (!ln::aligned_to(dy, dtype) || !ln::aligned_to(x, dtype) || !ln::aligned_to(dx, dtype) ||
        !ln::aligned_to(weight, weight_dtype) || !ln::aligned_to(dweight, weight_dtype) ||
        !ln::aligned_to(dbias, weight_dtype) || !ln::aligned_to(mean, GEMM_DTYPE_F32) ||
        !ln::aligned_to(rstd, GEMM_DTYPE_F32) || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return GEMM_ERR_MISALIGNED;
    const bool columns = dweight || dbias;
    size_t need = 0;
    (void)layer_norm_backward_workspace(rows, cols, &need);
    if (columns && (!workspace || workspace_bytes < need))
        return GEMM_ERR_INVALID_ARG;
    int dev;
    const int st = device_checked(&dev);
    if (st != GEMM_OK)
        return st;
    ln::Backward p{rows, cols, dy, x, lddy, ldx, mean, rstd, weight, weight_dtype == GEMM_DTYPE_BF16, dx, lddx,
                   dweight, dbias, static_cast<float *>(workspace), ln::backward_parts(rows, device_sms())};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == GEMM_DTYPE_F32 ? ln::launch_backward<float>(p, s) : ln::launch_backward<__nv_bfloat16>(p, s);
}

} // extern "C"
