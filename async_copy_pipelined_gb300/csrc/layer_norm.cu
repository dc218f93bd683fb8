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

#include "layer_norm_internal.h"
#include "pipelined_train.h"

namespace pg {

namespace ln {

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

// dweight and dbias from the partial sums: 32 columns by 32 parts of threads,
// blockIdx.y choosing which of the two.  Eight loads of a thread in flight, so
// that the partial sums of 152 CTAs take one latency.
constexpr int kFinishRows = 32;

__global__ void __launch_bounds__(32 * kFinishRows) finish_kernel(const Backward p)
{
    __shared__ float s[kFinishRows][33];
    const int j = blockIdx.x * 32 + threadIdx.x;
    const int which = blockIdx.y;
    void *out = which == 0 ? p.dweight : p.dbias;
    const float *from = p.partial + static_cast<long long>(which) * p.cols + j;
    const long long pitch = 2ll * p.cols;
    grid_wait();
    if (!out)
        return;
    float sum = 0.0f;
    for (int k = threadIdx.y; k < p.parts && j < p.cols; k += 8 * kFinishRows) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = k + u * kFinishRows < p.parts ? from[(k + u * kFinishRows) * pitch] : 0.0f;
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    // A warp a column.
    const float t = warp_sum(s[threadIdx.x][threadIdx.y]);
    const int column = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && column < p.cols)
        store_f32(out, p.weight_bf16, column, t);
}

// A gradient of few rows goes to one CTA, which needs no second kernel to add
// up column sums.  Each turn of the CTA's groups takes it 1.1 us, where all
// turns at once and the second kernel take the device 4 to 6 us whatever their
// number; but the second launch takes the host 3 to 4 us.  So one CTA has as
// many turns as cost the device no more than the launch costs the host.
// bfloat16, microseconds on the device (a call in a loop), one CTA and two
// kernels:
//   turns      2                      4                       8
//   64 columns 4.2 (20.3)  3.9 (24.5) 8.1 (20.0)  4.1 (23.4) 12.5 (20.0) 4.2 (23.2)
//   1024       5.7 (19.5)  5.0 (23.2) 8.9 (19.9)  5.1 (23.9) 13.2 (20.1) 5.4 (22.7)
//   2048       6.5 (20.6)  5.0 (23.2) 9.8 (20.3)  5.0 (23.3) 14.0 (20.6) 5.2 (24.0)
//   4096       8.3 (19.5)  5.7 (23.4) 12.0 (20.3) 5.9 (23.4) 16.9 (20.0) 6.1 (23.2)
// Of longer rows only one by itself (a second kernel would add up nothing).
bool one_cta(int rows, int cols)
{
    const int at_once = kBackwardThreads / ((cols + 16 * 32 - 1) / (16 * 32) * 32);
    return rows <= (cols <= 1024 ? 4 : 2) * at_once;
}

// Most partial sums of a column that any variant makes.
int backward_parts(int rows, int sms)
{
    const int most = 2 * sms;
    return rows < most ? (rows < 1 ? 1 : rows) : most;
}

// Elements per thread `e`, rows at a time, and where they come from.  The
// ring pays once a group has several rows to run ahead over; below that the
// threads load their own.  `ctas`: how many share the rows.  `full`: there is
// a variant for rows without a rest.  `ragged`: how the ring takes unaligned
// rows.
Plan spread(long long rows, int cols, int e, int max_threads, int streams, int parameters, bool vectors, bool full,
            Source ragged, size_t size, const Device &d, int ctas)
{
    Plan plan = {};
    const int tpr = (cols + e * 32 - 1) / (e * 32) * 32;
    if (tpr > max_threads)
        return plan;
    plan.elements = e;
    const int groups = std::max(1, static_cast<int>(std::min<long long>(max_threads / tpr, (rows + ctas - 1) / ctas)));
    const long long trips = (rows + groups - 1) / groups;
    const int row_bytes = cols * static_cast<int>(size);
    // An unaligned row's last piece is read with the granule after it.
    const int slot_bytes = vectors ? row_bytes : (row_bytes + 15 + 15) / 16 * 16 + 16;
    const int fixed = parameters * parameter_floats(cols) * 4;
    const int layer = groups * streams * slot_bytes; // one slot of every group
    const int slots = std::min({kMaxSlots, std::max(2, kRingBytes / layer), (kSmemBytes - fixed) / layer});
    const bool ring = trips > 2 * ctas && slots >= 2;
    plan.source = !ring ? (vectors ? kVector : kScalar)
                  : !vectors ? ragged
                  : cols == tpr * e && full ? kRingFull : kRingVector;
    plan.shape = Shape{tpr, groups, slots, slot_bytes, d.status, call_wait_limit_ns(), call_withhold()};
    plan.grid = static_cast<int>(std::min<long long>(trips, ctas));
    plan.smem = ring ? fixed + slots * groups * streams * slot_bytes : 0;
    return plan;
}

bool vector_rows(const void *p, long long ld, int rows, size_t size)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (ld * static_cast<long long>(size)) % 16 == 0);
}

bool vector_parameter(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class T>
int launch_forward(const Forward &p, const Device &d, cudaStream_t s)
{
    constexpr bool kBf16 = sizeof(T) == 2;
    const bool vectors = p.cols % Vec16<T>::kElements == 0 && vector_rows(p.x, p.ldx, p.rows, sizeof(T)) &&
                         vector_rows(p.y, p.ldy, p.rows, sizeof(T)) && vector_parameter(p.weight) &&
                         vector_parameter(p.bias);
    // 16 elements a thread give a single row the most threads; 32 give many
    // rows the most groups, whose reductions overlap.
    const int e = p.cols <= 512 || (p.rows <= 2 * d.sms && p.cols <= 8192) ? 16 : 32;
    Plan plan = spread(p.rows, p.cols, e, forward_threads(e), 1, 2, vectors, true, kRingShifted, sizeof(T), d, d.sms);
    if (plan.source == kScalar && e == 32 && p.cols <= 8192)
        plan = spread(p.rows, p.cols, 16, forward_threads(16), 1, 2, vectors, true, kRingShifted, sizeof(T), d, d.sms);
    if (plan.elements != 0) {
        if (!from_ring(plan.source)) // no ring to keep the memory system busy: every CTA that fits
            plan.grid = std::min((p.rows + plan.shape.groups - 1) / plan.shape.groups, 4 * d.sms);
        return launch_forward_rows(p, kBf16, plan, d, s);
    }
    const int grid = p.rows < 65536 ? p.rows : 65536;
    forward_any_kernel<T><<<grid, kAnyThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

int launch_finish(const Backward &p, bool overlap, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.cols + 31) / 32), 2);
    cfg.blockDim = dim3(32, kFinishRows);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, finish_kernel, p) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <class T>
int launch_backward(Backward p, const Device &d, cudaStream_t s)
{
    constexpr bool kBf16 = sizeof(T) == 2;
    const bool columns = p.dweight || p.dbias;
    const bool vectors = p.cols % Vec16<T>::kElements == 0 && vector_rows(p.x, p.ldx, p.rows, sizeof(T)) &&
                         vector_rows(p.dy, p.lddy, p.rows, sizeof(T)) && vector_rows(p.dx, p.lddx, p.rows, sizeof(T)) &&
                         vector_parameter(p.weight);
    // 16 elements leave room for the two column sums of each in registers.
    const int e = p.cols <= 8192 ? 16 : 32;
    const int ctas = one_cta(p.rows, p.cols) ? 1 : d.sms;
    Plan plan = spread(p.rows, p.cols, e, kBackwardThreads, 2, 1, vectors, e == 16, backward_unaligned(sizeof(T)),
                       sizeof(T), d, ctas);
    if (plan.elements != 0 && p.rows > 0) {
        p.parts = plan.grid;
        const int st = launch_backward_rows(p, kBf16, plan, d, s);
        return st != GEMM_OK || !columns || p.parts == 1 ? st : launch_finish(p, true, s);
    }
    if (columns) {
        const unsigned column_blocks = static_cast<unsigned>((p.cols + 31) / 32);
        columns_kernel<T><<<dim3(column_blocks, p.parts), dim3(32, kColumnRows), 0, s>>>(p);
        const int st = launch_finish(p, false, s);
        if (st != GEMM_OK)
            return st;
    }
    const int grid = p.rows < 65536 ? p.rows : 65536;
    if (grid > 0)
        backward_any_kernel<T><<<grid, kAnyThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// The current device, and what its kernels need to know.
int enter(Device *d)
{
    const int st = device_checked(&d->index);
    if (st != GEMM_OK)
        return st;
    d->sms = device_sms();
    d->ctx = current_context_id();
    d->status = device_status_word(d->index, d->ctx);
    return d->status ? GEMM_OK : GEMM_ERR_CUDA;
}

constexpr int kMaxCols = 1 << 28; // a row's bytes and columns are counted in an int

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
    if (cols > ln::kMaxCols)
        return GEMM_ERR_UNSUPPORTED;
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
    ln::Device d;
    const int st = ln::enter(&d);
    if (st != GEMM_OK)
        return st;
    if (rows == 0)
        return GEMM_OK;
    const ln::Forward p{rows, cols, x, ldx, weight, bias, weight_dtype == GEMM_DTYPE_BF16, y, ldy, mean, rstd, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == GEMM_DTYPE_F32 ? ln::launch_forward<float>(p, d, s) : ln::launch_forward<__nv_bfloat16>(p, d, s);
}

int layer_norm_backward_workspace(int rows, int cols, size_t *bytes)
{
    if (rows < 0 || cols < 1 || !bytes)
        return GEMM_ERR_INVALID_ARG;
    if (cols > ln::kMaxCols)
        return GEMM_ERR_UNSUPPORTED;
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
    if (cols > ln::kMaxCols)
        return GEMM_ERR_UNSUPPORTED;
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
    ln::Device d;
    const int st = ln::enter(&d);
    if (st != GEMM_OK)
        return st;
    const ln::Backward p{rows, cols, dy, x, lddy, ldx, mean, rstd, weight, weight_dtype == GEMM_DTYPE_BF16, dx, lddx,
                   dweight, dbias, static_cast<float *>(workspace), ln::backward_parts(rows, d.sms)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == GEMM_DTYPE_F32 ? ln::launch_backward<float>(p, d, s) : ln::launch_backward<__nv_bfloat16>(p, d, s);
}

} // extern "C"
