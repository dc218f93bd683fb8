// The layer norm calls between their entry points (layer_norm.cu) and the
// kernels for rows a CTA holds in registers.
#pragma once

#include <algorithm>
#include <cstdint>

#include "gemm_internal.h"
#include "row_kernels.cuh"

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

// How a call is spread out.  `elements` 0: the row is too long to be held, and
// the kernels for rows of any length take it.
struct Plan {
    int elements; // per thread
    Source source;
    Shape shape;
    int grid, smem;
};

// Threads of a CTA: what leaves each the registers it needs.  Forward, 16384
// rows of 4096 bfloat16: 55.6 us with 512 threads of 32 elements, 56.0 with
// 640, 63 with 768 (which spill).
constexpr int forward_threads(int elements) { return elements > 16 ? 512 : 768; }
constexpr int kBackwardThreads = 512;

// How the gradient takes unaligned rows.
constexpr Source backward_unaligned(size_t size) { return size == 4 ? kRingElement : kRingShifted; }

struct Device {
    int index, sms;
    unsigned long long ctx;
    unsigned int *status;
};

int launch_forward_rows(const Forward &p, bool bf16, const Plan &plan, const Device &d, cudaStream_t s);
int launch_backward_rows(const Backward &p, bool bf16, const Plan &plan, const Device &d, cudaStream_t s);

} // namespace ln

} // namespace pg
