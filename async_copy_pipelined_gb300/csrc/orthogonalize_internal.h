// What the orthogonalisation's kernels share: how G is read and normalised,
// how values are kept as float16 planes, and the call as its entry point
// (orthogonalize.cu) hands it on.
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>

#include "gemm_internal.h"
#include "pipelined_train.h"
#include "ptx.cuh"
#include "tma_ring.cuh"
#include "vector_io.cuh"

namespace pg {

namespace orth {

// Powers of two the planes are scaled by: the largest magnitudes they must
// hold under float16's 65504 are X 4, A + (b / 2c) I 8, Q 32 (orthogonalize()
// refuses coefficients that reach further), and nothing that matters at the
// other end falls below its 2^-14.
constexpr float kScaleX = 16384.0f, kScaleA = 8192.0f, kScaleQ = 2048.0f;

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_f16(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// A batch of row-major matrices to read.
struct Matrix {
    const void *G;
    int bf16;
    int m, n;
    long long ld, batch_pitch; // elements
    int vec;                   // rows can be read eight elements at a time
};

// Eight consecutive elements j .. j+7 of a row of n, zero past its end.
__device__ __forceinline__ void load8(const Matrix &p, long long row_at, int j, float (&v)[8])
{
    if (p.vec && j + 8 <= p.n) {
        if (p.bf16) {
            Vec16<__nv_bfloat16>::unpack(
                *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.G) + row_at + j), v);
        } else {
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p.G) + row_at + j);
            const uint4 a = q[0], b = q[1];
            Vec16<float>::unpack(a, v);
            Vec16<float>::unpack(b, v + 4);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = j + e < p.n ? load_f32(p.G, p.bf16, row_at + j + e) : 0.0f;
    }
}

// Sums of squares: of the elements, and of 2^-96 and 2^96 times them, for the
// norm of a G whose squares overflow float32 or vanish in it.
constexpr float kDown = 1.26217744835361889e-29f; // 2^-96
constexpr float kUp = 7.92281625142643376e28f;    // 2^96

// 2^k for |k| below 127.
__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((127 + k) << 23); }

struct Squares {
    float plain = 0.0f;
    unsigned long long scaled = 0ull; // down, up

    __device__ __forceinline__ void add(float v)
    {
        plain = fmaf(v, v, plain);
        const unsigned long long d = mul2(pair(v, v), pair(kDown, kUp));
        scaled = fma2(d, d, scaled);
    }
    __device__ __forceinline__ void add(const float4 &v)
    {
        plain += v.x;
        scaled = add2(scaled, pair(v.y, v.z));
    }
    __device__ __forceinline__ void add_up_warp()
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            plain += __shfl_xor_sync(0xffffffffu, plain, o);
            scaled = add2(scaled, __shfl_xor_sync(0xffffffffu, scaled, o));
        }
    }
    __device__ __forceinline__ float4 sums() const
    {
        float down, up;
        split(scaled, down, up);
        return make_float4(plain, down, up, 0.0f);
    }
};

// Below this sum what vanished of the squares can show; their like in 2^96
// times the elements stay below 2^122.
constexpr float kSmallSum = 8.47032947254300339e-22f; // 2^-70

// The planes hold X up to a factor, X = g Y: Y is G times a power of two that
// depends on |G|_F alone, so that its norm is in (1/2, 1] however eps compares
// with |G|_F and float16 keeps its bits; g = 2^-e / (|G|_F + eps), at most 2,
// goes into the products' epilogues in float32.
//
// From the sums: g, and in *e the power of two with kScaleX.  An infinite or
// NaN norm makes g, and so every element that comes of it, NaN.
__device__ __forceinline__ float split_scale(const Squares &squares, float eps, int *e)
{
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
    const float4 s = squares.sums();
    const bool big = !(s.x < inf), small = s.x < kSmallSum;
    const float unit = big ? kDown : small ? kUp : 1.0f; // `norm` is so many times |G|_F
    const float norm = sqrtf(big ? s.y : small ? s.z : s.x);
    *e = 0;
    if (!(norm < inf))
        return nan;
    if (norm == 0.0f)
        return eps > 0.0f ? 1.0f : nan;
    // norm is a normal number between 2^-54 and 2^64: 2^k norm in (1/2, 1].
    const int bits = __float_as_int(norm), k = 127 - (bits >> 23) - ((bits & 0x7fffff) != 0 ? 1 : 0);
    *e = k + (big ? -96 : small ? 96 : 0) + 14; // kScaleX
    // eps unit may be infinite: then g is zero, and |G|_F / eps below 2^-67.
    return power_of_two(-k) / (norm + eps * unit);
}

// What a step's epilogues multiply by: A = X X^T by g g, Q by rho, so that the
// next X is (g / rho) (rho Q) Y and Y becomes rho Q Y.  As soon as g is not
// small Q takes all of it, and from then on X is Y.  Until then X is so small
// that Q is nearly a I, and rho keeps Y from growing.
struct alignas(8) Factors {
    float g, rho;
};
constexpr float kSmallG = 0.0625f;

// How large Q can be while singular values are at most kSmallG, and 1 / that.
struct Slow {
    float most, inverse;
};
inline Slow slow_step(const float *coefficients)
{
    const float most = std::max(1.0f, std::fabs(coefficients[0]) + std::fabs(coefficients[1]) * 0x1p-8f +
                                          std::fabs(coefficients[2]) * 0x1p-16f);
    return Slow{most, 1.0f / most};
}
// This step's factors; g becomes the next step's.
__device__ __forceinline__ Factors step_factors(float &g, const Slow &slow)
{
    const bool small = g < kSmallG;
    const Factors f{g, small ? slow.inverse : g};
    g = small ? g * slow.most : 1.0f;
    return f;
}

constexpr int kMaxSteps = 32;
constexpr int kFactors = kMaxSteps + 1; // per matrix: each step's, and the result's

// `overlap`: the kernel may start while the one before it ends (it calls
// grid_wait()); `cluster`: CTAs per cluster.
template <class Kernel, class... Args>
int launch(Kernel kernel, dim3 grid, int threads, int smem, bool overlap, int cluster, cudaStream_t s,
           const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2] = {};
    unsigned n = 0;
    if (overlap) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

struct Device {
    int index, sms;
    unsigned long long ctx;
};

struct Call {
    int batch, m, n;
    const void *G;
    long long ldg, g_batch;
    int dtype;
    void *out;
    long long ldo, o_batch;
    int out_dtype;
    int steps;
    const float *coefficients;
    float eps;

    Matrix matrix() const
    {
        const long long size = dtype == GEMM_DTYPE_BF16 ? 2 : 4;
        const bool vec = (reinterpret_cast<uintptr_t>(G) & 15u) == 0 && (ldg * size) % 16 == 0 &&
                         (batch == 1 || (g_batch * size) % 16 == 0);
        return Matrix{G, dtype == GEMM_DTYPE_BF16, m, n, ldg, g_batch, vec};
    }
};

// bfloat16 results of matrices whose shorter side is at most 128 and whose
// longer one a cluster of eight CTAs holds (orthogonalize_small.cu).
bool fits_small(int m, int n, int out_dtype);
// Clusters of `ranks` CTAs, each alone on its SM, that run at once; 0 if unknown.
int cluster_room(int ranks, const Device &d);
int run_small(const Call &call, const Device &d, unsigned int *status, cudaStream_t s);

} // namespace orth

} // namespace pg
