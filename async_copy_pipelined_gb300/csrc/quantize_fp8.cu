// Quantisation to 8-bit floating point numbers with one scale for 128 elements
// of a row, 128 of a column, or a block of 128 x 128.
//
//   scale = max(max |x| / MAX, 2^-126),  q = nearest(x / scale)
//
// One pass: a group stays in registers between its maximum and its quotients,
// so the bytes of x and q bound it.  A quotient is bracketed by x * (1 / scale)
// times 1 -+ 2^-21, two products in float32 whose own errors are at most half
// of that; where both ends convert to the same value, so does the exact quotient.
// Elsewhere (2^-16 of the elements of a continuous distribution, one in 300 of
// bfloat16 numbers, which meet borders exactly) the sign of x - scale * (the
// middle of the two values) decides, which one FMA gives exactly, so that the
// result is the definition's everywhere.
//
// 8192 x 8192 bfloat16 by rows 46 us on the device (4.4 TB/s; 49 a call among others),
// by columns 60 (61.5), in blocks 50: three of four issue slots are busy, two thirds of
// them on the integer pipe, which also converts.  float32 by rows runs at 5.4 TB/s.
#include <algorithm>
#include <cstdint>
#include <cuda_fp16.h>

#include "gemm_internal.h"
#include "pipelined_ffn.h"
#include "vector_io.cuh"

namespace pg {
namespace quantize {

constexpr int kGroup = 128;

struct Call {
    int rows, cols;
    const void *x;
    long long ldx;
    uint8_t *q;
    long long ldq;
    float *scale;
    long long lds;
    bool x_vectors; // 16-byte loads of x
    int q_vectors;  // bytes that q's rows are aligned to: 16, 8 or fewer (0)
};

template <int Format>
struct Fp8;
template <>
struct Fp8<GEMM_FP8_E4M3> {
    static constexpr float kMost = 448.0f;
    // The values nearest to lo and hi, in the lower and upper byte.
    static __device__ __forceinline__ uint32_t convert(float lo, float hi)
    {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
        return r;
    }
    // What the two low bytes stand for.
    static __device__ __forceinline__ __half2 values(uint32_t bytes)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(bytes)));
        return *reinterpret_cast<const __half2 *>(&r);
    }
};
template <>
struct Fp8<GEMM_FP8_E5M2> {
    static constexpr float kMost = 57344.0f;
    static __device__ __forceinline__ uint32_t convert(float lo, float hi)
    {
        uint16_t r;
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
        return r;
    }
    // What the two low bytes stand for.
    static __device__ __forceinline__ __half2 values(uint32_t bytes)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(bytes)));
        return *reinterpret_cast<const __half2 *>(&r);
    }
};

// Of the largest magnitude's bits.
template <int Format>
__device__ __forceinline__ float scale_of(uint32_t largest)
{
    const float s = __uint_as_float(largest) / Fp8<Format>::kMost;
    return s < 0x1p-126f ? 0x1p-126f : s; // a NaN stays
}

// Ends of the bracket around 1 / s.
struct Inverse {
    float low, high;
};

__device__ __forceinline__ Inverse inverse_of(float s)
{
    float r; // off by at most one unit in its last place
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return Inverse{r * (1.0f - 0x1p-21f), r * (1.0f + 0x1p-21f)};
}

// Four elements whose bracket's ends convert to the bytes of `low`, the smaller
// in magnitude, and `high`: equal, or neighbouring values, whose codes differ by
// one.  |x| - s * (the middle of the two values), which one FMA rounds without
// losing its sign, says which is nearer; none to the even code.
template <int Format>
__device__ __forceinline__ uint32_t settle4(const float (&v)[4], const float (&s)[4], uint32_t low, uint32_t high)
{
    using F = Fp8<Format>;
    const __half2 half = __float2half2_rn(0.5f);
    uint32_t up = 0;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        // Of magnitudes; halves of the formats' values and their sums are exact.
        const uint32_t a = low >> (8 * e) & 0x7F7Fu, b = high >> (8 * e) & 0x7F7Fu;
        const float2 middle = __half22float2(__hfma2(F::values(a), half, __hmul2(F::values(b), half)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x = fabsf(v[e + i]), scale = s[e + i];
            if (scale < 0x1p-40f) { // together, so that no difference vanishes
                x *= 0x1p64f;
                scale *= 0x1p64f;
            }
            const int beyond = __float_as_int(fmaf(i == 0 ? -middle.x : -middle.y, scale, x));
            const int odd = static_cast<int>(low >> (8 * (e + i)) & 1u);
            up |= beyond + odd > 0 ? 1u << (8 * (e + i)) : 0u;
        }
    }
    return low + (up & (high - low));
}

// Eight elements, of which the pair k is v[k]; low(k) and high(k) are the pair's
// brackets, and scale(e) is element e's.
template <int Format, class Low, class High, class Scale>
__device__ __forceinline__ uint2 quantize8(const unsigned long long (&v)[4], Low low, High high, Scale scale)
{
    using F = Fp8<Format>;
    auto convert = [&](int k, unsigned long long r) {
        float a, b;
        split(mul2(v[k], r), a, b);
        return F::convert(a, b);
    };
    uint32_t q[2], other[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        q[h] = convert(2 * h, low(2 * h)) | convert(2 * h + 1, low(2 * h + 1)) << 16;
        other[h] = convert(2 * h, high(2 * h)) | convert(2 * h + 1, high(2 * h + 1)) << 16;
    }
    // Four at a time, most often in one pass whichever four a lane has to settle.
    while (q[0] != other[0] || q[1] != other[1]) {
        const bool second = q[0] == other[0];
        float x[4], s[4];
        split(second ? v[2] : v[0], x[0], x[1]);
        split(second ? v[3] : v[1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[e] = scale(second ? 4 + e : e);
        const uint32_t settled = settle4<Format>(x, s, second ? q[1] : q[0], second ? other[1] : other[0]);
        if (second)
            q[1] = other[1] = settled;
        else
            q[0] = other[0] = settled;
    }
    return make_uint2(q[0], q[1]);
}

// Eight consecutive elements of a row as they lie in memory, zero from the
// matrix's end on.
template <class T>
struct Raw8 {
    static constexpr int kPieces = 8 / Vec16<T>::kElements;
    uint4 piece[kPieces];

    __device__ __forceinline__ void load(const Call &p, long long row, int col)
    {
        const T *from = static_cast<const T *>(p.x) + row * p.ldx + col;
        if (p.x_vectors && col + 8 <= p.cols) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                piece[k] = __ldcs(reinterpret_cast<const uint4 *>(from) + k);
        } else {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = col + e < p.cols ? to_f32(from[e]) : 0.0f;
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                piece[k] = Vec16<T>::pack(v + k * Vec16<T>::kElements);
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            piece[k] = make_uint4(0, 0, 0, 0);
    }
    // As pairs.
    __device__ __forceinline__ void unpack(unsigned long long (&v)[4]) const
    {
        float one[8];
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            Vec16<T>::unpack(piece[k], one + k * Vec16<T>::kElements);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = pair(one[2 * k], one[2 * k + 1]);
    }
    __device__ __forceinline__ uint32_t word(int i) const
    {
        const uint4 &q = piece[i / 4];
        return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
    }
};

// Magnitudes of elements as they lie in memory, as whole numbers that order them,
// with infinity and every NaN on top: two bfloat16 ones in a word, or one float32.
template <class T>
struct Magnitude;
template <>
struct Magnitude<float> {
    static constexpr int kWords = 8; // of eight elements
    static __device__ __forceinline__ uint32_t of(uint32_t word) { return word & 0x7FFFFFFFu; }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
    // The largest of a word as a float32's bits, and element i's of one.
    static __device__ __forceinline__ uint32_t largest(uint32_t m) { return m; }
    static __device__ __forceinline__ uint32_t element(uint32_t m, int) { return m; }
};
template <>
struct Magnitude<__nv_bfloat16> {
    static constexpr int kWords = 4;
    static __device__ __forceinline__ uint32_t of(uint32_t word) { return word & 0x7FFF7FFFu; }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
    static __device__ __forceinline__ uint32_t largest(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t element(uint32_t m, int i) { return i == 0 ? m << 16 : m & 0xFFFF0000u; }
};

__device__ __forceinline__ void store8(const Call &p, long long row, int col, uint2 v)
{
    uint8_t *to = p.q + row * p.ldq + col;
    if (p.q_vectors && col + 8 <= p.cols) {
        *reinterpret_cast<uint2 *>(to) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < p.cols)
                to[e] = static_cast<uint8_t>((e < 4 ? v.x : v.y) >> (8 * (e & 3)));
    }
}

// ------------------------------------------------------------- row groups
// A lane has kPieces times eight consecutive elements (32 bytes) of a group, so
// that eight lanes share one of bfloat16 numbers and sixteen one of float32; a
// warp's lanes are side by side in a row, kAhead such runs loaded before the first
// maximum.  With sixteen lanes to a group of bfloat16 numbers its reduction and
// scale cost as much as its elements (8192 x 8192: 57 us).
constexpr int kRowThreads = 256;

template <class T, int Format>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const Call p)
{
    using M = Magnitude<T>;
    constexpr int kPieces = 4 / sizeof(T), kAhead = 4 / kPieces;
    constexpr int kRun = 32 * 8 * kPieces, kLanes = kGroup / (8 * kPieces);
    const int runs = (p.cols + kRun - 1) / kRun;
    const long long total = static_cast<long long>(p.rows) * runs;
    const int lane = threadIdx.x & 31;
    const int warps = static_cast<int>(gridDim.x) * (kRowThreads / 32);
    const int start = static_cast<int>(blockIdx.x) * (kRowThreads / 32) + static_cast<int>(threadIdx.x) / 32;
    // A warp's runs lie `warps` apart.
    const int step_rows = warps / runs, step_runs = warps - step_rows * runs;
    int next_row = start / runs, next_run = start - next_row * runs;
    for (long long first = start; first < total; first += static_cast<long long>(warps) * kAhead) {
        Raw8<T> raw[kAhead][kPieces];
        int row[kAhead], col[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            row[k] = next_row;
            col[k] = next_run * kRun + lane * 8 * kPieces;
            if (next_row < p.rows) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    raw[k][i].load(p, row[k], col[k] + 8 * i);
            }
            next_row += step_rows;
            next_run += step_runs;
            if (next_run >= runs) {
                next_run -= runs;
                ++next_row;
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (row[k] >= p.rows)
                break; // warp-uniform
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < kPieces * M::kWords; ++i)
                most = M::larger(most, M::of(raw[k][i / M::kWords].word(i % M::kWords)));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
                most = M::larger(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float scale = scale_of<Format>(M::largest(most));
            const Inverse inverse = inverse_of(scale);
            const unsigned long long low = pair(inverse.low, inverse.low), high = pair(inverse.high, inverse.high);
            uint2 q[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                unsigned long long v[4];
                raw[k][i].unpack(v);
                q[i] = quantize8<Format>(v, [&](int) { return low; }, [&](int) { return high; },
                                         [&](int) { return scale; });
            }
            if (kPieces == 2 && p.q_vectors == 16 && col[k] + 16 <= p.cols) {
                *reinterpret_cast<uint4 *>(p.q + row[k] * p.ldq + col[k]) =
                    make_uint4(q[0].x, q[0].y, q[kPieces - 1].x, q[kPieces - 1].y);
            } else {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    store8(p, row[k], col[k] + 8 * i, q[i]);
            }
            if (lane % kLanes == 0 && col[k] < p.cols)
                p.scale[row[k] * p.lds + col[k] / kGroup] = scale;
        }
    }
}

// ------------------------------------------------ column groups and blocks
// A CTA per 128 rows x Columns columns (column groups: 64, so that more CTAs
// share an SM and one's loads overlap another's arithmetic; blocks: 128), each
// thread eight columns of four rows.
constexpr int kTileSteps = 4;

template <int Columns>
constexpr int tile_threads()
{
    return Columns / 8 * (kGroup / kTileSteps);
}

template <class T, int Format, int Columns>
__global__ void __launch_bounds__(tile_threads<Columns>(), (sizeof(T) == 2 ? 1024 : 768) / tile_threads<Columns>())
    tile_kernel(const Call p)
{
    constexpr bool kBlock = Columns == kGroup;
    constexpr int kAcross = Columns / 8, kDown = kGroup / kTileSteps, kWarps = tile_threads<Columns>() / 32;
    using M = Magnitude<T>;
    constexpr int kWords = Columns * M::kWords / 8; // of a row of magnitudes
    __shared__ uint32_t most_of[kWarps][kWords];
    __shared__ uint32_t most_of_words[(kWords + 31) / 32];
    __shared__ float scales[Columns];
    // Of pairs of columns.
    __shared__ float2 lows[Columns / 2], highs[Columns / 2];
    const int across = threadIdx.x % kAcross, down = threadIdx.x / kAcross;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int tiles_n = (p.cols + Columns - 1) / Columns;
    const long long tiles = static_cast<long long>((p.rows + kGroup - 1) / kGroup) * tiles_n;
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        const long long tm = t / tiles_n;
        const int tn = static_cast<int>(t - tm * tiles_n);
        const int col = tn * Columns + across * 8;
        Raw8<T> raw[kTileSteps];
#pragma unroll
        for (int k = 0; k < kTileSteps; ++k) {
            const long long row = tm * kGroup + k * kDown + down;
            if (row < p.rows)
                raw[k].load(p, row, col);
            else
                raw[k].clear();
        }
        uint32_t most[M::kWords];
#pragma unroll
        for (int i = 0; i < M::kWords; ++i) {
            most[i] = M::of(raw[0].word(i));
#pragma unroll
            for (int k = 1; k < kTileSteps; ++k)
                most[i] = M::larger(most[i], M::of(raw[k].word(i)));
            // Lanes kAcross apart hold the same columns.
#pragma unroll
            for (int o = kAcross; o < 32; o *= 2)
                most[i] = M::larger(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
            if (lane < kAcross)
                most_of[warp][lane * M::kWords + i] = most[i];
        }
        __syncthreads();
        if (threadIdx.x < kWords) {
            uint32_t m = most_of[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                m = M::larger(m, most_of[w][threadIdx.x]);
            if (kBlock) {
                m = __reduce_max_sync(0xffffffffu, M::largest(m));
                if (lane == 0)
                    most_of_words[warp] = m;
            } else {
                // Each column's scale once, where all its threads find it.
                constexpr int kPerWord = Columns / kWords;
#pragma unroll
                for (int i = 0; i < kPerWord; ++i) {
                    const int c = static_cast<int>(threadIdx.x) * kPerWord + i;
                    const float scale = scale_of<Format>(M::element(m, i));
                    const Inverse inverse = inverse_of(scale);
                    scales[c] = scale;
                    reinterpret_cast<float *>(lows)[c] = inverse.low;
                    reinterpret_cast<float *>(highs)[c] = inverse.high;
                    if (tn * Columns + c < p.cols)
                        p.scale[tm * p.lds + tn * Columns + c] = scale;
                }
            }
        }
        __syncthreads();
        unsigned long long low[kBlock ? 1 : 4], high[kBlock ? 1 : 4];
        float block_scale = 0.0f;
        if (kBlock) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < (kWords + 31) / 32; ++w)
                m = max(m, most_of_words[w]);
            block_scale = scale_of<Format>(m);
            const Inverse inverse = inverse_of(block_scale);
            low[0] = pair(inverse.low, inverse.low);
            high[0] = pair(inverse.high, inverse.high);
            if (threadIdx.x == 0)
                p.scale[tm * p.lds + tn] = block_scale;
        } else {
#pragma unroll
            for (int k = 0; k < (kBlock ? 1 : 4); ++k) {
                const float2 a = lows[across * 4 + k], b = highs[across * 4 + k];
                low[k] = pair(a.x, a.y);
                high[k] = pair(b.x, b.y);
            }
        }
#pragma unroll
        for (int k = 0; k < kTileSteps; ++k) {
            const long long row = tm * kGroup + k * kDown + down;
            unsigned long long v[4];
            raw[k].unpack(v);
            const uint2 q = quantize8<Format>(v, [&](int i) { return low[kBlock ? 0 : i]; },
                                              [&](int i) { return high[kBlock ? 0 : i]; },
                                              [&](int e) { return kBlock ? block_scale : scales[across * 8 + e]; });
            if (row < p.rows)
                store8(p, row, col, q);
        }
        __syncthreads(); // the maxima and scales are read before the next tile's
    }
}

template <class T, int Format>
int launch(const Call &p, int group, int sms, cudaStream_t s)
{
    if (group == GEMM_FP8_ROW) {
        const int run = static_cast<int>(32 * 8 * (4 / sizeof(T)));
        const long long warps = static_cast<long long>(p.rows) * ((p.cols + run - 1) / run);
        const long long blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
        const unsigned grid = static_cast<unsigned>(std::min<long long>(blocks, 16ll * sms));
        row_kernel<T, Format><<<grid, kRowThreads, 0, s>>>(p);
    } else {
        const bool block = group == GEMM_FP8_BLOCK;
        const int columns = block ? kGroup : kGroup / 2;
        const long long tiles = (static_cast<long long>(p.rows) + kGroup - 1) / kGroup * ((p.cols + columns - 1) / columns);
        const unsigned grid = static_cast<unsigned>(std::min<long long>(tiles, 1ll << 30));
        if (block)
            tile_kernel<T, Format, kGroup><<<grid, tile_threads<kGroup>(), 0, s>>>(p);
        else
            tile_kernel<T, Format, kGroup / 2><<<grid, tile_threads<kGroup / 2>(), 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

constexpr int kMaxSide = 1 << 30;

} // namespace quantize
} // namespace pg

using namespace pg;

extern "C" int quantize_fp8(int rows, int cols, const void *x, long long ldx, int dtype, int group, int format, void *q,
                            long long ldq, float *scale, long long lds, void *stream)
{
    using namespace quantize;
    if (rows < 0 || cols < 0 || (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16) || group < GEMM_FP8_ROW ||
        group > GEMM_FP8_BLOCK || (format != GEMM_FP8_E4M3 && format != GEMM_FP8_E5M2))
        return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxSide || cols > kMaxSide)
        return GEMM_ERR_UNSUPPORTED;
    const bool empty = rows == 0 || cols == 0;
    const size_t size = dtype == GEMM_DTYPE_F32 ? 4 : 2;
    if (!empty) {
        const int scale_rows = group == GEMM_FP8_ROW ? rows : (rows + kGroup - 1) / kGroup;
        const int scale_cols = group == GEMM_FP8_COLUMN ? cols : (cols + kGroup - 1) / kGroup;
        if (!x || !q || !scale || (rows > 1 && (ldx < cols || ldq < cols)) || (scale_rows > 1 && lds < scale_cols))
            return GEMM_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(x) & (size - 1)) != 0 || (reinterpret_cast<uintptr_t>(scale) & 3u) != 0)
            return GEMM_ERR_MISALIGNED;
    }
    int dev;
    const int st = device_checked(&dev);
    if (st != GEMM_OK || empty)
        return st;
    Call p = {};
    p.rows = rows;
    p.cols = cols;
    p.x = x;
    p.ldx = ldx;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.scale = scale;
    p.lds = lds;
    p.x_vectors = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (rows <= 1 || (ldx * static_cast<long long>(size)) % 16 == 0);
    const uintptr_t q_low = reinterpret_cast<uintptr_t>(q) | (rows > 1 ? static_cast<uintptr_t>(ldq) : 0);
    p.q_vectors = (q_low & 15u) == 0 ? 16 : (q_low & 7u) == 0 ? 8 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int sms = device_sms();
    if (dtype == GEMM_DTYPE_F32)
        return format == GEMM_FP8_E4M3 ? launch<float, GEMM_FP8_E4M3>(p, group, sms, s)
                                       : launch<float, GEMM_FP8_E5M2>(p, group, sms, s);
    return format == GEMM_FP8_E4M3 ? launch<__nv_bfloat16, GEMM_FP8_E4M3>(p, group, sms, s)
                                   : launch<__nv_bfloat16, GEMM_FP8_E5M2>(p, group, sms, s);
}
