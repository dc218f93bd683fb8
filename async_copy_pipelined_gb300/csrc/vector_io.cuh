// Loads and stores of float32 and bfloat16 elements as float32 values, and
// arithmetic on pairs of them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace pg {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Element j of a vector whose type is known at run time.
__device__ __forceinline__ float load_f32(const void *base, bool bf16, long long j)
{
    return bf16 ? to_f32(static_cast<const __nv_bfloat16 *>(base)[j]) : static_cast<const float *>(base)[j];
}

__device__ __forceinline__ void store_f32(void *base, bool bf16, long long j, float v)
{
    if (bf16)
        static_cast<__nv_bfloat16 *>(base)[j] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(base)[j] = v;
}

// Sixteen bytes as float32 values, and back.
template <class T>
struct Vec16;

template <>
struct Vec16<float> {
    static constexpr int kElements = 4;
    static __device__ __forceinline__ void unpack(const uint4 &q, float *v)
    {
        v[0] = __uint_as_float(q.x);
        v[1] = __uint_as_float(q.y);
        v[2] = __uint_as_float(q.z);
        v[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *v)
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

// Two bfloat16 values in a word.
__device__ __forceinline__ void unpack_bf16(uint32_t w, float *v)
{
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
}

template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int kElements = 8;
    static __device__ __forceinline__ void unpack(const uint4 &q, float *v)
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            unpack_bf16(w[e], v + 2 * e);
    }
    static __device__ __forceinline__ uint4 pack(const float *v)
    {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Two float32 values in one 64-bit register, added and multiplied by one
// instruction.
__device__ __forceinline__ unsigned long long pair(float a, float b)
{
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void split(unsigned long long v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float both(unsigned long long v)
{
    float a, b;
    split(v, a, b);
    return a + b;
}

} // namespace pg
