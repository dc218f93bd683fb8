// Loads and stores of float32 and bfloat16 elements as float32 values.
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

} // namespace pg
