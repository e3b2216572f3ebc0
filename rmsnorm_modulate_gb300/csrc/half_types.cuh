// Conversions between stored 16-bit types (bf16, fp16) and fp32, two values of a word at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"

namespace rmsmod {

// exact
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w);
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// rounded to nearest, ties to even
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float lo, float hi)
{
    return pack_bf2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// the sum of two words' values, one rounding each (what fp32's sum rounds to as well)
template <typename T>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t add2<__nv_bfloat16>(uint32_t a, uint32_t b)
{
    return bf2_add(a, b);
}
template <>
__device__ __forceinline__ uint32_t add2<__half>(uint32_t a, uint32_t b)
{
    return h2_add(a, b);
}

// widening and rounding of packed fp32 pairs
template <typename T>
__device__ __forceinline__ u64 widen(uint32_t w)
{
    const float2 v = widen2<T>(w);
    return f2_pack(v.x, v.y);
}

template <typename T>
__device__ __forceinline__ uint32_t narrow(u64 v)
{
    float lo, hi;
    f2_unpack(v, lo, hi);
    return narrow2<T>(lo, hi);
}

}  // namespace rmsmod
