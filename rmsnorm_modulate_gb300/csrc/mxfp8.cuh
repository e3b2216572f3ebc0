// Microscaled 8-bit blocks and the activations whose inputs they keep, on the device.
//
// A block is 32 values that stand side by side in a row: e4m3 codes (sign, four exponent bits, three
// mantissa bits; largest 448, smallest 2^-9) under one e8m0 scale, the least 2^e with
// max|x| <= 448 * 2^e and e >= -127, so no value saturates.  A code is x * 2^-e rounded to nearest,
// ties to even; x * 2^-e is exact in fp32 wherever the code is not zero, so a block is its
// definition's own whatever the order of the work.
#pragma once

#include "half_types.cuh"

namespace rmsmod {

// Scale byte of a block whose largest magnitude has the fp32 pattern `bits`: the exponent of the
// least power of two with max <= 448 * 2^e (448 = 1.75 * 2^8), biased by 127; 255 (NaN) for a block
// that holds Inf or NaN.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t bits)
{
    if (bits >= 0x7F800000u)
        return 255u;
    const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}

// 2^-e of a scale byte that mx8_scale_byte gave (at most 247, or 255: then 0).
__device__ __forceinline__ float mx8_inverse(uint32_t byte)
{
    return __uint_as_float((254u - (byte == 255u ? 254u : byte)) << 23);
}

// What a scale byte stands for.
__device__ __forceinline__ float mx8_scale(uint32_t byte)
{
    return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23));
}

__device__ __forceinline__ uint32_t magnitude_bits(float v)
{
    // as integers magnitudes order like the values, with Inf and NaN on top
    return __float_as_uint(v) & 0x7FFFFFFFu;
}

// Four e4m3 codes, element 0 in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_code(float v)
{
    return e4m3x4(v, 0.0f, 0.0f, 0.0f) & 0xFFu;
}

// Two codes (the low 16 bits) as packed fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return h;
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes)
{
    const uint32_t h = e4m3x2_half2(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Where the scale byte of row r, block k of a matrix of `tiles` block tiles (128 values) a row stands.
__device__ __forceinline__ int64_t mx8_scale_at(int64_t r, int64_t k, int64_t tiles)
{
    return ((r >> 7) * tiles + (k >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (k & 3);
}

// Thirty-two neighbours that one thread holds, to codes and their scale byte.
__device__ __forceinline__ uint32_t quantize32(const float (&v)[32], uint4 (&codes)[2])
{
    uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 32; ++i)
        m[i & 3] = max(m[i & 3], magnitude_bits(v[i]));
    const uint32_t byte = mx8_scale_byte(max(max(m[0], m[1]), max(m[2], m[3])));
    const float inv = mx8_inverse(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        word(codes[i >> 2], i & 3) =
            e4m3x4(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv),
                   __fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv));
    return byte;
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// SiLU z p(z); GELU z Phi(z); its tanh form z p(2 sqrt(2 / pi) (z + 0.044715 z^3)), since
// (1 + tanh(a / 2)) / 2 = p(a); p(a) = 1 / (1 + e^-a).
enum Activation : int { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3 };

// p(a), and q = p(a) (1 - p(a)), from t = e^-|a| <= 1: nothing overflows on either side.  The
// approximate instructions are good to 2^-22 each and the exponent's rounding to |a| 2^-24, so p is
// good to 2^-18 where it is 2^-40 and better above: far inside a step of what its products are
// rounded to.
__device__ __forceinline__ float logistic(float a, float& q)
{
    float t, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(__fmul_rn(fabsf(a), -1.4426950408889634f)));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, t)));
    const float s = __fmul_rn(t, r);
    q = __fmul_rn(s, r);
    return a >= 0.0f || a != a ? r : s;
}

constexpr float kGeluSlope = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float gelu_argument(float z)
{
    const float zz = __fmul_rn(z, z);
    return __fmul_rn(kGeluSlope, __fmaf_rn(__fmul_rn(kGeluCubic, zz), z, z));
}

template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    float q;
    if (ACT == kActSilu)
        return __fmul_rn(z, logistic(z, q));
    if (ACT == kActGeluTanh)
        return __fmul_rn(z, logistic(gelu_argument(z), q));
    if (ACT == kActGelu)
        return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(z, -0.70710678118654752f)));
    return z;
}

// The activation and, in `slope`, its derivative.
template <int ACT>
__device__ __forceinline__ float activate(float z, float& slope)
{
    if (ACT == kActSilu || ACT == kActGeluTanh) {
        float q, rise = 1.0f;
        const float p = logistic(ACT == kActSilu ? z : gelu_argument(z), q);
        if (ACT == kActGeluTanh)
            rise = __fmul_rn(kGeluSlope, __fmaf_rn(3.0f * kGeluCubic, __fmul_rn(z, z), 1.0f));
        // (q is 0 before z^2 leaves fp32's range)
        slope = q > 0.0f ? __fmaf_rn(__fmul_rn(z, q), rise, p) : p;
        return __fmul_rn(z, p);
    }
    if (ACT == kActGelu) {
        const float phi = __fmul_rn(0.5f, erfcf(__fmul_rn(z, -0.70710678118654752f)));
        float t;  // e^(-z^2 / 2)
        asm("ex2.approx.f32 %0, %1;"
            : "=f"(t)
            : "f"(__fmul_rn(__fmul_rn(z, z), -0.72134752044448170f)));
        slope = t > 0.0f ? __fmaf_rn(__fmul_rn(z, 0.39894228040143268f), t, phi) : phi;
        return __fmul_rn(z, phi);
    }
    slope = 1.0f;
    return z;
}

}  // namespace rmsmod
