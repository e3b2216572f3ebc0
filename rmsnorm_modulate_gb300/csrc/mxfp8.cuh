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
// least power of two with max <= 448 * 2^e (448 = 1.75 * 2^8: past its mantissa the sum carries into the
// exponent), biased by 127; 255 (NaN) for a block that holds Inf or NaN.  `inverse`: 2^-e.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t bits, float& inverse)
{
    const int e = max(static_cast<int>((bits + 0x1FFFFFu) >> 23) - 8, 0);
    inverse = __uint_as_float(0x7F000000u - (static_cast<uint32_t>(e) << 23));
    return bits >= 0x7F800000u ? 255u : static_cast<uint32_t>(e);
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

// max(m, |v.lo|, |v.hi|), NaN if one is.
__device__ __forceinline__ float absmax2(float m, u64 v)
{
    float lo, hi, r;
    f2_unpack(v, lo, hi);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(lo), "f"(hi));
    return r;
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

__device__ __forceinline__ uint32_t e4m3x4(u64 ab, u64 cd)
{
    float a, b, c, d;
    f2_unpack(ab, a, b);
    f2_unpack(cd, c, d);
    return e4m3x4(a, b, c, d);
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

// Four codes as two pairs of fp32, exact.
__device__ __forceinline__ void e4m3x4_values(uint32_t codes, u64& lo, u64& hi)
{
    lo = widen<__half>(e4m3x2_half2(codes & 0xFFFFu));
    hi = widen<__half>(e4m3x2_half2(codes >> 16));
}

// Where the scale byte of row r, block k of a matrix of `tiles` block tiles (128 values) a row stands.
__device__ __forceinline__ int64_t mx8_scale_at(int64_t r, int64_t k, int64_t tiles)
{
    return ((r >> 7) * tiles + (k >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (k & 3);
}

// 2 * N neighbours of a block that LANES lanes share, each with as many, to codes and the block's scale
// byte.
template <int N, int LANES>
__device__ __forceinline__ uint32_t quantize_pairs(const u64 (&v)[N], uint32_t (&codes)[N / 2])
{
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i)
        m[i & 1] = absmax2(m[i & 1], v[i]);
    uint32_t bits = max(__float_as_uint(m[0]), __float_as_uint(m[1]));
#pragma unroll
    for (int off = 1; off < LANES; off *= 2)
        bits = max(bits, __shfl_xor_sync(kFullMask, bits, off));
    float inverse;
    const uint32_t byte = mx8_scale_byte(bits, inverse);
    const u64 inv = f2_splat(inverse);
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        codes[i] = e4m3x4(f2_mul(v[2 * i], inv), f2_mul(v[2 * i + 1], inv));
    return byte;
}

// ---------------------------------------------------------------------------
// activations, two values at a time
// ---------------------------------------------------------------------------

// SiLU z p(z); GELU z Phi(z); its tanh form z p(2 sqrt(2 / pi) (z + 0.044715 z^3)), since
// (1 + tanh(a / 2)) / 2 = p(a); p(a) = 1 / (1 + e^-a).
enum Activation : int { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3 };

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ u64 rcp2(u64 v)
{
    float lo, hi;
    f2_unpack(v, lo, hi);
    return f2_pack(rcp(lo), rcp(hi));
}

// `a` where z >= 0 (or is NaN), else b.
__device__ __forceinline__ u64 by_sign(u64 z, u64 a, u64 b)
{
    float zl, zh, al, ah, bl, bh;
    f2_unpack(z, zl, zh);
    f2_unpack(a, al, ah);
    f2_unpack(b, bl, bh);
    return f2_pack(zl < 0.0f ? bl : al, zh < 0.0f ? bh : ah);
}

constexpr float kLog2e = 1.4426950408889634f;

// p(a) for a = -x log(2), and q = p(a) (1 - p(a)), from t = 2^x = e^-a, at most 2^127: then t p is 1 - p
// without a difference, and nothing overflows on either side.  (Past 2^126 p is 0, which the reciprocal
// flushes to.)
// The approximate instructions are good to 2^-22 each and x to its own rounding, |x| 2^-24, and those of
// its factors (four or so for the cubic argument): z p is good to (16 + 4 |ln p|) 2^-24, which is 2^-19
// where p >= 1/2 and 2^-17 where it is 2^-40, far inside a step of 8- and 16-bit results.  fp32 results
// have no more than that either.  A NaN is left to the factors z.
__device__ __forceinline__ u64 logistic2(u64 x, u64& q)
{
    float lo, hi;
    f2_unpack(x, lo, hi);
    const u64 t = f2_pack(ex2(fminf(lo, 127.0f)), ex2(fminf(hi, 127.0f)));
    const u64 p = rcp2(f2_add(t, f2_splat(1.0f)));
    q = f2_mul(f2_mul(t, p), p);
    return p;
}

constexpr float kGeluSlope = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// -log2(e) times the logistic's argument.
__device__ __forceinline__ u64 gelu_argument(u64 z, u64 zz)
{
    constexpr float c = -kGeluSlope * kLog2e;
    return f2_mul(z, f2_fma(zz, f2_splat(c * kGeluCubic), f2_splat(c)));
}

// Phi(z), and e^(-z^2 / 2).  With t = 1 / (1 + c |z|) and P a polynomial,
//     Phi(-|z|) = e^(-z^2 / 2) t P(t):
// e^(z^2 / 2) Phi(-|z|) is smooth in t, and goes like t for large |z|.  P is the least maximum of the
// relative error over |z| <= 19.8, 2^-25.2, found by weighted least squares against erfcx in 64 bits; in
// fp32 the product is good to 2^-21 (and e^(-z^2 / 2) to z^2 2^-24).  Beyond 19.8 it is 0.
__device__ __forceinline__ u64 normal2(u64 z, u64 zz, u64& e)
{
    constexpr float c = 0.26870057f;
    constexpr float P[9] = {0.10720491409301758f,  0.10697222501039505f,  0.10184260457754135f,
                            0.06984031200408936f,  0.1136091947555542f,   -0.07841922342777252f,
                            0.17966914176940918f,  -0.1299300491809845f,  0.02921086549758911f};
    float lo, hi;
    f2_unpack(z, lo, hi);
    const u64 az = f2_pack(fminf(fabsf(lo), 19.75f), fminf(fabsf(hi), 19.75f));
    const u64 t = rcp2(f2_fma(az, f2_splat(c), f2_splat(1.0f)));
    u64 p = f2_splat(P[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i)
        p = f2_fma(p, t, f2_splat(P[i]));
    f2_unpack(f2_mul(zz, f2_splat(-0.5f * kLog2e)), lo, hi);
    e = f2_pack(ex2(lo), ex2(hi));
    const u64 tail = f2_mul(f2_mul(p, t), e);
    return by_sign(z, f2_sub(f2_splat(1.0f), tail), tail);
}

template <int ACT>
__device__ __forceinline__ u64 activate2(u64 z)
{
    u64 unused;
    if (ACT == kActSilu)
        return f2_mul(z, logistic2(f2_mul(z, f2_splat(-kLog2e)), unused));
    if (ACT == kActGelu)
        return f2_mul(z, normal2(z, f2_mul(z, z), unused));
    if (ACT == kActGeluTanh)
        return f2_mul(z, logistic2(gelu_argument(z, f2_mul(z, z)), unused));
    return z;
}

// act'(z), and act(z) / z in `part`.  |z| up to 2^60: the derivative's factors stay finite.
template <int ACT>
__device__ __forceinline__ u64 slope2(u64 z, u64& part)
{
    if (ACT == kActNone) {
        part = f2_splat(1.0f);
        return part;
    }
    const u64 zz = f2_mul(z, z);
    if (ACT == kActGelu) {
        u64 e;
        part = normal2(z, zz, e);
        return f2_fma(f2_mul(z, f2_splat(0.39894228040143268f)), e, part);
    }
    u64 q;
    if (ACT == kActSilu) {
        part = logistic2(f2_mul(z, f2_splat(-kLog2e)), q);
        return f2_fma(z, q, part);
    }
    part = logistic2(gelu_argument(z, zz), q);
    const u64 rise = f2_fma(zz, f2_splat(3.0f * kGeluCubic * kGeluSlope), f2_splat(kGeluSlope));
    return f2_fma(f2_mul(z, q), rise, part);
}

}  // namespace rmsmod
