// Microscaled 4-bit floating point rows: quantisation and its inverse.
//
// A row is cut into blocks of 32 values.  A block holds 32 e2m1 codes (sign, two exponent bits,
// one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) under one e8m0 scale, a power of two.  The scale
// is the least 2^e with max|x| <= 6 * 2^e, so no value saturates; the codes are x * 2^-e rounded
// to nearest, ties to the even code.  x * 2^-e is exact in fp32, so the result is the definition's
// own whatever the order of the work.
//
// Layout (what the block-scaled tensor core instructions read):
//   packed   [rows, K / 2] bytes, the even element in the low half
//   scales   tiles of 128 rows by 4 blocks, 512 bytes each, [row tile][block tile]; in a tile row r
//            and block k stand at byte (r % 32) * 16 + (r / 32) * 4 + k.  Bytes of rows and blocks
//            that the matrix does not have are zero.

#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp4.h"

namespace rmsmod {

namespace {

// Eight e2m1 codes of eight fp32 (nearest, ties to even), element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
          "f"(v[7]));
    return d;
}

// The two values of a byte of codes, exact in fp16.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h)
        : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Scale byte of a block whose largest magnitude has the fp32 pattern `bits`: the exponent of the
// least power of two with max <= 6 * 2^e (6 = 1.5 * 2^2), biased by 127; 255 (NaN) for a block
// that holds Inf or NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits)
{
    if (bits >= 0x7F800000u)
        return 255u;
    const int e = static_cast<int>(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}

__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23));
}

constexpr int kThreads = 256;
constexpr int kUnitsPerCta = kThreads / 16;

// A unit is the 128 values of one block tile in the four rows r, r + 32, r + 64, r + 96 of a row tile,
// whose sixteen scale bytes are neighbours; 16 lanes take a unit, eight values of each row, so four
// lanes share a block and a unit's scales are one store.  Neighbouring units are neighbours in the
// rows.  Bound by HBM: 4216 x 16384 bf16 quantised in 28.0 us and back in 27.0, 0.92 and 0.95 of the
// measured copy peak (both together 49 us; with a unit for each row, whose scales are stores of four
// bytes, 62).
struct Unit {
    uint32_t tile, row, scale_word;
};

__device__ __forceinline__ Unit unit_of(const Mxfp4RowsArgs& a, uint32_t u)
{
    Unit t;
    const uint32_t line = a.by_tiles.div(u);  // (row tile, r)
    t.tile = u - line * a.by_tiles.d;
    t.row = (line >> 5) * 128 + (line & 31);
    t.scale_word = ((line >> 5) * a.by_tiles.d + t.tile) * 32 + (line & 31);  // of 16 bytes
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Mxfp4RowsArgs a)
{
    grid_dependency_sync();
    const int lane = threadIdx.x & 31;
    const uint32_t sub = threadIdx.x & 15;  // which eight of the tile's 128 values
    const Unit t = unit_of(a, blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4));
    const uint32_t col = t.tile * 16 + sub;
    const uint4* __restrict__ x = static_cast<const uint4*>(a.values);
    uint32_t* __restrict__ packed = static_cast<uint32_t*>(a.packed);
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = t.row + 32 * i;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < a.rows && col < a.Kv)
            v[i] = ld_stream(x + static_cast<int64_t>(row) * a.Kv + col);
    }
    uint4 four;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[8];
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = widen2<T>(word(v[i], j));
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
            // as integers magnitudes order like the values, with Inf and NaN on top
            bits = max(bits, __float_as_uint(p.x) & 0x7FFFFFFFu);
            bits = max(bits, __float_as_uint(p.y) & 0x7FFFFFFFu);
        }
        bits = max(bits, __shfl_xor_sync(kFullMask, bits, 1));
        bits = max(bits, __shfl_xor_sync(kFullMask, bits, 2));
        const uint32_t byte = scale_byte(bits);
        const float inv = __uint_as_float((254u - (byte == 255u ? 254u : byte)) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = __fmul_rn(f[j], inv);
        const uint32_t codes = e2m1x8(f);
        // the row's four scale bytes, from lanes 0, 4, 8 and 12 of the unit
        const int base = lane & 16;
        uint32_t w = __shfl_sync(kFullMask, byte, base);
        w |= __shfl_sync(kFullMask, byte, base + 4) << 8;
        w |= __shfl_sync(kFullMask, byte, base + 8) << 16;
        w |= __shfl_sync(kFullMask, byte, base + 12) << 24;
        word(four, i) = w;
        const uint32_t row = t.row + 32 * i;
        if (row < a.rows && col < a.Kv)
            packed[static_cast<int64_t>(row) * a.Kv + col] = codes;
    }
    if (sub == 0 && t.row < a.rows_padded)
        static_cast<uint4*>(a.scales)[t.scale_word] = four;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Mxfp4RowsArgs a)
{
    grid_dependency_sync();
    const uint32_t sub = threadIdx.x & 15;
    const Unit t = unit_of(a, blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4));
    const uint32_t col = t.tile * 16 + sub;
    if (t.row >= a.rows || col >= a.Kv)
        return;
    const uint32_t* __restrict__ packed = static_cast<const uint32_t*>(a.packed);
    uint4* __restrict__ out = static_cast<uint4*>(a.values);
    const uint4 four = ld_cached(static_cast<const uint4*>(a.scales) + t.scale_word);
    uint32_t codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = t.row + 32 * i;
        codes[i] = row < a.rows ? ld_cached(packed + static_cast<int64_t>(row) * a.Kv + col) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = t.row + 32 * i;
        const float s = scale_value((word(four, i) >> (8 * (sub >> 2))) & 0xFFu);
        uint4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = e2m1x2_values((codes[i] >> (8 * j)) & 0xFFu);
            word(o, j) = narrow2<T>(__fmul_rn(p.x, s), __fmul_rn(p.y, s));
        }
        if (row < a.rows)
            st_stream(out + static_cast<int64_t>(row) * a.Kv + col, o);
    }
}

}  // namespace

cudaError_t launch_mxfp4_rows(bool quantize, const Mxfp4RowsArgs& a, cudaStream_t stream)
{
    const uint32_t units = a.rows_padded / 4 * a.by_tiles.d;
    const int grid = static_cast<int>((units + kUnitsPerCta - 1) / kUnitsPerCta);
    if (quantize)
        return launch_dependent(a.f16 ? quantize_kernel<__half> : quantize_kernel<__nv_bfloat16>,
                                grid, kThreads, 0, stream, a);
    return launch_dependent(a.f16 ? dequantize_kernel<__half> : dequantize_kernel<__nv_bfloat16>,
                            grid, kThreads, 0, stream, a);
}

}  // namespace rmsmod
