// Microscaled 8-bit rows: quantisation and its inverse, their blocks laid out anew along the other
// axis, and the gradient of an activation whose input they keep.
//
// Layout (what the block-scaled tensor core instructions read):
//   codes    [rows, K] bytes, e4m3
//   scales   tiles of 128 rows by 4 blocks, 512 bytes each, [row tile][block tile]; in a tile row r
//            and block k stand at byte (r % 32) * 16 + (r / 32) * 4 + k.  Bytes of rows and blocks
//            that the matrix does not have are zero.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp8.cuh"
#include "mxfp8.h"
#include "sectors.cuh"

namespace rmsmod {

namespace {

constexpr int kThreads = 256;
constexpr int kUnitsPerCta = kThreads / 16;

// ---------------------------------------------------------------------------
// rows to blocks and back
// ---------------------------------------------------------------------------

// A unit is the 128 values of one block tile in the four rows r, r + 32, r + 64, r + 96 of a row tile,
// whose sixteen scale bytes are neighbours; 16 lanes take a unit, eight values of each row, so four
// lanes share a block and a unit's scales are one store.  Neighbouring units are neighbours in the
// rows.  Bound by HBM: at 4216 x 16384 33 to 36 us to codes and 32 back, of 31; at 4216 x 4096 (in part
// from L2) 11 and 9.
struct Unit {
    uint32_t tile, row;
    int64_t scale_word;  // of 16 bytes
};

__device__ __forceinline__ Unit unit_of(const Mxfp8RowsArgs& a, uint32_t u)
{
    Unit t;
    const uint32_t line = a.by_tiles.div(u);  // (row tile, r)
    t.tile = u - line * a.by_tiles.d;
    t.row = (line >> 5) * 128 + (line & 31);
    t.scale_word = (static_cast<int64_t>(line >> 5) * a.by_tiles.d + t.tile) * 32 + (line & 31);
    return t;
}

// The four scale bytes of a row's block tile, of which each of its sixteen lanes has its block's.
__device__ __forceinline__ uint32_t join_bytes(uint32_t byte, int lane)
{
    uint32_t w = byte << (2 * (lane & 12));
    w |= __shfl_xor_sync(kFullMask, w, 4);
    w |= __shfl_xor_sync(kFullMask, w, 8);
    return w;
}

__device__ __forceinline__ void values8(uint2 codes, float scale, u64 (&f)[4])
{
    e4m3x4_values(codes.x, f[0], f[1]);
    e4m3x4_values(codes.y, f[2], f[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = f2_mul(f[j], f2_splat(scale));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize8_kernel(const Mxfp8RowsArgs a)
{
    grid_dependency_sync();
    const int lane = threadIdx.x & 31;
    const uint32_t sub = threadIdx.x & 15;  // which eight of the tile's 128 values
    const Unit t = unit_of(a, blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4));
    const uint32_t col = t.tile * 16 + sub;
    const uint4* __restrict__ x = static_cast<const uint4*>(a.values);
    uint2* __restrict__ codes = static_cast<uint2*>(a.codes);
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
        u64 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = widen<T>(word(v[i], j));
        uint32_t c[2];
        word(four, i) = join_bytes(quantize_pairs<4, 4>(f, c), lane);
        const uint32_t row = t.row + 32 * i;
        if (row < a.rows && col < a.Kv)
            codes[static_cast<int64_t>(row) * a.Kv + col] = make_uint2(c[0], c[1]);
    }
    if (sub == 0 && t.row < a.rows_padded)
        static_cast<uint4*>(a.scales)[t.scale_word] = four;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize8_kernel(const Mxfp8RowsArgs a)
{
    grid_dependency_sync();
    const uint32_t sub = threadIdx.x & 15;
    const Unit t = unit_of(a, blockIdx.x * kUnitsPerCta + (threadIdx.x >> 4));
    const uint32_t col = t.tile * 16 + sub;
    if (t.row >= a.rows || col >= a.Kv)
        return;
    const uint2* __restrict__ codes = static_cast<const uint2*>(a.codes);
    uint4* __restrict__ out = static_cast<uint4*>(a.values);
    const uint4 four = ld_cached(static_cast<const uint4*>(a.scales) + t.scale_word);
    uint2 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = t.row + 32 * i;
        c[i] = make_uint2(0u, 0u);
        if (row < a.rows)
            c[i] = ld_stream2(codes + static_cast<int64_t>(row) * a.Kv + col);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = t.row + 32 * i;
        u64 f[4];
        values8(c[i], mx8_scale((word(four, i) >> (8 * (sub >> 2))) & 0xFFu), f);
        uint4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            word(o, j) = narrow<T>(f[j]);
        if (row < a.rows)
            st_stream(out + static_cast<int64_t>(row) * a.Kv + col, o);
    }
}

// ---------------------------------------------------------------------------
// blocks along the other axis
// ---------------------------------------------------------------------------

// 128 x 128 codes by 128 threads: a thread takes four columns (one word of each row) of 32 rows, which
// are four of the result's blocks, whole.
//
// With the largest scale 2^E of the 32 rows' blocks, a value times 2^(7 - E) is at most 448 * 2^7: an
// fp16 number, exact down to 2^-24.  So in packed fp16 a column's largest magnitude costs a product and
// a maximum for two values, and its codes one more product, by the power of two that brings it under
// the new scale 2^x.  That is the definition's own result while the largest is 2^-3 or more: x is then
// -11 or more, so what has a code that is not zero is at least 2^(x - 10) = 2^-21 and keeps its four
// bits.  Else (a column far below its rows' largest, scales 2^32 apart, NaN, the least scale)
// turn_slowly() goes by whole numbers and fp32.
//
// 30 us at 4216 x 16384, whose bytes take 21 (six CTAs an SM; five 33, seven 36, eight 39).  Neither its
// instructions (56% of the issue slots) nor HBM (37%) bound it: a CTA loads, turns and stores one after
// the other, which only the CTAs beside it on the SM hide.
constexpr int kTurn = 128;

__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return (w >> (8 * i)) & 0xFFu; }

__device__ __forceinline__ uint32_t h2_absmax(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t e4m3x2_of_half2(uint32_t h)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

// Order of the two codes' magnitudes (halves of the result), with e8 = 8 * scale byte; zero codes come
// last.  `nan`: bits 8 and 24 where the code is NaN.
__device__ __forceinline__ uint32_t order2(uint32_t half2, uint32_t e8, uint32_t& nan)
{
    const uint32_t k = (half2 >> 7) & 0x00FF00FFu;
    nan = (k + 0x00010001u) & 0x01000100u;  // NaN: all of the eight bits
    return k + (((k + 0x00FF00FFu) >> 8) & 0x00010001u) * e8;
}

// Four rows of four columns to four columns of four rows, at word q of each column.
__device__ __forceinline__ void turn4(const uint32_t (&w)[4], uint32_t (&out)[4][8], int q)
{
    const uint32_t a01 = __byte_perm(w[0], w[1], 0x5140), b01 = __byte_perm(w[0], w[1], 0x7362);
    const uint32_t a23 = __byte_perm(w[2], w[3], 0x5140), b23 = __byte_perm(w[2], w[3], 0x7362);
    out[0][q] = __byte_perm(a01, a23, 0x5410);
    out[1][q] = __byte_perm(a01, a23, 0x7632);
    out[2][q] = __byte_perm(b01, b23, 0x5410);
    out[3][q] = __byte_perm(b01, b23, 0x7632);
}

// For any codes and scales.  A value is (1 + m / 8) * 2^(E + e), from a code's fp16 form (every e4m3
// value is a normal fp16 number) and its scale's exponent: 8 E + m + 8 e, a whole number, orders the
// magnitudes, so the block's scale is found without rounding whatever the exponents' spread.  Moving a
// value to the new scale 2^n multiplies it by 2^(e - n), exact in fp32 where the result is not zero.
__device__ __noinline__ void turn_slowly(const uint32_t* words, const uint32_t* scale_words, int block,
                                         uint32_t (&bytes)[4], uint32_t (&out)[4][8])
{
    uint32_t top[2] = {0u, 0u}, nan = 0u;
    for (int r = 0; r < 32; ++r) {
        const uint32_t w = words[r * 32], e = byte_of(scale_words[r * 4], block);
        uint32_t n01, n23;
        top[0] = __vmaxu2(top[0], order2(e4m3x2_half2(w & 0xFFFFu), e * 8u, n01));
        top[1] = __vmaxu2(top[1], order2(e4m3x2_half2(w >> 16), e * 8u, n23));
        nan |= n01 | (n23 << 1);
        if (e == 255u)
            nan = 0x03000300u;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t k = (top[c >> 1] >> (16 * (c & 1))) & 0xFFFFu;
        const int e = static_cast<int>(k >> 3) - 23 + ((k & 7u) == 7u ? 1 : 0);
        bytes[c] = e > 0 ? static_cast<uint32_t>(e) : 0u;
        if (nan & (0x100u << (16 * (c & 1)) << (c >> 1)))
            bytes[c] = 255u;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        uint32_t w4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * q + i;
            const int e = static_cast<int>(byte_of(scale_words[r * 4], block));
            u64 lo, hi;
            e4m3x4_values(words[r * 32], lo, hi);
            float v[4];
            f2_unpack(lo, v[0], v[1]);
            f2_unpack(hi, v[2], v[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // 2^(e - n): at most 2^17 where the code is not zero
                const int d = min(max(e - static_cast<int>(bytes[c]), -126), 17);
                v[c] = __fmul_rn(v[c], __uint_as_float(static_cast<uint32_t>(d + 127) << 23));
            }
            w4[i] = e4m3x4(v[0], v[1], v[2], v[3]);
        }
        turn4(w4, out, q);
    }
}

__global__ void __launch_bounds__(kTurn, 6) transpose8_kernel(const Mxfp8TransposeArgs a)
{
    __shared__ __align__(16) uint32_t tile[kTurn * kTurn / 4];
    __shared__ __align__(16) uint32_t scale_in[128], scale_out[128];
    __shared__ uint32_t factors[4][32][4];  // [rows][row][block], in both halves
    grid_dependency_sync();
    const int64_t tiles_k = (a.K + 127) / 128, tiles_r = (a.rows + 127) / 128;
    const uint32_t across = blockIdx.x / static_cast<uint32_t>(tiles_k);
    const int64_t tr = across, tk = blockIdx.x - across * static_cast<uint32_t>(tiles_k);
    const int64_t r0 = tr * 128, k0 = tk * 128;
    const int64_t padded = (a.rows + 31) / 32 * 32;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint8_t* __restrict__ codes = static_cast<const uint8_t*>(a.codes);
    uint4 in[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 16 + (t >> 3), k = k0 + (t & 7) * 16;
        in[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.rows && k < a.K)
            in[i] = ld_stream(reinterpret_cast<const uint4*>(codes + r * a.K + k));
    }
    {  // word t: row t / 4 + 32 * (t % 4)
        const int64_t r = r0 + (t >> 2) + 32 * (t & 3);
        scale_in[t] = r < a.rows ? ld_cached(static_cast<const uint32_t*>(a.scales) +
                                         (tr * tiles_k + tk) * 128 + t)
                                 : 0u;
        scale_out[t] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint4*>(tile)[i * kTurn + t] = in[i];
    __syncthreads();
    // rows r0 + 32 * warp ..., columns k0 + 4 * lane ...
    const int block = lane >> 3;
    uint32_t top_byte = 0u;  // of this thread's blocks
    uint32_t far = 0u;       // a bit for each block tile's: a factor that fp16 lacks would count
    {
        const uint32_t w = scale_in[lane * 4 + warp];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t e = byte_of(w, k), most = __reduce_max_sync(kFullMask, e);
            // 2^(7 - (most - e)): fp16 ends at 2^-24, what counts (448 * 2^-30 > 2^-22) later
            const int x = 22 - static_cast<int>(most - e);  // biased exponent
            const uint32_t f = x > 0 ? static_cast<uint32_t>(x) << 10 : x >= -9 ? 1u << (9 + x) : 0u;
            far |= (x < -9 && x >= -15 ? 1u : 0u) << k;
            factors[warp][lane][k] = f * 0x00010001u;
            if (k == block)
                top_byte = most;
        }
    }
    far = __reduce_or_sync(kFullMask, far);
    __syncwarp();
    const uint32_t* words = tile + warp * 32 * 32 + lane;
    uint32_t v[32][2], top[2], any = 0u;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const uint32_t w = words[r * 32], f = factors[warp][r][block];
        any |= w;
        v[r][0] = h2_mul(e4m3x2_half2(w & 0xFFFFu), f);
        v[r][1] = h2_mul(e4m3x2_half2(w >> 16), f);
        // (begun with the first row: against a constant zero a negative row's magnitude was lost)
        top[0] = r ? h2_absmax(top[0], v[r][0]) : v[r][0];
        top[1] = r ? h2_absmax(top[1], v[r][1]) : v[r][1];
    }
    uint32_t bytes[4], g[2] = {0u, 0u};
    bool slow = top_byte == 255u || (far >> block & 1u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t h = (top[c >> 1] >> (16 * (c & 1))) & 0x7FFFu;
        // least x with the largest <= 448 * 2^x (448 = 1.75 * 2^8), and 2^-x in fp16
        const int x = static_cast<int>(h >> 10) - 23 + ((h & 0x3FFu) > 0x300u ? 1 : 0);
        const int byte = static_cast<int>(top_byte) - 7 + x;
        if (((any >> (8 * c)) & 0x7Fu) == 0u) {  // zeros, with either sign
            bytes[c] = 0u;
            g[c >> 1] |= 0x3C00u << (16 * (c & 1));
        } else {
            slow = slow || h < 0x3000u || h >= 0x7C00u || byte < 0;
            bytes[c] = static_cast<uint32_t>(byte);
            g[c >> 1] |= (static_cast<uint32_t>(15 - x) << 10 & 0x7C00u) << (16 * (c & 1));
        }
    }
    uint32_t out[4][8];
    if (slow) {
        uint32_t slow_bytes[4], slow_out[4][8];
        turn_slowly(words, scale_in + warp, block, slow_bytes, slow_out);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            bytes[c] = slow_bytes[c];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                out[c][q] = slow_out[c][q];
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint32_t w4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w4[i] = e4m3x2_of_half2(h2_mul(v[4 * q + i][0], g[0])) |
                        e4m3x2_of_half2(h2_mul(v[4 * q + i][1], g[1])) << 16;
            turn4(w4, out, q);
        }
    }
    const int64_t r = r0 + warp * 32;
    const bool wide = reinterpret_cast<uintptr_t>(a.out_codes) % 32 == 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int kk = 4 * lane + c;
        const int64_t k = k0 + kk;
        if (k < a.K && r < padded) {
            const uint4 two[2] = {make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]),
                                  make_uint4(out[c][4], out[c][5], out[c][6], out[c][7])};
            store_pair(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out_codes) + k * padded + r),
                       true, wide, two);
            reinterpret_cast<uint8_t*>(scale_out)[(kk & 31) * 16 + (kk >> 5) * 4 + warp] =
                static_cast<uint8_t>(bytes[c]);
        }
    }
    __syncthreads();
    static_cast<uint32_t*>(a.out_scales)[(tk * tiles_r + tr) * 128 + t] = scale_out[t];
}

// ---------------------------------------------------------------------------
// the gradient of an activation
// ---------------------------------------------------------------------------

// An item is 128 rows of one batch by 128 columns; sixteen lanes a row, eight columns each, so that a
// thread's columns stay the same and their sums are in registers.  The rows of a batch are counted from
// its first, so a batch's sums do not depend on what stands before it.
//
// With an activation the instructions bound it: a derivative worked out for every value made it 72 us
// at 4216 x 16384 with the tanh form of GELU and 92 with the exact one.  But a scale has 256 values only,
// so persistent CTAs, four to an SM, work out the derivatives of the kRows scales 2^-16 ... 2^3 (blocks
// whose largest is between 0.004 and 3584) once, by the same function, while the kernel before them
// ends, and look them up; four rows of a warp with a block under any other scale work out their own.
// Faster at all sizes: 5.1 against 6.0 us at 77 x 4096, 19.3 against 20.9 at 4216 x 4096, 57.7 against
// 67.0 at 4096 x 16384.  With a gate whose gradient is taken as well there would be two values to look
// up: 134 us, against 80 of working them out.
//
// Now at 4216 x 16384: 56 us (GELU's tanh form; 54 the exact one; HBM's time 41), without an activation
// 39 (z is not read: 31), with a gate and its gradient 63 (41), with both 80.  Some 18 instructions a
// value are issued, a fourth of them for an item's start and its sums.  Rows copied ahead to shared
// memory: 76 us (tanh form), by TMA 78.
constexpr int kRows = 20, kFirstByte = 127 - 16;

struct ActWalk {
    FastDiv tiles, chunks;  // items: [batch][chunk][tile]
};

__device__ __forceinline__ float table_value(uint32_t address)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(address));
    return v;
}

// (a call of its own: the registers of the rows that look theirs up are theirs)
template <int ACT>
__device__ __noinline__ u64 slope_apart(u64 z)
{
    u64 unused;
    return slope2<ACT>(z, unused);
}

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, GATED && ACT != kActNone ? 3 : 4)
    activation_backward_kernel(const Mxfp8ActBwdArgs a, ActWalk walk, int items, int parts)
{
    constexpr bool TABLE = ACT != kActNone && !GATED;
    extern __shared__ uint8_t dynamic[];
    __shared__ float sums[2][kThreads / 32][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = threadIdx.x & 15, hw = threadIdx.x >> 4;
    // [kRows][256] derivatives, on a border of 1024 bytes
    const uint32_t table =
        (static_cast<uint32_t>(__cvta_generic_to_shared(dynamic)) + 1023u) & ~1023u;
    if (TABLE) {
        for (int i = threadIdx.x; i < kRows * 64; i += kThreads) {  // four neighbours at a time
            const uint32_t code = (i & 63) * 0x04040404u + 0x03020100u;
            const float scale = mx8_scale(kFirstByte + (i >> 6));
            u64 z[2], unused;
            e4m3x4_values(code, z[0], z[1]);
            float4 v;
            f2_unpack(slope2<ACT>(f2_mul(z[0], f2_splat(scale)), unused), v.x, v.y);
            f2_unpack(slope2<ACT>(f2_mul(z[1], f2_splat(scale)), unused), v.z, v.w);
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                         :
                         : "r"(table + i * 16), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                         : "memory");
        }
        __syncthreads();
    }
    grid_dependency_sync();
    const int tiles = static_cast<int>((a.N + 127) / 128), N = static_cast<int>(a.N);
    const int64_t M = a.B * a.S;
    const uint32_t* __restrict__ z_scales = static_cast<const uint32_t*>(a.z_scales);
    uint8_t* grad_scales = static_cast<uint8_t*>(a.grad_z_scales);
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t unit = walk.tiles.div(item), tile = item - unit * tiles;
        const uint32_t batch = walk.chunks.div(unit), chunk = unit - batch * walk.chunks.d;
        const int64_t n = static_cast<int64_t>(tile) * 128 + sub * 8;
        const int64_t begin = batch * a.S + static_cast<int64_t>(chunk) * 128;
        const int64_t end = min(begin + 128, (batch + int64_t{1}) * a.S);
        // all rows of a row tile are this CTA's: its scales are stored four rows at a time
        const bool whole = begin % 128 == 0 && (end == begin + 128 || end == M);
        const bool has = n < a.N;
        const uint8_t* __restrict__ z = static_cast<const uint8_t*>(a.z) + begin * N + n;
        const T* __restrict__ grad = static_cast<const T*>(a.grad_out) + begin * N + n;
        uint8_t* grad_z = static_cast<uint8_t*>(a.grad_z) + begin * N + n;
        const int rows = static_cast<int>(end - begin), live = has ? rows : 0;  // (m * N is under 2^27)
        const bool partial = rows < 128;
        u64 gate[4], sb[4], sg[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gate[j] = f2_splat(1.0f);
            sb[j] = sg[j] = 0ull;
        }
        if (GATED && has) {
            const uint4 g = ld_cached(reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.gate) + batch * a.gate_bstride + n));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                gate[j] = widen<T>(word(g, j));
        }
#pragma unroll 1
        for (int i0 = 0; i0 < 2; ++i0) {
            const int r = hw + 16 * i0;
            uint2 c[4];
            uint4 g[4];
            uint32_t e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = r + 32 * i;
                c[i] = make_uint2(0u, 0u);
                g[i] = make_uint4(0u, 0u, 0u, 0u);
                e[i] = 0x7F7F7F7Fu;
                if (m < live) {
                    c[i] = ld_stream2(reinterpret_cast<const uint2*>(z + m * N));
                    g[i] = ld_stream(reinterpret_cast<const uint4*>(grad + m * N));
                }
            }
            if (whole) {
                const uint4 w = ld_cached(reinterpret_cast<const uint4*>(z_scales) +
                                          (begin / 128 * tiles + tile) * 32 + r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + 32 * i < live)
                        e[i] = word(w, i);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + 32 * i < live)
                        e[i] = ld_cached(z_scales +
                                     mx8_scale_at(begin + r + 32 * i, tile * 4, tiles) / 4);
            }
            uint32_t mine = 0u;  // the scale byte of row r + 32 * (sub % 4), which this lane stores
            const auto finish = [&](int i, u64(&d)[4]) {
                const int m = r + 32 * i;
                // rows that there are not: 0 * gate is NaN under a gate that is not finite
                if (GATED && partial && m >= live)
                    d[0] = d[1] = d[2] = d[3] = 0ull;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sb[j] = f2_add(sb[j], d[j]);
                uint32_t out[2];
                const uint32_t byte = quantize_pairs<4, 4>(d, out);
                mine = (sub & 3) == i ? byte : mine;
                if (m < live)
                    *reinterpret_cast<uint2*>(grad_z + m * N) = make_uint2(out[0], out[1]);
            };
            bool near = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = (e[i] >> (8 * (sub >> 2))) & 0xFFu;
                near = near && e[i] - kFirstByte < kRows;
            }
            if (TABLE && __all_sync(kFullMask, near)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t row = table + (e[i] - kFirstByte) * 1024;
                    u64 d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t two = j < 2 ? c[i].x : c[i].y;
                        const uint32_t lo = (j & 1) ? two >> 14 : two << 2;
                        const uint32_t hi = (j & 1) ? two >> 22 : two >> 6;
                        d[j] = f2_mul(widen<T>(word(g[i], j)),
                                      f2_pack(table_value((lo & 0x3FCu) | row),
                                              table_value((hi & 0x3FCu) | row)));
                    }
                    finish(i, d);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // Past 2^32 the derivative is 1 or 0 all the same, and so is act(z) / z: such a z
                    // is taken down to there, and only act(z) has the rest of its scale.
                    const bool far = ACT != kActNone && e[i] > 159u && e[i] != 255u;
                    const float scale = mx8_scale(far ? 159u : e[i]);
                    const u64 rest = f2_splat(far ? mx8_scale(e[i] - 32u) : 1.0f);
                    u64 f[4], d[4];
                    if (ACT != kActNone || GATED)
                        values8(c[i], scale, f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u64 go = widen<T>(word(g[i], j));
                        u64 part;
                        d[j] = ACT == kActNone ? go
                               : TABLE         ? f2_mul(go, slope_apart<ACT>(f[j]))
                                               : f2_mul(go, slope2<ACT>(f[j], part));
                        if (GATED) {
                            d[j] = f2_mul(d[j], gate[j]);
                            if (parts & 2)
                                sg[j] = ACT == kActNone
                                            ? f2_fma(go, f[j], sg[j])
                                            : f2_fma(f2_mul(go, f2_mul(f[j], part)), rest, sg[j]);
                        }
                    }
                    finish(i, d);
                }
            }
            const int m = r + 32 * (sub & 3);
            if (whole || m < rows)
                grad_scales[mx8_scale_at(begin + m, tile * 4 + (sub >> 2), tiles)] =
                    static_cast<uint8_t>(mine);
        }
        if (!whole && end == M)  // rows behind the last one
            for (int64_t m = M + threadIdx.x; m < (M + 127) / 128 * 128; m += kThreads)
                reinterpret_cast<uint32_t*>(grad_scales)[mx8_scale_at(m, tile * 4, tiles) / 4] = 0u;
        if (!parts)
            continue;
        __syncthreads();  // the last item's sums have been read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4 v;
            f2_unpack(sb[j], v.x, v.y);
            f2_unpack(sg[j], v.z, v.w);
            v.x = __fadd_rn(v.x, __shfl_xor_sync(kFullMask, v.x, 16));
            v.y = __fadd_rn(v.y, __shfl_xor_sync(kFullMask, v.y, 16));
            if (GATED) {
                v.z = __fadd_rn(v.z, __shfl_xor_sync(kFullMask, v.z, 16));
                v.w = __fadd_rn(v.w, __shfl_xor_sync(kFullMask, v.w, 16));
            }
            if (lane < 16) {
                *reinterpret_cast<float2*>(&sums[0][warp][sub * 8 + 2 * j]) = make_float2(v.x, v.y);
                if (GATED)
                    *reinterpret_cast<float2*>(&sums[1][warp][sub * 8 + 2 * j]) =
                        make_float2(v.z, v.w);
            }
        }
        __syncthreads();
        const int part = threadIdx.x >> 7, col = threadIdx.x & 127;
        // parts: bit 0 the bias's sums, bit 1 the gate's
        if ((parts >> part & 1) && tile * 128 + col < N) {
            float v = sums[part][0][col];
#pragma unroll
            for (int k = 1; k < kThreads / 32; ++k)
                v = __fadd_rn(v, sums[part][k][col]);
            const int each = parts == 3 ? 2 : 1;
            a.partials[(static_cast<int64_t>(unit) * each + (parts == 3 ? part : 0)) * N +
                       tile * 128 + col] = v;
        }
    }
}

// Sums of the chunks' parts: those of all batches for the bias, of one for a row of the gate's
// gradient; eight warps take every eighth, 128 columns a CTA.
__global__ void __launch_bounds__(kThreads)
    activation_columns_kernel(const Mxfp8ActBwdArgs a, int64_t chunks, int64_t batches, int parts)
{
    __shared__ float4 join[kThreads / 32][32];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tiles = (a.N + 127) / 128;
    const int64_t which = blockIdx.x / tiles;
    const bool bias = which == 0 && a.grad_bias;
    const int64_t slice = which - (a.grad_bias ? 1 : 0);  // of the gate's gradient
    const int each = parts == 3 ? 2 : 1, part = parts == 3 && !bias ? 1 : 0;
    const int64_t first = bias ? 0 : slice * chunks;
    const int64_t count = bias ? batches * chunks : chunks;
    const int64_t n = (blockIdx.x - which * tiles) * 128 + lane * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n < a.N)
        for (int64_t i = warp; i < count; i += kThreads / 32) {
            const float4 p = *reinterpret_cast<const float4*>(
                a.partials + ((first + i) * each + part) * a.N + n);
            s = make_float4(__fadd_rn(s.x, p.x), __fadd_rn(s.y, p.y), __fadd_rn(s.z, p.z),
                            __fadd_rn(s.w, p.w));
        }
    join[warp][lane] = s;
    __syncthreads();
    if (warp || n >= a.N)
        return;
#pragma unroll
    for (int k = 1; k < kThreads / 32; ++k) {
        const float4 p = join[k][lane];
        s = make_float4(__fadd_rn(s.x, p.x), __fadd_rn(s.y, p.y), __fadd_rn(s.z, p.z),
                        __fadd_rn(s.w, p.w));
    }
    *reinterpret_cast<float4*>((bias ? a.grad_bias : a.grad_gate + slice * a.N) + n) = s;
}

// Batches as the sums see them: one where no gate tells them apart.
int64_t sum_batches(int64_t B, bool per_batch) { return per_batch ? B : 1; }

int64_t sum_chunks(int64_t B, int64_t S, bool per_batch)
{
    return ((per_batch ? S : B * S) + 127) / 128;
}

template <typename T, int ACT>
cudaError_t launch_activation(const Mxfp8ActBwdArgs& a, int items, ActWalk walk, int parts,
                              const DeviceInfo& dev, cudaStream_t stream)
{
    if (a.gate)
        return launch_dependent(activation_backward_kernel<T, ACT, true>, items, kThreads, 0, stream,
                                a, walk, items, parts);
    const int resident = 4 * dev.sms;
    return ACT == kActNone
               ? launch_dependent(activation_backward_kernel<T, ACT, false>, items, kThreads, 0,
                                  stream, a, walk, items, parts)
               : launch_dependent(activation_backward_kernel<T, ACT, false>,
                                  items < resident ? items : resident, kThreads, kRows * 1024 + 1024,
                                  stream, a, walk, items, parts);
}

template <typename T>
cudaError_t launch_activation(const Mxfp8ActBwdArgs& a, int items, ActWalk walk, int parts,
                              const DeviceInfo& dev, cudaStream_t stream)
{
    switch (a.activation) {
    case kActSilu:
        return launch_activation<T, kActSilu>(a, items, walk, parts, dev, stream);
    case kActGelu:
        return launch_activation<T, kActGelu>(a, items, walk, parts, dev, stream);
    case kActGeluTanh:
        return launch_activation<T, kActGeluTanh>(a, items, walk, parts, dev, stream);
    default:
        return launch_activation<T, kActNone>(a, items, walk, parts, dev, stream);
    }
}

}  // namespace

cudaError_t launch_mxfp8_rows(bool quantize, const Mxfp8RowsArgs& a, cudaStream_t stream)
{
    const uint32_t units = a.rows_padded / 4 * a.by_tiles.d;
    const int grid = static_cast<int>((units + kUnitsPerCta - 1) / kUnitsPerCta);
    if (quantize)
        return launch_dependent(a.f16 ? quantize8_kernel<__half> : quantize8_kernel<__nv_bfloat16>,
                                grid, kThreads, 0, stream, a);
    return launch_dependent(a.f16 ? dequantize8_kernel<__half> : dequantize8_kernel<__nv_bfloat16>,
                            grid, kThreads, 0, stream, a);
}

cudaError_t launch_mxfp8_transpose(const Mxfp8TransposeArgs& a, cudaStream_t stream)
{
    const int64_t tiles = (a.K + 127) / 128 * ((a.rows + 127) / 128);
    if (tiles > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_dependent(transpose8_kernel, static_cast<int>(tiles), kTurn, 0, stream, a);
}

size_t mxfp8_activation_backward_workspace_bytes(int64_t B, int64_t S, int64_t N, bool per_batch,
                                                 int parts)
{
    return static_cast<size_t>(sum_batches(B, per_batch) * sum_chunks(B, S, per_batch) * parts * N) *
           4;
}

cudaError_t launch_mxfp8_activation_backward(const Mxfp8ActBwdArgs& args, const DeviceInfo& dev,
                                             cudaStream_t stream)
{
    Mxfp8ActBwdArgs a = args;
    const bool per_batch = a.gate && a.gate_bstride != 0;
    if (!per_batch) {
        a.S *= a.B;
        a.B = 1;
    }
    const int64_t chunks = (a.S + 127) / 128, tiles = (a.N + 127) / 128;
    const int parts = (a.grad_bias ? 1 : 0) + (a.grad_gate ? 2 : 0);
    if (a.B * chunks * tiles > INT32_MAX - 4 * dev.sms)
        return cudaErrorInvalidValue;
    const int items = static_cast<int>(a.B * chunks * tiles);
    const ActWalk walk{FastDiv::make(static_cast<uint32_t>(tiles)),
                       FastDiv::make(static_cast<uint32_t>(chunks))};
    const cudaError_t e = a.f16
                              ? launch_activation<__half>(a, items, walk, parts, dev, stream)
                              : launch_activation<__nv_bfloat16>(a, items, walk, parts, dev, stream);
    if (e != cudaSuccess || !parts)
        return e;
    const int64_t slices = (a.grad_bias ? 1 : 0) + (a.grad_gate ? a.B : 0);
    if (slices * tiles > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_dependent(activation_columns_kernel, static_cast<int>(slices * tiles), kThreads, 0,
                            stream, a, chunks, a.B, parts);
}

}  // namespace rmsmod
