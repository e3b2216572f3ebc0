// The product of two microscaled 8-bit matrices on the block-scaled tensor core instructions
// (tcgen05.mma, kind::mxf8f6f4), with a projection's epilogue:
//   acc[m, n] = sum_k a[m, k] * b[n, k]          (fp32 accumulators in tensor memory)
//   z = acc + bias;  y = residual + gate_b * act(z)
// y is stored with one rounding, to the type of bias, gate and residual or to 8-bit blocks along n;
// z, for the backward pass, to 8-bit blocks.
//
// Operand tiles are 128 values (128 bytes) of every row, brought by TMA (128-byte swizzle), with one
// scale tile for each 128 rows; one thread copies the scales to tensor memory and starts four
// products of 32 values.
//
// pair_kernel (more than 128 rows of a): two CTAs of a cluster share a 256 x BN tile
// (cta_group::2), each with its 128 rows of a and half of b's rows.  Persistent, with two
// accumulators: eight warps finish one tile's rows while the next tile's products run.  A thread of
// theirs holds 32 columns of a row at a time, which are one block: quantising needs no other thread.
// 4216 x 16384 x 4096 171-175 us (146 at twice the bf16 rate of a library product; the products alone,
// without copies or epilogue, 160 under the power limit), with the activation and two 8-bit results
// 177-188; 16384 x 4096 x 4224 to fp32 197-202, joined to a residual 232-238.
//
// few_kernel (up to 128 rows of a, where reading b is what counts): b's rows take the 128-row side of
// the instruction, a's rows the other.  A cluster of up to eight CTAs splits K, and joins its parts in
// the CTAs' order through distributed shared memory.  A warp's lanes are 32 columns: a block.
// 8 x 4096 x 4096 7.4 us (2.6 of HBM time: launch, first copies and join are the rest), 8 x 16384 x 4096
// 15 (10.2), 128 x 4096 x 4096 10.7.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp8.cuh"
#include "mxfp8.h"
#include "tensor_core.cuh"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

constexpr int kStepK = 128;       // values, and bytes, of a row per operand tile
constexpr int kTileBytes = 128 * kStepK;
constexpr int kScaleBytes = 512;  // an operand tile's scales of 128 rows
constexpr uint32_t kPairTmemCols = 512, kFewTmemCols = 256;

template <bool PAIR>
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
            "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
            "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
            : "memory");
}

// Instruction descriptor: e4m3 operands, e8m0 scales.
__host__ __device__ constexpr uint32_t instruction(int M, int N)
{
    return (static_cast<uint32_t>(N / 8) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M / 16) << 24);
}

// The products of one step of SUBS * 128 values: `parts` of 32 values each, four to an operand tile
// (b's are b_tile bytes apart), whose scales are copied before them: a tile of four blocks for each
// 128 rows.  A product takes one of a column's four scales.
template <bool PAIR, int B_TILES, int SUBS>
__device__ __forceinline__ void step_products(uint32_t acc, uint32_t sfa_col, uint32_t sfb_col,
                                              uint32_t sa, uint32_t sb, uint32_t b_tile,
                                              uint32_t sfa, uint32_t sfb, uint32_t idesc,
                                              int parts, bool first)
{
#pragma unroll
    for (int p = 0; p < 4 * SUBS; ++p)
        if (p < parts) {
            const int h = p >> 2;  // operand tile
            const uint32_t id = p & 3;
            if (id == 0) {
                copy_scales<PAIR>(sfa_col + h % 2 * 4, scale_desc(sfa + h * kScaleBytes));
#pragma unroll
                for (int i = 0; i < B_TILES; ++i)
                    copy_scales<PAIR>(sfb_col + h % 2 * (4 * B_TILES) + i * 4,
                                      scale_desc(sfb + (i * SUBS + h) * kScaleBytes));
            }
            mma_mxf8<PAIR>(acc, operand_desc(sa + h * kTileBytes + id * 32),
                           operand_desc(sb + h * b_tile + id * 32), idesc | (id << 4) | (id << 29),
                           sfa_col + h % 2 * 4, sfb_col + h % 2 * (4 * B_TILES), !first || p > 0);
        }
}

// Products (of 32 values) of step t.
template <int SUBS>
__device__ __forceinline__ int parts_of(int64_t K, int t)
{
    const int64_t left = K - static_cast<int64_t>(t) * (SUBS * kStepK);
    return left >= SUBS * kStepK ? 4 * SUBS : static_cast<int>(left / 32);
}

struct Maps {
    CUtensorMap a, a_scales, b, b_scales;
};

// The tiles in the pairs' order: groups of some twelve rows of tiles, whose columns come one after the
// other, so that the pairs that run at a time share few rows of a and of b (16384 x 4096 x 4224, 64 rows
// of tiles, 197 us; in one group, 213).
struct Raster {
    int tiles_m, tiles_n, group;

    __device__ __forceinline__ void at(int tile, int& m, int& n) const
    {
        const int per_group = group * tiles_n, g = tile / per_group, rest = tile - g * per_group;
        const int first = g * group, rows = tiles_m - first < group ? tiles_m - first : group;
        n = rest / rows;
        m = first + rest - n * rows;
    }
};

// ---------------------------------------------------------------------------
// the epilogue
// ---------------------------------------------------------------------------

// Eight values, exact in fp32.
template <typename T>
__device__ __forceinline__ void widen8(const uint4* v, u64 (&f)[4])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = f2_pack(__uint_as_float(word(v[i >> 1], i % 2 * 2)),
                           __uint_as_float(word(v[i >> 1], i % 2 * 2 + 1)));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = widen<T>(word(v[0], i));
    }
}

template <typename T>
__device__ __forceinline__ void narrow8(const u64* f, uint4* v)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(f[i], lo, hi);
            word(v[i >> 1], i % 2 * 2) = __float_as_uint(lo);
            word(v[i >> 1], i % 2 * 2 + 1) = __float_as_uint(hi);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            word(v[0], i) = narrow<T>(f[i]);
    }
}

template <int ACT>
__device__ __forceinline__ void activate32(u64 (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = activate2<ACT>(v[i]);
}

__device__ __forceinline__ void activate32(int act, u64 (&v)[16])
{
    switch (act) {
    case kActSilu:
        return activate32<kActSilu>(v);
    case kActGelu:
        return activate32<kActGelu>(v);
    case kActGeluTanh:
        return activate32<kActGeluTanh>(v);
    default:
        return;
    }
}

template <int ACT>
__device__ __forceinline__ void activate4(float (&v)[4])
{
    const u64 a = activate2<ACT>(f2_pack(v[0], v[1])), b = activate2<ACT>(f2_pack(v[2], v[3]));
    f2_unpack(a, v[0], v[1]);
    f2_unpack(b, v[2], v[3]);
}

__device__ __forceinline__ void activate4(int act, float (&v)[4])
{
    switch (act) {
    case kActSilu:
        return activate4<kActSilu>(v);
    case kActGelu:
        return activate4<kActGelu>(v);
    case kActGeluTanh:
        return activate4<kActGeluTanh>(v);
    default:
        return;
    }
}

// A block's codes at row m, column n of a matrix of N columns.
__device__ __forceinline__ void store_codes(void* codes, int64_t m, int64_t N, int64_t n,
                                            bool wide, const uint32_t (&c)[8])
{
    const uint4 two[2] = {make_uint4(c[0], c[1], c[2], c[3]), make_uint4(c[4], c[5], c[6], c[7])};
    store_pair(reinterpret_cast<uint4*>(static_cast<uint8_t*>(codes) + m * N + n), true, wide, two);
}

// ---------------------------------------------------------------------------
// more than 128 rows
// ---------------------------------------------------------------------------

// Two operand tiles to a step: the issuing thread waits and passes on half as often.
constexpr int kPairSubs = 2;

template <int BN>
struct Pair {
    static constexpr int kBBytes = BN / 2 * kStepK;  // of one operand tile
    static constexpr int kBTiles = BN / 128;
    static constexpr int kStageBytes =
        kPairSubs * (kTileBytes + kBBytes + kScaleBytes * (1 + kBTiles));
    static constexpr int kStages = (kSmemMax - 2048) / kStageBytes;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
    static constexpr int kAccs = 2;
    // Two accumulators of 256 columns and the scales are more than tensor memory's 512: the second
    // one begins in the last 32 columns of the first, which the epilogue reads before the others.
    static constexpr bool kOverlap = BN == 256;
    static constexpr uint32_t kAccStep = kOverlap ? BN - 32 : BN;
    static constexpr uint32_t kSfaCol = kAccStep + BN;
    static constexpr uint32_t kSfbCol = kSfaCol + 8;
    static constexpr int kCols = BN / 2;  // of an accumulator row in one epilogue thread
    static_assert(kSfbCol + 8 * kBTiles <= kPairTmemCols, "tensor memory");
    static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

constexpr int kEpilogueWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpilogueWarps;  // producer, issuer, epilogue

// The scale bytes of a thread's blocks of one row (two or four neighbours of a tile); zeros for rows
// and blocks that the matrix does not have.
template <int COLS>
__device__ __forceinline__ void store_scales(void* scales, int64_t m, int64_t M, int64_t n,
                                             int64_t N, uint32_t bytes)
{
    if (m >= (M + 127) / 128 * 128 || n >= (N + 127) / 128 * 128)
        return;
    uint8_t* at = static_cast<uint8_t*>(scales) + mx8_scale_at(m, n / 32, (N + 127) / 128);
    if (COLS == 128)
        *reinterpret_cast<uint32_t*>(at) = m < M ? bytes : 0u;
    else
        *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(m < M ? bytes : 0u);
}

template <typename T, int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const Mxfp8MatmulArgs a, const __grid_constant__ Maps maps, const Raster raster)
{
    using P = Pair<BN>;
    constexpr int kVecs = sizeof(T) / 2;  // 16-byte vectors of eight columns
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) unsigned long long full[P::kStages], empty[P::kStages];
    __shared__ __align__(8) unsigned long long acc_full[P::kAccs], acc_empty[P::kAccs], shared_read;
    __shared__ uint32_t tmem_base;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    const int steps = static_cast<int>((a.K + kPairSubs * kStepK - 1) / (kPairSubs * kStepK));
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = raster.tiles_m * raster.tiles_n;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P::kStages; ++s) {
            mbar_init(smem_addr(&full[s]), 1u);
            mbar_init(smem_addr(&empty[s]), 1u);
        }
        for (int s = 0; s < P::kAccs; ++s) {
            mbar_init(smem_addr(&acc_full[s]), 1u);
            mbar_init(smem_addr(&acc_empty[s]), 2u * kEpilogueWarps);
        }
        mbar_init(smem_addr(&shared_read), kEpilogueWarps);  // half of the warps of each CTA
        mbar_init_fence();
    }
    if (warp == 1)
        tmem_alloc<true, kPairTmemCols>(smem_addr(&tmem_base));
    before_sync();
    cluster_barrier();
    after_sync();
    grid_dependency_sync();
    const uint32_t tmem = tmem_base;

    bool broken = false;
    auto gave_up = [&](bool ok) {
        if (!ok && !broken) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
    };

    if (warp == 0) {
        if (elect_one()) {
            // both CTAs' copies are counted on the first one's barriers
            const int block_tiles = static_cast<int>((a.K + 127) / 128);
            int s = 0;
            uint32_t phase = 1;
            for (int tile = pair; tile < tiles; tile += pairs) {
                int m0, n0;
                raster.at(tile, m0, n0);
                m0 = m0 * 256 + static_cast<int>(rank) * 128;
                n0 *= BN;
                for (int t = 0; t < steps; ++t) {
                    if (!broken)
                        gave_up(step_wait(smem_addr(&empty[s]), phase));
                    const uint32_t bar = in_cta(smem_addr(&full[s]), 0);
                    const uint32_t dst = ring + s * P::kStageBytes;
                    if (rank == 0)
                        mbar_expect_tx(smem_addr(&full[s]), 2 * P::kStageBytes);
                    // (operand tiles past K: zeros, which nothing reads)
#pragma unroll
                    for (int h = 0; h < kPairSubs; ++h) {
                        const int x = (kPairSubs * t + h) * kStepK;
                        tma_box<true>(dst + h * kTileBytes, &maps.a, x, m0, bar);
                        tma_box<true>(dst + kPairSubs * kTileBytes + h * P::kBBytes, &maps.b, x,
                                      n0 + static_cast<int>(rank) * (BN / 2), bar);
                    }
                    const uint32_t sf = dst + kPairSubs * (kTileBytes + P::kBBytes);
                    tma_box<true>(sf, &maps.a_scales, 0,
                                  2 * (m0 / 128 * block_tiles + kPairSubs * t), bar);
#pragma unroll
                    for (int i = 0; i < P::kBTiles; ++i)
                        tma_box<true>(sf + (1 + i) * kPairSubs * kScaleBytes, &maps.b_scales, 0,
                                      2 * ((n0 / 128 + i) * block_tiles + kPairSubs * t), bar);
                    if (++s == P::kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no arrival is left on its way when this CTA's shared memory goes
            for (int i = 0; i < P::kStages; ++i) {
                if (!broken)
                    gave_up(step_wait(smem_addr(&empty[s]), phase));
                if (++s == P::kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t kIdesc = instruction(256, BN);
            int s = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 1, read_phase = 1;
            for (int tile = pair; tile < tiles; tile += pairs) {
                if (!broken)
                    gave_up(step_wait(smem_addr(&acc_empty[acc]), acc_phase));
                if (P::kOverlap) {  // the last tile's part of the columns that both have
                    if (!broken)
                        gave_up(step_wait(smem_addr(&shared_read), read_phase));
                    read_phase ^= 1u;
                }
                after_sync();
                for (int t = 0; t < steps; ++t) {
                    if (!broken)
                        gave_up(step_wait(smem_addr(&full[s]), phase));
                    after_sync();
                    const uint32_t sa = ring + s * P::kStageBytes;
                    const uint32_t sb = sa + kPairSubs * kTileBytes;
                    const uint32_t sfa = sb + kPairSubs * P::kBBytes;
                    step_products<true, P::kBTiles, kPairSubs>(
                        tmem + acc * P::kAccStep, tmem + P::kSfaCol, tmem + P::kSfbCol, sa, sb,
                        P::kBBytes, sfa, sfa + kPairSubs * kScaleBytes, kIdesc,
                        parts_of<kPairSubs>(a.K, t), t == 0);
                    commit<true>(smem_addr(&empty[s]));
                    if (++s == P::kStages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                commit<true>(smem_addr(&acc_full[acc]));
                if (++acc == P::kAccs) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    } else {
        // a warp reads the 32 lanes of tensor memory that its index selects, half of the columns
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const T* __restrict__ bias = static_cast<const T*>(a.bias);
        const T* __restrict__ gate = static_cast<const T*>(a.gate);
        const T* __restrict__ residual = static_cast<const T*>(a.residual);
        int acc = 0;
        uint32_t phase = 0;
        for (int tile = pair; tile < tiles; tile += pairs) {
            if (!broken)
                gave_up(step_wait(smem_addr(&acc_full[acc]), phase));
            int tile_m, tile_n;
            raster.at(tile, tile_m, tile_n);
            const int64_t m = static_cast<int64_t>(tile_m) * 256 + rank * 128 + quarter * 32 + lane;
            const int64_t n0 = static_cast<int64_t>(tile_n) * BN + half * P::kCols;
            const T* gate_b = gate && m < a.M ? gate + m / a.S * a.gate_bstride : gate;
            const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                  acc * P::kAccStep + half * P::kCols;
            uint32_t out_bytes = 0, keep_bytes = 0;
            // 32 columns at a time, from the side that the other accumulator has too
            const bool shares = P::kOverlap && half != acc;
#pragma unroll 1
            for (int k0 = 0; k0 < P::kCols / 32; ++k0) {
                const int c = P::kOverlap && acc == 0 ? P::kCols / 32 - 1 - k0 : k0;
                uint32_t acc_bits[32];
                __syncwarp();
                after_sync();
                tmem_load32(from + 32 * c, acc_bits);
                // the residual, on its way meanwhile
                const int64_t n = n0 + 32 * c;
                uint4 rv[4 * kVecs];
                if (residual && m < a.M) {
                    const uint4* r = reinterpret_cast<const uint4*>(residual + m * a.N + n);
#pragma unroll
                    for (int k = 0; k < 4 * kVecs; k += 2)
                        if (n + k * (8 / kVecs) < a.N)
                            load_pair(r + k, n + (k + 1) * (8 / kVecs) < a.N, a.wide, rv + k);
                }
                tmem_loads_done();
                if (k0 + 1 == P::kCols / 32 || (shares && k0 == 0)) {
                    before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (shares && k0 == 0)
                            arrive_remote(in_cta(smem_addr(&shared_read), 0));
                        if (k0 + 1 == P::kCols / 32)
                            arrive_remote(in_cta(smem_addr(&acc_empty[acc]), 0));
                    }
                }
                if (m >= a.M || n >= a.N)
                    continue;
                u64 v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = f2_pack(__uint_as_float(acc_bits[2 * i]),
                                   __uint_as_float(acc_bits[2 * i + 1]));
                if (bias)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n + 8 * k < a.N) {
                            uint4 q[kVecs];
                            u64 f[4];
#pragma unroll
                            for (int i = 0; i < kVecs; ++i)
                                q[i] = ld_cached(reinterpret_cast<const uint4*>(bias + n + 8 * k) + i);
                            widen8<T>(q, f);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[4 * k + i] = f2_add(v[4 * k + i], f[i]);
                        }
                uint32_t codes[8];
                if (a.keep) {
                    keep_bytes |= quantize_pairs<16, 1>(v, codes) << (8 * c);
                    store_codes(a.keep, m, a.N, n, a.wide, codes);
                }
                activate32(a.activation, v);
                if (gate)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n + 8 * k < a.N) {
                            uint4 q[kVecs];
                            u64 f[4];
#pragma unroll
                            for (int i = 0; i < kVecs; ++i)
                                q[i] = ld_cached(reinterpret_cast<const uint4*>(gate_b + n + 8 * k) + i);
                            widen8<T>(q, f);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[4 * k + i] = f2_mul(v[4 * k + i], f[i]);
                        }
                if (residual)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        u64 f[4];
                        widen8<T>(rv + k * kVecs, f);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[4 * k + i] = f2_add(v[4 * k + i], f[i]);
                    }
                if (a.out_scales) {
                    out_bytes |= quantize_pairs<16, 1>(v, codes) << (8 * c);
                    store_codes(a.out, m, a.N, n, a.wide, codes);
                    continue;
                }
                uint4 o[4 * kVecs];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    narrow8<T>(v + 4 * k, o + k * kVecs);
                uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + m * a.N + n);
#pragma unroll
                for (int k = 0; k < 4 * kVecs; k += 2)
                    if (n + k * (8 / kVecs) < a.N) {
                        const uint4 two[2] = {o[k], o[k + 1]};
                        store_pair(to + k, n + (k + 1) * (8 / kVecs) < a.N, a.wide, two);
                    }
            }
            if (a.keep)
                store_scales<P::kCols>(a.keep_scales, m, a.M, n0, a.N, keep_bytes);
            if (a.out_scales)
                store_scales<P::kCols>(a.out_scales, m, a.M, n0, a.N, out_bytes);
            if (++acc == P::kAccs) {
                acc = 0;
                phase ^= 1u;
            }
        }
    }
    // after a timeout: a bounded pause for the copies still in flight
    if (broken)
        drain_pause();
    before_sync();
    cluster_barrier();
    after_sync();
    if (warp == 1)
        tmem_free<true, kPairTmemCols>(tmem);
}

// ---------------------------------------------------------------------------
// up to 128 rows
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 320;  // eight epilogue warps, producer, issuer
constexpr int kFewMaxStages = 10;
constexpr uint32_t kFewSfwCol = 128;            // accumulators in columns 0..127
constexpr uint32_t kFewSfxCol = kFewSfwCol + 8;

struct Few {
    int NX;           // a's rows as the instruction takes them: 16, 32, 64 or 128
    int stages;
    int stage_bytes;
    int split;        // CTAs of a cluster, each with a range of the steps
};

// Sums over the cluster's SPLIT parts, in their order, of four rows (the last one again past M).
template <int SPLIT>
__device__ __forceinline__ void join4(float (&v)[4], uint32_t at, int m0, int step, int M)
{
    float p[4][SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
        const uint32_t from = in_cta(at, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(p[i][k])
                         : "r"(from + min(m0 + i * step, M - 1) * 512));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = p[i][0];
#pragma unroll
        for (int k = 1; k < SPLIT; ++k)
            v[i] = __fadd_rn(v[i], p[i][k]);
    }
}

// Rows of a that come in 16 bits (RAW, up to kMxfp8DirectRows of them): the operand tile and scales of
// step t, as quantisation and the copies would have laid them.  One warp; sixteen lanes a row.
template <typename T>
__device__ __forceinline__ void quantize_step(const Mxfp8MatmulArgs& a, int NX, int t, uint32_t tile,
                                              uint32_t scales)
{
    const int lane = threadIdx.x & 31, sub = lane & 15;
    const int64_t k = static_cast<int64_t>(t) * kStepK + sub * 8;
    const T* x = static_cast<const T*>(a.a);
#pragma unroll 1
    for (int r0 = 0; r0 < NX; r0 += 16) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 2 * i + (lane >> 4);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < a.M && k < a.K)
                v[i] = ld_stream(reinterpret_cast<const uint4*>(x + r * a.K + k));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 2 * i + (lane >> 4);
            u64 f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = widen<T>(word(v[i], j));
            uint32_t o[2];
            uint32_t w = quantize_pairs<4, 4>(f, o) << (2 * (lane & 12));
            w |= __shfl_xor_sync(kFullMask, w, 4);
            w |= __shfl_xor_sync(kFullMask, w, 8);
            // rows of 128 bytes, whose 16-byte chunks are swizzled by the row
            const uint32_t at = tile + r * kStepK + (((sub >> 1) ^ (r & 7)) << 4) + (sub & 1) * 8;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(o[0]), "r"(o[1])
                         : "memory");
            if (sub == 0)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(scales + r * 16), "r"(w) : "memory");
        }
    }
    fence_proxy_async();
}

template <typename T, bool RAW>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const Mxfp8MatmulArgs a, const __grid_constant__ Maps maps, const Few f)
{
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) unsigned long long full[kFewMaxStages], empty[kFewMaxStages], done;
    __shared__ uint32_t tmem_base;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t rank = f.split > 1 ? cluster_rank() : 0u;
    const int n0 = static_cast<int>(blockIdx.x) / f.split * 128;
    const int all = static_cast<int>((a.K + kStepK - 1) / kStepK);
    const int begin = static_cast<int>(static_cast<int64_t>(all) * rank / f.split);
    const int end = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / f.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < f.stages; ++s) {
            mbar_init(smem_addr(&full[s]), RAW ? 2u : 1u);
            mbar_init(smem_addr(&empty[s]), 1u);
        }
        mbar_init(smem_addr(&done), 1u);
        mbar_init_fence();
    }
    if (warp == 9)
        tmem_alloc<false, kFewTmemCols>(smem_addr(&tmem_base));
    before_sync();
    __syncthreads();
    after_sync();
    grid_dependency_sync();
    const uint32_t tmem = tmem_base;

    bool broken = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!broken && !mbar_wait(bar, parity, kWaitLimitNs)) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
    };

    if (warp == 8) {
        if (elect_one()) {
            const int block_tiles = static_cast<int>((a.K + 127) / 128);
            int s = 0;
            uint32_t phase = 1;
            for (int t = begin; t < end; ++t) {
                wait(smem_addr(&empty[s]), phase);
                const uint32_t bar = smem_addr(&full[s]);
                const uint32_t dst = ring + s * f.stage_bytes;
                mbar_expect_tx(bar, RAW ? kTileBytes + kScaleBytes : f.stage_bytes);
                tma_box<false>(dst, &maps.b, t * kStepK, n0, bar);
                tma_box<false>(dst + kTileBytes, &maps.b_scales, 0,
                               2 * (n0 / 128 * block_tiles + t), bar);
                if (!RAW) {
                    tma_box<false>(dst + kTileBytes + kScaleBytes, &maps.a_scales, 0, 2 * t, bar);
                    tma_box<false>(dst + kTileBytes + 2 * kScaleBytes, &maps.a, t * kStepK, 0, bar);
                }
                if (++s == f.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 9) {
        if (elect_one()) {
            const uint32_t idesc = instruction(128, f.NX);
            int s = 0;
            uint32_t phase = 0;
            for (int t = begin; t < end; ++t) {
                wait(smem_addr(&full[s]), phase);
                after_sync();
                const uint32_t sw = ring + s * f.stage_bytes, sfw = sw + kTileBytes;
                step_products<false, 1, 1>(tmem, tmem + kFewSfwCol, tmem + kFewSfxCol, sw,
                                           sfw + 2 * kScaleBytes, 0u, sfw, sfw + kScaleBytes, idesc,
                                           parts_of<1>(a.K, t), t == begin);
                commit<false>(smem_addr(&empty[s]));
                if (++s == f.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            commit<false>(smem_addr(&done));
        }
    } else if (RAW) {
        // the warps that finish the rows later: each takes every eighth step
        for (int i = warp; i < end - begin; i += 8) {
            const int s = i % f.stages;
            wait(smem_addr(&empty[s]), (i / f.stages & 1) ^ 1);
            const uint32_t sx = ring + s * f.stage_bytes + kTileBytes + kScaleBytes;
            if constexpr (sizeof(T) == 2)
                quantize_step<T>(a, f.NX, begin + i, sx + kScaleBytes, sx);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&full[s]));
        }
    }
    // ---- lane n of tensor memory, column m: to shared memory, sixteen columns at a time, dealt to the
    // two warps that see a lane
    const int quarter = warp & 3, half = warp >> 2;
    const int n_in = quarter * 32 + lane;
    const int64_t n = n0 + n_in;
    const bool epilogue = warp < 8, has = epilogue && n < a.N;
    const T* bias = static_cast<const T*>(a.bias);
    const T* gate = static_cast<const T*>(a.gate);
    const T* residual = static_cast<const T*>(a.residual);
    const int M = static_cast<int>(a.M), S = static_cast<int>(a.S);
    const float bias_n = has && bias ? static_cast<float>(bias[n]) : 0.0f;
    // scale bytes of rows that the matrix does not have
    if (epilogue && half == 0 && rank == 0)
        for (void* scales : {a.keep ? a.keep_scales : nullptr, a.out_scales})
            if (scales && n_in >= M)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(scales) + n0 / 128 * 512ll +
                                             n_in % 32 * 16 + n_in / 32 * 4) = 0u;
    float* part = reinterpret_cast<float*>(raw + (ring - smem_addr(raw)));  // [m][128]
    if (epilogue) {
        wait(smem_addr(&done), 0);
        __syncwarp();
        after_sync();
        for (int c = half * 16; c < M; c += 32) {
            uint32_t v[16];
            tmem_load16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, v);
            tmem_loads_done();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                part[(c + j) * 128 + n_in] = __uint_as_float(v[j]);
        }
        before_sync();
    }
    if (broken)
        drain_pause();
    if (f.split > 1)
        cluster_barrier();
    else
        __syncthreads();
    if (epilogue) {
        const int64_t scale_tile = static_cast<int64_t>(n0 / 128) * 512 + quarter;
        // a warp's 32 values of row m as a block
        auto block = [&](void* codes, void* scales, int m, float v) {
            float inverse;
            const uint32_t byte =
                mx8_scale_byte(__reduce_max_sync(kFullMask, magnitude_bits(v)), inverse);
            const uint32_t code = e4m3_code(__fmul_rn(v, inverse));
            if (has)
                static_cast<uint8_t*>(codes)[m * a.N + n] = static_cast<uint8_t>(code);
            if (lane == 0)
                static_cast<uint8_t*>(scales)[scale_tile + m % 32 * 16 + m / 32 * 4] =
                    static_cast<uint8_t>(has ? byte : 0u);
        };
        // this CTA's rows of a, four at a time (all their loads on the way at once), the parts of K in
        // order
        const uint32_t at = smem_addr(part) + n_in * 4;
        const int step = 2 * f.split;
#pragma unroll 1
        for (int m0 = static_cast<int>(rank) * 2 + half; m0 < M; m0 += 4 * step) {
            float g[4], r[4], v[4];
            if (gate)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = min(m0 + i * step, M - 1);
                    g[i] = has ? static_cast<float>(gate[m / S * a.gate_bstride + n]) : 0.0f;
                }
            if (residual)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = min(m0 + i * step, M - 1);
                    r[i] = has ? static_cast<float>(residual[m * a.N + n]) : 0.0f;
                }
            switch (f.split) {
            case 1:
                join4<1>(v, at, m0, step, M);
                break;
            case 2:
                join4<2>(v, at, m0, step, M);
                break;
            case 4:
                join4<4>(v, at, m0, step, M);
                break;
            default:
                join4<8>(v, at, m0, step, M);
            }
            if (bias)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = __fadd_rn(v[i], bias_n);
            if (a.keep)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (m0 + i * step < M)
                        block(a.keep, a.keep_scales, m0 + i * step, v[i]);
            activate4(a.activation, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + i * step;
                if (m >= M)
                    continue;
                if (gate)
                    v[i] = __fmul_rn(v[i], g[i]);
                if (residual)
                    v[i] = __fadd_rn(v[i], r[i]);
                if (a.out_scales)
                    block(a.out, a.out_scales, m, v[i]);
                else if (has)
                    static_cast<T*>(a.out)[m * a.N + n] = static_cast<T>(v[i]);
            }
        }
    }
    if (f.split > 1)
        cluster_barrier();
    else
        __syncthreads();
    if (warp == 9) {
        after_sync();
        tmem_free<false, kFewTmemCols>(tmem);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// An 8-bit matrix: its codes in boxes of `box_rows` rows, and its scale tiles as rows of 256 bytes, in
// boxes of the tiles of `subs` * 128 values.
cudaError_t matrix_maps(CUtensorMap& codes, CUtensorMap& scales, const void* p, const void* sp,
                        int64_t rows, int64_t K, int box_rows, int subs)
{
    const cudaError_t e = bytes_map(codes, p, rows, K, kStepK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (rows + 127) / 128 * ((K + 127) / 128);
    return bytes_map(scales, sp, tiles * 2, 256, 256, 2 * subs, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <typename T, int BN>
cudaError_t launch_pair(const Mxfp8MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    using P = Pair<BN>;
    static PerDeviceInt ready;
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(pair_kernel<T, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    P::kSmemBytes);
    });
    if (e != cudaSuccess)
        return e;
    Maps maps;
    if ((e = matrix_maps(maps.a, maps.a_scales, a.a, a.a_scales, a.M, a.K, 128, kPairSubs)) !=
            cudaSuccess ||
        (e = matrix_maps(maps.b, maps.b_scales, a.b, a.b_scales, a.N, a.K, BN / 2, kPairSubs)) !=
            cudaSuccess)
        return e;
    const int64_t tiles_m = (a.M + 255) / 256, tiles = tiles_m * ((a.N + BN - 1) / BN);
    if (tiles > INT32_MAX)
        return cudaErrorInvalidValue;
    const int pairs = static_cast<int>(tiles < dev.sms / 2 ? tiles : dev.sms / 2);
    Raster r;
    r.tiles_m = static_cast<int>(tiles_m);
    r.tiles_n = static_cast<int>((a.N + BN - 1) / BN);
    const int groups = r.tiles_m < 18 ? 1 : (r.tiles_m + 6) / 12;
    r.group = (r.tiles_m + groups - 1) / groups;
    return launch_clusters(pair_kernel<T, BN>, 2 * pairs, 2, kPairThreads, P::kSmemBytes, stream, a,
                           maps, r);
}

template <typename T, bool RAW>
cudaError_t launch_few(const Mxfp8MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    static PerDeviceInt ready;
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(few_kernel<T, RAW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemMax - 1024);
    });
    if (e != cudaSuccess)
        return e;
    Few f;
    f.NX = 16;
    while (f.NX < a.M)
        f.NX *= 2;
    f.stage_bytes = kTileBytes + 2 * kScaleBytes + f.NX * kStepK;
    // parts of K until the GPU is full: they depend on N and K alone, so that a row's result does
    // not depend on the rows beside it (of up to 128: the pairs sum K without parts, so that the
    // same row among more may differ in its last bits)
    const int64_t tiles = (a.N + 127) / 128, steps = (a.K + kStepK - 1) / kStepK;
    f.split = 1;
    while (f.split < 8 && 2 * f.split * tiles <= 152 && 2 * f.split <= steps)
        f.split *= 2;
    const int most = static_cast<int>((steps + f.split - 1) / f.split);
    f.stages = (kSmemMax - 4096) / f.stage_bytes;
    f.stages = f.stages > kFewMaxStages ? kFewMaxStages : f.stages;
    f.stages = f.stages > most ? most : f.stages;
    // the parts to be joined (or one part on its way to its rows) take the ring's place
    int smem = f.stages * f.stage_bytes;
    if (smem < f.NX * 512)
        smem = f.NX * 512;
    // more than half of an SM's shared memory: two CTAs that wait for one another's tensor memory
    // and for the rest of their clusters would never end
    if (smem < kSmemMax / 2 + 2048)
        smem = kSmemMax / 2 + 2048;
    Maps maps{};
    if ((!RAW && (e = matrix_maps(maps.a, maps.a_scales, a.a, a.a_scales, a.M, a.K, f.NX, 1)) !=
                     cudaSuccess) ||
        (e = matrix_maps(maps.b, maps.b_scales, a.b, a.b_scales, a.N, a.K, 128, 1)) !=
            cudaSuccess)
        return e;
    return launch_clusters(few_kernel<T, RAW>, static_cast<int>(tiles * f.split), f.split, kFewThreads,
                           smem + 1024, stream, a, maps, f);
}

template <typename T>
cudaError_t launch(const Mxfp8MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    // What the instruction's other side holds; one border for all N and K, so that a row's bits change
    // at one number of rows.  At 128 rows of 4096 values the pairs take 11.6 us for N = 4096, these 10.7;
    // for N = 16384 20.0 and 24.6.  At 32 rows and N = 4096 10.9 and 7.7.
    // (K = N = 4096, us, and with the rows quantised by a launch of their own: one row 7.2, 8.5; 32 rows
    // 9.3, 9.5)
    if (!a.a_scales) {
        if constexpr (sizeof(T) == 2)
            return launch_few<T, true>(a, dev, stream);
        return cudaErrorInvalidValue;
    }
    if (a.M <= 128)
        return launch_few<T, false>(a, dev, stream);
    // Narrower tiles where the wide ones leave half of the SMs without work (N = K = 4096, us: 512 rows,
    // 32 wide tiles, narrow 12.1, wide 15.4; 768 rows, 48 tiles, 18.2 and 16.1; 2048 rows 31.4 and 27.4).
    const int64_t wide = (a.M + 255) / 256 * ((a.N + 255) / 256);
    return wide <= dev.sms / 4 ? launch_pair<T, 128>(a, dev, stream)
                               : launch_pair<T, 256>(a, dev, stream);
}

}  // namespace

cudaError_t launch_mxfp8_matmul(Mxfp8MatmulArgs a, const DeviceInfo& dev, cudaStream_t stream)
{
    const auto on32 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; };
    // (rows of 8-bit results are a multiple of 32 bytes)
    const int64_t row = a.N * (a.out_scales ? 1 : a.type == kTypeF32 ? 4 : 2);
    a.wide = row % 32 == 0 && on32(a.out) && on32(a.keep) && on32(a.residual) &&
             (!a.residual || a.N % 16 == 0);
    if (a.type == kTypeF32)
        return launch<float>(a, dev, stream);
    return a.type == kTypeF16 ? launch<__half>(a, dev, stream) : launch<__nv_bfloat16>(a, dev, stream);
}

cudaError_t mxfp8_matmul_error(unsigned* bits, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_error, sizeof(unsigned));
    if (e == cudaSuccess && clear && *bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_error, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace rmsmod
