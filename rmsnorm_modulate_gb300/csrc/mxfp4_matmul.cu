// The product of two microscaled 4-bit matrices, out = a b^T, on the block-scaled tensor core
// instructions (tcgen05.mma, kind::mxf4), with bias, gate and residual in its epilogue:
//   acc[m, n] = sum_k a[m, k] * b[n, k]          (fp32 accumulators in tensor memory)
//   out       = R(residual + gate_b * (acc + bias)),  one rounding
//
// Operand tiles are 256 values (128 bytes) of every row, brought by TMA (128-byte swizzle), with two
// scale tiles for each 128 rows; one thread copies the scales to tensor memory and starts four
// products of 64 values.
//
// pair_kernel (more than 128 rows of a): two CTAs of a cluster share a 256 x BN tile
// (cta_group::2), each with its 128 rows of a and half of b's rows.  256 values of K take 512 cycles of
// products (BN = 256), in which 35 KB arrive in each SM, 68 bytes a cycle: about what an SM takes from
// L2, and the next bound beside the products.  (BN = 192 brings 31.7 KB for 384 cycles: 93 us where
// this takes 85, 4214 x 4096 x 16384; a CTA alone would bring half as much again.)  Persistent, with two
// accumulators: eight warps finish one tile's rows while the next tile's products run.  Without the
// copies the products take 73 us, without the epilogue 81; at 4216 x 16384 x 4096, where a tile has a
// quarter of the steps, 104 us in all, 77 and 94.
//
// few_kernel (up to 128 rows of a, where reading b is what counts): b's rows take the 128-row side of
// the instruction, a's rows the other.  A cluster of up to eight CTAs splits K, and joins its parts in
// the CTAs' order through distributed shared memory.
#include <cuda.h>
#include <mutex>

#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp4.h"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

constexpr int kStepBytes = 128;   // of a row per step
constexpr int kStepK = 256;       // values per step
constexpr int kTileBytes = 128 * kStepBytes;
constexpr int kScaleBytes = 1024;  // a step's scales of 128 rows
constexpr uint32_t kPairTmemCols = 512, kFewTmemCols = 256;
constexpr int kSmemMax = 227 * 1024;

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// A shared-memory address of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

// mbar_wait for a loop of short steps: the clock is read once for many tries.  (Copies, products and
// tensor-memory reads order themselves: the barriers need no acquire beyond the CTA's, whose cluster
// form costs each step some hundred cycles.)
__device__ __forceinline__ bool step_wait(uint32_t bar, uint32_t parity)
{
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity))
            return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity))
                return true;
        if (global_ns() - t0 > kWaitLimitNs)
            return false;
    }
}

// Box of a 2-D tensor map into this CTA's shared memory.  PAIR: the barrier may be the other CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t bar)
{
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx"
            "::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

// Shared-memory matrix descriptors.  Operand tiles: rows of 128 bytes, swizzled, eight rows
// (1024 bytes) to a group.  Scale tiles: 32 rows of 16 bytes, eight rows (128 bytes) to a group.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (8ull << 16) | (8ull << 32) |
           (1ull << 46);
}

// 512 bytes of scales to 32 lanes x 4 columns, repeated for the four groups of lanes.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    if (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                     : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
            "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
            "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
            : "memory");
}

// Arrives on `bar` (in both CTAs of a pair) when what this thread has started is done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
            ".b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t to)
{
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to),
                     "r"(kPairTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to),
                     "r"(kFewTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem)
{
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kPairTmemCols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kFewTmemCols));
}

__device__ __forceinline__ void before_sync()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void after_sync()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_loads_done()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Instruction descriptor: e2m1 operands, e8m0 scales, K = 64.
__host__ __device__ constexpr uint32_t instruction(int M, int N)
{
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N / 8) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M / 16) << 24);
}

// The products of one step of SUBS * 256 values: `parts` of 64 values each, four to an operand tile
// (b's are b_tile bytes apart).  Scales: two tiles (of four blocks each) for each 128 rows and 256
// values, copied before each four products; a product takes two of a column's four scales.
template <bool PAIR, int B_TILES, int SUBS>
__device__ __forceinline__ void step_products(uint32_t acc, uint32_t sfa_col, uint32_t sfb_col,
                                              uint32_t sa, uint32_t sb,
                                              uint32_t b_tile, uint32_t sfa, uint32_t sfb,
                                              uint32_t idesc, int parts, bool first)
{
#pragma unroll
    for (int p = 0; p < 4 * SUBS; ++p)
        if (p < parts) {
            const int h = p >> 1;  // scale tile
            if (p % 2 == 0) {
                copy_scales<PAIR>(sfa_col + h % 2 * 4, scale_desc(sfa + h * 512));
#pragma unroll
                for (int i = 0; i < B_TILES; ++i)
                    copy_scales<PAIR>(sfb_col + h % 2 * (4 * B_TILES) + i * 4,
                                      scale_desc(sfb + i * (SUBS * kScaleBytes) + h * 512));
            }
            const uint32_t id = (p & 1) * 2u;
            mma_mxf4<PAIR>(acc, operand_desc(sa + (p >> 2) * kTileBytes + (p & 3) * 32),
                           operand_desc(sb + (p >> 2) * b_tile + (p & 3) * 32),
                           idesc | (id << 4) | (id << 29), sfa_col + h % 2 * 4,
                           sfb_col + h % 2 * (4 * B_TILES), !first || p > 0);
        }
}

// Products (of 64 values) of step t.
template <int SUBS>
__device__ __forceinline__ int parts_of(int64_t K, int t)
{
    const int64_t left = K - static_cast<int64_t>(t) * (SUBS * kStepK);
    return left >= SUBS * kStepK ? 4 * SUBS : static_cast<int>((left + 63) / 64);
}

struct Maps {
    CUtensorMap a, a_scales, b, b_scales;
};

// ---------------------------------------------------------------------------
// more than 128 rows
// ---------------------------------------------------------------------------

// Two operand tiles to a step: waiting for one and passing it on takes the issuing thread as long as
// several products (one tile to a step: 121 us where two take 100, 4216 x 16384 x 4096).
constexpr int kPairSubs = 2;

template <int BN>
struct Pair {
    static constexpr int kBBytes = BN / 2 * kStepBytes;  // of one operand tile
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

// 32 bytes (a whole sector) at once where rows start on 32 bytes, else 16 and 16.
__device__ __forceinline__ void load_pair(const uint4* p, bool both, bool wide, uint4* v)
{
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                       "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
    } else {
        v[0] = ld_stream(p);
        if (both)
            v[1] = ld_stream(p + 1);
    }
}

__device__ __forceinline__ void store_pair(uint4* p, bool both, bool wide, const uint4 (&v)[2])
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0].x),
                     "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
                     "r"(v[1].w)
                     : "memory");
    } else {
        st_stream(p, v[0]);
        if (both)
            st_stream(p + 1, v[1]);
    }
}

// Eight columns of one row.
template <typename T>
__device__ __forceinline__ uint4 finish8(const uint32_t* acc, bool bias, bool gate, bool residual,
                                         const uint4& bv, const uint4& gv, const uint4& rv)
{
    uint4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float lo = __uint_as_float(acc[2 * j]), hi = __uint_as_float(acc[2 * j + 1]);
        if (bias) {
            const float2 v = widen2<T>(word(bv, j));
            lo += v.x;
            hi += v.y;
        }
        if (gate) {
            const float2 v = widen2<T>(word(gv, j));
            lo *= v.x;
            hi *= v.y;
        }
        if (residual) {
            const float2 v = widen2<T>(word(rv, j));
            lo += v.x;
            hi += v.y;
        }
        word(o, j) = narrow2<T>(lo, hi);
    }
    return o;
}

template <typename T, int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const Mxfp4MatmulArgs a, const __grid_constant__ Maps maps, int tiles_m, int tiles)
{
    using P = Pair<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) unsigned long long full[P::kStages], empty[P::kStages];
    __shared__ __align__(8) unsigned long long acc_full[P::kAccs], acc_empty[P::kAccs], shared_read;
    __shared__ uint32_t tmem_base;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    const int steps = static_cast<int>((a.K + kPairSubs * kStepK - 1) / (kPairSubs * kStepK));
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

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
        tmem_alloc<true>(smem_addr(&tmem_base));
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
                const int m0 = tile % tiles_m * 256 + static_cast<int>(rank) * 128;
                const int n0 = tile / tiles_m * BN;
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
                        const int x = (kPairSubs * t + h) * kStepBytes;
                        tma_box<true>(dst + h * kTileBytes, &maps.a, x, m0, bar);
                        tma_box<true>(dst + kPairSubs * kTileBytes + h * P::kBBytes, &maps.b, x,
                                      n0 + static_cast<int>(rank) * (BN / 2), bar);
                    }
                    const uint32_t sf = dst + kPairSubs * (kTileBytes + P::kBBytes);
                    tma_box<true>(sf, &maps.a_scales, 0,
                                  2 * (m0 / 128 * block_tiles + 2 * kPairSubs * t), bar);
#pragma unroll
                    for (int i = 0; i < P::kBTiles; ++i)
                        tma_box<true>(sf + (1 + i) * kPairSubs * kScaleBytes, &maps.b_scales, 0,
                                      2 * ((n0 / 128 + i) * block_tiles + 2 * kPairSubs * t), bar);
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
        const uint4* __restrict__ bias = static_cast<const uint4*>(a.bias);
        const uint4* __restrict__ gate = static_cast<const uint4*>(a.gate);
        const uint4* __restrict__ residual = static_cast<const uint4*>(a.residual);
        const int64_t Nv = a.N / 8;
        int acc = 0;
        uint32_t phase = 0;
        for (int tile = pair; tile < tiles; tile += pairs) {
            if (!broken)
                gave_up(step_wait(smem_addr(&acc_full[acc]), phase));
            const int64_t m = static_cast<int64_t>(tile % tiles_m) * 256 + rank * 128 +
                              quarter * 32 + lane;
            const int64_t n0 = (static_cast<int64_t>(tile / tiles_m) * BN + half * P::kCols) / 8;
            const int64_t gate_at = (gate && m < a.M ? m / a.S * a.gate_bstride : 0) / 8;
            const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                  acc * P::kAccStep + half * P::kCols;
            // 32 columns at a time, from the side that the other accumulator has too
            const bool shares = P::kOverlap && half != acc;
#pragma unroll 1
            for (int k0 = 0; k0 < P::kCols / 32; ++k0) {
                const int c = P::kOverlap && acc == 0 ? P::kCols / 32 - 1 - k0 : k0;
                uint32_t v[32];
                __syncwarp();
                after_sync();
                tmem_load32(from + 32 * c, v);
                // what they take beside the accumulators, on its way meanwhile
                const int64_t n = n0 + 4 * c;
                uint4 bv[4], gv[4], rv[4];
                if (m < a.M) {
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
                        if (residual && n + k < Nv)
                            load_pair(residual + m * Nv + n + k, n + k + 1 < Nv, a.wide, rv + k);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (bias && n + k < Nv)
                            bv[k] = ld_cached(bias + n + k);
                        if (gate && n + k < Nv)
                            gv[k] = ld_cached(gate + gate_at + n + k);
                    }
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
                if (m < a.M)
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        uint4 o[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            o[i] = finish8<T>(v + 8 * (k + i), bias, gate, residual, bv[k + i],
                                              gv[k + i], rv[k + i]);
                        if (n + k < Nv)
                            store_pair(static_cast<uint4*>(a.out) + m * Nv + n + k, n + k + 1 < Nv,
                                       a.wide, o);
                    }
            }
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
        tmem_free<true>(tmem);
}

// ---------------------------------------------------------------------------
// up to 128 rows
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 192;  // four epilogue warps, producer, issuer
constexpr int kFewMaxStages = 10;
constexpr uint32_t kFewSfwCol = 128;            // accumulators in columns 0..127
constexpr uint32_t kFewSfxCol = kFewSfwCol + 8;

struct Few {
    int NX;           // a's rows as the instruction takes them: 16, 32, 64 or 128
    int stages;
    int stage_bytes;
    int split;        // CTAs of a cluster, each with a range of the steps
};

template <typename T>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const Mxfp4MatmulArgs a, const __grid_constant__ Maps maps, const Few f)
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
            mbar_init(smem_addr(&full[s]), 1u);
            mbar_init(smem_addr(&empty[s]), 1u);
        }
        mbar_init(smem_addr(&done), 1u);
        mbar_init_fence();
    }
    if (warp == 5)
        tmem_alloc<false>(smem_addr(&tmem_base));
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

    if (warp == 4) {
        if (elect_one()) {
            const int block_tiles = static_cast<int>((a.K + 127) / 128);
            int s = 0;
            uint32_t phase = 1;
            for (int t = begin; t < end; ++t) {
                wait(smem_addr(&empty[s]), phase);
                const uint32_t bar = smem_addr(&full[s]);
                const uint32_t dst = ring + s * f.stage_bytes;
                mbar_expect_tx(bar, f.stage_bytes);
                tma_box<false>(dst, &maps.b, t * kStepBytes, n0, bar);
                tma_box<false>(dst + kTileBytes, &maps.b_scales, 0,
                               2 * (n0 / 128 * block_tiles + 2 * t), bar);
                tma_box<false>(dst + kTileBytes + kScaleBytes, &maps.a_scales, 0, 4 * t, bar);
                tma_box<false>(dst + kTileBytes + 2 * kScaleBytes, &maps.a, t * kStepBytes, 0, bar);
                if (++s == f.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 5) {
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
    }
    // ---- lane n of tensor memory, column m
    const int n_in = warp * 32 + lane;
    const int64_t n = n0 + n_in;
    const T* bias = static_cast<const T*>(a.bias);
    const T* gate = static_cast<const T*>(a.gate);
    const T* residual = static_cast<const T*>(a.residual);
    T* out = static_cast<T*>(a.out);
    const int M = static_cast<int>(a.M), S = static_cast<int>(a.S);
    auto finish = [&](int m, float v, float bias_n) {
        v += bias_n;
        if (gate)
            v *= static_cast<float>(gate[m / S * a.gate_bstride + n]);
        if (residual)
            v += static_cast<float>(residual[m * a.N + n]);
        out[m * a.N + n] = static_cast<T>(v);
    };
    const float bias_n = warp < 4 && n < a.N && bias ? static_cast<float>(bias[n]) : 0.0f;
    float* part = reinterpret_cast<float*>(raw + (ring - smem_addr(raw)));  // [m][128]
    if (warp < 4) {
        wait(smem_addr(&done), 0);
        __syncwarp();
        after_sync();
        for (int c = 0; c < M; c += 16) {
            uint32_t v[16];
            tmem_load16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
            tmem_loads_done();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (f.split > 1)
                    part[(c + j) * 128 + n_in] = __uint_as_float(v[j]);
                else if (c + j < M && n < a.N)
                    finish(c + j, __uint_as_float(v[j]), bias_n);
            }
        }
        before_sync();
    }
    if (broken)
        drain_pause();
    if (f.split > 1) {
        cluster_barrier();
        if (warp < 4 && n < a.N) {
            // this CTA's rows of a, four at a time (all their loads on the way at once), the parts of
            // K in order
            const uint32_t at = smem_addr(part) + n_in * 4;
            for (int m = static_cast<int>(rank); m < M; m += 4 * f.split) {
                float p[4][8];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (r < f.split && m + i * f.split < M)
                            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                         : "=f"(p[i][r])
                                         : "r"(in_cta(at + (m + i * f.split) * 512, r)));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (m + i * f.split < M) {
                        float v = p[i][0];
#pragma unroll
                        for (int r = 1; r < 8; ++r)
                            if (r < f.split)
                                v += p[i][r];
                        finish(m + i * f.split, v, bias_n);
                    }
            }
        }
        cluster_barrier();
    } else {
        __syncthreads();
    }
    if (warp == 5) {
        after_sync();
        tmem_free<false>(tmem);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once.
cudaError_t encoder(EncodeTiled& fn)
{
    static std::mutex mu;
    static EncodeTiled cached = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                               cudaEnableDefault, &q);
        if (e != cudaSuccess)
            return e;
        if (q != cudaDriverEntryPointSuccess || !p)
            return cudaErrorNotSupported;
        cached = reinterpret_cast<EncodeTiled>(p);
    }
    fn = cached;
    return cudaSuccess;
}

// `rows` rows of `row_bytes` bytes; boxes of `box_bytes` by `box_rows`, zeros outside the matrix.
cudaError_t bytes_map(CUtensorMap& map, const void* p, int64_t rows, int64_t row_bytes,
                      int box_bytes, int box_rows, CUtensorMapSwizzle swizzle)
{
    EncodeTiled fn = nullptr;
    const cudaError_t e = encoder(fn);
    if (e != cudaSuccess)
        return e;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes),
                               static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r =
        fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A 4-bit matrix: its codes in boxes of `box_rows` rows, and its scale tiles as rows of 256 bytes, in
// boxes of the tiles of `subs` * 256 values (two for each 256).
cudaError_t matrix_maps(CUtensorMap& codes, CUtensorMap& scales, const void* p, const void* sp,
                        int64_t rows, int64_t K, int box_rows, int subs)
{
    const cudaError_t e =
        bytes_map(codes, p, rows, K / 2, kStepBytes, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (rows + 127) / 128 * ((K + 127) / 128);
    return bytes_map(scales, sp, tiles * 2, 256, 256, 4 * subs, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <typename K, typename... Args>
cudaError_t launch_clusters(K kern, int grid, int cluster, int threads, int smem,
                            cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int BN>
cudaError_t launch_pair(const Mxfp4MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
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
    return launch_clusters(pair_kernel<T, BN>, 2 * pairs, 2, kPairThreads, P::kSmemBytes, stream, a,
                           maps, static_cast<int>(tiles_m), static_cast<int>(tiles));
}

template <typename T>
cudaError_t launch_few(const Mxfp4MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    static PerDeviceInt ready;
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(few_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemMax - 1024);
    });
    if (e != cudaSuccess)
        return e;
    Few f;
    f.NX = 16;
    while (f.NX < a.M)
        f.NX *= 2;
    f.stage_bytes = kTileBytes + 2 * kScaleBytes + f.NX * kStepBytes;
    // parts of K until the GPU is full: they depend on N and K alone, so that a row's result does
    // not depend on the rows beside it (of up to 128: the pairs sum K without parts, so that the
    // same row among more may differ in its last bits).  A power of two leaves up to half of the SMs
    // without a part; what 8 rows take with K = 4096 shows little of it: N = 9728 (152 CTAs) 7.9 us,
    // 9856 (77) 8.2, 11008 (86) 8.3.
    const int64_t tiles = (a.N + 127) / 128, steps = (a.K + kStepK - 1) / kStepK;
    f.split = 1;
    while (f.split < 8 && 2 * f.split * tiles <= 152 && 2 * f.split <= steps)
        f.split *= 2;
    const int most = static_cast<int>((steps + f.split - 1) / f.split);
    f.stages = (kSmemMax - 4096) / f.stage_bytes;
    f.stages = f.stages > kFewMaxStages ? kFewMaxStages : f.stages;
    f.stages = f.stages > most ? most : f.stages;
    // the parts to be joined take the ring's place
    int smem = f.stages * f.stage_bytes;
    if (f.split > 1 && smem < f.NX * 512)
        smem = f.NX * 512;
    // more than half of an SM's shared memory: two CTAs that wait for one another's tensor memory
    // and for the rest of their clusters would never end
    if (smem < kSmemMax / 2 + 2048)
        smem = kSmemMax / 2 + 2048;
    Maps maps;
    if ((e = matrix_maps(maps.a, maps.a_scales, a.a, a.a_scales, a.M, a.K, f.NX, 1)) !=
            cudaSuccess ||
        (e = matrix_maps(maps.b, maps.b_scales, a.b, a.b_scales, a.N, a.K, 128, 1)) !=
            cudaSuccess)
        return e;
    return launch_clusters(few_kernel<T>, static_cast<int>(tiles * f.split), f.split, kFewThreads,
                           smem + 1024, stream, a, maps, f);
}

template <typename T>
cudaError_t launch(const Mxfp4MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    // What the instruction's other side holds.  With K = 4096, N = 4096 and 16 rows 5.6 us against the
    // pairs' 8.2, 64 rows 7.4 and 8.2, 96 rows 8.6 and 8.4, 128 rows 9.8 and 8.4; with N = 16384
    // 64 rows 11.0 and 12.8, 128 rows 13.0 and 13.3.  One border for all N and K, so that a row's bits
    // change at one number of rows.
    if (a.M <= 128)
        return launch_few<T>(a, dev, stream);
    // narrower tiles where the wide ones leave half of the SMs without work: 256 and 512 rows
    // (N = K = 4096) 8.7 and 9.3 us against 10.8 and 11.4; 1024 rows 13.1 and 12.2
    const int64_t wide = (a.M + 255) / 256 * ((a.N + 255) / 256);
    return wide <= dev.sms / 4 ? launch_pair<T, 128>(a, dev, stream)
                               : launch_pair<T, 256>(a, dev, stream);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(Mxfp4MatmulArgs a, const DeviceInfo& dev, cudaStream_t stream)
{
    const auto on32 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; };
    a.wide = a.N % 16 == 0 && on32(a.out) && on32(a.residual);
    return a.f16 ? launch<__half>(a, dev, stream) : launch<__nv_bfloat16>(a, dev, stream);
}

cudaError_t mxfp4_matmul_error(unsigned* bits, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_error, sizeof(unsigned));
    if (e == cudaSuccess && clear && *bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_error, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace rmsmod
