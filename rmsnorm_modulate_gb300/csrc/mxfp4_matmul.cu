// The product of two microscaled 4-bit matrices, out = a b^T, on the block-scaled tensor core
// instructions (tcgen05.mma, kind::mxf4), with bias, gate and residual in its epilogue:
//   acc[m, n] = sum_k a[m, k] * b[n, k]          (fp32 accumulators in tensor memory)
//   out       = R(residual + gate_b * (acc + bias)),  one rounding
//
// One CTA per 128 x 256 tile of the output.  A producer warp brings 128 bytes (256 values) of
// every row of a and b per step by TMA (128-byte swizzle), and the scale tiles as they lie; the
// issuing thread copies the scales into tensor memory and starts four products of 64 values each;
// four warps read the accumulators back and finish the rows.
#include <cuda.h>
#include <mutex>

#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp4.h"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kStepBytes = 128;  // of a row per step
constexpr int kStepK = 256;      // values per step
constexpr int kStages = 4;
constexpr int kABytes = kBM * kStepBytes;
constexpr int kBBytes = kBN * kStepBytes;
constexpr int kSfaBytes = 1024;                // 128 rows x 8 blocks
constexpr int kSfbBytes = kBN / 128 * 1024;
constexpr int kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kThreads = 192;    // four epilogue warps, producer, issuer
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfaCol = 256;  // accumulators in columns 0..255
constexpr uint32_t kSfbCol = kSfaCol + 8;

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// Tile of a 2-D tensor map into shared memory.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar)
{
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
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::
                     "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32])
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

struct Maps {
    CUtensorMap a, b;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
    matmul_kernel(const Mxfp4MatmulArgs a, const __grid_constant__ Maps maps)
{
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) unsigned long long full[kStages], empty[kStages], done;
    __shared__ uint32_t tmem_base;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kBM;
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kBN;
    const int steps = static_cast<int>((a.K + kStepK - 1) / kStepK);
    const int64_t block_tiles = (a.K + 127) / 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&full[s]), 1u);
            mbar_init(smem_addr(&empty[s]), 1u);
        }
        mbar_init(smem_addr(&done), 1u);
        mbar_init_fence();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
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
            // row tiles of b's scales that exist under this tile
            const int64_t b_tiles = (a.N + 127) / 128;
            const int sfb_tiles = static_cast<int>(b_tiles - n0 / 128 < kBN / 128
                                                       ? b_tiles - n0 / 128 : kBN / 128);
            const uint8_t* sfa = static_cast<const uint8_t*>(a.a_scales) +
                                 blockIdx.x * block_tiles * 512;
            const uint8_t* sfb = static_cast<const uint8_t*>(a.b_scales) +
                                 n0 / 128 * block_tiles * 512;
            for (int t = 0; t < steps; ++t) {
                const int s = t % kStages;
                if (t >= kStages)
                    wait(smem_addr(&empty[s]), ((t / kStages) & 1) ^ 1);
                const uint32_t bar = smem_addr(&full[s]);
                const uint32_t dst = ring + s * kStageBytes;
                const uint32_t sf_bytes = block_tiles - 2 * t >= 2 ? 1024u : 512u;
                mbar_expect_tx(bar, kABytes + kBBytes + sf_bytes * (1 + sfb_tiles));
                tma_tile(dst, &maps.a, t * kStepBytes, static_cast<int>(m0), bar);
                tma_tile(dst + kABytes, &maps.b, t * kStepBytes, static_cast<int>(n0), bar);
                bulk_g2s(dst + kABytes + kBBytes, sfa + t * 1024, sf_bytes, bar);
                for (int i = 0; i < sfb_tiles; ++i)
                    bulk_g2s(dst + kABytes + kBBytes + kSfaBytes + i * 1024,
                             sfb + i * block_tiles * 512 + t * 1024, sf_bytes, bar);
            }
        }
    } else if (warp == 5) {
        if (elect_one()) {
            // e2m1 operands, e8m0 scales, M = 128, N = 256
            constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((kBN / 8) << 17) | (1u << 23) |
                                        ((kBM / 16) << 24);
            for (int t = 0; t < steps; ++t) {
                const int s = t % kStages;
                wait(smem_addr(&full[s]), (t / kStages) & 1);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sa = ring + s * kStageBytes, sb = sa + kABytes;
                const uint32_t sfa = sb + kBBytes, sfb = sfa + kSfaBytes;
                const int64_t left = a.K - static_cast<int64_t>(t) * kStepK;
                const int parts = left >= kStepK ? 4 : static_cast<int>((left + 63) / 64);
                // a step's scales: two tiles of four blocks for each 128 rows
                for (int h = 0; h < (parts + 1) / 2; ++h) {
                    copy_scales(tmem + kSfaCol + h * 4, scale_desc(sfa + h * 512));
                    for (int i = 0; i < kBN / 128; ++i)
                        copy_scales(tmem + kSfbCol + h * (kBN / 32) + i * 4,
                                    scale_desc(sfb + i * 1024 + h * 512));
                }
                for (int p = 0; p < parts; ++p) {
                    const uint32_t id = (p & 1) * 2u;  // which two of a column's four scales
                    mma_mxf4(tmem, operand_desc(sa + p * 32), operand_desc(sb + p * 32),
                             kIdesc | (id << 4) | (id << 29), tmem + kSfaCol + (p >> 1) * 4,
                             tmem + kSfbCol + (p >> 1) * (kBN / 32), t > 0 || p > 0);
                }
                commit(smem_addr(&empty[s]));
            }
            commit(smem_addr(&done));
        }
    } else {
        wait(smem_addr(&done), 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const int64_t m = m0 + warp * 32 + lane;
        const uint4* __restrict__ bias = static_cast<const uint4*>(a.bias);
        const uint4* __restrict__ gate = static_cast<const uint4*>(a.gate);
        const uint4* __restrict__ residual = static_cast<const uint4*>(a.residual);
        const int64_t gate_row = (m < a.M ? m / a.S : 0) * (a.gate_bstride / 8);
        for (int c = 0; c < kBN; c += 32) {
            if (n0 + c >= a.N)
                break;
            uint32_t acc[32];
            __syncwarp();
            tmem_load32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, acc);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t n = n0 + c + q * 8;
                if (m >= a.M || n >= a.N)
                    continue;
                const uint4 bv = bias ? ld_cached(bias + n / 8) : make_uint4(0u, 0u, 0u, 0u);
                const uint4 gv = gate ? ld_cached(gate + gate_row + n / 8) : bv;
                const uint4 rv = residual ? ld_stream(residual + (m * a.N + n) / 8) : bv;
                uint4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo = __uint_as_float(acc[q * 8 + 2 * j]);
                    float hi = __uint_as_float(acc[q * 8 + 2 * j + 1]);
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
                st_stream(static_cast<uint4*>(a.out) + (m * a.N + n) / 8, o);
            }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    // after a timeout: a bounded pause for the copies still in flight
    if (broken)
        drain_pause();
    __syncthreads();
    if (warp == 5) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols));
    }
}

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

// Rows of K / 2 bytes; boxes of 128 bytes by `box_rows`, zeros outside the matrix.
cudaError_t rows_map(CUtensorMap& map, const void* p, int64_t rows, int64_t K, int box_rows)
{
    EncodeTiled fn = nullptr;
    const cudaError_t e = encoder(fn);
    if (e != cudaSuccess)
        return e;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
    const cuuint32_t box[2] = {kStepBytes, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r =
        fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch(const Mxfp4MatmulArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    static PerDeviceInt ready;
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(matmul_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemBytes);
    });
    if (e != cudaSuccess)
        return e;
    Maps maps;
    if ((e = rows_map(maps.a, a.a, a.M, a.K, kBM)) != cudaSuccess ||
        (e = rows_map(maps.b, a.b, a.N, a.K, kBN)) != cudaSuccess)
        return e;
    const dim3 grid(static_cast<unsigned>((a.M + kBM - 1) / kBM),
                    static_cast<unsigned>((a.N + kBN - 1) / kBN));
    return launch_dependent(matmul_kernel<T>, grid, kThreads, kSmemBytes, stream, a, maps);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(const Mxfp4MatmulArgs& a, const DeviceInfo& dev,
                                cudaStream_t stream)
{
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
