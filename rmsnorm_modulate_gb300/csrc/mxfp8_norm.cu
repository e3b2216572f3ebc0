// The norm before a projection in 8 bits, and its gradients from an 8-bit checkpoint of its input.
//
//   forward   res  = R(x + update)
//             r    = 1 / sqrt(mean(res^2) + eps)
//             out  = Q((res * r) * m + shift),               m = weight * (1 + scale)
//             keep = Q(res)
//   backward  hh   = kept * r
//             dx   = R(r * (go * m - hh * c) + gr),          c = mean(go * m * hh)
//             sums over the tokens of go and go * hh, from which a last launch forms the gradients
//             of shift, scale and weight
//
// fp32 throughout, one rounding per stored value (Q: mxfp8.cuh).  Sums run in an order that D (and,
// over tokens, S) alone fixes.  7 to 8 bytes a value forward, 7 backward: the forward pass is bound by HBM,
// the backward pass by its instructions and their latency about as much.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp8.cuh"
#include "mxfp8.h"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

// 1 / sqrt(sum / n + eps) to half a step and little more, where the sum and the root are normal: every
// value of a row has its error in common, and what is rounded to e4m3 a step off in it is then on the
// other side of a border that much more often.  The quotient has its remainder added; one Newton step from
// the approximate root, whose products' low parts are kept.
__device__ __forceinline__ float rstd_fast(float sum, float n, float inv_n, float eps)
{
    const float q = __fmul_rn(sum, inv_n);
    const float ms = __fadd_rn(__fmaf_rn(__fmaf_rn(-q, n, sum), inv_n, q), eps);
    const float y = rsqrtf(ms);
    const float h = __fmul_rn(ms, y), l = __fmaf_rn(ms, y, -h);
    const float e = __fmaf_rn(-l, y, __fmaf_rn(-h, y, 1.0f));  // 1 - ms y^2
    return __fmaf_rn(__fmul_rn(0.5f, y), e, y);
}

__device__ __forceinline__ float4 floats(u64 a, u64 b)
{
    float4 f;
    f2_unpack(a, f.x, f.y);
    f2_unpack(b, f.z, f.w);
    return f;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kFullMask, v, off));
    return v;
}

// The parts of a row's sum that a group's warps leave, zeros behind the last, and their sum in an order
// that the number of warps fixes: a few wide loads of the same words in every lane, which are sooner done
// than four exchanges.
struct __align__(16) Parts {
    float of[16];

    __device__ __forceinline__ float joined(int warps) const
    {
        const float4* p = reinterpret_cast<const float4*>(of);
        auto four = [&](int i) {
            const float4 v = p[i];
            return __fadd_rn(__fadd_rn(v.x, v.y), __fadd_rn(v.z, v.w));
        };
        float s = four(0);
        if (warps > 4)
            s = __fadd_rn(s, four(1));
        if (warps > 8)
            s = __fadd_rn(s, __fadd_rn(four(2), four(3)));
        return s;
    }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// One CTA per SM, whose sixteen warps form groups that take a row each, up to V vectors of eight values
// a thread.  A CTA has a range of rows, dealt to its groups in turn, and a group a ring of bulk copies
// ahead of it.  A row is in registers when its sum over the group's warps is joined, so its slot is filled
// again from there on.  Sixteen lanes' blocks are a block tile, whose scales in the row are one store of
// four bytes.  (Rows 32 apart in turn, whose scales are neighbours, and one store for four of them: no
// faster, and a CTA that has two batches' rows changes its row vectors with every row.)
//
// 4 x 1 x 4096 2.9 us; 1 x 4216 x 4096 29.2 with `keep` and 25.7 without (20.5 and 17.9 of HBM time: the
// rest is the launch, the first rows' latency and the last rows' stores); 17024 x 4096 80 (72).
constexpr int kFwdWarps = 16;
constexpr int kFwdThreads = 32 * kFwdWarps;
constexpr int kFwdMaxStages = 8;
constexpr int kFwdSmem = 224 * 1024;

struct FwdPlan {
    FastDiv by_S;
    uint32_t rows;  // those behind the last one, which have scales, among them
    int warps;      // of a group
    int groups;
    int stages;     // of a group's ring
    int row_bytes;  // of a slot
};

template <typename T, int V>
__global__ void __launch_bounds__(kFwdThreads, 1)
    norm_kernel(const Mxfp8NormArgs a, const FwdPlan plan)
{
    constexpr bool kWide = V > 2;  // the row vectors' products in shared memory, for each group
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) unsigned long long full[kFwdWarps][kFwdMaxStages];
    __shared__ Parts part[2][kFwdWarps];  // [group]

    const int lane = threadIdx.x & 31;
    const int group = (threadIdx.x >> 5) / plan.warps;
    const int warp = (threadIdx.x >> 5) - group * plan.warps;
    const int Dv = a.D / 8;
    const uint32_t tiles = (a.D + 127) / 128;
    const bool leader = warp == 0 && lane == 0;
    if (group >= plan.groups)
        return;  // (no barrier of the whole CTA)
    auto group_sync = [&]() {
        if (plan.warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(plan.warps * 32) : "memory");
    };
    if (leader) {
        for (int s = 0; s < plan.stages; ++s)
            mbar_init(smem_addr(&full[group][s]), 1u);
        mbar_init_fence();
    }
    if (warp == 0 && lane < 16)
        part[0][group].of[lane] = part[1][group].of[lane] = 0.0f;
    group_sync();
    grid_dependency_sync();

    // kWide: the multipliers [Dv], [Dv], and the shifts [Dv]
    float4* m_lo = reinterpret_cast<float4*>(smem + (kWide ? group * a.D * 6 : 0));
    uint4* shifts = reinterpret_cast<uint4*>(m_lo + 2 * Dv);
    uint8_t* ring = smem + (kWide ? plan.groups * a.D * 6 : 0) +
                    static_cast<size_t>(group) * plan.stages * plan.row_bytes;

    // the CTA's rows: ranges whose lengths differ by one at most
    const uint32_t each = plan.rows / gridDim.x, more = plan.rows - each * gridDim.x;
    const uint32_t first = blockIdx.x * each + (blockIdx.x < more ? blockIdx.x : more);
    const uint32_t last = first + each + (blockIdx.x < more ? 1u : 0u);
    const uint32_t filled = last < a.rows ? last : a.rows;

    uint32_t ahead = first + group;
    int put = 0;
    auto issue = [&]() {  // the leader
        if (ahead >= filled)
            return;
        const uint32_t bar = smem_addr(&full[group][put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(put) * plan.row_bytes);
        const int64_t from = static_cast<int64_t>(ahead) * a.D * 2;
        fence_proxy_async();
        mbar_expect_tx(bar, static_cast<uint32_t>(plan.row_bytes));
        bulk_g2s(dst, static_cast<const uint8_t*>(a.x) + from, a.D * 2, bar);
        if (a.update)
            bulk_g2s(dst + a.D * 2, static_cast<const uint8_t*>(a.update) + from, a.D * 2, bar);
        put = put + 1 == plan.stages ? 0 : put + 1;
        ahead += plan.groups;
    };
    if (leader)
        for (int s = 0; s < plan.stages; ++s)
            issue();

    int at[V];  // a thread's vectors
    bool has[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        at[j] = (j * plan.warps + warp) * 32 + lane;
        has[j] = at[j] < Dv;
    }
    const float n = static_cast<float>(a.D), inv_n = __fdiv_rn(1.0f, n);
    u64 m[kWide ? 1 : V][4], shift[kWide ? 1 : V][4];
    const uint32_t tile0 = static_cast<uint32_t>(at[0]) >> 4;  // of its vector 0 among a row's block tiles
    uint32_t batch = 0xFFFFFFFFu, phase = 0;
    int get = 0, odd = 0;
    bool broken = false;
    for (uint32_t row = first + group; row < last; row += plan.groups) {
        // the scales of a thread's sixteen lanes' block tile of vector j
        const int64_t scales_at = mx8_scale_at(row, 0, tiles) / 4;
        auto put_word = [&](void* scales, int j, uint32_t w) {
            const uint32_t t = tile0 + 2 * j * plan.warps;
            if ((lane & 15) == 0 && t < tiles)
                static_cast<uint32_t*>(scales)[scales_at + t * 128] = w;
        };
        if (row >= a.rows) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                put_word(a.out_scales, j, 0u);
                if (a.keep)
                    put_word(a.keep_scales, j, 0u);
            }
            continue;
        }
        const uint32_t b = plan.by_S.div(row);
        if (b != batch) {
            batch = b;  // (a thread reads the products that it has written)
            const int64_t mod = static_cast<int64_t>(b) * a.mod_bstride;
            auto vec = [&](const void* p, int64_t off, int j) {
                return ld_cached(
                    reinterpret_cast<const uint4*>(static_cast<const T*>(p) + off) + at[j]);
            };
#pragma unroll
            for (int j = 0; j < V; ++j) {
                u64 t[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    t[k] = f2_splat(1.0f);
                uint4 sh = make_uint4(0u, 0u, 0u, 0u);
                if (has[j] && a.weight) {
                    const uint4 w = vec(a.weight, 0, j);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        t[k] = widen<T>(word(w, k));
                }
                if (has[j] && a.scale) {
                    const uint4 w = vec(a.scale, mod, j);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        t[k] = f2_mul(t[k], f2_add(f2_splat(1.0f), widen<T>(word(w, k))));
                }
                if (has[j] && a.shift)
                    sh = vec(a.shift, mod, j);
                if (kWide) {
                    if (has[j]) {
                        m_lo[at[j]] = floats(t[0], t[1]);
                        m_lo[Dv + at[j]] = floats(t[2], t[3]);
                        shifts[at[j]] = sh;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        m[kWide ? 0 : j][k] = t[k];
                        shift[kWide ? 0 : j][k] = widen<T>(word(sh, k));
                    }
                }
            }
        }
        // ---- the row: R(x + update), and the sum of its squares
        if (!broken && !mbar_wait(smem_addr(&full[group][get]), phase, kWaitLimitNs)) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
        const uint4* slot = reinterpret_cast<const uint4*>(
            ring + static_cast<size_t>(get) * plan.row_bytes);
        if (++get == plan.stages) {
            get = 0;
            phase ^= 1u;
        }
        u64 f[V][4], s[2] = {0ull, 0ull};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (has[j]) {
                x = slot[at[j]];
                if (a.update) {
                    const uint4 u = slot[Dv + at[j]];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        word(x, k) = add2<T>(word(x, k), word(u, k));
                    st_stream(static_cast<uint4*>(a.res_out) +
                                  static_cast<int64_t>(row) * Dv + at[j], x);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[j][k] = widen<T>(word(x, k));
                s[k & 1] = f2_fma(f[j][k], f[j][k], s[k & 1]);
            }
        }
        float lo, hi;
        f2_unpack(f2_add(s[0], s[1]), lo, hi);
        float sum = warp_sum(__fadd_rn(lo, hi));
        if (plan.warps > 1) {
            if (lane == 0)
                part[odd][group].of[warp] = sum;  // two places in turn
            group_sync();
            sum = part[odd][group].joined(plan.warps);
            odd ^= 1;
        } else {
            __syncwarp();
        }
        if (leader)  // every warp is past this row's slot
            issue();
        float rstd, stored;
        u64 down = f2_splat(1.0f);  // of scaled rows, before rstd
        // past 2^120, or so small that a tiny eps leaves it to decide (uniform over the row)
        const bool extreme = sum > 1.3e36f || (sum < 8e-25f && a.eps < 1e-18f);
        if (!extreme) {
            rstd = stored = rstd_fast(sum, n, inv_n, a.eps);
        } else {
            // again over the power of two of the largest magnitude, mean and root in fp64; the next row's
            // place takes the largest, and then this row's, which every warp has read, the sums
            Parts& tops = part[odd][group];
            Parts& sums = part[odd ^ 1][group];
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = absmax2(top, f[j][k]);
            uint32_t bits = __reduce_max_sync(kFullMask, __float_as_uint(top));
            if (lane == 0)
                tops.of[warp] = __uint_as_float(bits);
            group_sync();
            bits = 0u;
            for (int k = 0; k < plan.warps; ++k)
                bits = max(bits, __float_as_uint(tops.of[k]));
            // (Inf, or nothing but zeros: the sum says it all)
            const bool scaled = bits != 0u && bits < 0x7F800000u;
            const int e = scaled ? max(ilogbf(__uint_as_float(bits)), -126) : 0;
            float t = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float u, v;
                    f2_unpack(f[j][k], u, v);
                    u = scalbnf(u, -e);
                    v = scalbnf(v, -e);
                    t = __fadd_rn(t, __fadd_rn(__fmul_rn(u, u), __fmul_rn(v, v)));
                }
            t = warp_sum(t);
            if (lane == 0)
                sums.of[warp] = t;
            group_sync();
            if (scaled) {
                const double ms = scalbn(static_cast<double>(sums.joined(plan.warps)) / a.D, 2 * e);
                const double r = 1.0 / sqrt(ms + static_cast<double>(a.eps));
                // without eps 1 / rms of the smallest rows is past fp32, not so its product with
                // them
                stored = static_cast<float>(r);
                rstd = static_cast<float>(scalbn(r, e));
                down = f2_splat(scalbnf(1.0f, -e));
            } else {
                stored = rstd =
                    __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), a.eps)));
            }
        }
        if (leader && a.rstd_out)
            a.rstd_out[row] = stored;
        // ---- its blocks
        const u64 r2 = f2_splat(rstd);
        const int64_t base = static_cast<int64_t>(row) * Dv;
        auto store = [&](const u64 (&v)[4], int j, void* codes, void* scales) {
            uint32_t o[2];
            const uint32_t byte = quantize_pairs<4, 4>(v, o);
            if (has[j])
                static_cast<uint2*>(codes)[base + at[j]] = make_uint2(o[0], o[1]);
            // the four blocks of sixteen lanes' tile
            uint32_t t = has[j] ? byte << (2 * (lane & 12)) : 0u;
            t |= __shfl_xor_sync(kFullMask, t, 4);
            t |= __shfl_xor_sync(kFullMask, t, 8);
            put_word(scales, j, t);
        };
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (a.keep)
                store(f[j], j, a.keep, a.keep_scales);
            if (extreme)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    f[j][k] = f2_mul(f[j][k], down);
            u64 mm[4], sh[4];
            if (kWide) {
                float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), q = p;
                uint4 t = make_uint4(0u, 0u, 0u, 0u);
                if (has[j]) {
                    p = m_lo[at[j]];
                    q = m_lo[Dv + at[j]];
                    t = shifts[at[j]];
                }
                mm[0] = f2_pack(p.x, p.y);
                mm[1] = f2_pack(p.z, p.w);
                mm[2] = f2_pack(q.x, q.y);
                mm[3] = f2_pack(q.z, q.w);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sh[k] = widen<T>(word(t, k));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mm[k] = m[kWide ? 0 : j][k];
                    sh[k] = shift[kWide ? 0 : j][k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[j][k] = f2_fma(f2_mul(f[j][k], r2), mm[k], sh[k]);
            store(f[j], j, a.out, a.out_scales);
        }
    }
    if (broken)
        drain_pause();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// One CTA per SM, whose sixteen warps form groups that take a row each, up to V vectors of eight values
// a thread.  A CTA takes runs of rows of one batch, dealt to its groups in turn; a group has a ring of
// bulk copies ahead of it and keeps its columns' sums in registers; at a run's end the groups' sums are
// joined and left as a part for the last launch.  Up to two vectors a thread a row is in registers when
// its sum over the group's warps is joined, so its slot is filled again from there on.
//
// At 1 x 4216 x 4096 30.9 us, 4 of them the last launch; its bytes are 17.9 of HBM time, and twice the rows
// take 24.3 more.  No one part bounds it: without the loads of the scales 29.5, without the reduction over
// the row 29.2, without the columns' sums 30.1, without all three 26.2.
constexpr int kBwdWarps = 16;
constexpr int kBwdThreads = 32 * kBwdWarps;
constexpr int kBwdMaxStages = 8;
constexpr int kBwdJoin = kBwdThreads * 16;  // bytes a vector
constexpr int kBwdSmem = 224 * 1024;  // (and 3 KB of barriers and sums)

struct BwdPlan {
    FastDiv per_batch;  // runs of a batch
    uint32_t chunk;     // rows of a run
    uint32_t count;     // runs
    int warps;          // of a group
    int groups;
    int stages;         // of a group's ring
    int row_bytes;      // of a slot
};

// Vectors a thread, us measured: 16384 x 256 one 12.9, two 14.0; 16384 x 1024 two 30.0, one 35.5; 2108 x
// 8192 two 31.9, four 34.2; past that two would not hold a row.  (Eight warps with 255 registers, four
// vectors a thread and every value widened once: 4216 x 4096 32.6, against the 30.9 of sixteen with two.)
int row_vectors(int64_t D) { return D <= 256 ? 1 : D <= 8192 ? 2 : 4; }

int row_warps(int64_t D)
{
    const int V = row_vectors(D);
    return static_cast<int>((D / 8 + 32 * V - 1) / (32 * V));
}

int row_groups(int64_t D) { return kBwdWarps / row_warps(D); }

// Rows of a run: that 152 CTAs have one each, but two for each group at least.  It depends on S and D
// alone, so a batch's sums do not depend on the batches beside it.  One row a group is sooner done where
// there is one batch (154 x 1024: 7.6 us, two 8.8, four 11.4) and later where the runs of several are then
// more than the SMs (4 x 512 x 1024: 13.3, two 9.6, four 11.6).
int64_t bwd_chunk(int64_t S, int64_t D)
{
    const int64_t c = (S + 151) / 152, least = 2 * row_groups(D);
    return c < least ? least : c;
}

template <typename T, int V>
__global__ void __launch_bounds__(kBwdThreads, 1)
    norm_backward_kernel(const Mxfp8NormBwdArgs a, const BwdPlan plan)
{
    // four vectors a thread: the multipliers stand in shared memory, and the row is read again after
    // its sum
    constexpr bool kWide = V > 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) unsigned long long full[kBwdWarps][kBwdMaxStages];
    __shared__ Parts part[2][kBwdWarps];  // [group]

    const int lane = threadIdx.x & 31;
    const int group = (threadIdx.x >> 5) / plan.warps;
    const int warp = (threadIdx.x >> 5) - group * plan.warps;
    const int Dv = a.D / 8;
    const bool leader = warp == 0 && lane == 0;
    if (group >= plan.groups)
        return;  // (barriers count the groups' threads)
    const int threads = plan.groups * plan.warps * 32;
    auto group_sync = [&]() {
        if (plan.warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(plan.warps * 32) : "memory");
    };
    auto cta_sync = [&]() { asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory"); };
    if (leader) {
        for (int s = 0; s < plan.stages; ++s)
            mbar_init(smem_addr(&full[group][s]), 1u);
        mbar_init_fence();
    }
    if (warp == 0 && lane < 16)
        part[0][group].of[lane] = part[1][group].of[lane] = 0.0f;
    cta_sync();
    grid_dependency_sync();

    // the multipliers (kWide), or the groups' sums on their way to one another; then the rings
    float4* m_lo = reinterpret_cast<float4*>(smem);
    float4* join = reinterpret_cast<float4*>(smem);
    uint8_t* ring = smem + (kWide ? a.D * 4 : plan.groups > 1 ? kBwdJoin * V : 0) +
                    static_cast<size_t>(group) * plan.stages * plan.row_bytes;
    const uint8_t* kept = static_cast<const uint8_t*>(a.kept);
    const uint8_t* scales = static_cast<const uint8_t*>(a.kept_scales);
    const uint32_t tiles = (a.D + 127) / 128;

    // a walk over this group's rows
    struct Walk {
        uint32_t item, row, left;
    };
    auto open = [&](Walk& w) {  // the first run from w.item on that has a row for the group
        for (; w.item < plan.count; w.item += gridDim.x) {
            const uint32_t batch = plan.per_batch.div(w.item);
            const uint32_t S = static_cast<uint32_t>(a.S), last = (batch + 1) * S;
            const uint32_t begin = batch * S + (w.item - batch * plan.per_batch.d) * plan.chunk;
            const uint32_t rows = last - begin < plan.chunk ? last - begin : plan.chunk;
            if (rows > static_cast<uint32_t>(group)) {
                w.row = begin + group;
                w.left = (rows - group + plan.groups - 1) / plan.groups;
                return;
            }
        }
    };
    auto advance = [&](Walk& w) {
        w.row += plan.groups;
        if (--w.left == 0) {
            w.item += gridDim.x;
            open(w);
        }
    };
    Walk now{blockIdx.x, 0u, 0u};
    open(now);
    Walk ahead = now, soon = now;  // `soon`: whose scales and rstd are loaded next
    int put = 0;
    auto issue = [&]() {  // the leader
        if (ahead.item >= plan.count)
            return;
        const uint32_t bar = smem_addr(&full[group][put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(put) * plan.row_bytes);
        const int64_t at = static_cast<int64_t>(ahead.row) * a.D;
        fence_proxy_async();
        mbar_expect_tx(bar, static_cast<uint32_t>(plan.row_bytes));
        bulk_g2s(dst, kept + at, a.D, bar);
        bulk_g2s(dst + a.D, static_cast<const uint8_t*>(a.grad_out) + 2 * at, 2 * a.D, bar);
        if (a.grad_res)
            bulk_g2s(dst + 3 * a.D, static_cast<const uint8_t*>(a.grad_res) + 2 * at, 2 * a.D, bar);
        put = put + 1 == plan.stages ? 0 : put + 1;
        advance(ahead);
    };
    if (leader)
        for (int s = 0; s < plan.stages; ++s)
            issue();

    // a thread's vectors, and their scale bytes, which stand apart from a row's first one by as much in
    // every row
    int at[V];
    bool has[V];
    uint32_t scale_off[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        at[j] = (j * plan.warps + warp) * 32 + lane;
        has[j] = at[j] < Dv;
        const uint32_t block = static_cast<uint32_t>(at[j]) / 4;
        scale_off[j] = (block >> 2) * 512 + (block & 3);
    }
    // what the next two rows need beside the ring
    struct Beside {
        uint32_t byte[V];
        float rstd;
    };
    auto fetch = [&](Beside& e) {
        if (soon.item >= plan.count)
            return;
        e.rstd = ld_cached(a.rstd + soon.row);
        const uint8_t* from = scales + mx8_scale_at(soon.row, 0, tiles);
#pragma unroll
        for (int j = 0; j < V; ++j)
            e.byte[j] = has[j] ? ld_cached(from + scale_off[j]) : 0u;
        advance(soon);
    };
    Beside first{}, second{};
    fetch(first);
    fetch(second);

    u64 m[kWide ? 1 : V][4];
    u64 hats[V][4], gos[V][4];  // column sums of go * hat and of go
    const float inv_n = __fdiv_rn(1.0f, static_cast<float>(a.D));
    uint32_t batch = 0xFFFFFFFFu, phase = 0;
    int get = 0, odd = 0;
    bool broken = false, waiting = false;
    for (uint32_t item = blockIdx.x; item < plan.count; item += gridDim.x) {
        const uint32_t b = plan.per_batch.div(item);
        if (b != batch) {
            batch = b;  // (a thread reads the multipliers that it has written)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                u64 t[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    t[k] = f2_splat(1.0f);
                if (has[j] && a.weight) {
                    const uint4 w = ld_cached(static_cast<const uint4*>(a.weight) + at[j]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        t[k] = widen<T>(word(w, k));
                }
                if (has[j] && a.scale) {
                    const uint4 w = ld_cached(reinterpret_cast<const uint4*>(
                                                  static_cast<const T*>(a.scale) +
                                                  b * a.mod_bstride) + at[j]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        t[k] = f2_mul(t[k], f2_add(f2_splat(1.0f), widen<T>(word(w, k))));
                }
                if (kWide) {
                    if (has[j]) {
                        m_lo[at[j]] = floats(t[0], t[1]);
                        m_lo[Dv + at[j]] = floats(t[2], t[3]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        m[kWide ? 0 : j][k] = t[k];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                hats[j][k] = gos[j][k] = 0ull;
        while (now.item == item) {
            const uint32_t row = now.row;
            advance(now);
            const float r = first.rstd;
            float factor[V];  // of a code's value, to hat: a vector's eight are of one block
#pragma unroll
            for (int j = 0; j < V; ++j)
                factor[j] = __fmul_rn(mx8_scale(first.byte[j]), r);
            first = second;
            fetch(second);
            if (!broken && !mbar_wait(smem_addr(&full[group][get]), phase, kWaitLimitNs)) {
                broken = true;
                atomicOr(&g_error, kErrCopyTimeout);
            }
            const uint8_t* slot = ring + static_cast<size_t>(get) * plan.row_bytes;
            if (++get == plan.stages) {
                get = 0;
                phase ^= 1u;
            }
            uint2 x[V];
            uint4 g[V], gr[V];
            auto read = [&](int j) {
                x[j] = reinterpret_cast<const uint2*>(slot)[at[j]];
                g[j] = reinterpret_cast<const uint4*>(slot + a.D)[at[j]];
            };
            auto read_stream = [&](int j) {
                gr[j] = make_uint4(0u, 0u, 0u, 0u);
                if (a.grad_res)
                    gr[j] = reinterpret_cast<const uint4*>(slot + 3 * a.D)[at[j]];
            };
            auto value = [&](int j, int k) {
                return widen<__half>(
                    e4m3x2_half2(((k < 2 ? x[j].x : x[j].y) >> (16 * (k & 1))) & 0xFFFFu));
            };
            auto multipliers = [&](int j, u64 (&mm)[4]) {
                if (kWide) {
                    const float4 lo = m_lo[at[j]], hi = m_lo[Dv + at[j]];
                    mm[0] = f2_pack(lo.x, lo.y);
                    mm[1] = f2_pack(lo.z, lo.w);
                    mm[2] = f2_pack(hi.x, hi.y);
                    mm[3] = f2_pack(hi.z, hi.w);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mm[k] = m[kWide ? 0 : j][k];
                }
            };
            // ---- the sum over the row of go * m * hat, and the columns'
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (has[j]) {
                    read(j);
                    if (!kWide)
                        read_stream(j);
                    u64 mm[4], d = 0ull;
                    const u64 f = f2_splat(factor[j]);
                    multipliers(j, mm);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const u64 go = widen<T>(word(g[j], k));
                        const u64 p = f2_mul(go, value(j, k));
                        d = f2_fma(p, mm[k], d);
                        hats[j][k] = f2_fma(p, f, hats[j][k]);
                        gos[j][k] = f2_add(gos[j][k], go);
                    }
                    float lo, hi;
                    f2_unpack(d, lo, hi);
                    sum = __fmaf_rn(__fadd_rn(lo, hi), factor[j], sum);
                }
            sum = warp_sum(sum);
            if (plan.warps > 1) {
                if (lane == 0)
                    part[odd][group].of[warp] = sum;
                group_sync();
                sum = part[odd][group].joined(plan.warps);
                odd ^= 1;
            } else {
                __syncwarp();
            }
            // every warp is past this row's slot (kWide: past the one before it)
            if (leader && (!kWide || waiting))
                issue();
            waiting = true;
            if (!a.grad_x)
                continue;
            const float c = __fmul_rn(__fmul_rn(-sum, inv_n), r);
            const u64 rr = f2_splat(r);
            uint4* to = static_cast<uint4*>(a.grad_x) + static_cast<int64_t>(row) * Dv;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (has[j]) {
                    u64 mm[4];
                    multipliers(j, mm);
                    if (kWide) {
                        read(j);
                        read_stream(j);
                    }
                    const u64 f = f2_splat(__fmul_rn(factor[j], c));
                    uint4 o;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const u64 d = f2_fma(value(j, k), f, widen<T>(word(gr[j], k)));
                        word(o, k) = narrow<T>(
                            f2_fma(f2_mul(widen<T>(word(g[j], k)), mm[k]), rr, d));
                    }
                    st_stream(to + at[j], o);
                }
        }
        if (!a.sums)
            continue;
        float4* to = reinterpret_cast<float4*>(a.partials + static_cast<int64_t>(item) * 2 * a.D);
        if (plan.groups == 1) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (has[j]) {
                    float4* t = to + 2 * at[j];
                    t[0] = floats(hats[j][0], hats[j][1]);
                    t[1] = floats(hats[j][2], hats[j][3]);
                    t += 2 * Dv;
                    t[0] = floats(gos[j][0], gos[j][1]);
                    t[1] = floats(gos[j][2], gos[j][3]);
                }
            continue;
        }
        // half of each vector at a time, [vector][thread]: the sums of go * hat and then those of go
        const int per_group = plan.warps * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const u64(&mine)[4] = q >= 2 ? gos[j] : hats[j];
                join[j * kBwdThreads + threadIdx.x] = floats(mine[q % 2 * 2], mine[q % 2 * 2 + 1]);
            }
            cta_sync();
            for (int c = threadIdx.x; c < V * per_group; c += threads) {
                const int j = c >= per_group ? 1 : 0;  // (V is at most 2 where groups are joined)
                if (c < Dv) {
                    const float4* from = join + j * kBwdThreads + c - j * per_group;
                    float4 t = from[0];
                    for (int g = 1; g < plan.groups; ++g) {
                        const float4 p = from[g * per_group];
                        t = make_float4(__fadd_rn(t.x, p.x), __fadd_rn(t.y, p.y),
                                        __fadd_rn(t.z, p.z), __fadd_rn(t.w, p.w));
                    }
                    to[q / 2 * 2 * Dv + 2 * c + q % 2] = t;
                }
            }
            cta_sync();
        }
    }
    if (broken)
        drain_pause();
}

// The row vectors' gradients from the runs' parts, 64 columns a CTA, half a warp a part.  With one batch
// a CTA forms all of them from the same sums; else those of grad_weight are over all batches, each
// under its 1 + scale, and those of a row of grad_scale and grad_shift over one.
constexpr int kColumnThreads = 1024;
constexpr int kColumnWarps = kColumnThreads / 32;

template <typename T>
__global__ void __launch_bounds__(kColumnThreads)
    norm_columns_kernel(const Mxfp8NormBwdArgs a, FastDiv per_batch, uint32_t count)
{
    __shared__ float4 join[2][kColumnWarps][16];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tiles = (a.D + 63) / 64;
    const uint32_t which = blockIdx.x / tiles;
    const bool one = a.B == 1;
    const bool weight = !one && which == 0 && a.grad_weight;  // of several batches
    const uint32_t slice = one ? 0u : which - (a.grad_weight ? 1u : 0u);
    const uint32_t first = weight ? 0u : slice * per_batch.d;
    const uint32_t end = weight ? count : first + per_batch.d;
    const int n = static_cast<int>(blockIdx.x - which * tiles) * 64 + (lane & 15) * 4;
    auto add4 = [](float4 p, float4 q) {
        return make_float4(__fadd_rn(p.x, q.x), __fadd_rn(p.y, q.y), __fadd_rn(p.z, q.z),
                           __fadd_rn(p.w, q.w));
    };
    auto mul4 = [](float4 p, float4 q) {
        return make_float4(__fmul_rn(p.x, q.x), __fmul_rn(p.y, q.y), __fmul_rn(p.z, q.z),
                           __fmul_rn(p.w, q.w));
    };
    auto row4 = [&](const void* p, int64_t at) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(p) + at + n);
        const float2 lo = widen2<T>(w.x), hi = widen2<T>(w.y);
        return make_float4(lo.x, lo.y, hi.x, hi.y);
    };
    const float4 ones = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    auto under_scale = [&](float4 p, uint32_t batch) {
        return a.scale ? mul4(p, add4(ones, row4(a.scale, batch * a.mod_bstride))) : p;
    };
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), t = s;
    if (n < a.D) {
        constexpr uint32_t kStep = 2 * kColumnWarps;
        const float* from = a.partials + n;
        for (uint32_t i = first + 2 * warp + (lane >> 4); i < end; i += 4 * kStep) {
            float4 p[4], q[4];  // on their way at once
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p[k] = q[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i + k * kStep < end) {
                    const float* at = from + static_cast<int64_t>(i + k * kStep) * 2 * a.D;
                    p[k] = *reinterpret_cast<const float4*>(at);
                    if (!weight)
                        q[k] = *reinterpret_cast<const float4*>(at + a.D);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (weight && i + k * kStep < end)
                    p[k] = under_scale(p[k], per_batch.div(i + k * kStep));
                s = add4(s, p[k]);
                t = add4(t, q[k]);
            }
        }
    }
    auto halves = [&](float4 p) {
        return add4(p, make_float4(__shfl_xor_sync(kFullMask, p.x, 16),
                                   __shfl_xor_sync(kFullMask, p.y, 16),
                                   __shfl_xor_sync(kFullMask, p.z, 16),
                                   __shfl_xor_sync(kFullMask, p.w, 16)));
    };
    s = halves(s);
    t = halves(t);
    join[lane >> 4][warp][lane & 15] = lane >> 4 ? t : s;
    __syncthreads();
    if (warp)
        return;
    s = join[lane >> 4][0][lane & 15];  // lanes 16 and on: the sums of go
#pragma unroll
    for (int k = 1; k < kColumnWarps; ++k)
        s = add4(s, join[lane >> 4][k][lane & 15]);
    if (n >= a.D)
        return;
    const int64_t at = static_cast<int64_t>(slice) * a.D + n;
    if (lane >> 4) {
        if (!weight && a.grad_shift)
            *reinterpret_cast<float4*>(a.grad_shift + at) = s;
        return;
    }
    if (weight || (one && a.grad_weight))
        *reinterpret_cast<float4*>(a.grad_weight + n) = weight ? s : under_scale(s, 0);
    if (!weight && a.grad_scale)
        *reinterpret_cast<float4*>(a.grad_scale + at) = a.weight ? mul4(s, row4(a.weight, 0)) : s;
}

template <typename T, int V>
cudaError_t launch_backward_rows(const Mxfp8NormBwdArgs& a, BwdPlan p, const DeviceInfo& dev,
                                 cudaStream_t stream)
{
    const int fixed = V > 2 ? a.D * 4 : p.groups > 1 ? V * kBwdJoin : 0;
    const int slot = p.groups * p.row_bytes;
    p.stages = (kBwdSmem - fixed) / slot;
    p.stages = p.stages > kBwdMaxStages ? kBwdMaxStages : p.stages;
    if (p.stages < 2)  // (four vectors: that of the row before stays taken until this one is summed)
        return cudaErrorInvalidValue;
    static PerDeviceInt ready;
    int v = 0;
    const cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(norm_backward_kernel<T, V>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int grid = static_cast<int>(p.count) < dev.sms ? static_cast<int>(p.count) : dev.sms;
    return launch_dependent(norm_backward_kernel<T, V>, grid, kBwdThreads,
                            fixed + p.stages * slot, stream, a, p);
}

template <typename T>
cudaError_t launch_backward(const Mxfp8NormBwdArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const int64_t chunk = bwd_chunk(a.S, a.D);
    const int64_t per_batch = (a.S + chunk - 1) / chunk, count = a.B * per_batch;
    if (count > INT32_MAX)
        return cudaErrorInvalidValue;
    BwdPlan p{};
    p.per_batch = FastDiv::make(static_cast<uint32_t>(per_batch));
    p.chunk = static_cast<uint32_t>(chunk);
    p.count = static_cast<uint32_t>(count);
    p.warps = row_warps(a.D);
    p.groups = row_groups(a.D);
    p.row_bytes = a.D * (a.grad_res ? 5 : 3);
    const int V = row_vectors(a.D);
    const cudaError_t e = V == 1   ? launch_backward_rows<T, 1>(a, p, dev, stream)
                          : V == 2 ? launch_backward_rows<T, 2>(a, p, dev, stream)
                                   : launch_backward_rows<T, 4>(a, p, dev, stream);
    if (e != cudaSuccess || !a.sums)
        return e;
    const int64_t tiles = (a.D + 63) / 64;
    const int64_t slices =
        a.B == 1 ? 1 : (a.grad_weight ? 1 : 0) + (a.grad_scale || a.grad_shift ? a.B : 0);
    if (slices * tiles > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_dependent(norm_columns_kernel<T>, static_cast<int>(slices * tiles), kColumnThreads,
                            0, stream, a, p.per_batch, p.count);
}

template <typename T, int V>
cudaError_t launch_forward_rows(const Mxfp8NormArgs& a, FwdPlan p, const DeviceInfo& dev,
                                cudaStream_t stream)
{
    const int fixed = V > 2 ? p.groups * a.D * 6 : 0;
    p.stages = (kFwdSmem - fixed) / (p.groups * p.row_bytes);
    p.stages = p.stages > kFwdMaxStages ? kFwdMaxStages : p.stages;
    if (p.stages < 1)
        return cudaErrorInvalidValue;
    static PerDeviceInt ready;
    int v = 0;
    const cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(norm_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kFwdSmem);
    });
    if (e != cudaSuccess)
        return e;
    const int grid = static_cast<int>(p.rows < static_cast<uint32_t>(dev.sms) ? p.rows : dev.sms);
    return launch_dependent(norm_kernel<T, V>, grid, kFwdThreads,
                            fixed + p.groups * p.stages * p.row_bytes, stream, a, p);
}

template <typename T>
cudaError_t launch_forward(const Mxfp8NormArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    // Vectors a thread: few enough that a row is a warp's or that two groups share the CTA at least (one
    // works while the other waits for its sum), and past two those that leave fewer lanes idle.
    // Measured, us with `keep`: 16384 x 256 one 8.9, two 11.6; 4216 x 1024 two 8.0, one 9.5, four 8.3;
    // 3400 x 5120 (four by the rule) four 28.6, three 31.3, two 37.3; 2800 x 6144 (three) three 28.6,
    // four 30.8, two 33.1; 2108 x 8192 four 29.3, two 30.7, three 34.8.  At 4096 four would be faster in
    // the middle (4216 rows: 27.8 against 29.1) and slower at both ends (4 rows: 4.0 against 2.8; 17024
    // rows, not kept: 90.6 against 79.5).
    const int Dv = a.D / 8;
    const auto busy = [Dv](int V) { return 12 / V * (kFwdWarps / ((Dv + 32 * V - 1) / (32 * V))); };
    const int V = Dv <= 32 ? 1 : Dv <= 512 ? 2 : Dv <= 768 && busy(3) > busy(4) ? 3 : 4;
    FwdPlan p{};
    p.by_S = FastDiv::make(a.S);
    p.rows = (a.rows + 127u) / 128u * 128u;
    p.warps = (Dv + 32 * V - 1) / (32 * V);
    p.groups = kFwdWarps / p.warps;
    p.row_bytes = a.D * (a.update ? 4 : 2);
    return V == 1   ? launch_forward_rows<T, 1>(a, p, dev, stream)
           : V == 2 ? launch_forward_rows<T, 2>(a, p, dev, stream)
           : V == 3 ? launch_forward_rows<T, 3>(a, p, dev, stream)
                    : launch_forward_rows<T, 4>(a, p, dev, stream);
}

}  // namespace

cudaError_t launch_mxfp8_norm(const Mxfp8NormArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    return a.f16 ? launch_forward<__half>(a, dev, stream)
                 : launch_forward<__nv_bfloat16>(a, dev, stream);
}

size_t mxfp8_norm_backward_workspace_bytes(int64_t B, int64_t S, int64_t D)
{
    const auto runs = [D](int64_t b, int64_t s) {
        const int64_t c = bwd_chunk(s, D);
        return b * ((s + c - 1) / c);
    };
    const int64_t apart = runs(B, S), joined = runs(1, B * S);
    return static_cast<size_t>((apart > joined ? apart : joined) * 2 * D) * 4;
}

cudaError_t launch_mxfp8_norm_backward(const Mxfp8NormBwdArgs& args, const DeviceInfo& dev,
                                       cudaStream_t stream)
{
    Mxfp8NormBwdArgs a = args;
    if (a.mod_bstride == 0) {  // one row for all batches
        a.S *= a.B;
        a.B = 1;
    }
    if (!a.grad_x)
        a.grad_res = nullptr;  // (nothing to add it to: not read)
    return a.f16 ? launch_backward<__half>(a, dev, stream)
                 : launch_backward<__nv_bfloat16>(a, dev, stream);
}

cudaError_t mxfp8_norm_error(unsigned* bits, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_error, sizeof(unsigned));
    if (e == cudaSuccess && clear && *bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_error, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace rmsmod
