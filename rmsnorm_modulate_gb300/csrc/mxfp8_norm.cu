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
// over tokens, S) alone fixes.  Both are bound by HBM: 7 to 8 bytes a value forward, 7 backward.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "mxfp8.cuh"
#include "mxfp8.h"
#include "sectors.cuh"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

// The approximate root and one Newton step: within 2 * 2^-24 of the root.
__device__ __forceinline__ float rstd_fast(float sum, float inv_n, float eps)
{
    const float ms = __fmaf_rn(sum, inv_n, eps);
    const float y = rsqrtf(ms);
    return __fmaf_rn(__fmul_rn(0.5f, y), __fmaf_rn(__fmul_rn(-ms, y), y, 1.0f), y);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kFullMask, v, off));
    return v;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// A CTA takes the four rows r, r + 32, r + 64, r + 96 of a row tile, whose scale bytes are neighbours
// (they are stored 16 bytes at a time); `warps` warps take a row, each thread V chunks of 16
// neighbouring values, so that two lanes share a block.
constexpr int kRows = 4;
constexpr int kMaxRowWarps = 8;

template <typename T, int V>
__global__ void __launch_bounds__(kRows * kMaxRowWarps * 32)
    norm_kernel(const Mxfp8NormArgs a, int warps, FastDiv by_S)
{
    __shared__ __align__(16) float part[kRows][kMaxRowWarps];
    extern __shared__ uint32_t words[];  // [out, keep][block tile][row]
    const int tid = threadIdx.x, lane = tid & 31;
    const int i = (tid >> 5) / warps;          // which of the four rows
    const int warp = (tid >> 5) - i * warps;   // of the row
    const int at = warp * 32 + lane, step = warps * 32;
    const int chunks = a.D / 16, tiles = (a.D + 127) / 128;
    const uint32_t tile = blockIdx.x >> 5, r = blockIdx.x & 31;
    const uint32_t row = tile * 128 + r + 32 * i;
    const bool has = row < a.rows;
    if (warp == 0 && lane >= warps && lane < kMaxRowWarps)
        part[i][lane] = 0.0f;
    grid_dependency_sync();

    // ---- the row
    const int64_t base = static_cast<int64_t>(row) * a.D;
    uint4 x[V][2];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = j * step + at;
        x[j][0] = x[j][1] = make_uint4(0u, 0u, 0u, 0u);
        if (has && c < chunks)
            load_pair(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + base + c * 16), true,
                      a.wide, x[j]);
    }
    if (a.update) {
        uint4 u[V][2];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = j * step + at;
            u[j][0] = u[j][1] = make_uint4(0u, 0u, 0u, 0u);
            if (has && c < chunks)
                load_pair(reinterpret_cast<const uint4*>(static_cast<const T*>(a.update) + base +
                                                         c * 16),
                          true, a.wide, u[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 p = widen2<T>(word(x[j][k >> 2], k & 3));
                const float2 q = widen2<T>(word(u[j][k >> 2], k & 3));
                word(x[j][k >> 2], k & 3) = narrow2<T>(__fadd_rn(p.x, q.x), __fadd_rn(p.y, q.y));
            }
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 p = widen2<T>(word(x[j][k >> 2], k & 3));
            s[0] = __fmaf_rn(p.x, p.x, s[0]);
            s[1] = __fmaf_rn(p.y, p.y, s[1]);
        }
    const float mine = warp_sum(__fadd_rn(s[0], s[1]));
    if (lane == 0)
        part[i][warp] = mine;
    auto joined = [&](int which) {
        const float4 p = *reinterpret_cast<const float4*>(&part[which][0]);
        const float4 q = *reinterpret_cast<const float4*>(&part[which][4]);
        return __fadd_rn(__fadd_rn(__fadd_rn(p.x, p.y), __fadd_rn(p.z, p.w)),
                         __fadd_rn(__fadd_rn(q.x, q.y), __fadd_rn(q.z, q.w)));
    };
    // squares that leave fp32's comfortable range: past 2^120 (a warp's part past 2^117), or so small
    // that a tiny eps leaves them to decide
    const bool look = __syncthreads_or(mine > 1.6e35f || a.eps < 1e-18f);
    const float sum = joined(i);
    const float n = static_cast<float>(a.D);
    float rstd = rstd_fast(sum, __fdiv_rn(1.0f, n), a.eps);
    float stored = rstd, down = 1.0f;  // (of scaled rows the values are multiplied by `down` first)
    if (look) {
        // again over the power of two of the largest magnitude, joined in fp64
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 p = widen2<T>(word(x[j][k >> 2], k & 3));
                top = max(top, max(magnitude_bits(p.x), magnitude_bits(p.y)));
            }
        top = __reduce_max_sync(kFullMask, top);
        __syncthreads();
        if (lane == 0)
            part[i][warp] = __uint_as_float(top);
        __syncthreads();
        top = 0u;
#pragma unroll
        for (int k = 0; k < kMaxRowWarps; ++k)
            top = max(top, __float_as_uint(part[i][k]));
        // (Inf, NaN, or nothing but zeros: the sum says it all)
        const bool scaled = top != 0u && top < 0x7F800000u && (sum > 1.3e36f || sum < 8e-25f);
        const int e = scaled ? max(ilogbf(__uint_as_float(top)), -126) : 0;
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 p = widen2<T>(word(x[j][k >> 2], k & 3));
                const float u = scalbnf(p.x, -e), v = scalbnf(p.y, -e);
                t = __fadd_rn(t, __fadd_rn(__fmul_rn(u, u), __fmul_rn(v, v)));
            }
        t = warp_sum(t);
        __syncthreads();
        if (lane == 0)
            part[i][warp] = t;
        __syncthreads();
        if (scaled) {
            const double ms = scalbn(static_cast<double>(joined(i)) / a.D, 2 * e);
            const double r = 1.0 / sqrt(ms + static_cast<double>(a.eps));
            // without eps 1 / rms of the smallest rows is past fp32, not so its product with them
            stored = static_cast<float>(r);
            rstd = static_cast<float>(scalbn(r, e));
            down = scalbnf(1.0f, -e);
        } else if (top == 0u || top >= 0x7F800000u) {  // where Newton's step would multiply 0 by Inf
            stored = rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), a.eps)));
        }
    }
    if (has && a.rstd_out && warp == 0 && lane == 0)
        a.rstd_out[row] = stored;

    // ---- its blocks
    const int64_t mod = has ? by_S.div(row) * a.mod_bstride : 0;
    // a chunk's codes; the four scale bytes of its block tile go to shared memory
    auto store_chunk = [&](const float (&f)[16], int c, void* codes, int which) {
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            bits = max(bits, magnitude_bits(f[k]));
        bits = max(bits, __shfl_xor_sync(kFullMask, bits, 1));
        const uint32_t byte = mx8_scale_byte(bits);
        const float inv = mx8_inverse(byte);
        uint4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            word(o, k) = e4m3x4(__fmul_rn(f[4 * k], inv), __fmul_rn(f[4 * k + 1], inv),
                                __fmul_rn(f[4 * k + 2], inv), __fmul_rn(f[4 * k + 3], inv));
        if (has && c < chunks)
            st_stream(reinterpret_cast<uint4*>(static_cast<uint8_t*>(codes) + base + c * 16), o);
        uint32_t w = has && c < chunks ? byte << (8 * ((lane >> 1) & 3)) : 0u;
        w |= __shfl_xor_sync(kFullMask, w, 2);
        w |= __shfl_xor_sync(kFullMask, w, 4);
        if ((lane & 7) == 0 && c < tiles * 8)
            words[(which * tiles + c / 8) * kRows + i] = w;
    };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = j * step + at;
        float f[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 p = widen2<T>(word(x[j][k >> 2], k & 3));
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
        }
        if (has && c < chunks && a.update)
            store_pair(reinterpret_cast<uint4*>(static_cast<T*>(a.res_out) + base + c * 16), true,
                       a.wide, x[j]);
        if (a.keep)
            store_chunk(f, c, a.keep, 1);
        if (look)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                f[k] = __fmul_rn(f[k], down);
#pragma unroll
        for (int k = 0; k < 16; ++k)
            f[k] = __fmul_rn(f[k], rstd);
        if (has && c < chunks) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float m[8];
                if (a.weight) {
                    const uint4 w = ld_cached(reinterpret_cast<const uint4*>(
                        static_cast<const T*>(a.weight) + c * 16 + 8 * h));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = widen2<T>(word(w, k));
                        m[2 * k] = p.x;
                        m[2 * k + 1] = p.y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        m[k] = 1.0f;
                }
                if (a.scale) {
                    const uint4 w = ld_cached(reinterpret_cast<const uint4*>(
                        static_cast<const T*>(a.scale) + mod + c * 16 + 8 * h));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = widen2<T>(word(w, k));
                        m[2 * k] = __fmul_rn(m[2 * k], __fadd_rn(1.0f, p.x));
                        m[2 * k + 1] = __fmul_rn(m[2 * k + 1], __fadd_rn(1.0f, p.y));
                    }
                }
                if (a.shift) {
                    const uint4 w = ld_cached(reinterpret_cast<const uint4*>(
                        static_cast<const T*>(a.shift) + mod + c * 16 + 8 * h));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = widen2<T>(word(w, k));
                        f[8 * h + 2 * k] = __fmaf_rn(f[8 * h + 2 * k], m[2 * k], p.x);
                        f[8 * h + 2 * k + 1] = __fmaf_rn(f[8 * h + 2 * k + 1], m[2 * k + 1], p.y);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        f[8 * h + k] = __fmul_rn(f[8 * h + k], m[k]);
                }
            }
        }
        store_chunk(f, c, a.out, 0);
    }
    __syncthreads();
    for (int t = tid; t < tiles * (a.keep ? 2 : 1); t += blockDim.x) {
        const int which = t >= tiles ? 1 : 0;
        static_cast<uint4*>(which ? a.keep_scales : a.out_scales)
            [(static_cast<int64_t>(tile) * tiles + t - which * tiles) * 32 + r] =
                reinterpret_cast<const uint4*>(words)[t];
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// One CTA per SM, of sixteen warps in groups that take a row each (up to V vectors of eight values a
// thread); a group walks over runs of rows of one batch, with a ring of bulk copies ahead of it, and
// keeps its columns' sums in registers, to be left at the run's end as a part for the last launch.
constexpr int kBwdWarps = 16;
constexpr int kBwdThreads = kBwdWarps * 32;
constexpr int kBwdMaxStages = 8;
constexpr int kBwdSmem = 224 * 1024;  // (and 3 KB of barriers and sums)
constexpr int kBwdRing = 160 * 1024;  // what the rings take of it, where two slots a group allow

struct BwdPlan {
    FastDiv per_batch;  // runs of a batch
    uint32_t chunk;     // rows of a run
    uint32_t count;     // runs
    int warps;          // of a group
    int groups;
    int stages;
    int row_bytes;      // of a slot
};

// Vectors of a thread: as few as leave a row to one CTA.
int bwd_vectors(int64_t D) { return D <= 4096 ? 1 : D <= 8192 ? 2 : 4; }
int bwd_warps(int64_t D) { return static_cast<int>((D / 8 + 32 * bwd_vectors(D) - 1) / (32 * bwd_vectors(D))); }

// Rows of a run: that 152 CTAs' groups have one each, but eight at least, whose parts are then a
// quarter of the rows' bytes.
int64_t bwd_chunk(int64_t S, int64_t D)
{
    const int64_t slots = 152 * (kBwdWarps / bwd_warps(D));
    const int64_t c = (S + slots - 1) / slots;
    return c < 8 ? 8 : c;
}

template <typename T, int V>
__global__ void __launch_bounds__(kBwdThreads, 1)
    norm_backward_kernel(const Mxfp8NormBwdArgs a, const BwdPlan plan)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) unsigned long long full[kBwdWarps][kBwdMaxStages];
    __shared__ float part[kBwdWarps][2][kBwdWarps];
    constexpr bool kShared = V == 4;  // the multipliers in shared memory

    const int lane = threadIdx.x & 31;
    const int group = (threadIdx.x >> 5) / plan.warps;
    const int warp = (threadIdx.x >> 5) - group * plan.warps;
    if (group >= plan.groups)
        return;  // (no barrier of the whole CTA follows)
    const int Dv = a.D / 8;
    const bool leader = warp == 0 && lane == 0;
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
    group_sync();
    grid_dependency_sync();

    float4* m_lo = reinterpret_cast<float4*>(smem);  // kShared: [Dv] and [Dv]
    uint8_t* ring = smem + (kShared ? a.D * 4 : 0) +
                    static_cast<size_t>(group) * plan.stages * plan.row_bytes;
    const uint8_t* kept = static_cast<const uint8_t*>(a.kept);
    const uint8_t* scales = static_cast<const uint8_t*>(a.kept_scales);
    const int64_t tiles = (a.D + 127) / 128;

    // a walk over this group's rows
    struct Walk {
        uint32_t item, row, end;
    };
    const uint32_t stride = gridDim.x * plan.groups;
    auto open = [&](Walk& w) {
        if (w.item >= plan.count)
            return;
        const uint32_t batch = plan.per_batch.div(w.item);
        const uint32_t S = static_cast<uint32_t>(a.S);
        w.row = batch * S + (w.item - batch * plan.per_batch.d) * plan.chunk;
        const uint32_t last = (batch + 1) * S;
        w.end = last - w.row < plan.chunk ? last : w.row + plan.chunk;
    };
    auto next = [&](Walk& w) {
        if (++w.row < w.end)
            return;
        w.item += stride;
        open(w);
    };
    Walk now{blockIdx.x * plan.groups + group, 0u, 0u};
    open(now);
    Walk ahead = now;
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
        next(ahead);
    };
    if (leader)
        for (int s = 0; s < plan.stages; ++s)
            issue();

    // what a row needs beside the ring, one row ahead
    uint32_t byte[V];
    float rstd = 0.0f;
    auto fetch = [&](const Walk& w) {
        if (w.item >= plan.count)
            return;
        rstd = __ldg(a.rstd + w.row);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * plan.warps + warp) * 32 + lane;
            byte[j] = c < Dv ? __ldg(scales + mx8_scale_at(w.row, c / 4, tiles)) : 0u;
        }
    };
#pragma unroll
    for (int j = 0; j < V; ++j)
        byte[j] = 0u;
    fetch(now);

    float m[kShared ? 1 : V][8];
    float hats[V][8], gos[V][8];  // column sums of go * hat and of go
    const float inv_n = __fdiv_rn(1.0f, static_cast<float>(a.D));
    uint32_t batch = 0xFFFFFFFFu, phase = 0;
    int get = 0, odd = 0;
    bool broken = false;
    while (now.item < plan.count) {
        const uint32_t item = now.item;
        const uint32_t b = plan.per_batch.div(item);
        if (b != batch) {
            batch = b;
            if (kShared)
                group_sync();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * plan.warps + warp) * 32 + lane;
                float t[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    t[k] = c < Dv ? 1.0f : 0.0f;
                if (c < Dv && a.weight) {
                    const uint4 w = ld_cached(static_cast<const uint4*>(a.weight) + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = widen2<T>(word(w, k));
                        t[2 * k] = p.x;
                        t[2 * k + 1] = p.y;
                    }
                }
                if (c < Dv && a.scale) {
                    const uint4 w = ld_cached(reinterpret_cast<const uint4*>(
                                                  static_cast<const T*>(a.scale) +
                                                  b * a.mod_bstride) + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 p = widen2<T>(word(w, k));
                        t[2 * k] = __fmul_rn(t[2 * k], __fadd_rn(1.0f, p.x));
                        t[2 * k + 1] = __fmul_rn(t[2 * k + 1], __fadd_rn(1.0f, p.y));
                    }
                }
                if (kShared) {
                    if (c < Dv) {
                        m_lo[c] = make_float4(t[0], t[1], t[2], t[3]);
                        m_lo[Dv + c] = make_float4(t[4], t[5], t[6], t[7]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        m[kShared ? 0 : j][k] = t[k];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                hats[j][k] = gos[j][k] = 0.0f;
        while (now.item == item) {
            if (!broken && !mbar_wait(smem_addr(&full[group][get]), phase, kWaitLimitNs)) {
                broken = true;
                atomicOr(&g_error, kErrCopyTimeout);
            }
            const uint8_t* slot = ring + static_cast<size_t>(get) * plan.row_bytes;
            if (++get == plan.stages) {
                get = 0;
                phase ^= 1u;
            }
            const int64_t at = static_cast<int64_t>(now.row) * Dv;
            const float r = rstd;
            float scale[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                scale[j] = mx8_scale(byte[j]);
            next(now);
            fetch(now);
            // ---- hat and go * m: their product's sum over the row
            uint2 x[V];
            uint4 g[V];
            float dot[2] = {0.0f, 0.0f};
            auto values = [&](int j, float (&hat)[8], float (&go)[8], float (&mm)[8]) {
                const int c = (j * plan.warps + warp) * 32 + lane;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 p = e4m3x2_values(((k < 2 ? x[j].x : x[j].y) >> (16 * (k & 1))) &
                                                   0xFFFFu);
                    hat[2 * k] = __fmul_rn(__fmul_rn(p.x, scale[j]), r);
                    hat[2 * k + 1] = __fmul_rn(__fmul_rn(p.y, scale[j]), r);
                    const float2 q = widen2<T>(word(g[j], k));
                    go[2 * k] = q.x;
                    go[2 * k + 1] = q.y;
                }
                if (kShared) {
                    const float4 lo = c < Dv ? m_lo[c] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    const float4 hi = c < Dv ? m_lo[Dv + c] : lo;
                    mm[0] = lo.x;
                    mm[1] = lo.y;
                    mm[2] = lo.z;
                    mm[3] = lo.w;
                    mm[4] = hi.x;
                    mm[5] = hi.y;
                    mm[6] = hi.z;
                    mm[7] = hi.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mm[k] = m[kShared ? 0 : j][k];
                }
            };
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * plan.warps + warp) * 32 + lane;
                x[j] = make_uint2(0u, 0u);
                g[j] = make_uint4(0u, 0u, 0u, 0u);
                if (c < Dv) {
                    x[j] = reinterpret_cast<const uint2*>(slot)[c];
                    g[j] = reinterpret_cast<const uint4*>(slot + a.D)[c];
                }
                float hat[8], go[8], mm[8];
                values(j, hat, go, mm);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    dot[k & 1] = __fmaf_rn(__fmul_rn(go[k], mm[k]), hat[k], dot[k & 1]);
                    hats[j][k] = __fmaf_rn(go[k], hat[k], hats[j][k]);
                    gos[j][k] = __fadd_rn(gos[j][k], go[k]);
                }
            }
            float sum = warp_sum(__fadd_rn(dot[0], dot[1]));
            if (plan.warps > 1) {
                if (lane == 0)
                    part[group][odd][warp] = sum;
                group_sync();
                sum = 0.0f;
                for (int k = 0; k < plan.warps; ++k)
                    sum = __fadd_rn(sum, part[group][odd][k]);
                odd ^= 1;
            } else {
                __syncwarp();
            }
            const float c1 = __fmul_rn(sum, inv_n);
            if (a.grad_x) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = (j * plan.warps + warp) * 32 + lane;
                    if (c < Dv) {
                        float hat[8], go[8], mm[8];
                        values(j, hat, go, mm);
                        uint4 gr = make_uint4(0u, 0u, 0u, 0u);
                        if (a.grad_res)
                            gr = reinterpret_cast<const uint4*>(slot + 3 * a.D)[c];
                        uint4 o;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 q = widen2<T>(word(gr, k));
                            const float lo = __fmaf_rn(-hat[2 * k], c1, __fmul_rn(go[2 * k], mm[2 * k]));
                            const float hi = __fmaf_rn(-hat[2 * k + 1], c1,
                                                       __fmul_rn(go[2 * k + 1], mm[2 * k + 1]));
                            word(o, k) = narrow2<T>(__fmaf_rn(r, lo, q.x), __fmaf_rn(r, hi, q.y));
                        }
                        st_stream(static_cast<uint4*>(a.grad_x) + at + c, o);
                    }
                }
            }
            // the slot is free when all of the group's warps have read it
            group_sync();
            if (leader)
                issue();
        }
        if (a.sums) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * plan.warps + warp) * 32 + lane;
                if (c < Dv) {
                    float4* to = reinterpret_cast<float4*>(a.partials +
                                                           static_cast<int64_t>(item) * 2 * a.D) + 2 * c;
                    to[0] = make_float4(hats[j][0], hats[j][1], hats[j][2], hats[j][3]);
                    to[1] = make_float4(hats[j][4], hats[j][5], hats[j][6], hats[j][7]);
                    to += 2 * Dv;
                    to[0] = make_float4(gos[j][0], gos[j][1], gos[j][2], gos[j][3]);
                    to[1] = make_float4(gos[j][4], gos[j][5], gos[j][6], gos[j][7]);
                }
            }
        }
    }
    if (broken)
        drain_pause();
}

// The row vectors' gradients from the runs' parts: for grad_weight those of all batches, each under
// its 1 + scale, for a row of grad_scale and grad_shift those of one; eight warps take every eighth,
// 128 columns a CTA.
constexpr int kColumnThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kColumnThreads)
    norm_columns_kernel(const Mxfp8NormBwdArgs a, FastDiv per_batch, uint32_t count)
{
    __shared__ float4 join[2][kColumnThreads / 32][32];
    grid_dependency_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tiles = (a.D + 127) / 128;
    const uint32_t which = blockIdx.x / tiles;
    const bool weight = which == 0 && a.grad_weight;
    const uint32_t slice = which - (a.grad_weight ? 1u : 0u);
    const uint32_t first = weight ? 0u : slice * per_batch.d;
    const uint32_t end = weight ? count : first + per_batch.d;
    const int n = static_cast<int>(blockIdx.x - which * tiles) * 128 + lane * 4;
    auto row4 = [&](const void* p, int64_t at) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(p) + at + n);
        const float2 lo = widen2<T>(w.x), hi = widen2<T>(w.y);
        return make_float4(lo.x, lo.y, hi.x, hi.y);
    };
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), t = s;
    if (n < a.D)
        for (uint32_t i = first + warp; i < end; i += kColumnThreads / 32) {
            const float* from = a.partials + static_cast<int64_t>(i) * 2 * a.D + n;
            float4 p = *reinterpret_cast<const float4*>(from);
            if (weight) {
                if (a.scale) {
                    const float4 f = row4(a.scale, per_batch.div(i) * a.mod_bstride);
                    p = make_float4(__fmul_rn(p.x, __fadd_rn(1.0f, f.x)),
                                    __fmul_rn(p.y, __fadd_rn(1.0f, f.y)),
                                    __fmul_rn(p.z, __fadd_rn(1.0f, f.z)),
                                    __fmul_rn(p.w, __fadd_rn(1.0f, f.w)));
                }
            } else {
                const float4 q = *reinterpret_cast<const float4*>(from + a.D);
                t = make_float4(__fadd_rn(t.x, q.x), __fadd_rn(t.y, q.y), __fadd_rn(t.z, q.z),
                                __fadd_rn(t.w, q.w));
            }
            s = make_float4(__fadd_rn(s.x, p.x), __fadd_rn(s.y, p.y), __fadd_rn(s.z, p.z),
                            __fadd_rn(s.w, p.w));
        }
    join[0][warp][lane] = s;
    join[1][warp][lane] = t;
    __syncthreads();
    if (warp > 1 || n >= a.D || (warp == 1 && weight))
        return;
    s = join[warp][0][lane];
#pragma unroll
    for (int k = 1; k < kColumnThreads / 32; ++k) {
        const float4 p = join[warp][k][lane];
        s = make_float4(__fadd_rn(s.x, p.x), __fadd_rn(s.y, p.y), __fadd_rn(s.z, p.z),
                        __fadd_rn(s.w, p.w));
    }
    float* to = weight ? a.grad_weight : warp ? a.grad_shift : a.grad_scale;
    if (!to)
        return;
    if (!weight) {
        to += static_cast<int64_t>(slice) * a.D;
        if (warp == 0 && a.weight) {
            const float4 f = row4(a.weight, 0);
            s = make_float4(__fmul_rn(s.x, f.x), __fmul_rn(s.y, f.y), __fmul_rn(s.z, f.z),
                            __fmul_rn(s.w, f.w));
        }
    }
    *reinterpret_cast<float4*>(to + n) = s;
}

template <typename T, int V>
cudaError_t launch_backward_rows(const Mxfp8NormBwdArgs& a, const BwdPlan& plan, int grid, int smem,
                                 const DeviceInfo& dev, cudaStream_t stream)
{
    static PerDeviceInt ready;
    int v = 0;
    const cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(norm_backward_kernel<T, V>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    });
    if (e != cudaSuccess)
        return e;
    return launch_dependent(norm_backward_kernel<T, V>, grid, kBwdThreads, smem, stream, a, plan);
}

template <typename T>
cudaError_t launch_backward(const Mxfp8NormBwdArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const int64_t chunk = bwd_chunk(a.S, a.D);
    const int64_t per_batch = (a.S + chunk - 1) / chunk, count = a.B * per_batch;
    if (count > INT32_MAX)
        return cudaErrorInvalidValue;
    const int V = bwd_vectors(a.D);
    BwdPlan p{};
    p.per_batch = FastDiv::make(static_cast<uint32_t>(per_batch));
    p.chunk = static_cast<uint32_t>(chunk);
    p.count = static_cast<uint32_t>(count);
    p.warps = bwd_warps(a.D);
    p.groups = kBwdWarps / p.warps;
    p.row_bytes = a.D * (a.grad_res ? 5 : 3);
    const int fixed = V == 4 ? a.D * 4 : 0;
    p.stages = (kBwdRing - 0) / (p.groups * p.row_bytes);
    p.stages = p.stages < 2 ? 2 : p.stages > kBwdMaxStages ? kBwdMaxStages : p.stages;
    const int smem = fixed + p.groups * p.stages * p.row_bytes;
    if (smem > kBwdSmem)
        return cudaErrorInvalidValue;
    const int64_t ctas = (count + p.groups - 1) / p.groups;
    const int grid = static_cast<int>(ctas < dev.sms ? ctas : dev.sms);
    cudaError_t e;
    if (V == 1)
        e = launch_backward_rows<T, 1>(a, p, grid, smem, dev, stream);
    else if (V == 2)
        e = launch_backward_rows<T, 2>(a, p, grid, smem, dev, stream);
    else
        e = launch_backward_rows<T, 4>(a, p, grid, smem, dev, stream);
    if (e != cudaSuccess || !a.sums)
        return e;
    const int64_t tiles = (a.D + 127) / 128;
    const int64_t slices = (a.grad_weight ? 1 : 0) + (a.grad_scale || a.grad_shift ? a.B : 0);
    if (slices * tiles > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_dependent(norm_columns_kernel<T>, static_cast<int>(slices * tiles), kColumnThreads,
                            0, stream, a, p.per_batch, p.count);
}

template <typename T>
cudaError_t launch_forward(const Mxfp8NormArgs& a, cudaStream_t stream)
{
    // two chunks a thread while eight warps hold the row, one where a warp holds it that way
    const int chunks = a.D / 16;
    const int V = chunks <= 32 ? 1 : chunks <= 64 * kMaxRowWarps ? 2 : 4;
    const int warps = (chunks + 32 * V - 1) / (32 * V);
    const int grid = static_cast<int>((a.rows + 127u) / 128u * 32u);
    const int smem = (a.D + 127) / 128 * kRows * 4 * (a.keep ? 2 : 1);
    const FastDiv by_S = FastDiv::make(a.S);
    const int threads = kRows * warps * 32;
    if (V == 1)
        return launch_dependent(norm_kernel<T, 1>, grid, threads, smem, stream, a, warps, by_S);
    if (V == 2)
        return launch_dependent(norm_kernel<T, 2>, grid, threads, smem, stream, a, warps, by_S);
    return launch_dependent(norm_kernel<T, 4>, grid, threads, smem, stream, a, warps, by_S);
}

}  // namespace

cudaError_t launch_mxfp8_norm(Mxfp8NormArgs a, const DeviceInfo&, cudaStream_t stream)
{
    const auto on32 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; };
    a.wide = on32(a.x) && on32(a.update) && on32(a.res_out);
    return a.f16 ? launch_forward<__half>(a, stream) : launch_forward<__nv_bfloat16>(a, stream);
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
