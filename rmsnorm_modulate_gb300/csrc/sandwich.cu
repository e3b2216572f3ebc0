// The norms after and before a block, fused with its gate and residual scale, and their gradients.
//
//   forward   rp   = 1 / sqrt(mean(u^2) + post_eps)             u = update
//             v    = update_scale * gate * post_weight
//             res  = R(residual_scale * residual + (u * rp) * v)
//             r    = 1 / sqrt(mean(res^2) + eps)
//             out  = R((res * r) * m + shift),                  m = weight * (1 + scale)
//   backward  hh   = res * r, uh = u * rp, q = r * (go * m) + gr
//             dh   = q - r * c * hh,                            c  = mean(go * m * hh)
//             grad_residual = R(residual_scale * dh)
//             grad_update   = R(rp * (dh * v - cu * uh)),       cu = mean(dh * v * uh)
//             sums over the tokens of go, go * hh and dh * uh, from which a last launch forms the
//             gradients of shift, scale, weight, gate and post_weight
//
// All in fp32 with one rounding per stored value.  Sums run in an order that D (and, over tokens,
// S) alone fixes, so a result does not depend on the batch it stands in.
//
// Both are bound by HBM: 8 and 12 bytes per value.  A CTA takes a row at a time, two 16-byte vectors
// a thread; the rows come through a ring of bulk copies (TMA) that stays ahead of the arithmetic,
// the row vectors' products stay in registers for all rows of a batch.  Rows of more than 8192
// values are shared by a cluster of two CTAs, which exchange their partial sums through distributed
// shared memory.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "sandwich.h"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

constexpr int kV = 2;              // 16-byte vectors per thread
constexpr int kMaxStages = 8;
constexpr int kMaxThreads = 512;
constexpr int kMaxDvPerCta = kMaxThreads * kV;
constexpr int kSmemPerSm = 216 * 1024;

// ---------------------------------------------------------------------------
// sums over a row
// ---------------------------------------------------------------------------

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

__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t rank, float v)
{
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\t"
                 "st.shared::cluster.f32 [p], %2;\n\t}" ::"r"(addr),
                 "r"(rank), "f"(v)
                 : "memory");
}

template <bool CL>
__device__ __forceinline__ void row_barrier()
{
    if (CL)
        cluster_barrier();
    else
        __syncthreads();
}

// Where the warps of a row leave their partial values: [value][warp of the row, the other CTA's
// after this one's places]; zeros where the row has no warp.
constexpr int kMaxWarps = kMaxThreads / 32;

template <int N>
struct __align__(16) Exchange {
    float v[N][2 * kMaxWarps];
};

template <int N>
__device__ __forceinline__ void clear(Exchange<N>& ex)
{
    for (int i = threadIdx.x; i < N * 2 * kMaxWarps; i += blockDim.x)
        ex.v[0][i] = 0.0f;
}

// N sums (or maxima of magnitudes) over all threads of the row, in an order that the row's length
// fixes; every thread gets them.  One barrier: the same exchange may be used again after one more.
template <int N, bool CL, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&x)[N], Exchange<N>& ex, int warp, int lane,
                                           int warps, uint32_t rank)
{
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : __fadd_rn(a, b); };
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = join(x[i], __shfl_xor_sync(kFullMask, x[i], off));
    if (!CL && warps == 1)
        return;
    if (lane == 0) {
        const int at = static_cast<int>(rank) * kMaxWarps + warp;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ex.v[i][at] = x[i];
            if (CL)
                st_peer(smem_addr(&ex.v[i][at]), rank ^ 1u, x[i]);
        }
    }
    row_barrier<CL>();
    // four warps' values a load
    const int quads = CL ? 2 * kMaxWarps / 4 : (warps + 3) / 4;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* q = reinterpret_cast<const float4*>(ex.v[i]);
        float4 t = q[0];
        for (int k = 1; k < quads; ++k) {
            const float4 o = q[k];
            t = make_float4(join(t.x, o.x), join(t.y, o.y), join(t.z, o.z), join(t.w, o.w));
        }
        x[i] = join(join(t.x, t.y), join(t.z, t.w));
    }
}

template <typename T>
__device__ __forceinline__ float sum_squares(const uint4 (&x)[kV])
{
    u64 s = 0ull;
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u64 p = widen<T>(word(x[j], i));
            s = f2_fma(p, p, s);
        }
    float lo, hi;
    f2_unpack(s, lo, hi);
    return __fadd_rn(lo, hi);
}

// 1 / sqrt of a row whose fp32 sum of squares left fp32's comfortable range although its values are
// finite: squares of the values over the power of two of the largest, joined in fp64.
template <typename T, bool CL>
__device__ __noinline__ float rstd_scaled(const uint4 (&x)[kV], float sum, float n, float eps,
                                          Exchange<1>& e0, Exchange<1>& e1, int warp, int lane,
                                          int warps, uint32_t rank)
{
    float top[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = widen2<T>(word(x[j], i));
            top[0] = fmaxf(top[0], fmaxf(fabsf(p.x), fabsf(p.y)));
        }
    row_reduce<1, CL, true>(top, e0, warp, lane, warps, rank);
    // Inf, or nothing but zeros: the sum says it all.  (A NaN never gets here.)
    if (!(top[0] <= 3.4028235e38f) || top[0] == 0.0f)
        return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), eps)));
    const int e = ilogbf(top[0]);
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = widen2<T>(word(x[j], i));
            const float a = scalbnf(p.x, -e), b = scalbnf(p.y, -e);
            s[0] = __fadd_rn(s[0], __fadd_rn(__fmul_rn(a, a), __fmul_rn(b, b)));
        }
    row_reduce<1, CL>(s, e1, warp, lane, warps, rank);
    const double ms = scalbn(static_cast<double>(s[0]) / static_cast<double>(n), 2 * e);
    return static_cast<float>(1.0 / sqrt(ms + static_cast<double>(eps)));
}

template <typename T, bool CL>
__device__ __forceinline__ float rstd_of(const uint4 (&x)[kV], float sum, float n, float inv_n,
                                         float eps, Exchange<1> (&slow)[2], int warp, int lane, int warps,
                                         uint32_t rank)
{
    // past 2^120, or so small that a tiny eps leaves it to decide (uniform over the row)
    if (sum > 1.3e36f || (sum < 8e-25f && eps < 1e-18f))
        return rstd_scaled<T, CL>(x, sum, n, eps, slow[0], slow[1], warp, lane, warps, rank);
    // the approximate root and one Newton step: within 2 * 2^-24 of the root, in a tenth of the
    // instructions of a division and a square root, which every warp of a row repeats
    const float ms = __fmaf_rn(sum, inv_n, eps);
    const float y = rsqrtf(ms);
    return __fmaf_rn(__fmul_rn(0.5f, y), __fmaf_rn(__fmul_rn(-ms, y), y, 1.0f), y);
}

// ---------------------------------------------------------------------------
// rows of a CTA (or cluster): items blockIdx, blockIdx + grid, ... of `chunk` rows of one batch
// ---------------------------------------------------------------------------

struct Items {
    FastDiv per_batch;
    uint32_t chunk;
    uint32_t count;
    uint32_t S;
    int stages;
};

struct Cursor {
    uint32_t item, batch, row, end;

    __device__ __forceinline__ void open(const Items& it)
    {
        batch = it.per_batch.div(item);
        row = batch * it.S + (item - batch * it.per_batch.d) * it.chunk;
        const uint32_t left = (batch + 1) * it.S - row;
        end = row + (it.chunk < left ? it.chunk : left);
    }
    __device__ __forceinline__ bool valid(const Items& it) const { return item < it.count; }
    __device__ __forceinline__ void advance(const Items& it, uint32_t step)
    {
        if (++row < end)
            return;
        item += step;
        if (item < it.count)
            open(it);
    }
};

template <int MAXT>
constexpr int min_blocks() { return kMaxThreads / MAXT; }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

template <typename T, int MAXT, bool CL>
__global__ void __launch_bounds__(MAXT, min_blocks<MAXT>())
    sandwich_kernel(const SandwichArgs a, const Items items)
{
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ __align__(8) unsigned long long full[kMaxStages];
    __shared__ Exchange<1> ex[2], slow[2];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const uint32_t rank = CL ? cluster_rank() : 0u;
    const uint32_t step = CL ? gridDim.x / 2 : gridDim.x;
    const uint32_t first = CL ? blockIdx.x / 2 : blockIdx.x;
    // this CTA's vectors of a row
    const int half = CL ? (a.Dv + 1) / 2 : a.Dv;
    const int v0 = static_cast<int>(rank) * half;
    const int nv = a.Dv - v0 < half ? a.Dv - v0 : half;
    const uint32_t bytes = static_cast<uint32_t>(nv) * 16u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < items.stages; ++s)
            mbar_init(smem_addr(&full[s]), 1u);
        mbar_init_fence();
    }
    clear(ex[0]);
    clear(ex[1]);
    clear(slow[0]);
    clear(slow[1]);
    row_barrier<CL>();
    grid_dependency_sync();

    bool broken = false;
    const uint4* __restrict__ residual = static_cast<const uint4*>(a.residual) + v0;
    const uint4* __restrict__ update = static_cast<const uint4*>(a.update) + v0;
    uint4* res_out = static_cast<uint4*>(a.res_out) + v0;
    uint4* out = static_cast<uint4*>(a.out) + v0;

    Cursor ahead{first, 0, 0, 0};
    int put = 0;
    auto issue = [&]() {  // thread 0
        if (!ahead.valid(items))
            return;
        const uint32_t bar = smem_addr(&full[put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(put) * 2 * half);
        fence_proxy_async();
        mbar_expect_tx(bar, 2 * bytes);
        bulk_g2s(dst, update + static_cast<int64_t>(ahead.row) * a.Dv, bytes, bar);
        bulk_g2s(dst + half * 16, residual + static_cast<int64_t>(ahead.row) * a.Dv, bytes, bar);
        put = put + 1 == items.stages ? 0 : put + 1;
        ahead.advance(items, step);
    };
    Cursor at{first, 0, 0, 0};
    if (at.valid(items)) {
        at.open(items);
        ahead.open(items);
    }
    if (threadIdx.x == 0)
        for (int s = 0; s < items.stages; ++s)
            issue();

    u64 v[kV][4], m[kV][4], sh[kV][4];
    const u64 rs2 = f2_splat(a.residual_scale);
    const float inv_n = __fdiv_rn(1.0f, a.n);
    uint32_t batch = 0xFFFFFFFFu;
    int get = 0;
    uint32_t phase = 0;
    for (; at.valid(items); at.advance(items, step)) {
        const uint32_t b = at.batch;
        if (b != batch) {  // the row vectors of this batch
            batch = b;
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int c = j * blockDim.x + threadIdx.x;
                const bool in = c < nv;
                auto load = [&](const void* p, int64_t row) {
                    return in && p ? ld_cached(static_cast<const uint4*>(p) + row + v0 + c)
                                   : make_uint4(0u, 0u, 0u, 0u);
                };
                const uint4 wp = load(a.post_weight, 0), g = load(a.gate, b * a.gate_bstride);
                const uint4 w = load(a.weight, 0), sc = load(a.scale, b * a.mod_bstride);
                const uint4 sf = load(a.shift, b * a.mod_bstride);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u64 one = f2_splat(1.0f);
                    u64 t = f2_splat(a.update_scale);
                    if (a.post_weight)
                        t = f2_mul(t, widen<T>(word(wp, i)));
                    if (a.gate)
                        t = f2_mul(t, widen<T>(word(g, i)));
                    v[j][i] = t;
                    t = a.weight ? widen<T>(word(w, i)) : one;
                    m[j][i] = a.scale ? f2_mul(t, f2_add(one, widen<T>(word(sc, i)))) : t;
                    sh[j][i] = widen<T>(word(sf, i));
                }
            }
        }
        if (!broken && !mbar_wait(smem_addr(&full[get]), phase, kWaitLimitNs)) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
        const uint4* slot = ring + static_cast<size_t>(get) * 2 * half;
        uint4 u[kV], x[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            u[j] = x[j] = make_uint4(0u, 0u, 0u, 0u);
            if (c < nv) {
                u[j] = slot[c];
                x[j] = slot[half + c];
            }
        }
        float s[1] = {sum_squares<T>(u)};
        row_reduce<1, CL>(s, ex[0], warp, lane, warps, rank);
        // a barrier has passed (or this is the only warp): the slot has been read
        if (!CL && warps == 1)
            __syncwarp();
        if (threadIdx.x == 0)
            issue();
        const float rp = rstd_of<T, CL>(u, s[0], a.n, inv_n, a.post_eps, slow, warp, lane,
                                         warps, rank);
        const u64 rp2 = f2_splat(rp);
        const int64_t base = static_cast<int64_t>(at.row) * a.Dv;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                word(x[j], i) = narrow<T>(
                    f2_fma(widen<T>(word(x[j], i)), rs2,
                           f2_mul(f2_mul(widen<T>(word(u[j], i)), rp2), v[j][i])));
            if (c < nv)
                st_stream(res_out + base + c, x[j]);
            else
                x[j] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (threadIdx.x == 0 && rank == 0 && a.post_rstd_out)
            a.post_rstd_out[at.row] = rp;
        if (a.out) {
            s[0] = sum_squares<T>(x);
            row_reduce<1, CL>(s, ex[1], warp, lane, warps, rank);
            const float r = rstd_of<T, CL>(x, s[0], a.n, inv_n, a.eps, slow, warp, lane,
                                            warps, rank);
            const u64 r2 = f2_splat(r);
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int c = j * blockDim.x + threadIdx.x;
                uint4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    word(o, i) = narrow<T>(
                        f2_fma(f2_mul(widen<T>(word(x[j], i)), r2), m[j][i], sh[j][i]));
                if (c < nv)
                    st_stream(out + base + c, o);
            }
            if (threadIdx.x == 0 && rank == 0 && a.rstd_out)
                a.rstd_out[at.row] = r;
        } else {
            row_barrier<CL>();  // between two uses of ex[0]
        }
        if (++get == items.stages) {
            get = 0;
            phase ^= 1u;
        }
    }
    if (broken)
        drain_pause();
    if (CL)
        cluster_barrier();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// POST: the block's post norm takes part (update), OUT: the norm after the add does (grad_out).
template <typename T, int MAXT, bool CL, bool POST, bool OUT>
__global__ void __launch_bounds__(MAXT, min_blocks<MAXT>())
    sandwich_bwd_kernel(const SandwichBwdArgs a, const Items items)
{
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ __align__(8) unsigned long long full[kMaxStages];
    __shared__ Exchange<3> ex[2];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const uint32_t rank = CL ? cluster_rank() : 0u;
    const uint32_t step = CL ? gridDim.x / 2 : gridDim.x;
    const uint32_t first = CL ? blockIdx.x / 2 : blockIdx.x;
    const int half = CL ? (a.Dv + 1) / 2 : a.Dv;
    const int v0 = static_cast<int>(rank) * half;
    const int nv = a.Dv - v0 < half ? a.Dv - v0 : half;
    const uint32_t bytes = static_cast<uint32_t>(nv) * 16u;
    const bool has_gr = a.grad_res != nullptr;
    // rows of a slot: update, res, grad_out, grad_res
    const int k_res = POST ? 1 : 0, k_go = k_res + 1, k_gr = (POST ? 1 : 0) + (OUT ? 2 : 0);
    const int rows = k_gr + (has_gr ? 1 : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < items.stages; ++s)
            mbar_init(smem_addr(&full[s]), 1u);
        mbar_init_fence();
    }
    clear(ex[0]);
    clear(ex[1]);
    row_barrier<CL>();
    grid_dependency_sync();

    bool broken = false;
    Cursor ahead{first, 0, 0, 0};
    int put = 0;
    auto issue = [&]() {  // thread 0
        if (!ahead.valid(items))
            return;
        const uint32_t bar = smem_addr(&full[put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(put) * rows * half);
        const int64_t from = static_cast<int64_t>(ahead.row) * a.Dv + v0;
        auto bring = [&](int k, const void* p) {
            bulk_g2s(dst + k * half * 16, static_cast<const uint4*>(p) + from, bytes, bar);
        };
        fence_proxy_async();
        mbar_expect_tx(bar, rows * bytes);
        if (POST)
            bring(0, a.update);
        if (OUT) {
            bring(k_res, a.res);
            bring(k_go, a.grad_out);
        }
        if (has_gr)
            bring(k_gr, a.grad_res);
        put = put + 1 == items.stages ? 0 : put + 1;
        ahead.advance(items, step);
    };
    Cursor at{first, 0, 0, 0};
    if (at.valid(items)) {
        at.open(items);
        ahead.open(items);
    }
    // one slot less than the ring holds: a slot is refilled after the next row's barrier
    if (threadIdx.x == 0)
        for (int s = 0; s + 1 < items.stages; ++s)
            issue();

    constexpr int kParts = (OUT ? 2 : 0) + (POST ? 1 : 0);
    u64 v[kV][4], m[kV][4];
    u64 sum_go[kV][4], sum_gh[kV][4], sum_du[kV][4];
    auto restart = [&]() {
#pragma unroll
        for (int j = 0; j < kV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum_go[j][i] = sum_gh[j][i] = sum_du[j][i] = 0ull;
    };
    restart();
    const float inv_n = __fdiv_rn(1.0f, a.n);
    uint32_t batch = 0xFFFFFFFFu;
    int get = 0, par = 0;
    uint32_t phase = 0;
    float r = 0.0f, rp = 0.0f;
    if (at.valid(items)) {
        r = OUT ? a.rstd[at.row] : 0.0f;
        rp = POST ? a.post_rstd[at.row] : 0.0f;
    }
    while (at.valid(items)) {
        const uint32_t b = at.batch;
        if (b != batch) {
            batch = b;
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int c = j * blockDim.x + threadIdx.x;
                const bool in = c < nv;
                auto load = [&](const void* p, int64_t row) {
                    return in && p ? ld_cached(static_cast<const uint4*>(p) + row + v0 + c)
                                   : make_uint4(0u, 0u, 0u, 0u);
                };
                const u64 one = f2_splat(1.0f);
                if (POST) {
                    const uint4 wp = load(a.post_weight, 0), g = load(a.gate, b * a.gate_bstride);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u64 t = f2_splat(a.update_scale);
                        if (a.post_weight)
                            t = f2_mul(t, widen<T>(word(wp, i)));
                        if (a.gate)
                            t = f2_mul(t, widen<T>(word(g, i)));
                        v[j][i] = t;
                    }
                }
                if (OUT) {
                    const uint4 w = load(a.weight, 0), sc = load(a.scale, b * a.mod_bstride);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u64 t = a.weight ? widen<T>(word(w, i)) : one;
                        m[j][i] = a.scale ? f2_mul(t, f2_add(one, widen<T>(word(sc, i)))) : t;
                    }
                }
            }
        }
        if (!broken && !mbar_wait(smem_addr(&full[get]), phase, kWaitLimitNs)) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
        const uint4* slot = ring + static_cast<size_t>(get) * rows * half;
        const u64 r2 = f2_splat(r), rp2 = f2_splat(rp);
        // ---- the row's sums: s0 = sum go m hh, s1 = sum q p, s2 = sum hh p with p = v uh, from
        //      which both means follow (dh = q - r c hh)
        float s[3] = {0.0f, 0.0f, 0.0f};
        u64 t0 = 0ull, t1 = 0ull, t2 = 0ull;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nv) {
                uint4 uu, hh, go, gr;
                if (POST)
                    uu = slot[c];
                if (OUT) {
                    hh = slot[k_res * half + c];
                    go = slot[k_go * half + c];
                }
                if (POST && has_gr)
                    gr = slot[k_gr * half + c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u64 q = POST && has_gr ? widen<T>(word(gr, i)) : 0ull;
                    u64 h = 0ull;
                    if (OUT) {
                        h = f2_mul(widen<T>(word(hh, i)), r2);
                        const u64 d = f2_mul(widen<T>(word(go, i)), m[j][i]);
                        t0 = f2_fma(d, h, t0);
                        if (POST)
                            q = f2_fma(d, r2, q);
                    }
                    if (POST) {
                        const u64 p = f2_mul(f2_mul(widen<T>(word(uu, i)), rp2), v[j][i]);
                        t1 = f2_fma(q, p, t1);
                        if (OUT)
                            t2 = f2_fma(h, p, t2);
                    }
                }
            }
        }
        float lo, hi;
        f2_unpack(t0, lo, hi);
        s[0] = __fadd_rn(lo, hi);
        f2_unpack(t1, lo, hi);
        s[1] = __fadd_rn(lo, hi);
        f2_unpack(t2, lo, hi);
        s[2] = __fadd_rn(lo, hi);
        row_reduce<3, CL>(s, ex[par], warp, lane, warps, rank);
        par ^= 1;
        // every thread is past the previous row: its slot takes the next copies
        if (!CL && warps == 1)
            __syncwarp();
        if (threadIdx.x == 0)
            issue();
        // the next row's statistics, on their way during this row's second half
        Cursor next = at;
        next.advance(items, step);
        float r_next = 0.0f, rp_next = 0.0f;
        if (next.valid(items)) {
            r_next = OUT ? a.rstd[next.row] : 0.0f;
            rp_next = POST ? a.post_rstd[next.row] : 0.0f;
        }
        const float rc = __fmul_rn(r, __fmul_rn(s[0], inv_n));
        const float c_upd = __fmul_rn(__fmaf_rn(-rc, s[2], s[1]), inv_n);
        const u64 nrc2 = f2_splat(-rc), ncu2 = f2_splat(-c_upd);
        const u64 rs2 = f2_splat(a.residual_scale);
        // ---- the gradients of the row
        const int64_t base = static_cast<int64_t>(at.row) * a.Dv + v0;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = j * blockDim.x + threadIdx.x;
            if (c < nv) {
                uint4 uu, hh, go, gr, ox, ou;
                if (POST)
                    uu = slot[c];
                if (OUT) {
                    hh = slot[k_res * half + c];
                    go = slot[k_go * half + c];
                }
                if (has_gr)
                    gr = slot[k_gr * half + c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u64 dh = has_gr ? widen<T>(word(gr, i)) : 0ull;
                    if (OUT) {
                        const u64 g = widen<T>(word(go, i));
                        const u64 h = f2_mul(widen<T>(word(hh, i)), r2);
                        dh = f2_fma(f2_mul(g, m[j][i]), r2, dh);
                        dh = f2_fma(h, nrc2, dh);
                        sum_go[j][i] = f2_add(sum_go[j][i], g);
                        sum_gh[j][i] = f2_fma(g, h, sum_gh[j][i]);
                    }
                    word(ox, i) = narrow<T>(POST ? f2_mul(dh, rs2) : dh);
                    if (POST) {
                        const u64 uh = f2_mul(widen<T>(word(uu, i)), rp2);
                        sum_du[j][i] = f2_fma(dh, uh, sum_du[j][i]);
                        word(ou, i) = narrow<T>(
                            f2_mul(f2_fma(uh, ncu2, f2_mul(dh, v[j][i])), rp2));
                    }
                }
                if (a.grad_residual)
                    st_stream(static_cast<uint4*>(a.grad_residual) + base + c, ox);
                if (POST && a.grad_update)
                    st_stream(static_cast<uint4*>(a.grad_update) + base + c, ou);
            }
        }
        if (++get == items.stages) {
            get = 0;
            phase ^= 1u;
        }
        const uint32_t item = at.item;
        at = next;
        r = r_next;
        rp = rp_next;
        if (at.item != item) {  // the item's partial sums
            if (a.sums) {
                float4* to = reinterpret_cast<float4*>(a.partials) +
                             static_cast<int64_t>(item) * kParts * a.Dv * 2;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const int c = j * blockDim.x + threadIdx.x;
                    if (c >= nv)
                        continue;
                    auto leave = [&](int part, const u64 (&t)[4]) {
                        float4 f;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            f2_unpack(t[2 * h], f.x, f.y);
                            f2_unpack(t[2 * h + 1], f.z, f.w);
                            to[(static_cast<int64_t>(part) * a.Dv + v0 + c) * 2 + h] = f;
                        }
                    };
                    if (OUT) {
                        leave(0, sum_go[j]);
                        leave(1, sum_gh[j]);
                    }
                    if (POST)
                        leave(kParts - 1, sum_du[j]);
                }
            }
            restart();
        }
    }
    if (broken)
        drain_pause();
    if (CL)
        cluster_barrier();
}

// The gradients of the row vectors from the items' partial sums: 32 columns a CTA, the items of a
// batch dealt to its warps in turn and joined in the warps' order; batches in order.
constexpr int kColWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kColWarps)
    sandwich_columns_kernel(const SandwichBwdArgs a, int64_t per_batch, int parts)
{
    grid_dependency_sync();
    __shared__ float part[3][kColWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t D = static_cast<int64_t>(a.Dv) * 8;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const bool in = d < D;
    const bool out_on = a.grad_out != nullptr, post_on = a.update != nullptr;
    auto value = [&](const void* p, int64_t at, float none) {
        return p && in ? static_cast<float>(static_cast<const T*>(p)[at + d]) : none;
    };
    const float w = value(a.weight, 0, 1.0f);
    const float wp = __fmul_rn(value(a.post_weight, 0, 1.0f), a.update_scale);
    float g_w = 0.0f, g_wp = 0.0f, g_scale = 0.0f, g_shift = 0.0f, g_gate = 0.0f;
    for (int64_t b = 0; b < a.B; ++b) {
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (in) {
            const float* from = a.partials + b * per_batch * parts * D + d;
#pragma unroll 4
            for (int64_t k = warp; k < per_batch; k += kColWarps)
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    if (p < parts)
                        s[p] = __fadd_rn(s[p], __ldcs(from + (k * parts + p) * D));
        }
#pragma unroll
        for (int p = 0; p < 3; ++p)
            part[p][warp][lane] = s[p];
        __syncthreads();
        if (warp == 0 && in) {
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                s[p] = part[p][0][lane];
#pragma unroll
                for (int k = 1; k < kColWarps; ++k)
                    s[p] = __fadd_rn(s[p], part[p][k][lane]);
            }
            if (out_on) {
                const float one = __fadd_rn(1.0f, value(a.scale, b * a.mod_bstride * 8, 0.0f));
                g_w = __fmaf_rn(s[1], one, g_w);
                const float gs = __fmul_rn(s[1], w);
                if (a.mod_bstride != 0) {
                    if (a.grad_shift)
                        a.grad_shift[b * D + d] = s[0];
                    if (a.grad_scale)
                        a.grad_scale[b * D + d] = gs;
                } else {
                    g_shift = __fadd_rn(g_shift, s[0]);
                    g_scale = __fadd_rn(g_scale, gs);
                }
            }
            if (post_on) {
                const float du = out_on ? s[2] : s[0];
                const float g = value(a.gate, b * a.gate_bstride * 8, 1.0f);
                g_wp = __fmaf_rn(du, __fmul_rn(g, a.update_scale), g_wp);
                const float gg = __fmul_rn(du, wp);
                if (a.gate_bstride != 0) {
                    if (a.grad_gate)
                        a.grad_gate[b * D + d] = gg;
                } else {
                    g_gate = __fadd_rn(g_gate, gg);
                }
            }
        }
        __syncthreads();
    }
    if (warp != 0 || !in)
        return;
    if (a.grad_weight)
        a.grad_weight[d] = g_w;
    if (a.grad_post_weight)
        a.grad_post_weight[d] = g_wp;
    if (a.mod_bstride == 0) {
        if (a.grad_shift)
            a.grad_shift[d] = g_shift;
        if (a.grad_scale)
            a.grad_scale[d] = g_scale;
    }
    if (a.gate_bstride == 0 && a.grad_gate)
        a.grad_gate[d] = g_gate;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

struct Shape {
    bool cluster;
    int threads;
    int row_bytes;  // of one CTA's part of a row
};

Shape shape_of(int Dv)
{
    Shape s;
    s.cluster = Dv > kMaxDvPerCta;
    const int nv = s.cluster ? (Dv + 1) / 2 : Dv;
    s.threads = (nv + 32 * kV - 1) / (32 * kV) * 32;
    s.row_bytes = nv * 16;
    return s;
}

// CTAs that share an SM: as many as 512 threads make up.
int ctas_per_sm(const Shape& s)
{
    const int n = kMaxThreads / s.threads;
    return n > 16 ? 16 : n;
}

int ring_stages(const Shape& s, int rows_per_slot)
{
    const int budget = kSmemPerSm / ctas_per_sm(s) - 2048;
    const int n = budget / (s.row_bytes * rows_per_slot);
    return n > kMaxStages ? kMaxStages : (n < 2 ? 2 : n);
}

template <typename K, typename A>
cudaError_t launch_rows(K kern, const A& a, const Items& items, const Shape& s, int rows_per_slot,
                        PerDeviceInt& ready, const DeviceInfo& dev, cudaStream_t stream)
{
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
    });
    if (e != cudaSuccess)
        return e;
    const int64_t cap = static_cast<int64_t>(dev.sms) * ctas_per_sm(s) / (s.cluster ? 2 : 1);
    const int64_t groups = static_cast<int64_t>(items.count) < cap ? items.count : cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(groups * (s.cluster ? 2 : 1)));
    cfg.blockDim = dim3(static_cast<unsigned>(s.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(items.stages) * rows_per_slot * s.row_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, items);
}

Items items_of(int64_t B, int64_t S, int64_t chunk)
{
    Items it;
    const int64_t per_batch = (S + chunk - 1) / chunk;
    it.per_batch = FastDiv::make(static_cast<uint32_t>(per_batch));
    it.chunk = static_cast<uint32_t>(chunk);
    it.count = static_cast<uint32_t>(B * per_batch);
    it.S = static_cast<uint32_t>(S);
    it.stages = 2;
    return it;
}

// Rows of a batch in items that spread over the GPU.
Items spread(int64_t B, int64_t S, int64_t cap)
{
    int64_t per = cap / B;
    per = per < 1 ? 1 : (per > S ? S : per);
    return items_of(B, S, (S + per - 1) / per);
}

template <typename T, int MAXT, bool CL>
cudaError_t launch_fwd(const SandwichArgs& a, const Shape& s, const DeviceInfo& dev,
                       cudaStream_t stream)
{
    static PerDeviceInt ready;
    Items it = spread(a.rows / a.S, a.S,
                      static_cast<int64_t>(dev.sms) * ctas_per_sm(s) / (CL ? 2 : 1));
    it.stages = ring_stages(s, 2);
    return launch_rows(sandwich_kernel<T, MAXT, CL>, a, it, s, 2, ready, dev, stream);
}

template <typename T>
cudaError_t launch_fwd_t(const SandwichArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const Shape s = shape_of(a.Dv);
    if (s.cluster)
        return launch_fwd<T, 512, true>(a, s, dev, stream);
    if (s.threads > 256)
        return launch_fwd<T, 512, false>(a, s, dev, stream);
    return launch_fwd<T, 256, false>(a, s, dev, stream);
}

// Items of the backward pass: their rows depend on S and D alone, so that the token sums do not
// depend on the batch.  152 SMs.
Items backward_items(int64_t B, int64_t S, int Dv)
{
    const Shape s = shape_of(Dv);
    const int64_t spread_over = 152 * ctas_per_sm(s) / (s.cluster ? 2 : 1);
    const int64_t chunk = (S + spread_over - 1) / spread_over;
    return items_of(B, S, chunk > 64 ? 64 : chunk);
}

template <typename T, int MAXT, bool CL, bool POST, bool OUT>
cudaError_t launch_bwd(const SandwichBwdArgs& a, const Shape& s, Items it, const DeviceInfo& dev,
                       cudaStream_t stream)
{
    static PerDeviceInt ready;
    const int rows = (POST ? 1 : 0) + (OUT ? 2 : 0) + (a.grad_res ? 1 : 0);
    it.stages = ring_stages(s, rows);
    return launch_rows(sandwich_bwd_kernel<T, MAXT, CL, POST, OUT>, a, it, s, rows, ready, dev,
                       stream);
}

template <typename T, bool POST, bool OUT>
cudaError_t launch_bwd_t(const SandwichBwdArgs& a, const Items& it, const DeviceInfo& dev,
                         cudaStream_t stream)
{
    const Shape s = shape_of(a.Dv);
    if (s.cluster)
        return launch_bwd<T, 512, true, POST, OUT>(a, s, it, dev, stream);
    if (s.threads > 256)
        return launch_bwd<T, 512, false, POST, OUT>(a, s, it, dev, stream);
    return launch_bwd<T, 256, false, POST, OUT>(a, s, it, dev, stream);
}

template <typename T>
cudaError_t launch_columns(const SandwichBwdArgs& a, const Items& it, cudaStream_t stream)
{
    const int parts = (a.grad_out ? 2 : 0) + (a.update ? 1 : 0);
    const int grid = (a.Dv * 8 + 31) / 32;
    return launch_dependent(sandwich_columns_kernel<T>, grid, 32 * kColWarps, 0, stream, a,
                            static_cast<int64_t>(it.per_batch.d), parts);
}

template <typename T>
cudaError_t launch_sandwich_t(const SandwichBwdArgs& a, const Items& it, const DeviceInfo& dev,
                              cudaStream_t stream)
{
    const cudaError_t e = a.grad_out ? launch_bwd_t<T, true, true>(a, it, dev, stream)
                                     : launch_bwd_t<T, true, false>(a, it, dev, stream);
    return e == cudaSuccess && a.sums ? launch_columns<T>(a, it, stream) : e;
}

}  // namespace

cudaError_t launch_sandwich(const SandwichArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    return a.f16 ? launch_fwd_t<__half>(a, dev, stream)
                 : launch_fwd_t<__nv_bfloat16>(a, dev, stream);
}

size_t sandwich_backward_workspace_bytes(int64_t B, int64_t S, int64_t D, int parts)
{
    return static_cast<size_t>(backward_items(B, S, static_cast<int>(D / 8)).count) * parts * D *
           sizeof(float);
}

cudaError_t launch_sandwich_backward(const SandwichBwdArgs& a, const DeviceInfo& dev,
                                     cudaStream_t stream)
{
    const Items it = backward_items(a.B, a.S, a.Dv);
    if (a.update)
        return a.f16 ? launch_sandwich_t<__half>(a, it, dev, stream)
                     : launch_sandwich_t<__nv_bfloat16>(a, it, dev, stream);
    // the norm alone: rmsnorm_modulate is bf16
    const cudaError_t e = launch_bwd_t<__nv_bfloat16, false, true>(a, it, dev, stream);
    return e == cudaSuccess && a.sums ? launch_columns<__nv_bfloat16>(a, it, stream) : e;
}

cudaError_t sandwich_error(unsigned* bits, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_error, sizeof(unsigned));
    if (e == cudaSuccess && clear && *bits) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_error, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace rmsmod
