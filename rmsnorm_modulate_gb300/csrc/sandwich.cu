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
// Both are bound by HBM: 8 and 12 bytes per value.  One CTA per SM, of up to 16 warps (forward) or 8
// (backward, whose column sums take twice the registers); its warps form groups that take a row each,
// up to four 16-byte vectors a thread, and every group has a ring of bulk copies (TMA) that stays
// ahead of the arithmetic.  The products of a
// batch's row vectors lie in shared memory for all groups.  A row's values are in registers when its
// slot is refilled, before its sums are known.  Rows of more than 8192 values are shared by a
// cluster of two CTAs, which exchange their partial sums through distributed shared memory.
#include "device_common.cuh"
#include "half_types.cuh"
#include "launch.h"
#include "sandwich.h"

namespace rmsmod {

namespace {

__device__ unsigned int g_error;

constexpr int kMaxWarps = 16;      // of a CTA
// Of a CTA of the backward pass: eight, with 255 registers, for three or four vectors a thread (sixteen
// of two: 46.4 us where these take 43.8 at 4216 x 4096, 186 and 147 at 4256 x 16384); sixteen for rows
// of up to 512 values, which have one or two (eight: 62.2 us for 60000 x 256, these 48.2).
constexpr int backward_warps(int V) { return V <= 2 ? kMaxWarps : kMaxWarps / 2; }
constexpr int kMaxThreads = 32 * kMaxWarps;
constexpr int kMaxDvPerCta = 1024; // vectors of a row that one CTA takes
constexpr int kMaxStages = 4;      // of a group's ring
constexpr int kSmemBytes = 222 * 1024;

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

// Stores v at the other CTA's `addr`, where it completes four bytes of the phase of `bar`.
__device__ __forceinline__ void send(uint32_t addr, uint32_t bar, uint32_t rank, float v)
{
    asm volatile(
        "{\n\t.reg .b32 p, q;\n\tmapa.shared::cluster.u32 p, %0, %2;\n\t"
        "mapa.shared::cluster.u32 q, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [p], %3, [q];\n\t}" ::"r"(addr),
        "r"(bar), "r"(rank), "r"(__float_as_uint(v))
        : "memory");
}

// The threads of a CTA (or of the two CTAs of a cluster) that share rows.
struct Group {
    int warps;       // of a group in this CTA
    int index;       // of this group in its CTA
    int warp;        // of this thread in its group
    int lane;
    uint32_t rank;   // of the CTA in its cluster
    uint32_t bars;   // the group's barriers with the other CTA's warps (kJoint)

    __device__ __forceinline__ bool leader() const { return warp == 0 && lane == 0; }
    __device__ __forceinline__ int at(int j) const { return (j * warps + warp) * 32 + lane; }
};

// Who shares a row: a group of one CTA, or one group of each of two.
enum Sharing : int { kAlone = 0, kJoint = 1 };

constexpr int kGroupBars = 6;
constexpr uint32_t kGaveUp = 1u << 31;  // among the phases: a wait ran out, no more are made

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = global_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
            if (ok)
                return true;
        }
        if (global_ns() - t0 > kWaitLimitNs)
            return false;
    }
}

__device__ __forceinline__ void joint_wait(const Group& g, int which, uint32_t& phases)
{
    if (!(phases & kGaveUp) && !mbar_wait_cluster(g.bars + 8u * which, (phases >> which) & 1u)) {
        phases |= kGaveUp;
        atomicOr(&g_error, kErrCopyTimeout);
    }
    phases ^= 1u << which;
}

// Of the threads that share a row; kJoint: the warps of both CTAs arrive on barrier `which` of each,
// and `phases` has a bit for each barrier's next phase.
template <int CL>
__device__ __forceinline__ void group_barrier(const Group& g, int which, uint32_t& phases)
{
    if (CL == kJoint) {
        const uint32_t bar = g.bars + 8u * which;
        __syncwarp();
        if (g.lane == 0) {
            mbar_arrive(bar);
            asm volatile(
                "{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\t"
                "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [p];\n\t}" ::"r"(bar),
                "r"(g.rank ^ 1u)
                : "memory");
        }
        joint_wait(g, which, phases);
    } else if (g.warps == 1) {
        __syncwarp();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"(g.index + 1), "r"(g.warps * 32) : "memory");
    }
}

// Where the warps of a row leave their partial values: per value kPlaces, a group's warps from a
// multiple of four on (in a cluster a group's warps of both CTAs, one CTA's after the other's); zeros
// where there is no warp.  32 places, but for three groups of eight in each of two CTAs (kJoint).
template <int N>
struct __align__(16) Exchange {
    static constexpr int kPlaces = N == 1 ? 48 : 32;
    float v[N][kPlaces];
};

template <int N>
__device__ __forceinline__ void clear(Exchange<N>& ex)
{
    for (int i = threadIdx.x; i < N * Exchange<N>::kPlaces; i += blockDim.x)
        ex.v[i / Exchange<N>::kPlaces][i % Exchange<N>::kPlaces] = 0.0f;
}

// N sums (or maxima of magnitudes) over all threads of the row, in an order that the row's length
// fixes; every thread gets them.  One barrier: the same exchange may be used again after one more.
template <int N, int CL, bool MAX = false>
__device__ __forceinline__ void row_reduce(float (&x)[N], Exchange<N>& ex, const Group& g,
                                           int which, uint32_t& phases)
{
    auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : __fadd_rn(a, b); };
    // a group's warps in one CTA have (g.warps + 3) & ~3 places, the other CTA's follow them.  (Worked
    // out where they are used: held over the exchanges, the place costs the backward pass 5%.)
    const int first = g.index * ((g.warps + 3) & ~3) * (CL ? 2 : 1);
    auto mine = [&]() {
        return first + g.warp + (CL ? static_cast<int>(g.rank) * ((g.warps + 3) & ~3) : 0);
    };
    if constexpr (N == 3) {
        // three sums in six exchanges: each step halves the values that a lane still carries, so
        // lanes 0-7, 8-15 and 16-23 end with one sum each
        const bool up = g.lane & 16, odd = g.lane & 8;
        float a = join(up ? x[2] : x[0], __shfl_xor_sync(kFullMask, up ? x[0] : x[2], 16));
        const float b = join(up ? 0.0f : x[1], __shfl_xor_sync(kFullMask, up ? x[1] : 0.0f, 16));
        a = join(odd ? b : a, __shfl_xor_sync(kFullMask, odd ? a : b, 8));
#pragma unroll
        for (int off = 4; off > 0; off >>= 1)
            a = join(a, __shfl_xor_sync(kFullMask, a, off));
        if (!CL && g.warps == 1) {
            x[0] = __shfl_sync(kFullMask, a, 0);
            x[1] = __shfl_sync(kFullMask, a, 8);
            x[2] = __shfl_sync(kFullMask, a, 16);
            return;
        }
        if ((g.lane & 7) == 0 && g.lane < 24) {
            float* to = &ex.v[g.lane >> 3][mine()];
            *to = a;
            if (CL)
                send(smem_addr(to), g.bars + 8u * which, g.rank ^ 1u, a);
        }
        if (CL) {
            __syncwarp();
            if (g.lane == 0)
                mbar_expect_tx(g.bars + 8u * which, 12u);
        }
    } else {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = join(x[i], __shfl_xor_sync(kFullMask, x[i], off));
        if (!CL && g.warps == 1)
            return;
        if (g.lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float* to = &ex.v[i][mine()];
                *to = x[i];
                if (CL)
                    st_peer(smem_addr(to), g.rank ^ 1u, x[i]);
            }
        }
    }
    if (CL && N == 3)
        joint_wait(g, which, phases);
    else
        group_barrier<CL>(g, which, phases);
    // four warps' values a load
    const int quads = (g.warps + 3) / 4 * (CL ? 2 : 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* q = reinterpret_cast<const float4*>(&ex.v[i][first]);
        float4 t = q[0];
        for (int k = 1; k < quads; ++k) {
            const float4 o = q[k];
            t = make_float4(join(t.x, o.x), join(t.y, o.y), join(t.z, o.z), join(t.w, o.w));
        }
        x[i] = join(join(t.x, t.y), join(t.z, t.w));
    }
}

// One sum over a row's threads in two CTAs (kJoint), in two halves for work between them.  A warp
// arrives on its own CTA's barrier alone; its value in the other CTA completes a part of that one's
// transaction count.  (An arrival there with release semantics would first wait for the warp's
// stores of the row.)  A barrier is used for every other row: nothing for its next phase is sent
// before both CTAs have seen this one complete.
__device__ __forceinline__ void joint_give(float x, Exchange<1>& ex, const Group& g, int which)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        x = __fadd_rn(x, __shfl_xor_sync(kFullMask, x, off));
    __syncwarp();
    if (g.lane == 0) {
        const int part = (g.warps + 3) & ~3;
        float* to = &ex.v[0][(2 * g.index + static_cast<int>(g.rank)) * part + g.warp];
        const uint32_t bar = g.bars + 8u * which;
        *to = x;
        mbar_expect_tx(bar, 4u);
        send(smem_addr(to), bar, g.rank ^ 1u, x);
    }
}

__device__ __forceinline__ float joint_take(const Exchange<1>& ex, const Group& g, int which,
                                            uint32_t& phases)
{
    joint_wait(g, which, phases);
    const int quads = (g.warps + 3) / 4 * 2;
    const float4* q = reinterpret_cast<const float4*>(ex.v[0]) + g.index * quads;
    float4 t = q[0];
    for (int k = 1; k < quads; ++k) {
        const float4 o = q[k];
        t = make_float4(__fadd_rn(t.x, o.x), __fadd_rn(t.y, o.y), __fadd_rn(t.z, o.z),
                        __fadd_rn(t.w, o.w));
    }
    return __fadd_rn(__fadd_rn(t.x, t.y), __fadd_rn(t.z, t.w));
}

template <int V>
__device__ __forceinline__ float sum_squares(const u64 (&x)[V][4])
{
    u64 s[2] = {0ull, 0ull};
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i & 1] = f2_fma(x[j][i], x[j][i], s[i & 1]);
    float lo, hi;
    f2_unpack(f2_add(s[0], s[1]), lo, hi);
    return __fadd_rn(lo, hi);
}

// 1 / sqrt of a row whose fp32 sum of squares left fp32's comfortable range although its values are
// finite: squares of the values over the power of two of the largest, joined in fp64.  The thread's
// vectors are read again from `from`, so that the callers' registers need not outlive the sum.
struct Slow {
    float rstd;
    uint32_t phases;
};

template <typename T, int CL>
__device__ __noinline__ Slow rstd_scaled(const uint4* from, int nv, int vectors, float sum, float n,
                                         float eps, Exchange<1>* slow, const Group g,
                                         uint32_t phases)
{
    float top[1] = {0.0f};
    for (int j = 0; j < vectors; ++j)
        if (g.at(j) < nv) {
            const uint4 x = from[g.at(j)];
            for (int i = 0; i < 4; ++i) {
                const float2 p = widen2<T>(word(x, i));
                top[0] = fmaxf(top[0], fmaxf(fabsf(p.x), fabsf(p.y)));
            }
        }
    row_reduce<1, CL, true>(top, slow[0], g, 2, phases);
    // Inf, or nothing but zeros: the sum says it all.  (A NaN never gets here.)
    if (!(top[0] <= 3.4028235e38f) || top[0] == 0.0f)
        return {__fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), eps))), phases};
    const int e = ilogbf(top[0]);
    float s[1] = {0.0f};
    for (int j = 0; j < vectors; ++j)
        if (g.at(j) < nv) {
            const uint4 x = from[g.at(j)];
            for (int i = 0; i < 4; ++i) {
                const float2 p = widen2<T>(word(x, i));
                const float a = scalbnf(p.x, -e), b = scalbnf(p.y, -e);
                s[0] = __fadd_rn(s[0], __fadd_rn(__fmul_rn(a, a), __fmul_rn(b, b)));
            }
        }
    row_reduce<1, CL>(s, slow[1], g, 3, phases);
    const double ms = scalbn(static_cast<double>(s[0]) / static_cast<double>(n), 2 * e);
    return {static_cast<float>(1.0 / sqrt(ms + static_cast<double>(eps))), phases};
}

template <typename T, int CL>
__device__ __forceinline__ float rstd_of(const uint4* from, int nv, int vectors, float sum, float n,
                                         float inv_n, float eps, Exchange<1>* slow, const Group& g,
                                         uint32_t& phases)
{
    // past 2^120, or so small that a tiny eps leaves it to decide (uniform over the row)
    if (sum > 1.3e36f || (sum < 8e-25f && eps < 1e-18f)) {
        const Slow s = rstd_scaled<T, CL>(from, nv, vectors, sum, n, eps, slow, g, phases);
        phases = s.phases;
        return s.rstd;
    }
    // the approximate root and one Newton step: within 2 * 2^-24 of the root, in a tenth of the
    // instructions of a division and a square root, which every warp of a row repeats
    const float ms = __fmaf_rn(sum, inv_n, eps);
    const float y = rsqrtf(ms);
    return __fmaf_rn(__fmul_rn(0.5f, y), __fmaf_rn(__fmul_rn(-ms, y), y, 1.0f), y);
}

// ---------------------------------------------------------------------------
// rows of a CTA (or cluster): a range of items of `chunk` rows of one batch (neighbours, so that the
// row vectors change as seldom as they can), dealt to its groups in turn
// ---------------------------------------------------------------------------

struct Plan {
    FastDiv per_batch;
    uint32_t chunk;
    uint32_t count;
    uint32_t S;
    int groups;
    int warps;   // of a group
    int stages;  // of a group's ring
};

// The items of worker `w` of `workers`: their counts differ by one at most.
__device__ __forceinline__ uint32_t first_item(const Plan& p, uint32_t w, uint32_t workers)
{
    const uint32_t each = p.count / workers, more = p.count - each * workers;
    return w * each + (w < more ? w : more);
}

struct Span {  // an item
    uint32_t batch, begin, end;

    __device__ __forceinline__ Span(const Plan& p, uint32_t item)
    {
        batch = p.per_batch.div(item);
        begin = batch * p.S + (item - batch * p.per_batch.d) * p.chunk;
        const uint32_t left = (batch + 1) * p.S - begin;
        end = begin + (p.chunk < left ? p.chunk : left);
    }
};

// The rows of one group ahead of its arithmetic, in the ring's order.
struct Ahead {
    uint32_t item, last, row, end;
    int put;

    __device__ __forceinline__ bool any() const { return item < last; }
    __device__ __forceinline__ void seek(const Plan& p, int group)
    {
        for (; item < last; ++item) {
            const Span s(p, item);
            row = s.begin + group;
            end = s.end;
            if (row < end)
                return;
        }
    }
    __device__ __forceinline__ void advance(const Plan& p, int group)
    {
        put = put + 1 == p.stages ? 0 : put + 1;
        row += p.groups;
        if (row < end)
            return;
        ++item;
        seek(p, group);
    }
};

// Shared memory: per vector of the CTA's part of a row the fp32 products of the row vectors in two
// halves of four values (so that neighbouring lanes read neighbouring 16 bytes), then the rings.
__device__ __forceinline__ void put_pairs(float4* lo, float4* hi, const u64 (&t)[4])
{
    float4 f;
    f2_unpack(t[0], f.x, f.y);
    f2_unpack(t[1], f.z, f.w);
    *lo = f;
    f2_unpack(t[2], f.x, f.y);
    f2_unpack(t[3], f.z, f.w);
    *hi = f;
}

__device__ __forceinline__ void get_pairs(const float4* lo, const float4* hi, u64 (&t)[4])
{
    const float4 a = *lo, b = *hi;
    t[0] = f2_pack(a.x, a.y);
    t[1] = f2_pack(a.z, a.w);
    t[2] = f2_pack(b.x, b.y);
    t[3] = f2_pack(b.z, b.w);
}

// Product of a constant and up to two nullable row vectors at vector c.
template <typename T>
__device__ __forceinline__ void product(u64 (&t)[4], float k, const void* p, const void* q,
                                        int64_t q_at, int c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t[i] = f2_splat(k);
    if (p) {
        const uint4 w = ld_cached(static_cast<const uint4*>(p) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t[i] = f2_mul(t[i], widen<T>(word(w, i)));
    }
    if (q) {
        const uint4 w = ld_cached(static_cast<const uint4*>(q) + q_at + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t[i] = f2_mul(t[i], widen<T>(word(w, i)));
    }
}

// weight * (1 + scale)
template <typename T>
__device__ __forceinline__ void multiplier(u64 (&t)[4], const void* weight, const void* scale,
                                           int64_t scale_at, int c)
{
    product<T>(t, 1.0f, weight, nullptr, 0, c);
    if (scale) {
        const uint4 w = ld_cached(static_cast<const uint4*>(scale) + scale_at + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t[i] = f2_mul(t[i], f2_add(f2_splat(1.0f), widen<T>(word(w, i))));
    }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

constexpr int kFwdVectorBytes = 80;  // v and m in fp32, shift as stored

template <typename T, int V, int CL>
__global__ void __launch_bounds__(kMaxThreads, 1)
    sandwich_kernel(const SandwichArgs a, const Plan plan)
{
    extern __shared__ __align__(128) uint4 smem[];
    __shared__ __align__(8) unsigned long long full[kMaxWarps][kMaxStages];
    // of the update's sum and of the new residual's; kJoint: two of each, for rows in turn
    constexpr int kSets = CL == kJoint ? 2 : 1;
    __shared__ Exchange<1> ex[2 * kSets], slow[2 * kSets];
    __shared__ __align__(8) unsigned long long joint[CL == kJoint ? kMaxWarps : 1][kGroupBars];

    Group g;
    g.warps = plan.warps;
    g.index = (threadIdx.x >> 5) / plan.warps;
    g.warp = (threadIdx.x >> 5) - g.index * plan.warps;
    g.lane = threadIdx.x & 31;
    g.rank = CL ? cluster_rank() : 0u;
    g.bars = smem_addr(&joint[CL == kJoint ? g.index : 0][0]);
    const uint32_t worker = CL ? blockIdx.x / 2 : blockIdx.x;
    const uint32_t workers = CL ? gridDim.x / 2 : gridDim.x;
    const uint32_t first = first_item(plan, worker, workers);
    const uint32_t last = first_item(plan, worker + 1, workers);
    // this CTA's vectors of a row
    const int half = CL ? (a.Dv + 1) / 2 : a.Dv;
    const int v0 = static_cast<int>(g.rank) * half;
    const int nv = a.Dv - v0 < half ? a.Dv - v0 : half;
    const uint32_t bytes = static_cast<uint32_t>(nv) * 16u;
    float4* v_lo = reinterpret_cast<float4*>(smem);
    float4 *v_hi = v_lo + half, *m_lo = v_lo + 2 * half, *m_hi = v_lo + 3 * half;
    uint4* sh = smem + 4 * half;
    uint4* ring = smem + 5 * half + static_cast<size_t>(g.index) * plan.stages * 2 * half;

    if (g.leader()) {
        for (int s = 0; s < plan.stages; ++s)
            mbar_init(smem_addr(&full[g.index][s]), 1u);
        if (CL == kJoint)
            for (int i = 0; i < kGroupBars; ++i)
                mbar_init(g.bars + 8u * i, i == 2 || i == 3 ? 2u * g.warps : 1u * g.warps);
        mbar_init_fence();
    }
    for (int i = 0; i < 2 * kSets; ++i) {
        clear(ex[i]);
        clear(slow[i]);
    }
    if (CL)
        cluster_barrier();
    else
        __syncthreads();
    grid_dependency_sync();

    bool broken = false;
    const uint4* __restrict__ residual = static_cast<const uint4*>(a.residual) + v0;
    const uint4* __restrict__ update = static_cast<const uint4*>(a.update) + v0;
    uint4* res_out = static_cast<uint4*>(a.res_out) + v0;
    uint4* out = static_cast<uint4*>(a.out) + v0;
    const float inv_n = __fdiv_rn(1.0f, a.n);
    const u64 rs2 = f2_splat(a.residual_scale);

    Ahead ahead{first, last, 0u, 0u, 0};
    auto issue = [&]() {  // the group's leader
        if (!ahead.any())
            return;
        const uint32_t bar = smem_addr(&full[g.index][ahead.put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(ahead.put) * 2 * half);
        const int64_t from = static_cast<int64_t>(ahead.row) * a.Dv;
        fence_proxy_async();
        mbar_expect_tx(bar, 2 * bytes);
        bulk_g2s(dst, update + from, bytes, bar);
        bulk_g2s(dst + half * 16, residual + from, bytes, bar);
        ahead.advance(plan, g.index);
    };
    if (g.leader()) {
        ahead.seek(plan, g.index);
        for (int s = 0; s < plan.stages; ++s)
            issue();
    }

    // Seven rows into a long run its rings are left a slot or two shorter: reads that are too far
    // ahead get in the way of the stores.  What stays on its way is 56 KB an SM or more.  (With all
    // slots and with fewer: 17920 rows of 4096 values 105.7 and 94.8 us, 8960 of 8192 108 and 97.5, 24576
    // of 1024 37.6 and 36.6, 2 x 1777 of 6144 in fp16 without adaLN rows 31.5 and 31.3; 9830 of 2560
    // 37.2 and 38.2, 30000 of 512 22.9 and 23.4, 3554 of 6144 33.5 and 33.6.  From the first row on,
    // 4216 of 4096 take 27.2 where these take 26.4.  The exchange of kJoint rows holds them back by
    // itself; rows of 256 values are issue-bound.)
    constexpr bool kRest = CL == kAlone && V > 1;
    __shared__ uint32_t rest[kRest ? kMaxWarps : 1];  // a bit for each refill to come: not made
    if (kRest && g.leader()) {
        uint32_t bits = 0;
        for (int k = 1; (plan.stages - k) * 32 * half * plan.groups >= 56 * 1024; ++k)
            bits = bits * 2u + 64u;
        rest[g.index] = bits;
    }
    auto issue_or_rest = [&]() {
        if (kRest) {
            const uint32_t bits = rest[g.index];
            rest[g.index] = bits >> 1;
            if (bits & 1u)
                return;
        }
        issue();
    };

    uint32_t batch = 0xFFFFFFFFu, phase = 0, phases = 0;
    int get = 0;
    auto next_slot = [&]() {
        if (!broken && !mbar_wait(smem_addr(&full[g.index][get]), phase, kWaitLimitNs)) {
            broken = true;
            atomicOr(&g_error, kErrCopyTimeout);
        }
        const uint4* slot = ring + static_cast<size_t>(get) * 2 * half;
        if (++get == plan.stages) {
            get = 0;
            phase ^= 1u;
        }
        return slot;
    };
    u64 f[V][4];  // update, then res, in fp32: widened once each
    uint4 x[V];
    auto load_update = [&](const uint4* slot, u64 (&to)[V][4]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = g.at(j);
            const uint4 u = c < nv ? slot[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to[j][i] = widen<T>(word(u, i));
        }
    };
    auto load_residual = [&](const uint4* slot) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = g.at(j);
            x[j] = c < nv ? slot[half + c] : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto store_res = [&](int64_t base, float rp) {
        const u64 rp2 = f2_splat(rp);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = g.at(j);
            if (c < nv) {
                u64 t[4];
                get_pairs(v_lo + c, v_hi + c, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = narrow<T>(f2_fma(widen<T>(word(x[j], i)), rs2,
                                                        f2_mul(f2_mul(f[j][i], rp2), t[i])));
                    word(x[j], i) = w;
                    f[j][i] = widen<T>(w);
                }
                st_stream(res_out + base + c, x[j]);
            }
        }
    };
    auto store_out = [&](int64_t base, float r) {
        const u64 r2 = f2_splat(r);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = g.at(j);
            if (c < nv) {
                u64 t[4];
                get_pairs(m_lo + c, m_hi + c, t);
                const uint4 sf = sh[c];
                uint4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    word(o, i) =
                        narrow<T>(f2_fma(f2_mul(f[j][i], r2), t[i], widen<T>(word(sf, i))));
                st_stream(out + base + c, o);
            }
        }
    };
    const bool teller = g.leader() && g.rank == 0;
    // kJoint: the next row's first sum is given before this row's second is taken, so that neither
    // exchange is waited for in full (8512 rows of 16384 values: 177 us; 262 with both waited for
    // where they are needed, and arrivals at the other CTA that release the row's stores; 235 with
    // those arrivals alone).  Needs a ring of two slots, or no second row.
    uint32_t left = 0, set = 0;
    const uint4* slot = nullptr;
    auto begin_row = [&]() {
        slot = next_slot();
        u64 u[V][4];
        load_update(slot, u);
        joint_give(sum_squares<V>(u), ex[2 * set], g, set ? 4 : 0);
        --left;
    };
    if (CL == kJoint) {
        for (uint32_t item = first; item < last; ++item) {
            const Span span(plan, item);
            const uint32_t rows = span.end - span.begin + plan.groups - 1 - g.index;
            left += rows / plan.groups;
        }
        if (left)
            begin_row();
    }
    for (uint32_t item = first; item < last; ++item) {
        const Span span(plan, item);
        if (span.batch != batch) {  // the row vectors of this batch
            __syncthreads();
            batch = span.batch;
            for (int c = threadIdx.x; c < nv; c += blockDim.x) {
                u64 t[4];
                product<T>(t, a.update_scale, a.post_weight, a.gate, batch * a.gate_bstride,
                           v0 + c);
                put_pairs(v_lo + c, v_hi + c, t);
                multiplier<T>(t, a.weight, a.scale, batch * a.mod_bstride, v0 + c);
                put_pairs(m_lo + c, m_hi + c, t);
                sh[c] = a.shift ? ld_cached(static_cast<const uint4*>(a.shift) +
                                            batch * a.mod_bstride + v0 + c)
                                : make_uint4(0u, 0u, 0u, 0u);
            }
            __syncthreads();
        }
        for (uint32_t row = span.begin + g.index; row < span.end; row += plan.groups) {
            const int64_t base = static_cast<int64_t>(row) * a.Dv;
            if constexpr (CL == kJoint) {
                Exchange<1>* mine = ex + 2 * set;
                const int b0 = set ? 4 : 0, b1 = b0 + 1;
                float sum = joint_take(mine[0], g, b0, phases);
                const float rp = rstd_of<T, CL>(slot, nv, V, sum, a.n, inv_n, a.post_eps, slow, g,
                                                phases);
                load_update(slot, f);
                load_residual(slot);
                store_res(base, rp);
                if (teller && a.post_rstd_out)
                    a.post_rstd_out[row] = rp;
                joint_give(sum_squares<V>(f), mine[1], g, b1);
                set ^= 1u;
                if (left)
                    begin_row();
                sum = joint_take(mine[1], g, b1, phases);
                // all have read this row's slot
                if (g.leader())
                    issue();
                if (a.out) {
                    const float r = rstd_of<T, CL>(res_out + base, nv, V, sum, a.n, inv_n, a.eps,
                                                   slow + 2, g, phases);
                    store_out(base, r);
                    if (teller && a.rstd_out)
                        a.rstd_out[row] = r;
                }
            } else {
                const uint4* slot = next_slot();
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = g.at(j);
                    uint4 u = make_uint4(0u, 0u, 0u, 0u);
                    x[j] = u;
                    if (c < nv) {
                        u = slot[c];
                        x[j] = slot[half + c];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        f[j][i] = widen<T>(word(u, i));
                }
                float s[1] = {sum_squares<V>(f)};
                row_reduce<1, CL>(s, ex[0], g, 0, phases);
                const float rp =
                    rstd_of<T, CL>(slot, nv, V, s[0], a.n, inv_n, a.post_eps, slow, g, phases);
                // a barrier has passed (or a warp's exchange, for a group of one): the slot is read
                if (!CL && g.warps == 1)
                    __syncwarp();
                if (g.leader())
                    issue_or_rest();
                store_res(base, rp);
                if (teller && a.post_rstd_out)
                    a.post_rstd_out[row] = rp;
                if (a.out) {
                    s[0] = sum_squares<V>(f);
                    row_reduce<1, CL>(s, ex[1], g, 1, phases);
                    const float r = rstd_of<T, CL>(res_out + base, nv, V, s[0], a.n, inv_n, a.eps,
                                                   slow, g, phases);
                    store_out(base, r);
                    if (teller && a.rstd_out)
                        a.rstd_out[row] = r;
                } else {
                    group_barrier<CL>(g, 1, phases);  // between two uses of ex[0]
                }
            }
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

constexpr int kBwdVectorBytes = 64;  // v and m in fp32

// POST: the block's post norm takes part (update), OUT: the norm after the add does (grad_out).
template <typename T, int V, int CL, bool POST, bool OUT>
__global__ void __launch_bounds__(32 * backward_warps(V), 1)
    sandwich_bwd_kernel(const SandwichBwdArgs a, const Plan plan)
{
    extern __shared__ __align__(128) uint4 smem[];
    __shared__ __align__(8) unsigned long long full[kMaxWarps][kMaxStages];
    __shared__ Exchange<3> ex[2];
    __shared__ __align__(8) unsigned long long joint[CL == kJoint ? kMaxWarps : 1][kGroupBars];

    Group g;
    g.warps = plan.warps;
    g.index = (threadIdx.x >> 5) / plan.warps;
    g.warp = (threadIdx.x >> 5) - g.index * plan.warps;
    g.lane = threadIdx.x & 31;
    g.rank = CL ? cluster_rank() : 0u;
    g.bars = smem_addr(&joint[CL == kJoint ? g.index : 0][0]);
    const uint32_t worker = CL ? blockIdx.x / 2 : blockIdx.x;
    const uint32_t workers = CL ? gridDim.x / 2 : gridDim.x;
    const uint32_t first = first_item(plan, worker, workers);
    const uint32_t last = first_item(plan, worker + 1, workers);
    const int half = CL ? (a.Dv + 1) / 2 : a.Dv;
    const int v0 = static_cast<int>(g.rank) * half;
    const int nv = a.Dv - v0 < half ? a.Dv - v0 : half;
    const uint32_t bytes = static_cast<uint32_t>(nv) * 16u;
    const bool has_gr = a.grad_res != nullptr;
    // rows of a slot: update, res, grad_out, grad_res
    const int k_res = POST ? 1 : 0, k_go = k_res + 1, k_gr = (POST ? 1 : 0) + (OUT ? 2 : 0);
    const int rows = k_gr + (has_gr ? 1 : 0);
    float4* v_lo = reinterpret_cast<float4*>(smem);
    float4 *v_hi = v_lo + half, *m_lo = v_lo + 2 * half, *m_hi = v_lo + 3 * half;
    uint4* ring = smem + 4 * half + static_cast<size_t>(g.index) * plan.stages * rows * half;
    // where groups hand their sums on: a place for every two of them, behind the rings
    float4* handed = reinterpret_cast<float4*>(
        smem + 4 * half + static_cast<size_t>(plan.groups) * plan.stages * rows * half);

    if (g.leader()) {
        for (int s = 0; s < plan.stages; ++s)
            mbar_init(smem_addr(&full[g.index][s]), 1u);
        if (CL == kJoint)
            for (int i = 0; i < kGroupBars; ++i)
                mbar_init(g.bars + 8u * i, 1u * g.warps);
        mbar_init_fence();
    }
    clear(ex[0]);
    clear(ex[1]);
    if (CL)
        cluster_barrier();
    else
        __syncthreads();
    grid_dependency_sync();

    bool broken = false;
    const float inv_n = __fdiv_rn(1.0f, a.n);
    const u64 rs2 = f2_splat(a.residual_scale);
    Ahead ahead{first, last, 0u, 0u, 0};
    auto issue = [&]() {  // the group's leader
        if (!ahead.any())
            return;
        const uint32_t bar = smem_addr(&full[g.index][ahead.put]);
        const uint32_t dst = smem_addr(ring + static_cast<size_t>(ahead.put) * rows * half);
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
        ahead.advance(plan, g.index);
    };
    if (g.leader()) {
        ahead.seek(plan, g.index);
        for (int s = 0; s < plan.stages; ++s)
            issue();
    }

    constexpr int kParts = (OUT ? 2 : 0) + (POST ? 1 : 0);
    u64 sums[V][kParts][4];  // go, go * hh (OUT), dh * uh (POST)
    uint32_t batch = 0xFFFFFFFFu, phase = 0, phases = 0;
    int get = 0, par = 0;
    for (uint32_t item = first; item < last; ++item) {
        const Span span(plan, item);
        if (span.batch != batch) {
            __syncthreads();
            batch = span.batch;
            for (int c = threadIdx.x; c < nv; c += blockDim.x) {
                u64 t[4];
                if (POST) {
                    product<T>(t, a.update_scale, a.post_weight, a.gate, batch * a.gate_bstride,
                               v0 + c);
                    put_pairs(v_lo + c, v_hi + c, t);
                }
                if (OUT) {
                    multiplier<T>(t, a.weight, a.scale, batch * a.mod_bstride, v0 + c);
                    put_pairs(m_lo + c, m_hi + c, t);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[j][p][i] = 0ull;
        uint32_t row = span.begin + g.index;
        float r = 0.0f, rp = 0.0f;
        if (row < span.end) {
            r = OUT ? a.rstd[row] : 0.0f;
            rp = POST ? a.post_rstd[row] : 0.0f;
        }
        while (row < span.end) {
            if (!broken && !mbar_wait(smem_addr(&full[g.index][get]), phase, kWaitLimitNs)) {
                broken = true;
                atomicOr(&g_error, kErrCopyTimeout);
            }
            const uint4* slot = ring + static_cast<size_t>(get) * rows * half;
            if (++get == plan.stages) {
                get = 0;
                phase ^= 1u;
            }
            const u64 r2 = f2_splat(r), rp2 = f2_splat(rp);
            // ---- the row's sums: s0 = sum go m hh, s1 = sum q p, s2 = sum hh p with p = v uh, from
            //      which both means follow (dh = q - r c hh)
            u64 q[V][4];
            uint4 x[V], u[V];
            u64 t0 = 0ull, t1 = 0ull, t2 = 0ull;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = g.at(j);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[j][i] = 0ull;
                x[j] = u[j] = make_uint4(0u, 0u, 0u, 0u);
                if (c < nv) {
                    if (has_gr) {
                        const uint4 w = slot[k_gr * half + c];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[j][i] = widen<T>(word(w, i));
                    }
                    if (OUT) {
                        const uint4 go = slot[k_go * half + c];
                        x[j] = slot[k_res * half + c];
                        u64 m[4];
                        get_pairs(m_lo + c, m_hi + c, m);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const u64 y = widen<T>(word(go, i));
                            const u64 h = f2_mul(widen<T>(word(x[j], i)), r2);
                            const u64 d = f2_mul(y, m[i]);
                            t0 = f2_fma(d, h, t0);
                            q[j][i] = f2_fma(d, r2, q[j][i]);
                            sums[j][0][i] = f2_add(sums[j][0][i], y);
                            sums[j][1][i] = f2_fma(y, h, sums[j][1][i]);
                        }
                    }
                    if (POST) {
                        u[j] = slot[c];
                        u64 v[4];
                        get_pairs(v_lo + c, v_hi + c, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const u64 p = f2_mul(f2_mul(widen<T>(word(u[j], i)), rp2), v[i]);
                            t1 = f2_fma(q[j][i], p, t1);
                            if (OUT)
                                t2 = f2_fma(f2_mul(widen<T>(word(x[j], i)), r2), p, t2);
                        }
                    }
                }
            }
            float s[3], hi;
            f2_unpack(t0, s[0], hi);
            s[0] = __fadd_rn(s[0], hi);
            f2_unpack(t1, s[1], hi);
            s[1] = __fadd_rn(s[1], hi);
            f2_unpack(t2, s[2], hi);
            s[2] = __fadd_rn(s[2], hi);
            row_reduce<3, CL>(s, ex[par], g, par, phases);
            par ^= 1;
            // the row is in registers everywhere: its slot takes the next copies
            if (!CL && g.warps == 1)
                __syncwarp();
            if (g.leader())
                issue();
            const int64_t base = static_cast<int64_t>(row) * a.Dv + v0;
            const float rc = __fmul_rn(r, __fmul_rn(s[0], inv_n));
            const float c_upd = __fmul_rn(__fmaf_rn(-rc, s[2], s[1]), inv_n);
            // the next row's statistics, on their way during this row's second half
            row += plan.groups;
            float r_next = 0.0f, rp_next = 0.0f;
            if (row < span.end) {
                r_next = OUT ? a.rstd[row] : 0.0f;
                rp_next = POST ? a.post_rstd[row] : 0.0f;
            }
            // hh and uh once more from the stored values: held in fp32 they would not fit the registers
            const u64 nrc2 = f2_splat(-rc), ncu2 = f2_splat(-c_upd);
            // ---- the gradients of the row
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = g.at(j);
                if (c < nv) {
                    uint4 ox, ou;
                    u64 v[4];
                    if (POST)
                        get_pairs(v_lo + c, v_hi + c, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u64 dh =
                            OUT ? f2_fma(f2_mul(widen<T>(word(x[j], i)), r2), nrc2, q[j][i])
                                : q[j][i];
                        word(ox, i) = narrow<T>(POST ? f2_mul(dh, rs2) : dh);
                        if (POST) {
                            const u64 uh = f2_mul(widen<T>(word(u[j], i)), rp2);
                            sums[j][kParts - 1][i] = f2_fma(dh, uh, sums[j][kParts - 1][i]);
                            word(ou, i) =
                                narrow<T>(f2_mul(f2_fma(uh, ncu2, f2_mul(dh, v[i])), rp2));
                        }
                    }
                    if (a.grad_residual)
                        st_stream(static_cast<uint4*>(a.grad_residual) + base + c, ox);
                    if (POST && a.grad_update)
                        st_stream(static_cast<uint4*>(a.grad_update) + base + c, ou);
                }
            }
            r = r_next;
            rp = rp_next;
        }
        if (!a.sums)
            continue;
        // ---- the item's sums: groups hand theirs on in pairs, the first one stores the total
        for (int apart = 1; apart < plan.groups; apart *= 2) {
            const bool gives = (g.index & (2 * apart - 1)) == apart;
            const bool takes = (g.index & (2 * apart - 1)) == 0 && g.index + apart < plan.groups;
            float4* place = handed + static_cast<size_t>((gives ? g.index : g.index + apart) >> 1) *
                                         kParts * 2 * half;
            if (gives) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = g.at(j);
                    if (c < nv)
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
                            put_pairs(place + 2 * p * half + c, place + (2 * p + 1) * half + c,
                                      sums[j][p]);
                }
            }
            __syncthreads();
            if (takes) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = g.at(j);
                    if (c < nv)
#pragma unroll
                        for (int p = 0; p < kParts; ++p) {
                            u64 t[4];
                            get_pairs(place + 2 * p * half + c, place + (2 * p + 1) * half + c, t);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sums[j][p][i] = f2_add(sums[j][p][i], t[i]);
                        }
                }
            }
        }
        if (g.index == 0) {
            float4* to = reinterpret_cast<float4*>(a.partials) +
                         static_cast<int64_t>(item) * kParts * a.Dv * 2;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = g.at(j);
                if (c < nv)
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        float4* at = to + (static_cast<int64_t>(p) * a.Dv + v0 + c) * 2;
                        put_pairs(at, at + 1, sums[j][p]);
                    }
            }
        }
        if (plan.groups > 1)
            __syncthreads();  // the places are free for the next item
    }
    if (broken)
        drain_pause();
    if (CL)
        cluster_barrier();
}

// The gradients of the row vectors from the items' partial sums.  A CTA has 32 columns, a thread four
// of them in one of 64 slices: `ks` slices share the items of a batch (a power of two that the
// number of items fixes, 4 to 32), so 64 / ks batches are summed at a time.  A warp then joins a
// batch's slices in order, and the warps their batches.
constexpr int kColSlices = 64;
constexpr int kColWarps = kColSlices / 4;

template <typename T>
__global__ void __launch_bounds__(8 * kColSlices)
    sandwich_columns_kernel(const SandwichBwdArgs a, uint32_t per_batch, int parts, int ks)
{
    grid_dependency_sync();
    __shared__ float4 part[3][kColSlices][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quad = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int at_once = kColSlices / ks;
    const int64_t D = static_cast<int64_t>(a.Dv) * 8;
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 8 + quad;     // this thread's four columns
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;    // the one it joins
    const bool out_on = a.grad_out != nullptr, post_on = a.update != nullptr;
    const bool joins = warp < at_once && d < D;
    auto value = [&](const void* p, int64_t at, float none) {
        return p && joins ? static_cast<float>(static_cast<const T*>(p)[at + d]) : none;
    };
    const float w = value(a.weight, 0, 1.0f);
    const float wp = __fmul_rn(value(a.post_weight, 0, 1.0f), a.update_scale);
    float g[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};  // weight, post weight, scale, shift, gate
    for (int64_t b0 = 0; b0 < a.B; b0 += at_once) {
        const int64_t mine = b0 + slice / ks, b = b0 + warp;
        float4 s[3];
#pragma unroll
        for (int p = 0; p < 3; ++p)
            s[p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (q * 4 < D && mine < a.B) {
            const float4* from = reinterpret_cast<const float4*>(a.partials) +
                                 mine * per_batch * parts * (D / 4) + q;
#pragma unroll 5
            for (uint32_t k = slice & (ks - 1); k < per_batch; k += ks)
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    if (p < parts) {
                        const float4 f =
                            __ldcs(from + (static_cast<int64_t>(k) * parts + p) * (D / 4));
                        s[p] = make_float4(__fadd_rn(s[p].x, f.x), __fadd_rn(s[p].y, f.y),
                                           __fadd_rn(s[p].z, f.z), __fadd_rn(s[p].w, f.w));
                    }
        }
        const bool on = joins && b < a.B;
        const float one = on ? __fadd_rn(1.0f, value(a.scale, b * a.mod_bstride * 8, 0.0f)) : 0.0f;
        const float gt = on ? value(a.gate, b * a.gate_bstride * 8, 1.0f) : 0.0f;
#pragma unroll
        for (int p = 0; p < 3; ++p)
            part[p][slice][quad] = s[p];
        __syncthreads();
        if (on) {
            float t[3];
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const float* at = reinterpret_cast<const float*>(&part[p][warp * ks][0]) + lane;
                t[p] = at[0];
#pragma unroll 4
                for (int k = 1; k < ks; ++k)
                    t[p] = __fadd_rn(t[p], at[k * 32]);
            }
            if (out_on) {
                const float gs = __fmul_rn(t[1], w);
                g[0] = __fmaf_rn(t[1], one, g[0]);
                if (a.mod_bstride == 0) {
                    g[2] = __fadd_rn(g[2], gs);
                    g[3] = __fadd_rn(g[3], t[0]);
                } else {
                    if (a.grad_scale)
                        a.grad_scale[b * D + d] = gs;
                    if (a.grad_shift)
                        a.grad_shift[b * D + d] = t[0];
                }
            }
            if (post_on) {
                const float du = out_on ? t[2] : t[0];
                const float gg = __fmul_rn(du, wp);
                g[1] = __fmaf_rn(du, __fmul_rn(gt, a.update_scale), g[1]);
                if (a.gate_bstride == 0)
                    g[4] = __fadd_rn(g[4], gg);
                else if (a.grad_gate)
                    a.grad_gate[b * D + d] = gg;
            }
        }
        __syncthreads();
    }
    // the warps' batches, in the warps' order
    float* join = reinterpret_cast<float*>(&part[0][0][0]);
    const int warps = a.B < at_once ? static_cast<int>(a.B) : at_once;
    if (warp < warps)
#pragma unroll
        for (int i = 0; i < 5; ++i)
            join[(i * kColWarps + warp) * 32 + lane] = g[i];
    __syncthreads();
    if (warp >= 5 || d >= D)
        return;
    float* to = warp == 0 ? a.grad_weight
                          : (warp == 1 ? a.grad_post_weight
                                       : (warp == 2 ? a.grad_scale
                                                    : (warp == 3 ? a.grad_shift : a.grad_gate)));
    const bool shared = warp < 2 || (warp < 4 ? a.mod_bstride : a.gate_bstride) == 0;
    if (!to || !shared)
        return;
    float t = join[warp * kColWarps * 32 + lane];
    for (int k = 1; k < warps; ++k)
        t = __fadd_rn(t, join[(warp * kColWarps + k) * 32 + lane]);
    to[d] = t;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// How a CTA's warps share rows of Dv vectors, V a thread.
struct Shape {
    bool cluster;
    int nv;      // vectors of a CTA's part of a row
    int V;
    int warps;   // of a group
    int groups;
};

Shape shape_of(int Dv, bool backward)
{
    Shape s;
    s.cluster = Dv > kMaxDvPerCta;
    s.nv = s.cluster ? (Dv + 1) / 2 : Dv;
    auto with = [&](int V) {
        s.V = V;
        const int most = backward ? backward_warps(V) : kMaxWarps;
        s.warps = (s.nv + 32 * V - 1) / (32 * V);
        s.groups = most / s.warps;
        // rows' vectors in the CTA at a time: more is better used lanes
        return s.groups * s.nv * 12 / V;
    };
    // Rows of one 16-byte vector a lane or two take no more than that: 60000 rows of 256 values in
    // 29.1 us (forward) and 48.2 (backward) with one, 31.5 and 51.5 with two, 38.5 (forward) with
    // four; 30000 rows of 512 in 21.9 with two and 25.7 with four.
    if (s.nv <= 64) {
        with(s.nv <= 32 ? 1 : 2);
        return s;
    }
    // three or four, whichever leaves fewer lanes idle
    const int four = with(4);
    if (with(3) > four)  // (no group at all counts none)
        return s;
    with(4);
    return s;
}

Plan plan_of(int64_t B, int64_t S, int64_t chunk, const Shape& s)
{
    Plan p;
    const int64_t per_batch = (S + chunk - 1) / chunk;
    p.per_batch = FastDiv::make(static_cast<uint32_t>(per_batch));
    p.chunk = static_cast<uint32_t>(chunk);
    p.count = static_cast<uint32_t>(B * per_batch);
    p.S = static_cast<uint32_t>(S);
    p.groups = chunk < s.groups ? static_cast<int>(chunk) : s.groups;
    p.warps = s.warps;
    p.stages = 1;
    return p;
}

// `fixed` bytes of shared memory beside the rings, slots of `slot` bytes.
template <typename K, typename A>
cudaError_t launch_rows(K kern, const A& a, Plan p, const Shape& s, int fixed, int slot,
                        PerDeviceInt& ready, const DeviceInfo& dev, cudaStream_t stream)
{
    int v = 0;
    cudaError_t e = ready.get(dev.device, v, [&](int& n) -> cudaError_t {
        n = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    });
    if (e != cudaSuccess)
        return e;
    // rings no longer than the rows of a group in its only item need
    const int64_t cap = s.cluster ? dev.sms / 2 : dev.sms;
    const int rows = static_cast<int>((p.chunk + p.groups - 1) / p.groups);
    p.stages = (kSmemBytes - fixed) / (slot * p.groups);
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages;
    if (p.count <= cap && rows < p.stages)
        p.stages = rows;
    const int64_t clusters = static_cast<int64_t>(p.count) < cap ? p.count : cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * (s.cluster ? 2 : 1)));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * p.warps * p.groups));
    cfg.dynamicSmemBytes = static_cast<size_t>(fixed) + static_cast<size_t>(p.stages) * p.groups * slot;
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
    return cudaLaunchKernelEx(&cfg, kern, a, p);
}

template <typename T, int V, int CL>
cudaError_t launch_fwd(const SandwichArgs& a, const Shape& s, const DeviceInfo& dev,
                       cudaStream_t stream)
{
    static PerDeviceInt ready;
    // Items that spread over the GPU.  They are rows of one batch and as many for every batch, so a
    // number of batches just past half of the CTAs, or past all of them, leaves up to half without
    // work: 17024 rows of 4096 values take 89 us as 1, 4 or 152 batches, 95 as 39, 129 as 77 and 149 as
    // 153.  With fewer rows a batch than a CTA has groups the groups past them have none, and the row
    // vectors are staged for every batch, shared or not: 4096 rows take 25.8 us as one batch, 31 as 512
    // (36 with rows of their own) and 72 (106) as 4096.
    const int64_t B = a.rows / a.S;
    int64_t per = (CL ? dev.sms / 2 : dev.sms) / B;
    per = per < 1 ? 1 : (per > a.S ? a.S : per);
    Plan p = plan_of(B, a.S, (a.S + per - 1) / per, s);
    // groups without a row help to stage the row vectors: a lone group's threads would take several
    // rounds of loads (3 us of a call of four rows of 4096 values)
    p.groups = s.groups;
    return launch_rows(sandwich_kernel<T, V, CL>, a, p, s, s.nv * kFwdVectorBytes, s.nv * 32, ready,
                       dev, stream);
}

template <typename T>
cudaError_t launch_fwd_t(const SandwichArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    const Shape s = shape_of(a.Dv, false);
    if (s.cluster)
        return s.V == 3 ? launch_fwd<T, 3, kJoint>(a, s, dev, stream)
                        : launch_fwd<T, 4, kJoint>(a, s, dev, stream);
    switch (s.V) {
    case 1:
        return launch_fwd<T, 1, kAlone>(a, s, dev, stream);
    case 2:
        return launch_fwd<T, 2, kAlone>(a, s, dev, stream);
    case 3:
        return launch_fwd<T, 3, kAlone>(a, s, dev, stream);
    default:
        return launch_fwd<T, 4, kAlone>(a, s, dev, stream);
    }
}

// Items of the backward pass: their rows depend on S and D alone, so that the token sums do not
// depend on the batch.  152 SMs.
Plan backward_plan(int64_t B, int64_t S, int Dv)
{
    const Shape s = shape_of(Dv, true);
    // whole rounds of items, of at most 256 rows (whose sums stay within a few 2^-24); of at least
    // eight, and two for each group, so that the partial sums are some eighth of the rows' bytes.
    // A batch of fewer rows is an item of those: at S = 1 the partial sums (12 bytes a value, which is
    // the workspace too) are as many bytes as the rows, and the second launch adds 16 batches at a time.
    // 4096 rows of 4096 values take 42 us as one batch, 104 (127 with rows of their own) as 512, 163
    // (208) as 1024 and 535 (781, with a workspace of 201 MB) as 4096.
    const int64_t over = s.cluster ? 76 : 152;
    const int64_t rounds = (S + 256 * over - 1) / (256 * over);
    int64_t chunk = (S + rounds * over - 1) / (rounds * over);
    const int64_t least = s.groups > 4 ? 2 * s.groups : 8;
    chunk = chunk < least ? least : chunk;
    return plan_of(B, S, chunk < S ? chunk : S, s);
}

template <typename T, int V, int CL, bool POST, bool OUT>
cudaError_t launch_bwd(const SandwichBwdArgs& a, const Shape& s, const Plan& p,
                       const DeviceInfo& dev, cudaStream_t stream)
{
    static PerDeviceInt ready;
    const int rows = (POST ? 1 : 0) + (OUT ? 2 : 0) + (a.grad_res ? 1 : 0);
    const int parts = (OUT ? 2 : 0) + (POST ? 1 : 0);
    const int handed = a.sums ? p.groups / 2 * parts * 32 : 0;
    // an odd number of groups: the last one's place too
    const int odd = a.sums && p.groups > 1 && p.groups % 2 ? parts * 32 : 0;
    return launch_rows(sandwich_bwd_kernel<T, V, CL, POST, OUT>, a, p, s,
                       s.nv * (kBwdVectorBytes + handed + odd), s.nv * 16 * rows, ready, dev,
                       stream);
}

template <typename T, bool POST, bool OUT>
cudaError_t launch_bwd_t(const SandwichBwdArgs& a, const Plan& p, const DeviceInfo& dev,
                         cudaStream_t stream)
{
    const Shape s = shape_of(a.Dv, true);
    if (s.cluster)
        return s.V == 3 ? launch_bwd<T, 3, kJoint, POST, OUT>(a, s, p, dev, stream)
                        : launch_bwd<T, 4, kJoint, POST, OUT>(a, s, p, dev, stream);
    switch (s.V) {
    case 1:
        return launch_bwd<T, 1, kAlone, POST, OUT>(a, s, p, dev, stream);
    case 2:
        return launch_bwd<T, 2, kAlone, POST, OUT>(a, s, p, dev, stream);
    case 3:
        return launch_bwd<T, 3, kAlone, POST, OUT>(a, s, p, dev, stream);
    default:
        return launch_bwd<T, 4, kAlone, POST, OUT>(a, s, p, dev, stream);
    }
}

template <typename T>
cudaError_t launch_columns(const SandwichBwdArgs& a, const Plan& p, cudaStream_t stream)
{
    const int parts = (a.grad_out ? 2 : 0) + (a.update ? 1 : 0);
    const int grid = (a.Dv * 8 + 31) / 32;
    int ks = 4;
    while (ks < 32 && static_cast<uint32_t>(ks) < p.per_batch.d)
        ks *= 2;
    return launch_dependent(sandwich_columns_kernel<T>, grid, 8 * kColSlices, 0, stream, a,
                            p.per_batch.d, parts, ks);
}

template <typename T>
cudaError_t launch_sandwich_t(const SandwichBwdArgs& a, const Plan& p, const DeviceInfo& dev,
                              cudaStream_t stream)
{
    const cudaError_t e = a.grad_out ? launch_bwd_t<T, true, true>(a, p, dev, stream)
                                     : launch_bwd_t<T, true, false>(a, p, dev, stream);
    return e == cudaSuccess && a.sums ? launch_columns<T>(a, p, stream) : e;
}

}  // namespace

cudaError_t launch_sandwich(const SandwichArgs& a, const DeviceInfo& dev, cudaStream_t stream)
{
    return a.f16 ? launch_fwd_t<__half>(a, dev, stream)
                 : launch_fwd_t<__nv_bfloat16>(a, dev, stream);
}

size_t sandwich_backward_workspace_bytes(int64_t B, int64_t S, int64_t D, int parts)
{
    return static_cast<size_t>(backward_plan(B, S, static_cast<int>(D / 8)).count) * parts * D *
           sizeof(float);
}

cudaError_t launch_sandwich_backward(const SandwichBwdArgs& a, const DeviceInfo& dev,
                                     cudaStream_t stream)
{
    const Plan p = backward_plan(a.B, a.S, a.Dv);
    if (a.update)
        return a.f16 ? launch_sandwich_t<__half>(a, p, dev, stream)
                     : launch_sandwich_t<__nv_bfloat16>(a, p, dev, stream);
    // the norm alone: rmsnorm_modulate is bf16
    const cudaError_t e = launch_bwd_t<__nv_bfloat16, false, true>(a, p, dev, stream);
    return e == cudaSuccess && a.sums ? launch_columns<__nv_bfloat16>(a, p, stream) : e;
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
