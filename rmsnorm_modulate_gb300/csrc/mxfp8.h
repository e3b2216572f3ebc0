// Host-side launch interface of the microscaled 8-bit operators.  Internal to librmsmod.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace rmsmod {

enum Mxfp8Type : int { kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2 };

// One side of the (de)quantisation is `values` [rows, K] (bf16 or fp16), the other codes and scales.
struct Mxfp8RowsArgs {
    void* values;
    void* codes;
    void* scales;
    uint32_t rows;
    uint32_t rows_padded;  // a multiple of 128
    uint32_t Kv;           // K / 8
    FastDiv by_tiles;      // block tiles of a row: ceil(K / 128)
    int f16;
};

cudaError_t launch_mxfp8_rows(bool quantize, const Mxfp8RowsArgs& a, cudaStream_t stream);

// Rows [rows, K] in blocks along K to rows [K, rows up to a multiple of 32] in blocks along the rows.
struct Mxfp8TransposeArgs {
    const void* codes;
    const void* scales;
    void* out_codes;
    void* out_scales;
    int64_t rows;
    int64_t K;
};

cudaError_t launch_mxfp8_transpose(const Mxfp8TransposeArgs& a, cudaStream_t stream);

// z = a b^T + bias, y = residual + gate * act(z); y to `out` (rounded to the type, or to 8-bit blocks
// where out_scales are given), z to 8-bit blocks where `keep` is given.
constexpr int kMxfp8DirectRows = 32;

struct Mxfp8MatmulArgs {
    const void* a;        // codes [M, K], or up to kMxfp8DirectRows rows of bf16 or fp16
    const void* a_scales; // null: of those
    const void* b;        // codes [N, K]
    const void* b_scales;
    const void* bias;     // nullable [N]
    const void* gate;     // nullable, rows at gate + batch * gate_bstride
    int64_t gate_bstride; // in elements
    const void* residual; // nullable [M, N]
    void* out;            // [M, N]
    void* out_scales;     // nullable
    void* keep;           // nullable
    void* keep_scales;
    int64_t M;
    int64_t S;            // rows of one batch
    int64_t N;
    int64_t K;
    int type;
    int activation;
    bool wide;            // set by the launcher: rows of out and residual start on 32 bytes
};

cudaError_t launch_mxfp8_matmul(Mxfp8MatmulArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t mxfp8_matmul_error(unsigned* bits, bool clear);

// res = R(x + update) (x itself without update), out = Q(RMSNorm(res) * weight * (1 + scale) + shift),
// keep = Q(res).  Row vectors' strides in elements.
struct Mxfp8NormArgs {
    const void* x;
    const void* update;   // nullable
    const void* weight;   // nullable
    const void* scale;    // nullable
    const void* shift;    // nullable
    int64_t mod_bstride;
    void* res_out;        // with update
    void* out;
    void* out_scales;
    void* keep;           // nullable
    void* keep_scales;
    float* rstd_out;      // nullable
    uint32_t rows;
    uint32_t S;
    int D;
    float eps;
    int f16;
};

cudaError_t launch_mxfp8_norm(const Mxfp8NormArgs& a, const DeviceInfo& dev, cudaStream_t stream);

// Gradients of that norm by res and by its row vectors.
struct Mxfp8NormBwdArgs {
    const void* kept;
    const void* kept_scales;
    const void* weight;    // nullable
    const void* scale;     // nullable
    int64_t mod_bstride;
    const void* grad_out;
    const void* grad_res;  // nullable
    const float* rstd;
    void* grad_x;          // nullable
    float* grad_weight;    // [D], nullable
    float* grad_scale;     // [B or 1, D], nullable
    float* grad_shift;     // [B or 1, D], nullable
    bool sums;
    float* partials;       // [B][items][2][D]
    int64_t B;
    int64_t S;
    int D;
    int f16;
};

size_t mxfp8_norm_backward_workspace_bytes(int64_t B, int64_t S, int64_t D);
cudaError_t launch_mxfp8_norm_backward(const Mxfp8NormBwdArgs& a, const DeviceInfo& dev,
                                       cudaStream_t stream);
cudaError_t mxfp8_norm_error(unsigned* bits, bool clear);

// grad_z = Q(grad_out * gate * act'(z)); column sums of grad_out * gate * act'(z) and, for each batch,
// of grad_out * act(z).
struct Mxfp8ActBwdArgs {
    const void* z;
    const void* z_scales;
    const void* grad_out;
    const void* gate;      // nullable
    int64_t gate_bstride;
    void* grad_z;
    void* grad_z_scales;
    float* grad_bias;      // [N], nullable
    float* grad_gate;      // [B or 1, N], nullable
    float* partials;       // [batches][tiles][parts][N]
    int64_t B;
    int64_t S;
    int64_t N;
    int activation;
    int f16;
};

size_t mxfp8_activation_backward_workspace_bytes(int64_t B, int64_t S, int64_t N, bool per_batch,
                                                 int parts);
cudaError_t launch_mxfp8_activation_backward(const Mxfp8ActBwdArgs& a, const DeviceInfo& dev,
                                             cudaStream_t stream);

}  // namespace rmsmod
