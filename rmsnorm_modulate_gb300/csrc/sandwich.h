// Host-side launch interface of the sandwich norms and their gradients.  Internal to librmsmod.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace rmsmod {

// Row tensors [B*S, D] and row vectors of one 16-bit type; strides in 16-byte vectors.
struct SandwichArgs {
    const void* residual;
    const void* update;
    const void* post_weight;  // nullable
    const void* gate;         // nullable
    int64_t gate_bstride;
    const void* weight;       // nullable
    const void* scale;        // nullable
    const void* shift;        // nullable
    int64_t mod_bstride;
    void* res_out;
    void* out;                // nullable: no norm after the add
    float* post_rstd_out;     // nullable
    float* rstd_out;          // nullable
    int64_t rows;
    int64_t S;
    int Dv;                   // D / 8
    float n;                  // D
    float post_eps;
    float eps;
    float residual_scale;
    float update_scale;
    int f16;
};

cudaError_t launch_sandwich(const SandwichArgs& a, const DeviceInfo& dev, cudaStream_t stream);

struct SandwichBwdArgs {
    const void* update;       // null: the gradient of the norm alone
    const void* res;
    const void* post_weight;  // nullable
    const void* gate;         // nullable
    int64_t gate_bstride;
    const void* weight;       // nullable
    const void* scale;        // nullable
    int64_t mod_bstride;
    const void* grad_res;     // nullable
    const void* grad_out;     // null: the post norm's gradient alone
    const float* post_rstd;
    const float* rstd;
    void* grad_residual;      // nullable
    void* grad_update;        // nullable
    float* grad_post_weight;  // [D], nullable
    float* grad_gate;         // [B or 1, D], nullable
    float* grad_weight;       // [D], nullable
    float* grad_scale;        // [B or 1, D], nullable
    float* grad_shift;        // [B or 1, D], nullable
    bool sums;                // a row vector's gradient is wanted
    float* partials;          // then [B][items][parts][D]
    int64_t B;
    int64_t S;
    int Dv;
    float n;
    float residual_scale;
    float update_scale;
    int f16;
};

// Bytes of the partial sums for `parts` column sums (1 to 3); B, S > 0.
size_t sandwich_backward_workspace_bytes(int64_t B, int64_t S, int64_t D, int parts);
cudaError_t launch_sandwich_backward(const SandwichBwdArgs& a, const DeviceInfo& dev,
                                     cudaStream_t stream);

cudaError_t sandwich_error(unsigned* bits, bool clear);

}  // namespace rmsmod
