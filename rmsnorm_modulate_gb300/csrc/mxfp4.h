// Host-side launch interface of the microscaled 4-bit operators.  Internal to librmsmod.so.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace rmsmod {

// One side of the (de)quantisation is `values` [rows, K] (bf16 or fp16), the other the packed
// codes and the tiled scales.
struct Mxfp4RowsArgs {
    void* values;
    void* packed;
    void* scales;
    uint32_t rows;
    uint32_t rows_padded;  // a multiple of 128
    uint32_t Kv;           // K / 8
    FastDiv by_tiles;      // block tiles of a row: ceil(K / 128)
    int f16;
};

cudaError_t launch_mxfp4_rows(bool quantize, const Mxfp4RowsArgs& a, cudaStream_t stream);

// out = R(residual + gate * (a b^T + bias)), or R(a b^T + bias) without residual.
struct Mxfp4MatmulArgs {
    const void* a;        // packed [M, K / 2]
    const void* a_scales;
    const void* b;        // packed [N, K / 2]
    const void* b_scales;
    const void* bias;     // nullable [N]
    const void* gate;     // nullable, rows at gate + batch * gate_bstride
    int64_t gate_bstride; // in elements
    const void* residual; // nullable [M, N]
    void* out;            // [M, N]
    int64_t M;
    int64_t S;            // rows of one batch
    int64_t N;
    int64_t K;
    int f16;
    bool wide;            // set by the launcher: rows of out and residual start on 32 bytes
};

cudaError_t launch_mxfp4_matmul(Mxfp4MatmulArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t mxfp4_matmul_error(unsigned* bits, bool clear);

}  // namespace rmsmod
