// Host-side launch descriptors of the queries' and keys' head norms.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

constexpr int kNormMaxDim = 256;   // widest head: 32 lanes of 8 channels

struct QkNormArgs {
    const void* x[2];        // q, k
    const float* weight[2];  // or null
    const float* cos;        // (table_rows, rot / 2) or null
    const float* sin;
    const int32_t* positions;   // (B, L) or null: the token's index in its row
    const void* dy[2];       // backward: gradients at the outputs
    void* out[2];            // outputs, or (backward) gradients at the inputs
    float* dweight[2];       // or null
    float* parts;            // workspace of the weights' gradients
    int64_t ld_x[2], ld_dy[2];
    int heads[2];
    int64_t tokens, seqlen, table_rows;
    int dim, rot;
    float eps;
    bool rms, interleaved, bf16;
    bool vec;                // dim and rot multiples of 8, everything aligned to four values
    hipStream_t stream;
};

size_t qk_norm_bwd_workspace_bytes(int64_t tokens, int q_heads, int k_heads, int dim);
hipError_t launch_qk_norm_fwd(const QkNormArgs& a);
hipError_t launch_qk_norm_bwd(const QkNormArgs& a);

}  // namespace mamba
