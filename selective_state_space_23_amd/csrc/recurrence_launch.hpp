// Host-side launch descriptors of the gated linear recurrence and of the 8-bit
// activation checkpoints, shared by recurrence_api.cpp and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

constexpr int kRecChunk = 128;   // tokens between two saved states
constexpr int kPackBlock = 64;   // channels that share one scale

// One 8-bit checkpoint: codes (rows, D) and scales (ceil(D / 64), rows).
struct Packed {
    int8_t* q = nullptr;
    float* scale = nullptr;
};

namespace rec {
struct Chain;   // recurrence.hpp
}

struct RecFwdArgs {
    // inputs; with packed inputs (the backward's recomputation of the states) x,
    // gate_a and gate_x are null and `in` holds their checkpoints
    const void* x;
    const void* gate_a;
    const void* gate_x;
    const void* z;                 // or null
    Packed in[3];
    const float* a_param;
    const uint8_t* doc_start;      // or null
    const float* initial_state;    // (B, D) or null
    void* out;                     // or null: states only
    float* final_state;            // (B, D) or null
    float* states;                 // (B, ceil(L / 128), D) or null
    Packed save[4];                // q null: not written
    void* ws;
    const rec::Chain* chain;       // cleared already, in place of ws; or null
    int64_t batch, seqlen, dim;
    int ld_x, ld_a, ld_g, ld_z;       // elements between two tokens
    float c;
    bool bf16;
    bool aligned;                  // quads of channels: D, strides and pointers
    hipStream_t stream;
};

struct RecBwdArgs {
    const void* x;
    const void* gate_a;
    const void* gate_x;
    const void* z;
    Packed in[4];                  // q set: 8-bit inputs instead of the four above
    const float* a_param;
    const uint8_t* doc_start;
    const float* initial_state;
    const float* states;           // or null: recomputed in the workspace
    const void* dout;
    const float* d_final_state;    // or null
    void* dx;
    void* dgate_a;
    void* dgate_x;
    float* da_param;               // (D,)
    void* dz;                      // null iff there is no z
    float* d_initial_state;        // or null
    void* ws;
    int64_t batch, seqlen, dim;
    int ld_x, ld_a, ld_g, ld_z, ld_o;
    float c;
    bool bf16;
    bool aligned;
    bool has_z;
    hipStream_t stream;
};

struct RecUpdateArgs {
    float* state;                  // (B, D), in place
    const void* x;
    const void* gate_a;
    const void* gate_x;
    const void* z;
    const float* a_param;
    const uint8_t* reset;          // (B,) or null
    void* out;                     // (B, D)
    int64_t batch, dim;
    int64_t ld_x, ld_a, ld_g, ld_z;
    float c;
    bool bf16;
    bool aligned;
    hipStream_t stream;
};

size_t recurrence_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim);
size_t recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool have_states);
hipError_t launch_recurrence_fwd(const RecFwdArgs& a);
hipError_t launch_recurrence_bwd(const RecBwdArgs& a);
hipError_t launch_recurrence_update(const RecUpdateArgs& a);

// 8-bit checkpoints (checkpoint.hip): rows x dim values, `ld` elements between
// two rows of x; out is dense.
struct PackArgs {
    const void* x;
    void* out;
    Packed p;
    int64_t rows, dim, ld;
    bool bf16;
    bool aligned;
    hipStream_t stream;
};

// The conv backward (conv1d_bwd.hip) with its input read from a checkpoint.
struct ConvBwdArgs;
hipError_t launch_causal_conv1d_bwd_packed(const ConvBwdArgs& a, const Packed& in);

hipError_t launch_pack(const PackArgs& a);
hipError_t launch_unpack(const PackArgs& a);

}  // namespace mamba
