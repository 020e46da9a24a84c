// Host-side launch descriptors of the gated delta rule.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

constexpr int kDeltaChunk = 64;       // tokens of a chunk, and between two saved states
constexpr int kGroupFloats = kDeltaChunk * 16;
constexpr int kDeltaMaxHead = 128;    // widest key and value heads

// What every pass of one call shares.  Strides are elements between two tokens.
struct DeltaArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;             // (B, L, Hv) log decays, or null: none
    const float* beta;          // (B, L, Hv)
    const uint8_t* doc_start;   // (B, L) or null
    const float* initial_state; // (B, Hv, K, V) or null
    // forward
    void* out;
    float* final_state;
    float* states;              // (B, Hv, n, K, V): the states entering the chunks, or null
    // backward (states: read)
    const void* dout;
    const float* d_final_state;
    void* dq;
    void* dk;
    void* dv;
    float* dg;
    float* dbeta;
    float* d_initial_state;
    float* dstates;             // workspace: gradients at the chunks' end states
    float* dx;                  // and the dX of their columns, 16 at a time
    // workspace written by the first pass
    char* chunks;               // one record per (row, value head, chunk)
    char* solve;                // the solved triangles, in the order the matrix cores read them
    char* solve_t;              // the backward's, transposed
    char* pairs;                // scale D o Q K^T in the same order (forward), or its transpose (backward); or null
    int64_t batch, seqlen, ld_q, ld_k, ld_v, ld_o;
    int kheads, vheads, kdim, vdim;
    int kpitch;                 // channels from one head of q and k to the next: kdim, or more with zeros behind
    int nchunks;
    float scale;
    bool bf16;
    bool vec_k;                 // q and k: 16-byte pieces of eight channels
    bool vec_o;                 // dout and the states: the same
    hipStream_t stream;
};

struct DeltaUpdateArgs {
    float* state;
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const uint8_t* reset;
    void* out;
    int64_t batch, ld_q, ld_k, ld_v;
    int kheads, vheads, kdim, vdim;
    float scale;
    bool bf16;
    bool vec;                   // state rows in 16-byte pieces
    hipStream_t stream;
};

// Bytes of each workspace part for one (row, value head, chunk).
size_t delta_chunk_bytes();
size_t delta_solve_bytes();

// q's and k's heads of a.kdim channels to a.q and a.k, heads of a.kpitch (a multiple of 8) one behind the other, zeros behind.
hipError_t launch_delta_pad(const DeltaArgs& a, const void* q, const void* k, int64_t ld_q, int64_t ld_k);
hipError_t launch_delta_prepare(const DeltaArgs& a);
hipError_t launch_delta_fwd(const DeltaArgs& a);
hipError_t launch_delta_bwd_states(const DeltaArgs& a);
hipError_t launch_delta_bwd_grads(const DeltaArgs& a);
hipError_t launch_delta_update(const DeltaUpdateArgs& a);

}  // namespace mamba
