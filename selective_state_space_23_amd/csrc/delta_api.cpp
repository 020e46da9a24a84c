// C ABI of the gated delta rule: argument validation and dispatch.  Every check
// runs on the host before any launch.
#include "mamba_hip.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.hpp"
#include "delta_launch.hpp"
#include "fill.hpp"

static_assert(MAMBA_DELTA_CHUNK == mamba::kDeltaChunk, "the header and the kernels agree");

namespace {

using namespace mamba::api;

constexpr int64_t kMaxWidth = int64_t(1) << 21;   // channels and strides of a token: a chunk's offsets fit 32 bits
constexpr int64_t kMaxChunks = 8000000;           // chunks of all rows and heads

int hip_status(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

int64_t chunks_of(const mamba_delta_dims_t* d) { return ceil_div(d->seqlen, MAMBA_DELTA_CHUNK); }

// `max_ld`: of the one-token step's rows, which are addressed in 64 bits.
int check_dims(const mamba_delta_dims_t* d, int64_t max_ld = kMaxWidth) {
    if (!d) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->batch < 0 || d->seqlen < 0 || d->batch > 65535) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->key_heads <= 0 || d->value_heads <= 0 || d->key_dim <= 0 || d->value_dim <= 0 ||
        d->value_heads % d->key_heads != 0)
        return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->dtype != MAMBA_DTYPE_F32 && d->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(d->scale)) return MAMBA_ERR_INVALID_ARGUMENT;
    const int64_t kw = int64_t(d->key_heads) * d->key_dim, vw = int64_t(d->value_heads) * d->value_dim;
    const int64_t lds[][2] = {{d->ld_q, kw}, {d->ld_k, kw}, {d->ld_v, vw}, {d->ld_dout, vw}};
    for (const auto& ld : lds)
        if (ld[0] < 0 || (ld[0] != 0 && ld[0] < ld[1])) return MAMBA_ERR_INVALID_ARGUMENT;
    for (const auto& ld : lds)
        if (ld[0] > max_ld) return MAMBA_ERR_UNSUPPORTED;
    if (d->ld_dout > kMaxWidth) return MAMBA_ERR_UNSUPPORTED;
    if (d->key_dim > mamba::kDeltaMaxHead || d->value_dim > mamba::kDeltaMaxHead) return MAMBA_ERR_UNSUPPORTED;
    if (kw > kMaxWidth || vw > kMaxWidth || d->seqlen > kMaxSeqlen) return MAMBA_ERR_UNSUPPORTED;
    if (d->batch * d->value_heads * (chunks_of(d) > 0 ? chunks_of(d) : 1) > kMaxChunks) return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

struct Sizes {
    size_t esz, k, v, gate, state;   // bytes of q or k and of v if dense, of a (B, L, Hv) array, of a state
    int64_t tokens, ld_q, ld_k, ld_v, ld_o;
    int64_t kw, vw;
};

Sizes sizes(const mamba_delta_dims_t* d) {
    Sizes s{};
    s.esz = d->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    s.tokens = d->batch * d->seqlen;
    s.kw = int64_t(d->key_heads) * d->key_dim;
    s.vw = int64_t(d->value_heads) * d->value_dim;
    s.k = static_cast<size_t>(s.tokens * s.kw) * s.esz;
    s.v = static_cast<size_t>(s.tokens * s.vw) * s.esz;
    s.gate = static_cast<size_t>(s.tokens * d->value_heads) * 4;
    s.state = static_cast<size_t>(d->batch * s.vw) * d->key_dim * 4;
    s.ld_q = d->ld_q ? d->ld_q : s.kw;
    s.ld_k = d->ld_k ? d->ld_k : s.kw;
    s.ld_v = d->ld_v ? d->ld_v : s.vw;
    s.ld_o = d->ld_dout ? d->ld_dout : s.vw;
    return s;
}

// q and k may be read in 16-byte pieces of eight channels.
bool pieces(const void* p, int64_t ld, size_t esz, int dim) {
    return dim % 8 == 0 && aligned(p, 16) && ld * esz % 16 == 0;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t record_bytes(const mamba_delta_dims_t* d) {
    return round256(static_cast<size_t>(d->batch * d->value_heads * chunks_of(d)) * mamba::delta_chunk_bytes());
}
size_t solve_bytes(const mamba_delta_dims_t* d) {   // of the triangles, of their transposes and of P
    return round256(static_cast<size_t>(d->batch * d->value_heads * chunks_of(d)) * mamba::delta_solve_bytes());
}

// Rows of q and k that are not in whole 16-byte pieces of eight channels are copied to such, with zeros behind.
// (3 x 18380 tokens, 3 heads of 118 in bf16, states and documents, backward: 2.76 ms, 5.99 read element by element.)
int pitch_of(const mamba_delta_dims_t* d) { return (d->key_dim + 7) / 8 * 8; }
bool copied(const mamba_delta_dims_t* d) {
    const int64_t piece = d->dtype == MAMBA_DTYPE_BF16 ? 8 : 4;
    return d->key_dim % 8 != 0 || d->ld_q % piece != 0 || d->ld_k % piece != 0;
}
size_t copy_bytes(const mamba_delta_dims_t* d) {   // of q or of k
    return copied(d) ? round256(static_cast<size_t>(d->batch * d->seqlen * d->key_heads) * pitch_of(d) *
                                (d->dtype == MAMBA_DTYPE_BF16 ? 2 : 4))
                     : 0;
}

// What the passes over a sequence take: check_dims, and launches of fewer than 2^32 threads.  (The other kernels stay below
// that for as many chunks as check_dims takes.)
int check_sequence(const mamba_delta_dims_t* d) {
    const int st = check_dims(d);
    if (st != MAMBA_OK) return st;
    constexpr int64_t kThreads = int64_t(1) << 32;
    // bf16: 512 threads for 64 columns of a row and head, heads in eights
    const int64_t groups = (d->batch * d->value_heads + 7) / 8 * 8 * ((d->value_dim + 63) / 64);
    if (d->dtype == MAMBA_DTYPE_BF16 && groups * 512 >= kThreads) return MAMBA_ERR_UNSUPPORTED;
    if (copied(d) && d->batch * d->seqlen * d->key_heads * (pitch_of(d) / 8) > kThreads - 256) return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

size_t fwd_workspace(const mamba_delta_dims_t* d) {
    return d->batch * d->seqlen == 0 ? 0 : 2 * copy_bytes(d) + record_bytes(d) + 2 * solve_bytes(d);
}

size_t state_bytes(const mamba_delta_dims_t* d) {   // of every chunk
    return round256(static_cast<size_t>(d->batch * d->value_heads * chunks_of(d)) * d->key_dim * d->value_dim * 4);
}

size_t dx_bytes(const mamba_delta_dims_t* d) {   // whole groups of 16 columns
    return static_cast<size_t>(d->batch * d->value_heads * chunks_of(d)) * ((d->value_dim + 15) / 16) * mamba::kGroupFloats * 4;
}
size_t bwd_workspace(const mamba_delta_dims_t* d, bool have_states) {
    return d->batch * d->seqlen == 0 ? 0 : 2 * copy_bytes(d) + record_bytes(d) + 3 * solve_bytes(d) +
                                                dx_bytes(d) + (have_states ? 1 : 2) * state_bytes(d);
}

mamba::DeltaArgs base_args(const mamba_delta_dims_t* d, const Sizes& s, const void* q, const void* k, const void* v,
                           const float* g, const float* beta, const uint8_t* doc_start, const float* initial_state,
                           void* workspace, void* stream) {
    mamba::DeltaArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.doc_start = doc_start; a.initial_state = initial_state;
    a.chunks = static_cast<char*>(workspace) + 2 * copy_bytes(d);
    a.solve = a.chunks + record_bytes(d);
    a.batch = d->batch; a.seqlen = d->seqlen;
    a.ld_q = s.ld_q; a.ld_k = s.ld_k; a.ld_v = s.ld_v; a.ld_o = s.ld_o;
    a.kheads = d->key_heads; a.vheads = d->value_heads; a.kdim = d->key_dim; a.vdim = d->value_dim;
    a.nchunks = static_cast<int>(chunks_of(d));
    a.scale = d->scale;
    a.bf16 = d->dtype == MAMBA_DTYPE_BF16;
    a.vec_k = pieces(q, s.ld_q, s.esz, d->key_dim) && pieces(k, s.ld_k, s.esz, d->key_dim);
    a.stream = static_cast<hipStream_t>(stream);
    a.kpitch = d->key_dim;
    if (copied(d)) {
        a.kpitch = pitch_of(d);
        a.q = workspace;
        a.k = static_cast<char*>(workspace) + copy_bytes(d);
        a.ld_q = a.ld_k = int64_t(d->key_heads) * a.kpitch;
        a.vec_k = true;
    }
    return a;
}

// The copies of q and k, where the arguments read such.
hipError_t copy_rows(const mamba::DeltaArgs& a, const mamba_delta_dims_t* d, const Sizes& s, const void* q, const void* k) {
    return copied(d) ? mamba::launch_delta_pad(a, q, k, s.ld_q, s.ld_k) : hipSuccess;
}

}  // namespace

extern "C" {

int mamba_gated_delta_rule_workspace_bytes(const mamba_delta_dims_t* dims, size_t* bytes) {
    if (!bytes) return MAMBA_ERR_INVALID_ARGUMENT;
    *bytes = 0;
    const int st = check_sequence(dims);
    if (st != MAMBA_OK) return st;
    *bytes = fwd_workspace(dims);
    return MAMBA_OK;
}

int mamba_gated_delta_rule_fwd(const mamba_delta_dims_t* dims, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const uint8_t* doc_start,
                               const float* initial_state, void* out, float* final_state, float* states,
                               void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_sequence(dims);
    if (st != MAMBA_OK) return st;
    const float* f32s[] = {g, beta, initial_state, final_state, states};
    for (const float* p : f32s)
        if (p && !aligned(p, 4)) return MAMBA_ERR_MISALIGNED;
    const Sizes s = sizes(dims);
    if (dims->batch == 0) return MAMBA_OK;
    if (dims->seqlen == 0) {
        if (overlap(final_state, s.state, initial_state, s.state)) return MAMBA_ERR_INVALID_ARGUMENT;
        return hip_status(mamba::launch_fill(final_state, initial_state, static_cast<int64_t>(s.state / 4),
                                             static_cast<hipStream_t>(stream)));
    }
    if (!q || !k || !v || !beta || !out) return MAMBA_ERR_INVALID_ARGUMENT;
    if (!aligned(q, s.esz) || !aligned(k, s.esz) || !aligned(v, s.esz) || !aligned(out, s.esz))
        return MAMBA_ERR_MISALIGNED;
    const size_t need = fwd_workspace(dims);
    if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MAMBA_ERR_MISALIGNED;
    const Span ins[] = {{q, span(s.tokens, s.kw, s.ld_q, s.esz)}, {k, span(s.tokens, s.kw, s.ld_k, s.esz)},
                        {v, span(s.tokens, s.vw, s.ld_v, s.esz)}, {g, s.gate}, {beta, s.gate},
                        {doc_start, static_cast<size_t>(s.tokens)}, {initial_state, s.state}};
    const Span outs[] = {{out, s.v}, {final_state, s.state}, {states, s.state * chunks_of(dims)}, {workspace, need}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    mamba::DeltaArgs a = base_args(dims, s, q, k, v, g, beta, doc_start, initial_state, workspace, stream);
    a.pairs = a.solve + solve_bytes(dims);
    a.out = out; a.final_state = final_state; a.states = states;
    hipError_t e = copy_rows(a, dims, s, q, k);
    if (e == hipSuccess) e = mamba::launch_delta_prepare(a);
    return hip_status(e != hipSuccess ? e : mamba::launch_delta_fwd(a));
}

int mamba_gated_delta_rule_bwd_workspace_bytes(const mamba_delta_dims_t* dims, int32_t have_states, size_t* bytes) {
    if (!bytes) return MAMBA_ERR_INVALID_ARGUMENT;
    *bytes = 0;
    const int st = check_sequence(dims);
    if (st != MAMBA_OK) return st;
    *bytes = bwd_workspace(dims, have_states != 0);
    return MAMBA_OK;
}

int mamba_gated_delta_rule_bwd(const mamba_delta_dims_t* dims, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const uint8_t* doc_start,
                               const float* initial_state, const float* states, const void* dout,
                               const float* d_final_state, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                               float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
    const int st = check_sequence(dims);
    if (st != MAMBA_OK) return st;
    const float* f32s[] = {g, beta, initial_state, states, d_final_state, dg, dbeta, d_initial_state};
    for (const float* p : f32s)
        if (p && !aligned(p, 4)) return MAMBA_ERR_MISALIGNED;
    if (d_initial_state && !initial_state) return MAMBA_ERR_INVALID_ARGUMENT;
    const Sizes s = sizes(dims);
    if (dims->batch == 0) return MAMBA_OK;
    if (dims->seqlen == 0) {
        if (overlap(d_initial_state, s.state, d_final_state, s.state)) return MAMBA_ERR_INVALID_ARGUMENT;
        return hip_status(mamba::launch_fill(d_initial_state, d_final_state, static_cast<int64_t>(s.state / 4),
                                             static_cast<hipStream_t>(stream)));
    }
    if (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta || (g != nullptr) != (dg != nullptr))
        return MAMBA_ERR_INVALID_ARGUMENT;
    const void* acts[] = {q, k, v, dout, dq, dk, dv};
    for (const void* p : acts)
        if (!aligned(p, s.esz)) return MAMBA_ERR_MISALIGNED;
    const size_t need = bwd_workspace(dims, states != nullptr);
    if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MAMBA_ERR_MISALIGNED;
    const Span ins[] = {{q, span(s.tokens, s.kw, s.ld_q, s.esz)}, {k, span(s.tokens, s.kw, s.ld_k, s.esz)},
                        {v, span(s.tokens, s.vw, s.ld_v, s.esz)}, {dout, span(s.tokens, s.vw, s.ld_o, s.esz)},
                        {g, s.gate}, {beta, s.gate}, {doc_start, static_cast<size_t>(s.tokens)},
                        {initial_state, s.state}, {d_final_state, s.state}, {states, s.state * chunks_of(dims)}};
    const Span outs[] = {{dq, s.k}, {dk, s.k}, {dv, s.v}, {dg, s.gate}, {dbeta, s.gate}, {d_initial_state, s.state},
                         {workspace, need}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    mamba::DeltaArgs a = base_args(dims, s, q, k, v, g, beta, doc_start, initial_state, workspace, stream);
    a.solve_t = a.solve + solve_bytes(dims);
    a.pairs = a.solve_t + solve_bytes(dims);
    a.dx = reinterpret_cast<float*>(a.pairs + solve_bytes(dims));
    a.dstates = a.dx + dx_bytes(dims) / 4;
    a.states = states ? const_cast<float*>(states) : a.dstates + state_bytes(dims) / 4;
    a.dout = dout; a.d_final_state = d_final_state;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.d_initial_state = d_initial_state;
    a.vec_o = pieces(dout, s.ld_o, s.esz, dims->value_dim) && aligned(a.states, 16);
    hipError_t e = copy_rows(a, dims, s, q, k);
    if (e == hipSuccess) e = mamba::launch_delta_prepare(a);
    if (e == hipSuccess && !states) e = mamba::launch_delta_fwd(a);   // no output: the states alone
    if (e == hipSuccess) e = mamba::launch_delta_bwd_states(a);
    if (e == hipSuccess) e = mamba::launch_delta_bwd_grads(a);
    return hip_status(e);
}

int mamba_gated_delta_rule_update(const mamba_delta_dims_t* dims, float* state, const void* q, const void* k,
                                  const void* v, const float* g, const float* beta, const uint8_t* reset, void* out,
                                  void* stream) {
    const int st = check_dims(dims, kMaxElems);
    if (st != MAMBA_OK) return st;
    if (dims->seqlen != 1) return MAMBA_ERR_INVALID_ARGUMENT;
    if (dims->batch == 0) return MAMBA_OK;
    if (!state || !q || !k || !v || !beta || !out) return MAMBA_ERR_INVALID_ARGUMENT;
    const Sizes s = sizes(dims);
    if (!aligned(state, 4) || (g && !aligned(g, 4)) || !aligned(beta, 4) || !aligned(q, s.esz) ||
        !aligned(k, s.esz) || !aligned(v, s.esz) || !aligned(out, s.esz))
        return MAMBA_ERR_MISALIGNED;
    const Span ins[] = {{q, span(s.tokens, s.kw, s.ld_q, s.esz)}, {k, span(s.tokens, s.kw, s.ld_k, s.esz)},
                        {v, span(s.tokens, s.vw, s.ld_v, s.esz)}, {g, s.gate}, {beta, s.gate},
                        {reset, static_cast<size_t>(dims->batch)}};
    const Span outs[] = {{state, s.state}, {out, s.v}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    mamba::DeltaUpdateArgs a{};
    a.state = state; a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.reset = reset; a.out = out;
    a.batch = dims->batch;
    a.ld_q = s.ld_q; a.ld_k = s.ld_k; a.ld_v = s.ld_v;
    a.kheads = dims->key_heads; a.vheads = dims->value_heads; a.kdim = dims->key_dim; a.vdim = dims->value_dim;
    a.scale = dims->scale;
    a.bf16 = dims->dtype == MAMBA_DTYPE_BF16;
    a.vec = dims->value_dim % 4 == 0 && aligned(state, 16);
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_delta_update(a));
}

}  // extern "C"
