// C ABI of the gated linear recurrence and of the 8-bit activation checkpoints:
// argument validation and dispatch.  Every check runs on the host before any
// launch.
#include "mamba_hip.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.hpp"
#include "fill.hpp"
#include "recurrence_launch.hpp"

static_assert(MAMBA_PACK_BLOCK == mamba::kPackBlock && MAMBA_RECURRENCE_CHUNK == mamba::kRecChunk,
              "the header and the kernels agree");

namespace {

using namespace mamba::api;

constexpr int64_t kMaxWidth = int64_t(1) << 21;   // channels and strides: a tile's offsets fit 32 bits
constexpr int64_t kMaxRowStride = kMaxElems;      // the one-token step's, which addresses in 64 bits
constexpr int64_t kMaxTiles = 8000000;            // workgroups of one launch

// `max_ld`: of the step's own inputs (dout is none of them).
int check_rec_dims(const mamba_recurrence_dims_t* d, int64_t max_ld = kMaxWidth) {
    if (!d) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->batch < 0 || d->seqlen < 0 || d->dim < 0 || d->batch > 65535) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->dtype != MAMBA_DTYPE_F32 && d->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID_ARGUMENT;
    if (!(d->c > 0.0f) || !std::isfinite(d->c)) return MAMBA_ERR_INVALID_ARGUMENT;
    const int64_t lds[] = {d->ld_x, d->ld_gate_a, d->ld_gate_x, d->ld_z, d->ld_dout};
    for (int64_t ld : lds) {
        if (ld < 0 || (ld != 0 && ld < d->dim)) return MAMBA_ERR_INVALID_ARGUMENT;
        if (ld > max_ld) return MAMBA_ERR_UNSUPPORTED;
    }
    if (d->ld_dout > kMaxWidth) return MAMBA_ERR_UNSUPPORTED;
    if (d->dim > kMaxWidth || d->seqlen > kMaxSeqlen) return MAMBA_ERR_UNSUPPORTED;
    if (d->batch * ceil_div(d->seqlen, mamba::kRecChunk) * ceil_div(d->dim, mamba::kPackBlock) > kMaxTiles)
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

// `save` / `packed`: four checkpoints, the last only with z.
int check_packed(const mamba_packed_t* p, bool has_z) {
    if (!p) return MAMBA_OK;
    for (int i = 0; i < 4; ++i) {
        const bool want = i < 3 || has_z;
        if (want != (p[i].q != nullptr) || want != (p[i].scale != nullptr)) return MAMBA_ERR_INVALID_ARGUMENT;
        if (want && !aligned(p[i].scale, 4)) return MAMBA_ERR_MISALIGNED;
    }
    return MAMBA_OK;
}

// Pointers and strides that the vectorised kernels take: quads of channels.
bool quads(const void* p, int64_t ld, size_t esz) { return aligned(p, 4 * esz) && ld % 4 == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

int check_pack(const void* act, const int8_t* q, const float* scale, int64_t rows, int64_t dim, int64_t ld,
               int32_t dtype, bool* empty) {
    *empty = false;
    if (rows < 0 || dim < 0 || ld < 0 || (ld != 0 && ld < dim)) return MAMBA_ERR_INVALID_ARGUMENT;
    if (dtype != MAMBA_DTYPE_F32 && dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID_ARGUMENT;
    if (dim > kMaxWidth || ld > kMaxWidth || rows > kMaxElems) return MAMBA_ERR_UNSUPPORTED;
    if (rows == 0 || dim == 0) {
        *empty = true;
        return MAMBA_OK;
    }
    if (ceil_div(rows, 64) * ceil_div(dim, mamba::kPackBlock) > 2 * kMaxTiles) return MAMBA_ERR_UNSUPPORTED;
    if (!act || !q || !scale) return MAMBA_ERR_INVALID_ARGUMENT;
    const size_t esz = dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(act, esz) || !aligned(scale, 4)) return MAMBA_ERR_MISALIGNED;
    return MAMBA_OK;
}

}  // namespace

extern "C" {

int mamba_activation_pack(const void* x, int8_t* q, float* scale, int64_t rows, int64_t dim, int64_t ld,
                          int32_t dtype, void* stream) {
    bool empty;
    const int st = check_pack(x, q, scale, rows, dim, ld, dtype, &empty);
    if (st != MAMBA_OK || empty) return st;
    const size_t esz = dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    const int64_t step = ld ? ld : dim;
    const Span ins[] = {{x, span(rows, dim, step, esz)}};
    const Span outs[] = {{q, static_cast<size_t>(rows * dim)},
                         {scale, static_cast<size_t>(rows * ceil_div(dim, mamba::kPackBlock)) * 4}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    mamba::PackArgs a{};
    a.x = x; a.p.q = q; a.p.scale = scale;
    a.rows = rows; a.dim = dim; a.ld = step;
    a.bf16 = dtype == MAMBA_DTYPE_BF16;
    a.aligned = dim % 4 == 0 && quads(x, step, esz) && aligned(q, 4);
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_pack(a));
}

int mamba_activation_unpack(const int8_t* q, const float* scale, void* out, int64_t rows, int64_t dim,
                            int32_t dtype, void* stream) {
    bool empty;
    const int st = check_pack(out, q, scale, rows, dim, 0, dtype, &empty);
    if (st != MAMBA_OK || empty) return st;
    const size_t esz = dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    const Span ins[] = {{q, static_cast<size_t>(rows * dim)},
                        {scale, static_cast<size_t>(rows * ceil_div(dim, mamba::kPackBlock)) * 4}};
    const Span outs[] = {{out, static_cast<size_t>(rows * dim) * esz}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    mamba::PackArgs a{};
    a.out = out; a.p.q = const_cast<int8_t*>(q); a.p.scale = const_cast<float*>(scale);
    a.rows = rows; a.dim = dim; a.ld = dim;
    a.bf16 = dtype == MAMBA_DTYPE_BF16;
    a.aligned = dim % 4 == 0 && quads(out, dim, esz) && aligned(q, 4);
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_unpack(a));
}

int mamba_gated_recurrence_workspace_bytes(const mamba_recurrence_dims_t* dims, size_t* bytes) {
    if (!bytes) return MAMBA_ERR_INVALID_ARGUMENT;
    *bytes = 0;
    const int st = check_rec_dims(dims);
    if (st != MAMBA_OK) return st;
    if (dims->batch * dims->dim != 0)
        *bytes = mamba::recurrence_workspace_bytes(dims->batch, dims->seqlen, dims->dim);
    return MAMBA_OK;
}

int mamba_gated_recurrence_fwd(const mamba_recurrence_dims_t* dims, const void* x, const void* gate_a,
                               const void* gate_x, const float* a_param, const void* z, const uint8_t* doc_start,
                               const float* initial_state, void* out, float* final_state, float* states,
                               const mamba_packed_t* save, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_rec_dims(dims);
    if (st != MAMBA_OK) return st;
    const int64_t B = dims->batch, L = dims->seqlen, D = dims->dim;
    const size_t sb = static_cast<size_t>(B * D) * 4;
    if ((final_state && !aligned(final_state, 4)) || (initial_state && !aligned(initial_state, 4)) ||
        (states && !aligned(states, 4)))
        return MAMBA_ERR_MISALIGNED;
    if (B * L * D == 0) {
        if (L != 0 || B * D == 0) return MAMBA_OK;
        if (overlap(final_state, sb, initial_state, sb)) return MAMBA_ERR_INVALID_ARGUMENT;
        return hip_status(mamba::launch_fill(final_state, initial_state, B * D, static_cast<hipStream_t>(stream)));
    }
    if (!x || !gate_a || !gate_x || !a_param || !out) return MAMBA_ERR_INVALID_ARGUMENT;
    if ((st = check_packed(save, z != nullptr)) != MAMBA_OK) return st;
    const size_t esz = dims->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate_a, esz) || !aligned(gate_x, esz) || (z && !aligned(z, esz)) ||
        !aligned(out, esz) || !aligned(a_param, 4))
        return MAMBA_ERR_MISALIGNED;
    const size_t need = mamba::recurrence_workspace_bytes(B, L, D);
    if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return MAMBA_ERR_MISALIGNED;
    mamba::RecFwdArgs a{};
    a.ld_x = static_cast<int>(dims->ld_x ? dims->ld_x : D);
    a.ld_a = static_cast<int>(dims->ld_gate_a ? dims->ld_gate_a : D);
    a.ld_g = static_cast<int>(dims->ld_gate_x ? dims->ld_gate_x : D);
    a.ld_z = static_cast<int>(dims->ld_z ? dims->ld_z : D);
    const int64_t rows = B * L;
    const size_t scb = static_cast<size_t>(rows * ceil_div(D, mamba::kPackBlock)) * 4;
    const size_t qb = static_cast<size_t>(rows * D);
    const mamba_packed_t none[4] = {};
    const mamba_packed_t* sv = save ? save : none;
    const Span ins[] = {{x, span(rows, D, a.ld_x, esz)}, {gate_a, span(rows, D, a.ld_a, esz)},
                        {gate_x, span(rows, D, a.ld_g, esz)}, {z, span(rows, D, a.ld_z, esz)},
                        {a_param, static_cast<size_t>(D) * 4}, {doc_start, static_cast<size_t>(rows)},
                        {initial_state, sb}};
    const Span outs[] = {{out, qb * esz}, {final_state, sb},
                         {states, static_cast<size_t>(B * ceil_div(L, mamba::kRecChunk) * D) * 4},
                         {sv[0].q, qb}, {sv[1].q, qb}, {sv[2].q, qb}, {sv[3].q, qb},
                         {sv[0].scale, scb}, {sv[1].scale, scb}, {sv[2].scale, scb}, {sv[3].scale, scb},
                         {need ? workspace : nullptr, need}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.z = z;
    a.a_param = a_param; a.doc_start = doc_start; a.initial_state = initial_state;
    a.out = out; a.final_state = final_state; a.states = states; a.ws = workspace;
    bool codes = true;
    for (int i = 0; i < 4; ++i) {
        a.save[i].q = sv[i].q;
        a.save[i].scale = sv[i].scale;
        codes = codes && aligned(sv[i].q, 4);
    }
    a.batch = B; a.seqlen = L; a.dim = D;
    a.c = dims->c;
    a.bf16 = dims->dtype == MAMBA_DTYPE_BF16;
    a.aligned = D % 4 == 0 && quads(x, a.ld_x, esz) && quads(gate_a, a.ld_a, esz) && quads(gate_x, a.ld_g, esz) &&
                (!z || quads(z, a.ld_z, esz)) && aligned(out, 4 * esz) && codes;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_recurrence_fwd(a));
}

int mamba_gated_recurrence_bwd_workspace_bytes(const mamba_recurrence_dims_t* dims, int32_t have_states,
                                               size_t* bytes) {
    if (!bytes) return MAMBA_ERR_INVALID_ARGUMENT;
    *bytes = 0;
    const int st = check_rec_dims(dims);
    if (st != MAMBA_OK) return st;
    if (dims->batch * dims->seqlen * dims->dim != 0)
        *bytes = mamba::recurrence_bwd_workspace_bytes(dims->batch, dims->seqlen, dims->dim, have_states != 0);
    return MAMBA_OK;
}

int mamba_gated_recurrence_bwd(const mamba_recurrence_dims_t* dims, const void* x, const void* gate_a,
                               const void* gate_x, const float* a_param, const void* z, const uint8_t* doc_start,
                               const float* initial_state, const mamba_packed_t* packed, const float* states,
                               const void* dout, const float* d_final_state, void* dx, void* dgate_a, void* dgate_x,
                               float* da_param, void* dz, float* d_initial_state, void* workspace,
                               size_t workspace_bytes, void* stream) {
    int st = check_rec_dims(dims);
    if (st != MAMBA_OK) return st;
    const int64_t B = dims->batch, L = dims->seqlen, D = dims->dim;
    const size_t sb = static_cast<size_t>(B * D) * 4;
    const float* f32s[] = {a_param, initial_state, states, d_final_state, da_param, d_initial_state};
    for (const float* p : f32s)
        if (p && !aligned(p, 4)) return MAMBA_ERR_MISALIGNED;
    if (d_initial_state && !initial_state) return MAMBA_ERR_INVALID_ARGUMENT;
    if (B * L * D == 0) {
        const hipStream_t s = static_cast<hipStream_t>(stream);
        if (overlap(d_initial_state, sb, d_final_state, sb) || overlap(d_initial_state, sb, da_param, D * 4) ||
            overlap(da_param, D * 4, d_final_state, sb))
            return MAMBA_ERR_INVALID_ARGUMENT;
        if (mamba::launch_fill(da_param, nullptr, D, s) != hipSuccess) return MAMBA_ERR_HIP;
        if (L != 0) return MAMBA_OK;
        return hip_status(mamba::launch_fill(d_initial_state, d_final_state, B * D, s));
    }
    const bool has_z = packed ? packed[3].q != nullptr : z != nullptr;
    if (packed ? (x || gate_a || gate_x || z) : (!x || !gate_a || !gate_x)) return MAMBA_ERR_INVALID_ARGUMENT;
    if (!a_param || !dout || !dx || !dgate_a || !dgate_x || !da_param) return MAMBA_ERR_INVALID_ARGUMENT;
    if (has_z != (dz != nullptr)) return MAMBA_ERR_INVALID_ARGUMENT;
    if ((st = check_packed(packed, has_z)) != MAMBA_OK) return st;
    const size_t esz = dims->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    const void* acts[] = {x, gate_a, gate_x, z, dout, dx, dgate_a, dgate_x, dz};
    for (const void* p : acts)
        if (p && !aligned(p, esz)) return MAMBA_ERR_MISALIGNED;
    const size_t need = mamba::recurrence_bwd_workspace_bytes(B, L, D, states != nullptr);
    if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MAMBA_ERR_MISALIGNED;
    mamba::RecBwdArgs a{};
    a.ld_x = static_cast<int>(dims->ld_x ? dims->ld_x : D);
    a.ld_a = static_cast<int>(dims->ld_gate_a ? dims->ld_gate_a : D);
    a.ld_g = static_cast<int>(dims->ld_gate_x ? dims->ld_gate_x : D);
    a.ld_z = static_cast<int>(dims->ld_z ? dims->ld_z : D);
    a.ld_o = static_cast<int>(dims->ld_dout ? dims->ld_dout : D);
    const int64_t rows = B * L;
    const size_t scb = static_cast<size_t>(rows * ceil_div(D, mamba::kPackBlock)) * 4;
    const size_t qb = static_cast<size_t>(rows * D);
    const mamba_packed_t none[4] = {};
    const mamba_packed_t* pk = packed ? packed : none;
    const Span ins[] = {{x, span(rows, D, a.ld_x, esz)}, {gate_a, span(rows, D, a.ld_a, esz)},
                        {gate_x, span(rows, D, a.ld_g, esz)}, {z, span(rows, D, a.ld_z, esz)},
                        {dout, span(rows, D, a.ld_o, esz)}, {a_param, static_cast<size_t>(D) * 4},
                        {doc_start, static_cast<size_t>(rows)}, {initial_state, sb}, {d_final_state, sb},
                        {states, static_cast<size_t>(B * ceil_div(L, mamba::kRecChunk) * D) * 4},
                        {pk[0].q, qb}, {pk[1].q, qb}, {pk[2].q, qb}, {pk[3].q, qb},
                        {pk[0].scale, scb}, {pk[1].scale, scb}, {pk[2].scale, scb}, {pk[3].scale, scb}};
    const Span outs[] = {{dx, qb * esz}, {dgate_a, qb * esz}, {dgate_x, qb * esz}, {dz, qb * esz},
                         {da_param, static_cast<size_t>(D) * 4}, {d_initial_state, sb}, {workspace, need}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.z = z;
    bool vec = D % 4 == 0 && quads(dout, a.ld_o, esz) && aligned(dx, 4 * esz) && aligned(dgate_a, 4 * esz) &&
               aligned(dgate_x, 4 * esz) && aligned(dz, 4 * esz);
    for (int i = 0; i < 4; ++i) {
        a.in[i].q = pk[i].q;
        a.in[i].scale = pk[i].scale;
        vec = vec && aligned(pk[i].q, 4);
    }
    if (!packed)
        vec = vec && quads(x, a.ld_x, esz) && quads(gate_a, a.ld_a, esz) && quads(gate_x, a.ld_g, esz) &&
              (!z || quads(z, a.ld_z, esz));
    a.aligned = vec;
    a.a_param = a_param; a.doc_start = doc_start; a.initial_state = initial_state; a.states = states;
    a.dout = dout; a.d_final_state = d_final_state;
    a.dx = dx; a.dgate_a = dgate_a; a.dgate_x = dgate_x; a.da_param = da_param; a.dz = dz;
    a.d_initial_state = d_initial_state;
    a.ws = workspace;
    a.batch = B; a.seqlen = L; a.dim = D;
    a.c = dims->c;
    a.bf16 = dims->dtype == MAMBA_DTYPE_BF16;
    a.has_z = has_z;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_recurrence_bwd(a));
}

int mamba_gated_recurrence_update(const mamba_recurrence_dims_t* dims, float* state, const void* x,
                                  const void* gate_a, const void* gate_x, const float* a_param, const void* z,
                                  const uint8_t* reset, void* out, void* stream) {
    const int st = check_rec_dims(dims, kMaxRowStride);
    if (st != MAMBA_OK) return st;
    if (dims->seqlen != 1) return MAMBA_ERR_INVALID_ARGUMENT;
    const int64_t B = dims->batch, D = dims->dim;
    if (B * D == 0) return MAMBA_OK;
    if (!state || !x || !gate_a || !gate_x || !a_param || !out) return MAMBA_ERR_INVALID_ARGUMENT;
    const size_t esz = dims->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(state, 4) || !aligned(x, esz) || !aligned(gate_a, esz) || !aligned(gate_x, esz) ||
        (z && !aligned(z, esz)) || !aligned(out, esz) || !aligned(a_param, 4))
        return MAMBA_ERR_MISALIGNED;
    mamba::RecUpdateArgs a{};
    a.ld_x = dims->ld_x ? dims->ld_x : D;
    a.ld_a = dims->ld_gate_a ? dims->ld_gate_a : D;
    a.ld_g = dims->ld_gate_x ? dims->ld_gate_x : D;
    a.ld_z = dims->ld_z ? dims->ld_z : D;
    const Span ins[] = {{x, span(B, D, a.ld_x, esz)}, {gate_a, span(B, D, a.ld_a, esz)},
                        {gate_x, span(B, D, a.ld_g, esz)}, {z, span(B, D, a.ld_z, esz)},
                        {a_param, static_cast<size_t>(D) * 4}, {reset, static_cast<size_t>(B)}};
    const Span outs[] = {{state, static_cast<size_t>(B * D) * 4}, {out, static_cast<size_t>(B * D) * esz}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    a.state = state; a.x = x; a.gate_a = gate_a; a.gate_x = gate_x; a.z = z; a.a_param = a_param;
    a.reset = reset; a.out = out;
    a.batch = B; a.dim = D;
    a.c = dims->c;
    a.bf16 = dims->dtype == MAMBA_DTYPE_BF16;
    a.aligned = D % 4 == 0 && quads(x, a.ld_x, esz) && quads(gate_a, a.ld_a, esz) && quads(gate_x, a.ld_g, esz) &&
                (!z || quads(z, a.ld_z, esz)) && aligned(out, 4 * esz) && aligned(state, 16);
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_recurrence_update(a));
}

}  // extern "C"
