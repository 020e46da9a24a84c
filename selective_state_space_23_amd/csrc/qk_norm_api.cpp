// C ABI of the queries' and keys' head norms with position rotation: argument
// validation and dispatch.  Every check runs on the host before any launch.
#include "mamba_hip.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.hpp"
#include "fill.hpp"
#include "qk_norm_launch.hpp"

namespace {

using namespace mamba::api;

constexpr int64_t kMaxWidth = int64_t(1) << 21;    // channels of a token
constexpr int64_t kMaxTokens = int64_t(1) << 31;   // rows times tokens: counted in 32 bits
constexpr int64_t kMaxTable = int64_t(1) << 31;

int hip_status(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

int check_dims(const mamba_qk_norm_dims_t* d) {
    if (!d) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->batch < 0 || d->seqlen < 0 || d->batch > 65535) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->q_heads <= 0 || d->k_heads < 0 || d->head_dim <= 0) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->rotary_dim < 0 || d->rotary_dim % 2 != 0 || d->rotary_dim > d->head_dim) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->table_rows < 0 || (d->rotary_dim > 0 && d->table_rows == 0)) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->dtype != MAMBA_DTYPE_F32 && d->dtype != MAMBA_DTYPE_BF16) return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->norm != MAMBA_NORM_RMS && d->norm != MAMBA_NORM_L2) return MAMBA_ERR_INVALID_ARGUMENT;
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return MAMBA_ERR_INVALID_ARGUMENT;
    const int64_t qw = int64_t(d->q_heads) * d->head_dim, kw = int64_t(d->k_heads) * d->head_dim;
    const int64_t lds[][2] = {{d->ld_q, qw}, {d->ld_k, kw}, {d->ld_dq_out, qw}, {d->ld_dk_out, kw}};
    for (const auto& ld : lds)
        if (ld[0] < 0 || (ld[0] != 0 && ld[0] < ld[1])) return MAMBA_ERR_INVALID_ARGUMENT;
    for (const auto& ld : lds)
        if (ld[0] > kMaxElems) return MAMBA_ERR_UNSUPPORTED;
    if (d->head_dim > mamba::kNormMaxDim || qw > kMaxWidth || kw > kMaxWidth || d->seqlen > kMaxSeqlen)
        return MAMBA_ERR_UNSUPPORTED;
    if (d->batch * d->seqlen >= kMaxTokens || d->table_rows > kMaxTable) return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

// Checks what both directions take and fills it in.
int common(const mamba_qk_norm_dims_t* d, const void* q, const void* k, const float* q_weight, const float* k_weight,
           const float* cos, const float* sin, const int32_t* positions, mamba::QkNormArgs* a) {
    if (!q || (d->k_heads > 0) != (k != nullptr) || (d->k_heads == 0 && k_weight)) return MAMBA_ERR_INVALID_ARGUMENT;
    if ((d->rotary_dim > 0) != (cos != nullptr) || (d->rotary_dim > 0) != (sin != nullptr) ||
        (positions && d->rotary_dim == 0))
        return MAMBA_ERR_INVALID_ARGUMENT;
    if (d->rotary_dim > 0 && !positions && d->seqlen > d->table_rows) return MAMBA_ERR_INVALID_ARGUMENT;
    const size_t esz = d->dtype == MAMBA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(q, esz) || !aligned(k, esz)) return MAMBA_ERR_MISALIGNED;
    const void* words[] = {q_weight, k_weight, cos, sin, positions};
    for (const void* p : words)
        if (!aligned(p, 4)) return MAMBA_ERR_MISALIGNED;
    const int64_t qw = int64_t(d->q_heads) * d->head_dim, kw = int64_t(d->k_heads) * d->head_dim;
    a->x[0] = q; a->x[1] = k;
    a->weight[0] = q_weight; a->weight[1] = k_weight;
    a->cos = cos; a->sin = sin; a->positions = positions;
    a->ld_x[0] = d->ld_q ? d->ld_q : qw;
    a->ld_x[1] = d->ld_k ? d->ld_k : kw;
    a->ld_dy[0] = d->ld_dq_out ? d->ld_dq_out : qw;
    a->ld_dy[1] = d->ld_dk_out ? d->ld_dk_out : kw;
    a->heads[0] = d->q_heads; a->heads[1] = d->k_heads;
    a->tokens = d->batch * d->seqlen; a->seqlen = d->seqlen; a->table_rows = d->table_rows;
    a->dim = d->head_dim; a->rot = d->rotary_dim;
    a->eps = d->eps;
    a->rms = d->norm == MAMBA_NORM_RMS;
    a->interleaved = d->interleaved != 0;
    a->bf16 = d->dtype == MAMBA_DTYPE_BF16;
    // four channels at a time, eight where pairs are interleaved
    const size_t piece = (a->interleaved ? 8 : 4) * esz < 16 ? (a->interleaved ? 8 : 4) * esz : 16;
    a->vec = d->head_dim % 8 == 0 && d->rotary_dim % 8 == 0 && aligned(q, piece) && aligned(k, piece) &&
             a->ld_x[0] * esz % piece == 0 && a->ld_x[1] * esz % piece == 0 && aligned(q_weight, 16) &&
             aligned(k_weight, 16) && aligned(cos, 16) && aligned(sin, 16);
    return MAMBA_OK;
}

size_t table_bytes(const mamba_qk_norm_dims_t* d) { return static_cast<size_t>(d->table_rows) * d->rotary_dim * 2; }

}  // namespace

extern "C" {

int mamba_qk_norm_rotary_fwd(const mamba_qk_norm_dims_t* dims, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* cos, const float* sin, const int32_t* positions,
                             void* q_out, void* k_out, void* stream) {
    int st = check_dims(dims);
    if (st != MAMBA_OK) return st;
    if (dims->batch * dims->seqlen == 0) return MAMBA_OK;
    mamba::QkNormArgs a{};
    if ((st = common(dims, q, k, q_weight, k_weight, cos, sin, positions, &a)) != MAMBA_OK) return st;
    if (!q_out || (dims->k_heads > 0) != (k_out != nullptr)) return MAMBA_ERR_INVALID_ARGUMENT;
    const size_t esz = a.bf16 ? 2 : 4, wb = static_cast<size_t>(a.dim) * 4;
    if (!aligned(q_out, esz) || !aligned(k_out, esz)) return MAMBA_ERR_MISALIGNED;
    const int64_t qw = int64_t(a.heads[0]) * a.dim, kw = int64_t(a.heads[1]) * a.dim;
    const Span ins[] = {{q, span(a.tokens, qw, a.ld_x[0], esz)}, {k, span(a.tokens, kw, a.ld_x[1], esz)}, {q_weight, wb},
                        {k_weight, wb}, {cos, table_bytes(dims)}, {sin, table_bytes(dims)},
                        {positions, static_cast<size_t>(a.tokens) * 4}};
    const Span outs[] = {{q_out, static_cast<size_t>(a.tokens * qw) * esz}, {k_out, static_cast<size_t>(a.tokens * kw) * esz}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    a.out[0] = q_out; a.out[1] = k_out;
    a.vec = a.vec && aligned(q_out, 16) && aligned(k_out, 16);
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_qk_norm_fwd(a));
}

int mamba_qk_norm_rotary_bwd_workspace_bytes(const mamba_qk_norm_dims_t* dims, size_t* bytes) {
    if (!bytes) return MAMBA_ERR_INVALID_ARGUMENT;
    *bytes = 0;
    const int st = check_dims(dims);
    if (st != MAMBA_OK) return st;
    if (dims->batch * dims->seqlen != 0)
        *bytes = mamba::qk_norm_bwd_workspace_bytes(dims->batch * dims->seqlen, dims->q_heads, dims->k_heads, dims->head_dim);
    return MAMBA_OK;
}

int mamba_qk_norm_rotary_bwd(const mamba_qk_norm_dims_t* dims, const void* q, const void* k, const float* q_weight,
                             const float* k_weight, const float* cos, const float* sin, const int32_t* positions,
                             const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_dims(dims);
    if (st != MAMBA_OK) return st;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return MAMBA_ERR_MISALIGNED;
    const size_t wb = static_cast<size_t>(dims->head_dim) * 4;
    if (dims->batch * dims->seqlen == 0) {
        if (overlap(dq_weight, wb, dk_weight, wb)) return MAMBA_ERR_INVALID_ARGUMENT;
        const hipStream_t s = static_cast<hipStream_t>(stream);
        const hipError_t e = mamba::launch_fill(dq_weight, nullptr, dims->head_dim, s);
        return hip_status(e != hipSuccess ? e : mamba::launch_fill(dk_weight, nullptr, dims->head_dim, s));
    }
    mamba::QkNormArgs a{};
    if ((st = common(dims, q, k, q_weight, k_weight, cos, sin, positions, &a)) != MAMBA_OK) return st;
    const bool has_k = dims->k_heads > 0;
    if (!dq_out || !dq || has_k != (dk_out != nullptr) || has_k != (dk != nullptr)) return MAMBA_ERR_INVALID_ARGUMENT;
    if ((dq_weight != nullptr) != (q_weight != nullptr) || (dk_weight != nullptr) != (k_weight != nullptr))
        return MAMBA_ERR_INVALID_ARGUMENT;
    const size_t esz = a.bf16 ? 2 : 4;
    const void* acts[] = {dq_out, dk_out, dq, dk};
    for (const void* p : acts)
        if (!aligned(p, esz)) return MAMBA_ERR_MISALIGNED;
    const size_t need = dq_weight || dk_weight
        ? mamba::qk_norm_bwd_workspace_bytes(a.tokens, a.heads[0], a.heads[1], a.dim) : 0;
    if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return MAMBA_ERR_MISALIGNED;
    const int64_t qw = int64_t(a.heads[0]) * a.dim, kw = int64_t(a.heads[1]) * a.dim;
    const Span ins[] = {{q, span(a.tokens, qw, a.ld_x[0], esz)}, {k, span(a.tokens, kw, a.ld_x[1], esz)}, {q_weight, wb},
                        {k_weight, wb}, {cos, table_bytes(dims)}, {sin, table_bytes(dims)},
                        {positions, static_cast<size_t>(a.tokens) * 4}, {dq_out, span(a.tokens, qw, a.ld_dy[0], esz)},
                        {dk_out, span(a.tokens, kw, a.ld_dy[1], esz)}};
    const Span outs[] = {{dq, static_cast<size_t>(a.tokens * qw) * esz}, {dk, static_cast<size_t>(a.tokens * kw) * esz},
                         {dq_weight, wb}, {dk_weight, wb}, {need ? workspace : nullptr, need}};
    if (!disjoint(ins, outs)) return MAMBA_ERR_INVALID_ARGUMENT;
    a.dy[0] = dq_out; a.dy[1] = dk_out;
    a.out[0] = dq; a.out[1] = dk;
    a.dweight[0] = dq_weight; a.dweight[1] = dk_weight;
    a.parts = static_cast<float*>(workspace);
    a.vec = a.vec && aligned(dq_out, 16) && aligned(dk_out, 16) && aligned(dq, 16) && aligned(dk, 16) &&
            a.ld_dy[0] * esz % 16 == 0 && a.ld_dy[1] * esz % 16 == 0;
    a.stream = static_cast<hipStream_t>(stream);
    return hip_status(mamba::launch_qk_norm_bwd(a));
}

}  // extern "C"
