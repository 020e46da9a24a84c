// Backward of the gated linear recurrence (recurrence.hip), gfx950: the gradients
// of sum(dout out) + sum(d_final_state final_state).
//
// With dy = dout silu(z), v = i x and the adjoint
//     G_t = dy_t + e_{t+1},   e_t = a_t G_t  (0 at a document start),
// e after the last token being d_final_state:
//     dx = G w i,   dgate_x = G w v (1 - i),   dz = dout h silu'(z),
//     r dlog a = G (r a h_{t-1} - (r / w) a^2 v),
//     dgate_a = -c softplus(a_param) (1 - r) r dlog a,
//     da_param = -c sigmoid(a_param) sum r dlog a,   d_initial_state = e_0.
// r / w stays finite as r -> 0 (w goes with sqrt r), where dlog a alone does not;
// where w^2 is 0 (or denormal) its term is left out.
//
// The state entering every 128 tokens comes from the forward (or is recomputed
// by its kernels into the workspace), so a tile rebuilds its own states without
// looking left.  The adjoint's maps e -> P e + X compose from the right with the
// same decays P as the forward's.
#include "recurrence.hpp"

namespace mamba {

namespace {

using namespace rec;

constexpr int kK = 4;
constexpr int kWaves = kTileTokens / (4 * kK);
constexpr int kThreads = kWaves * 64;

enum { kAggregate = 0, kOutput = 1 };

__device__ __forceinline__ float silu_grad(float z, float sg) { return sg * __builtin_fmaf(z, 1.0f - sg, 1.0f); }

// kAggregate writes the tile's adjoint map (P, X) per channel; kOutput starts
// from the adjoint entering the tile from the right (adj) and writes the
// gradients and the tile's part of sum r dlog a.
template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, int MODE>
__global__ __launch_bounds__(kThreads, MODE == kOutput ? 2 : 4) void rec_bwd_kernel(const RecBwdArgs a, int nct, int ntiles,
                                                              float2* __restrict__ agg,
                                                              const float* __restrict__ adj,
                                                              float* __restrict__ part) {
    __shared__ float s_k2[kTileChannels];
    __shared__ float s_P[kWaves][kTileChannels], s_H[kWaves][kTileChannels], s_X[kWaves][kTileChannels];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, ts = lane >> 4;
    const unsigned nchain = static_cast<unsigned>(nct) * static_cast<unsigned>(a.batch);
    const unsigned chain = blockIdx.x % nchain;
    const int tile = ntiles - 1 - static_cast<int>(blockIdx.x / nchain);
    const int ct = static_cast<int>(chain % static_cast<unsigned>(nct));
    const int64_t b = chain / static_cast<unsigned>(nct);
    const int dim = static_cast<int>(a.dim);
    const int64_t t0 = static_cast<int64_t>(tile) * kTileTokens;
    const int64_t row_tok = b * a.seqlen + t0;
    const int64_t left = a.seqlen - t0;
    const int nv = left < kTileTokens ? static_cast<int>(left) : kTileTokens;
    const int tok = (wave * 4 + ts) * kK;
    const int c = ct * kTileChannels + 4 * li;
    const int c_ld = ALIGNED ? (c < dim ? c : dim - 4) : c;
    const int64_t rows = a.batch * a.seqlen;

    LaneIn<T, ALIGNED, PIN, kK> xi, ai, gi, zi;
    LaneIn<T, ALIGNED, false, kK> oi;
    ai.load(a.gate_a, a.in[1], row_tok, a.ld_a, tok, nv, c_ld, dim, ct, rows);
    oi.load(a.dout, a.in[0], row_tok, a.ld_o, tok, nv, c_ld, dim, ct, rows);
    if constexpr (HAS_Z) zi.load(a.z, a.in[3], row_tok, a.ld_z, tok, nv, c_ld, dim, ct, rows);
    if constexpr (MODE == kOutput) {
        gi.load(a.gate_x, a.in[2], row_tok, a.ld_g, tok, nv, c_ld, dim, ct, rows);
        xi.load(a.x, a.in[0], row_tok, a.ld_x, tok, nv, c_ld, dim, ct, rows);
    }
    const TileStarts starts = tile_starts(a.doc_start, b * a.seqlen, t0, a.seqlen);
    if (threadIdx.x < kTileChannels) {
        const int d = ct * kTileChannels + threadIdx.x;
        s_k2[threadIdx.x] = -a.c * softplus_exact(a.a_param[d < dim ? d : dim - 1]);
    }
    lds_barrier();
    float kc4[4];   // -c softplus(a_param)
#pragma unroll
    for (int j = 0; j < 4; ++j) kc4[j] = s_k2[4 * li + j];

    auto body = [&](auto gen) {
        constexpr bool GEN = decltype(gen)::value;
        const uint32_t st = GEN ? starts.bits(tok, kK) : 0u;
        float A[kK][4], B[kK][4];     // effective decays, inputs
        float P[4], H[4], X[4];
        static_for<kK>([&](auto kc) {
            constexpr int k = decltype(kc)::value;
            float ga[4], gx[4], x[4], dy[4], z[4];
            ai.template get<k>(ga);
            oi.template get<k>(dy);
            if constexpr (HAS_Z) zi.template get<k>(z);
            if constexpr (MODE == kOutput) {
                gi.template get<k>(gx);
                xi.template get<k>(x);
            }
            const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= nv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float al, om = 0.0f, bb = 0.0f;
                if constexpr (MODE == kOutput) {
                    decay_terms(kc4[j] * kLog2e * sigmoid_f(ga[j]), al, om);
                    bb = __builtin_amdgcn_sqrtf(om) * (sigmoid_f(gx[j]) * x[j]);
                } else {
                    al = exp2_fast(kc4[j] * kLog2e * sigmoid_f(ga[j]));
                }
                if constexpr (HAS_Z) dy[j] *= silu_f(z[j]);
                if constexpr (GEN) {
                    al = out ? 1.0f : al;
                    bb = out ? 0.0f : bb;
                    dy[j] = out ? 0.0f : dy[j];
                }
                A[k][j] = al;
                B[k][j] = bb;
                if constexpr (k == 0) {
                    P[j] = start ? -0.0f : al;
                    H[j] = bb;
                    X[j] = start ? 0.0f : al * dy[j];
                } else {
                    P[j] = start ? -0.0f : P[j] * al;
                    H[j] = start ? bb : __builtin_fmaf(al, H[j], bb);
                    X[j] = GEN && is_reset(P[j]) ? X[j] : __builtin_fmaf(P[j], dy[j], X[j]);
                }
            }
        });
        // prefixes (forward) and suffixes (adjoint) over the wave's four groups
        float fp[4], fh[4], rp[4], rx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float p = P[j], x = X[j];
            float p1 = __shfl_down(p, 16), x1 = __shfl_down(x, 16);
            if (ts <= 2) { x = apply(p, x, x1); p = is_reset(p) ? p : p * p1; }
            p1 = __shfl_down(p, 32); x1 = __shfl_down(x, 32);
            if (ts <= 1) { x = apply(p, x, x1); p = is_reset(p) ? p : p * p1; }
            if (ts == 0) {
                s_P[wave][4 * li + j] = p;
                s_X[wave][4 * li + j] = x;
            }
            p1 = __shfl_down(p, 16); x1 = __shfl_down(x, 16);
            rp[j] = ts <= 2 ? p1 : 1.0f;
            rx[j] = ts <= 2 ? x1 : 0.0f;
            if constexpr (MODE == kOutput) {
                p = P[j];
                float h = H[j];
                p1 = __shfl_up(p, 16);
                float h1 = __shfl_up(h, 16);
                if (ts >= 1) compose(p, h, p1, h1);
                p1 = __shfl_up(p, 32); h1 = __shfl_up(h, 32);
                if (ts >= 2) compose(p, h, p1, h1);
                if (ts == 3) s_H[wave][4 * li + j] = h;
                p1 = __shfl_up(p, 16); h1 = __shfl_up(h, 16);
                fp[j] = ts >= 1 ? p1 : 1.0f;
                fh[j] = ts >= 1 ? h1 : 0.0f;
            }
        }
        lds_barrier();
        if constexpr (MODE == kAggregate) {
            if (threadIdx.x < kTileChannels) {
                float p = s_P[kWaves - 1][threadIdx.x], x = s_X[kWaves - 1][threadIdx.x];
#pragma unroll
                for (int w = kWaves - 2; w >= 0; --w) {
                    const float pl = s_P[w][threadIdx.x];
                    x = apply(pl, s_X[w][threadIdx.x], x);
                    p = is_reset(pl) ? pl : pl * p;
                }
                const int d = ct * kTileChannels + threadIdx.x;
                if (d < dim) agg[(b * ntiles + tile) * a.dim + d] = make_float2(p, x);
            }
            return;
        } else {
            float hp[kK][4], e[4], sum[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = c + j < dim ? c + j : dim - 1;
                float h = a.states != nullptr ? a.states[(b * ntiles + tile) * a.dim + d]
                                              : (a.initial_state != nullptr ? a.initial_state[b * a.dim + d] : 0.0f);
                for (int w = 0; w < wave; ++w) h = apply(s_P[w][4 * li + j], s_H[w][4 * li + j], h);
                h = apply(fp[j], fh[j], h);
#pragma unroll
                for (int k = 0; k < kK; ++k) {
                    hp[k][j] = h;
                    h = GEN && ((st >> k) & 1u) ? B[k][j] : __builtin_fmaf(A[k][j], h, B[k][j]);
                }
                e[j] = ntiles > 1 ? adj[(b * ntiles + tile) * a.dim + d]
                                  : (a.d_final_state != nullptr ? a.d_final_state[b * a.dim + d] : 0.0f);
                for (int w = kWaves - 1; w > wave; --w) e[j] = apply(s_P[w][4 * li + j], s_X[w][4 * li + j], e[j]);
                e[j] = apply(rp[j], rx[j], e[j]);
                sum[j] = 0.0f;
            }
            const int64_t ob = row_tok * a.dim * Elem<T>::kBytes;
            static_for<kK>([&](auto kc) {
                constexpr int k = kK - 1 - decltype(kc)::value;
                float ga[4], gx[4], x[4], dy[4], z[4], dx[4], da[4], dg[4], dz[4];
                ai.template get<k>(ga);
                gi.template get<k>(gx);
                xi.template get<k>(x);
                oi.template get<k>(dy);
                if constexpr (HAS_Z) zi.template get<k>(z);
                const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= nv;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float r = sigmoid_f(ga[j]);
                    float al, om;
                    decay_terms(kc4[j] * kLog2e * r, al, om);
                    const float rw = om >= 0x1p-126f ? __builtin_amdgcn_rsqf(om) : 0.0f;   // denormals count as 0
                    const float w = om * rw;
                    const float ig = sigmoid_f(gx[j]);
                    const float v = ig * x[j];
                    const float ah = start ? 0.0f : A[k][j] * hp[k][j];
                    if constexpr (HAS_Z) {
                        const float sg = sigmoid_f(z[j]);
                        dz[j] = dy[j] * (start ? B[k][j] : ah + B[k][j]) * silu_grad(z[j], sg);
                        dy[j] *= z[j] * sg;
                    }
                    if constexpr (GEN) dy[j] = out ? 0.0f : dy[j];
                    const float G = dy[j] + e[j];
                    const float gw = G * w;
                    dx[j] = gw * ig;
                    dg[j] = gw * v * (1.0f - ig);
                    const float q = G * r * (ah - rw * (al * al) * v);
                    da[j] = kc4[j] * (1.0f - r) * q;
                    sum[j] += out ? 0.0f : q;
                    e[j] = start ? 0.0f : A[k][j] * G;
                }
                if (!GEN || !out) {
                    const uint32_t to = static_cast<uint32_t>(tok + k) * static_cast<uint32_t>(dim);
                    store4<T, ALIGNED>(static_cast<char*>(a.dx) + ob, to, c, dim, dx);
                    store4<T, ALIGNED>(static_cast<char*>(a.dgate_a) + ob, to, c, dim, da);
                    store4<T, ALIGNED>(static_cast<char*>(a.dgate_x) + ob, to, c, dim, dg);
                    if constexpr (HAS_Z) store4<T, ALIGNED>(static_cast<char*>(a.dz) + ob, to, c, dim, dz);
                }
            });
            if (tile == 0 && wave == 0 && ts == 0 && a.d_initial_state != nullptr) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < dim) a.d_initial_state[b * a.dim + c + j] = e[j];
            }
            lds_barrier();   // s_P is read above
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[j] += __shfl_xor(sum[j], 16);
                sum[j] += __shfl_xor(sum[j], 32);
                if (ts == 0) s_P[wave][4 * li + j] = sum[j];
            }
            lds_barrier();
            if (threadIdx.x < kTileChannels) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) s += s_P[w][threadIdx.x];
                const int d = ct * kTileChannels + threadIdx.x;
                if (d < dim) part[(b * ntiles + tile) * a.dim + d] = s;
            }
        }
    };
    if (starts.any() || nv < kTileTokens) body(std::true_type{});
    else body(std::false_type{});
}

// Adjoints entering every tile from the right.
__global__ __launch_bounds__(256) void rec_bwd_carry_kernel(const float2* __restrict__ agg,
                                                            const float* __restrict__ d_final_state,
                                                            float* __restrict__ adj, int64_t batch, int64_t dim,
                                                            int ntiles) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= batch * dim) return;
    const int64_t b = i / dim, d = i % dim;
    float e = d_final_state != nullptr ? d_final_state[i] : 0.0f;
    const int64_t base = b * ntiles * dim + d;
    for (int t = ntiles - 1; t >= 0; --t) {
        adj[base + t * dim] = e;
        if (t > 0) {
            const float2 u = agg[base + t * dim];
            e = apply(u.x, u.y, e);
        }
    }
}

// da_param (D,): the tiles' parts summed in a fixed order, 16 threads a channel.
__global__ __launch_bounds__(1024) void rec_bwd_reduce_kernel(const float* __restrict__ part,
                                                              const float* __restrict__ a_param,
                                                              float* __restrict__ da_param, int64_t nparts, int dim,
                                                              float c) {
    __shared__ float red[16][64];
    const int o = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int d = static_cast<int>(blockIdx.x) * 64 + o;
    float s = 0.0f;
    if (d < dim)
        for (int64_t i = g; i < nparts; i += 16) s += part[i * dim + d];
    red[g][o] = s;
    __syncthreads();
    if (g != 0 || d >= dim) return;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += red[k][o];
    da_param[d] = -c * t * sigmoid_f(a_param[d]);
}

struct BwdWs {
    size_t agg, adj, part, states, fwd, total;
};

BwdWs bwd_ws(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
    const size_t n = static_cast<size_t>(batch * ((seqlen + kRecChunk - 1) / kRecChunk) * dim);
    BwdWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) / 256 * 256; return o; };
    w.part = take(n * 4);
    w.agg = take(n * 8);
    w.adj = take(n * 4);
    w.states = take(have_states ? 0 : n * 4);
    w.fwd = take(have_states ? 0 : recurrence_workspace_bytes(batch, seqlen, dim, true));
    w.total = off;
    return w;
}

template <typename T, bool ALIGNED, bool PIN, bool HAS_Z>
hipError_t launch_bwd(const RecBwdArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const int ntiles = static_cast<int>((a.seqlen + kTileTokens - 1) / kTileTokens);
    const unsigned grid = static_cast<unsigned>(nct) * static_cast<unsigned>(a.batch) * static_cast<unsigned>(ntiles);
    const BwdWs w = bwd_ws(a.batch, a.seqlen, a.dim, a.states != nullptr);
    char* ws = static_cast<char*>(a.ws);
    float2* agg = reinterpret_cast<float2*>(ws + w.agg);
    float* adj = reinterpret_cast<float*>(ws + w.adj);
    float* part = reinterpret_cast<float*>(ws + w.part);
    RecBwdArgs b = a;
    hipError_t e;
    if (a.states == nullptr && ntiles > 1) {
        RecFwdArgs f{};
        f.x = a.x; f.gate_a = a.gate_a; f.gate_x = a.gate_x;
        for (int i = 0; i < 3; ++i) f.in[i] = a.in[i];
        f.a_param = a.a_param; f.doc_start = a.doc_start; f.initial_state = a.initial_state;
        f.states = reinterpret_cast<float*>(ws + w.states);
        f.ws = ws + w.fwd;
        f.batch = a.batch; f.seqlen = a.seqlen; f.dim = a.dim;
        f.ld_x = a.ld_x; f.ld_a = a.ld_a; f.ld_g = a.ld_g;
        f.c = a.c; f.bf16 = a.bf16; f.aligned = a.aligned; f.stream = a.stream;
        if ((e = launch_recurrence_fwd(f)) != hipSuccess) return e;
        b.states = f.states;
    }
    if (ntiles > 1) {
        hipLaunchKernelGGL((rec_bwd_kernel<T, ALIGNED, PIN, HAS_Z, kAggregate>), dim3(grid), dim3(kThreads), 0,
                           a.stream, b, nct, ntiles, agg, adj, part);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(rec_bwd_carry_kernel, dim3(static_cast<unsigned>((a.batch * a.dim + 255) / 256)), dim3(256),
                           0, a.stream, agg, a.d_final_state, adj, a.batch, a.dim, ntiles);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((rec_bwd_kernel<T, ALIGNED, PIN, HAS_Z, kOutput>), dim3(grid), dim3(kThreads), 0, a.stream, b,
                       nct, ntiles, agg, adj, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(rec_bwd_reduce_kernel, dim3(static_cast<unsigned>((a.dim + 63) / 64)), dim3(1024), 0, a.stream,
                       part, a.a_param, a.da_param, a.batch * ntiles, static_cast<int>(a.dim), a.c);
    return hipGetLastError();
}

template <typename T, bool ALIGNED>
hipError_t launch_bwd_typed(const RecBwdArgs& a) {
    if (a.in[0].q != nullptr)
        return a.has_z ? launch_bwd<T, ALIGNED, true, true>(a) : launch_bwd<T, ALIGNED, true, false>(a);
    return a.has_z ? launch_bwd<T, ALIGNED, false, true>(a) : launch_bwd<T, ALIGNED, false, false>(a);
}

}  // namespace

size_t recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
    return bwd_ws(batch, seqlen, dim, have_states).total;
}

hipError_t launch_recurrence_bwd(const RecBwdArgs& a) {
    if (a.bf16) return a.aligned ? launch_bwd_typed<bf16_t, true>(a) : launch_bwd_typed<bf16_t, false>(a);
    return a.aligned ? launch_bwd_typed<float, true>(a) : launch_bwd_typed<float, false>(a);
}

}  // namespace mamba
