// Gated linear recurrence, forward and one-token step, gfx950.
//
// With r = sigmoid(gate_a), i = sigmoid(gate_x), log a = -c softplus(a_param) r
// and w = sqrt(1 - a^2), per row and channel
//     h_t = a_t h_{t-1} + w_t i_t x_t,    out_t = h_t silu(z_t)   (h_t without z),
// where h_{t-1} is 0 at a document start.
//
// A token's map h -> a h + b composes as (P, H): h -> P h + H.  A document start
// is a map that ignores its input, marked by the sign of P (decays are never
// negative): selects on that sign, not products with zero, keep an infinite or
// NaN state of one document out of the next.
#include "recurrence.hpp"

namespace mamba {

namespace {

using namespace rec;

constexpr int kK = 4;                                // tokens a lane walks
constexpr int kWaves = kTileTokens / (4 * kK);       // 4 groups of 16 lanes a wave
constexpr int kThreads = kWaves * 64;

enum { kAggregate = 0, kOutput = 1 };

// One workgroup per tile.  kAggregate writes the tile's composed map (P, H) per
// channel; kOutput starts from the state entering the tile (a.states, or the
// initial state in a row of one tile) and writes out, the final state and the
// checkpoints.
template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, bool SAVE, int MODE>
__global__ __launch_bounds__(kThreads, 4) void rec_fwd_kernel(const RecFwdArgs a, int nct,
                                                                                    int ntiles,
                                                                                    float2* __restrict__ agg) {
    __shared__ float s_k2[kTileChannels];
    __shared__ float2 s_agg[kWaves][kTileChannels];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, ts = lane >> 4;
    const unsigned nchain = static_cast<unsigned>(nct) * static_cast<unsigned>(a.batch);
    const unsigned chain = blockIdx.x % nchain;
    const int tile = static_cast<int>(blockIdx.x / nchain);
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

    LaneIn<T, ALIGNED, PIN, kK> xi, ai, gi;
    LaneIn<T, ALIGNED, false, kK> zi;
    ai.load(a.gate_a, a.in[1], row_tok, a.ld_a, tok, nv, c_ld, dim, ct, rows);
    gi.load(a.gate_x, a.in[2], row_tok, a.ld_g, tok, nv, c_ld, dim, ct, rows);
    xi.load(a.x, a.in[0], row_tok, a.ld_x, tok, nv, c_ld, dim, ct, rows);
    if constexpr (HAS_Z && MODE != kAggregate) zi.load(a.z, a.in[0], row_tok, a.ld_z, tok, nv, c_ld, dim, ct, rows);
    const TileStarts starts = tile_starts(a.doc_start, b * a.seqlen, t0, a.seqlen);

    if (threadIdx.x < kTileChannels) {
        const int d = ct * kTileChannels + threadIdx.x;
        s_k2[threadIdx.x] = -a.c * kLog2e * softplus_exact(a.a_param[d < dim ? d : dim - 1]);
    }
    lds_barrier();
    float k2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k2[j] = s_k2[4 * li + j];

    if constexpr (SAVE) {
        if (a.save[0].q != nullptr) save_packed<T, ALIGNED, kK>(xi, a.save[0], row_tok, tok, nv, c, dim, ct, rows);
        if (a.save[1].q != nullptr) save_packed<T, ALIGNED, kK>(ai, a.save[1], row_tok, tok, nv, c, dim, ct, rows);
        if (a.save[2].q != nullptr) save_packed<T, ALIGNED, kK>(gi, a.save[2], row_tok, tok, nv, c, dim, ct, rows);
        if constexpr (HAS_Z)
            if (a.save[3].q != nullptr) save_packed<T, ALIGNED, kK>(zi, a.save[3], row_tok, tok, nv, c, dim, ct, rows);
    }

    auto body = [&](auto gen) {
        constexpr bool GEN = decltype(gen)::value;   // document starts or tokens past the row end in the tile
        const uint32_t st = GEN ? starts.bits(tok, kK) : 0u;
        float P[kK][4], H[kK][4];
        static_for<kK>([&](auto kc) {
            constexpr int k = decltype(kc)::value;
            float ga[4], gx[4], x[4];
            ai.template get<k>(ga);
            gi.template get<k>(gx);
            xi.template get<k>(x);
            const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= nv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float al, om;
                decay_terms(k2[j] * sigmoid_f(ga[j]), al, om);
                float bb = __builtin_amdgcn_sqrtf(om) * (sigmoid_f(gx[j]) * x[j]);
                if constexpr (GEN) {
                    al = out ? 1.0f : al;
                    bb = out ? 0.0f : bb;
                }
                if constexpr (k == 0) {
                    P[k][j] = al;
                    H[k][j] = bb;
                } else {
                    P[k][j] = P[k - 1][j] * al;
                    H[k][j] = __builtin_fmaf(al, H[k - 1][j], bb);
                }
                if constexpr (GEN) {
                    P[k][j] = start ? -0.0f : P[k][j];
                    H[k][j] = start ? bb : H[k][j];
                }
            }
        });
        // prefixes over the wave's four groups of lanes
        float wp[4], wh[4], ep[4], eh[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float p = P[kK - 1][j], h = H[kK - 1][j];
            float p1 = __shfl_up(p, 16), h1 = __shfl_up(h, 16);
            if (ts >= 1) compose(p, h, p1, h1);
            p1 = __shfl_up(p, 32); h1 = __shfl_up(h, 32);
            if (ts >= 2) compose(p, h, p1, h1);
            wp[j] = p; wh[j] = h;
            p1 = __shfl_up(p, 16); h1 = __shfl_up(h, 16);
            ep[j] = ts >= 1 ? p1 : 1.0f;
            eh[j] = ts >= 1 ? h1 : 0.0f;
        }
        if (ts == 3) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s_agg[wave][4 * li + j] = make_float2(wp[j], wh[j]);
        }
        lds_barrier();
        if constexpr (MODE == kAggregate) {
            if (threadIdx.x < kTileChannels) {
                float2 t = s_agg[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) {
                    float2 u = s_agg[w][threadIdx.x];
                    compose(u.x, u.y, t.x, t.y);
                    t = u;
                }
                const int d = ct * kTileChannels + threadIdx.x;
                if (d < dim) agg[(b * ntiles + tile) * a.dim + d] = t;
            }
            return;
        }
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int d = c + j < dim ? c + j : dim - 1;
            e[j] = ntiles > 1 ? a.states[(b * ntiles + tile) * a.dim + d]
                              : (a.initial_state != nullptr ? a.initial_state[b * a.dim + d] : 0.0f);
            for (int w = 0; w < wave; ++w) {
                const float2 u = s_agg[w][4 * li + j];
                e[j] = apply(u.x, u.y, e[j]);
            }
            e[j] = apply(ep[j], eh[j], e[j]);
        }
        char* ob = static_cast<char*>(a.out) + row_tok * a.dim * Elem<T>::kBytes;
        static_for<kK>([&](auto kc) {
            constexpr int k = decltype(kc)::value;
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = GEN ? apply(P[k][j], H[k][j], e[j]) : __builtin_fmaf(P[k][j], e[j], H[k][j]);
            if (k == kK - 1 && tile == ntiles - 1 && wave == kWaves - 1 && ts == 3 && a.final_state != nullptr) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < dim) a.final_state[b * a.dim + c + j] = o[j];
            }
            if constexpr (HAS_Z) {
                float z[4];
                zi.template get<k>(z);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] *= silu_f(z[j]);
            }
            if (!GEN || tok + k < nv)
                store4<T, ALIGNED>(ob, static_cast<uint32_t>(tok + k) * static_cast<uint32_t>(dim), c, dim, o);
        });
    };
    // the same in every wave of the workgroup: body holds a barrier
    if (starts.any() || nv < kTileTokens) body(std::true_type{});
    else body(std::false_type{});
}

// States entering every tile: each channel's maps applied in order.
__global__ __launch_bounds__(256) void rec_carry_kernel(const float2* __restrict__ agg,
                                                        const float* __restrict__ initial_state,
                                                        float* __restrict__ states, int64_t batch, int64_t dim,
                                                        int ntiles) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= batch * dim) return;
    const int64_t b = i / dim, d = i % dim;
    float h = initial_state != nullptr ? initial_state[i] : 0.0f;
    const int64_t base = b * ntiles * dim + d;
    for (int t = 0; t < ntiles; ++t) {
        states[base + t * dim] = h;
        if (t + 1 < ntiles) {
            const float2 u = agg[base + t * dim];
            h = apply(u.x, u.y, h);
        }
    }
}

template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, bool SAVE>
hipError_t launch_fwd(const RecFwdArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const int ntiles = static_cast<int>((a.seqlen + kTileTokens - 1) / kTileTokens);
    const unsigned grid = static_cast<unsigned>(nct) * static_cast<unsigned>(a.batch) * static_cast<unsigned>(ntiles);
    RecFwdArgs b = a;
    float2* agg = static_cast<float2*>(a.ws);
    hipError_t e;
    if (ntiles > 1) {
        if (b.states == nullptr) b.states = reinterpret_cast<float*>(agg + a.batch * ntiles * a.dim);
        hipLaunchKernelGGL((rec_fwd_kernel<T, ALIGNED, PIN, false, false, kAggregate>), dim3(grid), dim3(kThreads), 0,
                           a.stream, b, nct, ntiles, agg);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (ntiles > 1 || a.states != nullptr) {
        hipLaunchKernelGGL(rec_carry_kernel, dim3(static_cast<unsigned>((a.batch * a.dim + 255) / 256)), dim3(256), 0,
                           a.stream, agg, a.initial_state, b.states, a.batch, a.dim, ntiles);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.out == nullptr) return hipSuccess;   // the states alone (the backward's recomputation)
    if constexpr (!PIN) {
        hipLaunchKernelGGL((rec_fwd_kernel<T, ALIGNED, false, HAS_Z, SAVE, kOutput>), dim3(grid), dim3(kThreads), 0,
                           a.stream, b, nct, ntiles, agg);
        return hipGetLastError();
    }
    return hipSuccess;
}

template <typename T, bool ALIGNED>
hipError_t launch_fwd_typed(const RecFwdArgs& a) {
    if (a.in[0].q != nullptr) return launch_fwd<T, ALIGNED, true, false, false>(a);
    if (a.save[0].q != nullptr)
        return a.z != nullptr ? launch_fwd<T, ALIGNED, false, true, true>(a) : launch_fwd<T, ALIGNED, false, false, true>(a);
    return a.z != nullptr ? launch_fwd<T, ALIGNED, false, true, false>(a) : launch_fwd<T, ALIGNED, false, false, false>(a);
}

// One token per row: a thread per four channels.
template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void rec_update_kernel(const RecUpdateArgs a) {
    const int dim = static_cast<int>(a.dim);
    const int64_t quads = (a.dim + 3) / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.batch * quads) return;
    const int64_t b = i / quads;
    const int c = static_cast<int>(i % quads) * 4;
    float ga[4], gx[4], x[4], z[4], h[4];
    unpack4(load4<T, ALIGNED>(static_cast<const char*>(a.gate_a) + b * a.ld_a * Elem<T>::kBytes, 0, c, dim), ga);
    unpack4(load4<T, ALIGNED>(static_cast<const char*>(a.gate_x) + b * a.ld_g * Elem<T>::kBytes, 0, c, dim), gx);
    unpack4(load4<T, ALIGNED>(static_cast<const char*>(a.x) + b * a.ld_x * Elem<T>::kBytes, 0, c, dim), x);
    if (a.z != nullptr)
        unpack4(load4<T, ALIGNED>(static_cast<const char*>(a.z) + b * a.ld_z * Elem<T>::kBytes, 0, c, dim), z);
    char* sb = reinterpret_cast<char*>(a.state + b * a.dim);
    unpack4(load4<float, ALIGNED>(sb, 0, c, dim), h);
    const bool clear = a.reset != nullptr && a.reset[b] != 0;
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float k2 = -a.c * kLog2e * softplus_exact(a.a_param[c + j < dim ? c + j : dim - 1]);
        float al, om;
        decay_terms(k2 * sigmoid_f(ga[j]), al, om);
        const float bb = __builtin_amdgcn_sqrtf(om) * (sigmoid_f(gx[j]) * x[j]);
        h[j] = clear ? bb : __builtin_fmaf(al, h[j], bb);
        o[j] = a.z != nullptr ? h[j] * silu_f(z[j]) : h[j];
    }
    store4<float, ALIGNED>(sb, 0, c, dim, h);
    store4<T, ALIGNED>(static_cast<char*>(a.out) + b * a.dim * Elem<T>::kBytes, 0, c, dim, o);
}

}  // namespace

size_t recurrence_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
    const int64_t ntiles = (seqlen + kRecChunk - 1) / kRecChunk;
    if (ntiles <= 1) return 0;
    return static_cast<size_t>(batch * ntiles * dim) * (have_states ? 8 : 12);
}

hipError_t launch_recurrence_fwd(const RecFwdArgs& a) {
    if (a.bf16) return a.aligned ? launch_fwd_typed<bf16_t, true>(a) : launch_fwd_typed<bf16_t, false>(a);
    return a.aligned ? launch_fwd_typed<float, true>(a) : launch_fwd_typed<float, false>(a);
}

hipError_t launch_recurrence_update(const RecUpdateArgs& a) {
    const int64_t threads = a.batch * ((a.dim + 3) / 4);
    const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
    if (a.bf16) {
        if (a.aligned) hipLaunchKernelGGL((rec_update_kernel<bf16_t, true>), grid, dim3(256), 0, a.stream, a);
        else hipLaunchKernelGGL((rec_update_kernel<bf16_t, false>), grid, dim3(256), 0, a.stream, a);
    } else {
        if (a.aligned) hipLaunchKernelGGL((rec_update_kernel<float, true>), grid, dim3(256), 0, a.stream, a);
        else hipLaunchKernelGGL((rec_update_kernel<float, false>), grid, dim3(256), 0, a.stream, a);
    }
    return hipGetLastError();
}

}  // namespace mamba
