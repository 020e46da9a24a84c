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

constexpr int kK = 4;                              // tokens a lane walks
constexpr int kWaves = kTileTokens / (2 * kK);     // two halves of 32 lanes a wave
constexpr int kThreads = kWaves * 64;

struct RecBwdKernelArgs {
    RecBwdArgs a;
    Chain ch;
    float* part;       // (B * tiles, D): sum of r dlog a over a tile
    int nct, ntiles;
};

// One pass over the data, from the row ends back.  A workgroup works off tiles as
// the forward does; everything the gradients need of a token is formed once, before
// the adjoint entering the tile is known, and kept in registers.
template <typename T, bool ALIGNED, bool PIN, bool HAS_Z>
__global__ __launch_bounds__(kThreads) void rec_bwd_kernel(const RecBwdKernelArgs) {
    __shared__ float s_rate[kTileChannels];
    // the last row of an array takes what no one reads
    __shared__ float s_P[kWaves + 1][kTileChannels], s_H[kWaves + 1][kTileChannels], s_X[kWaves + 1][kTileChannels];
    __shared__ float s_in[kWaves][kTileChannels], s_adj[kTileChannels], s_sum[kWaves + 1][kTileChannels];
    __shared__ float2 s_suf[kWaves][kTileChannels];    // the adjoint maps of all behind a wave
    __shared__ int s_ticket;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane % kRow, half = lane / kRow;
    const auto first = kernel_args<RecBwdKernelArgs>();
    const int dim = static_cast<int>(first->a.dim), nct = first->nct, ntiles = first->ntiles;
    const int tok = (wave * 2 + half) * kK;
    Walk walk;
    walk.init(nct, ntiles, static_cast<int>(first->a.batch));
    auto draw = [&]() { return walk.draw(kernel_args<RecBwdKernelArgs>()->ch.next); };
    auto place = [&](int ticket) { return walk.place<true>(ticket, kernel_args<RecBwdKernelArgs>()->a.seqlen); };

    // The next tile's inputs: staged in LDS (each wave its own part) while a tile is
    // worked off; float32 (too large) and unaligned ones are loaded at its start.
    constexpr bool kStaged = sizeof(T) == 2 && ALIGNED;
    using In = LaneIn<T, ALIGNED, PIN, kK>;
    using Plain = LaneIn<T, ALIGNED, false, kK>;
    constexpr int kStage = (HAS_Z ? 4 : 3) * In::kStageBytes + Plain::kStageBytes;
    __shared__ __attribute__((aligned(16))) char s_stage[kStaged ? kWaves * kStage : 16];
    char* const stage = s_stage + (kStaged ? wave * kStage : 0);
    In xi, ai, gi, zi;
    Plain oi;
    StartFlags fl;
    float rate[kV];
    auto fetch = [&](const Tile& t) {
        const int c = t.ct * kTileChannels + kV * li;
        const auto p = kernel_args<RecBwdKernelArgs>();
        const auto& a = p->a;
        const int64_t rows = a.batch * a.seqlen;
        if constexpr (kStaged) {
            ai.stage(stage, a.gate_a, a.in[1], t, a.ld_a, wave, dim, rows);
            gi.stage(stage + In::kStageBytes, a.gate_x, a.in[2], t, a.ld_g, wave, dim, rows);
            xi.stage(stage + 2 * In::kStageBytes, a.x, a.in[0], t, a.ld_x, wave, dim, rows);
            oi.stage(stage + 3 * In::kStageBytes, a.dout, a.in[0], t, a.ld_o, wave, dim, rows);
            if constexpr (HAS_Z)
                zi.stage(stage + 3 * In::kStageBytes + Plain::kStageBytes, a.z, a.in[3], t, a.ld_z, wave, dim, rows);
            if constexpr (PIN) {
                ai.load_scale(a.in[1], t, tok, rows);
                gi.load_scale(a.in[2], t, tok, rows);
                xi.load_scale(a.in[0], t, tok, rows);
                if constexpr (HAS_Z) zi.load_scale(a.in[3], t, tok, rows);
            }
        } else {
            ai.load(a.gate_a, a.in[1], t, a.ld_a, tok, c, dim, rows);
            gi.load(a.gate_x, a.in[2], t, a.ld_g, tok, c, dim, rows);
            xi.load(a.x, a.in[0], t, a.ld_x, tok, c, dim, rows);
            oi.load(a.dout, a.in[0], t, a.ld_o, tok, c, dim, rows);
            if constexpr (HAS_Z) zi.load(a.z, a.in[3], t, a.ld_z, tok, c, dim, rows);
        }
        fl.load(a.doc_start, t.row_tok, t.nv);
        if (ntiles > 1) {
            const float2 r = *reinterpret_cast<const float2*>(p->ch.rate + c);   // padded to whole channel tiles
            rate[0] = r.x; rate[1] = r.y;
        }
    };

    int cur, next;
    if (ntiles > 1) {
        if (wave == 0) s_ticket = draw();
        lds_barrier();
        cur = __builtin_amdgcn_readfirstlane(s_ticket);
        lds_barrier();
        if (wave == 0) s_ticket = draw();
        if (cur >= walk.tickets) return;
        if constexpr (kStaged) fetch(place(cur));
        lds_barrier();
        next = __builtin_amdgcn_readfirstlane(s_ticket);
        lds_barrier();
    } else {
        cur = static_cast<int>(blockIdx.x);
        next = 0x7fffffff;
        const Tile t = place(cur);
        fetch(t);
        if (threadIdx.x < kTileChannels) {
            const int d = t.ct * kTileChannels + threadIdx.x;
            s_rate[threadIdx.x] = -first->a.c * kLog2e * softplus_exact(first->a.a_param[d < dim ? d : dim - 1]);
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < kV; ++j) rate[j] = s_rate[kV * li + j];
    }

    // A tile's part of sum r dlog a: its waves' sums added by one wave behind the
    // next barrier.
    int64_t part_row = -1;
    int part_channel = 0;
    auto add_part = [&]() {
        if (part_row < 0) return;
        float s = 0.0f;
#pragma unroll 4
        for (int w = 0; w < kWaves; ++w) s += s_sum[w][lane];
        row_store(kernel_args<RecBwdKernelArgs>()->part, part_row, dim, part_channel + lane, s);
    };

    if constexpr (kStaged) wait_all_but<0>();
    for (;;) {
        const Tile t = place(cur);
        const int c = t.ct * kTileChannels + kV * li;
        if constexpr (!kStaged) {
            if (ntiles > 1) fetch(t);
        }
        const TileStarts starts = fl.starts();
        const bool general = starts.any() || t.nv < kTileTokens;   // the same in the whole workgroup
        const uint32_t st = starts.bits(tok, kK);
        In xc = xi, ac = ai, gc = gi, zc = zi;
        Plain oc = oi;
        float rc[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) rc[j] = rate[j];
        if constexpr (kStaged) {
            ac.read(stage, half, li);
            gc.read(stage + In::kStageBytes, half, li);
            xc.read(stage + 2 * In::kStageBytes, half, li);
            oc.read(stage + 3 * In::kStageBytes, half, li);
            if constexpr (HAS_Z) zc.read(stage + 3 * In::kStageBytes + Plain::kStageBytes, half, li);
            wait_lds_reads();
            fetch(place(next));   // past the last ticket: a tile of no tokens, nothing is read
        }
        // Of every token: a, r, w v, w i, 1 - i, (r / w) a^2 v, dy and dout silu'(z).
        float A[kK][kV], R[kK][kV], B[kK][kV], W[kK][kV], O[kK][kV], U[kK][kV], Y[kK][kV], Z[kK][kV];
        float P[kV], H[kV], X[kV];
        auto maps = [&](auto gen) {
            constexpr bool GEN = decltype(gen)::value;
            static_for<kK>([&](auto kcc) {
                constexpr int k = decltype(kcc)::value;
                float ga[kV], gx[kV], x[kV], z[kV];
                ac.template take<k>(ga);
                gc.template take<k>(gx);
                xc.template take<k>(x);
                oc.template take<k>(Y[k]);
                if constexpr (HAS_Z) zc.template take<k>(z);
                const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= t.nv;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float r = sigmoid_f(ga[j]);
                    float al, om;
                    decay_terms(rc[j] * r, al, om);
                    float rw = __builtin_amdgcn_rsqf(om);
                    asm volatile("" : "+v"(rw));
                    rw = om >= 0x1p-126f ? rw : 0.0f;   // denormals count as 0
                    const float w = om * rw;
                    const float ig = sigmoid_f(gx[j]);
                    const float v = ig * x[j];
                    if constexpr (HAS_Z) {
                        const float sg = sigmoid_f(z[j]);
                        Z[k][j] = Y[k][j] * (sg * __builtin_fmaf(z[j], 1.0f - sg, 1.0f));
                        Y[k][j] *= z[j] * sg;
                    }
                    R[k][j] = r;
                    W[k][j] = w * ig;
                    O[k][j] = 1.0f - ig;
                    U[k][j] = (r * rw) * (al * al) * v;
                    float bb = w * v;
                    if constexpr (GEN) {
                        al = out ? 1.0f : al;
                        bb = out ? 0.0f : bb;
                        Y[k][j] = out ? 0.0f : Y[k][j];
                    }
                    A[k][j] = al;
                    B[k][j] = bb;
                    if constexpr (k == 0) {
                        P[j] = start ? -0.0f : al;
                        H[j] = bb;
                        X[j] = start ? 0.0f : al * Y[k][j];
                    } else {
                        P[j] = start ? -0.0f : P[j] * al;
                        H[j] = start ? bb : __builtin_fmaf(al, H[j], bb);
                        X[j] = apply<GEN>(P[j], X[j], Y[k][j]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        if (general) maps(std::true_type{});
        else maps(std::false_type{});

        // what the wave's other half does before (forward) or after (adjoint), and the wave's maps
        float fp[kV], fh[kV], rp[kV], rx[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float p1 = __shfl_xor(P[j], 32), h1 = __shfl_xor(H[j], 32), x1 = __shfl_xor(X[j], 32);
            const int row = half ? wave : kWaves, rev = half ? kWaves : wave;
            s_P[row][kV * li + j] = is_reset(P[j]) ? P[j] : P[j] * p1;
            s_H[row][kV * li + j] = apply(P[j], H[j], h1);
            s_X[rev][kV * li + j] = apply(P[j], X[j], x1);
            fp[j] = half ? p1 : 1.0f;   // the first half's map, for the second
            fh[j] = half ? h1 : 0.0f;
            rp[j] = half ? 1.0f : p1;   // the second half's adjoint map, for the first
            rx[j] = half ? 0.0f : x1;
        }
        lds_barrier();
        if (wave == 0) {   // a lane per channel: the adjoint entering the tile from the right, and its waves
            const int d = t.ct * kTileChannels + lane;
            const auto p = kernel_args<RecBwdKernelArgs>();
            const auto& a = p->a;
            const ChainWords words = walk.words(Chain{p->ch.map, p->ch.value, p->ch.next, p->ch.rate}, t);
            float e = row_load(a.d_final_state, t.b, a.dim, d);
            float mp = s_P[kWaves - 1][lane], mx = s_X[kWaves - 1][lane];
            s_suf[kWaves - 1][lane] = make_float2(1.0f, 0.0f);
#pragma unroll 3
            for (int w = kWaves - 2; w >= 0; --w) {
                s_suf[w][lane] = make_float2(mp, mx);
                const float q = s_P[w][lane];
                mx = apply(q, s_X[w][lane], mx);
                mp = is_reset(q) ? q : q * mp;
            }
            if (t.pos + 1 < ntiles) words.publish_map(t.pos, mp, mx);
            e = words.look_back(t.pos, e);
            const float leaving = apply(mp, mx, e);
            if (t.pos + 1 < ntiles) words.publish_value(t.pos, leaving);
            if (t.tile == 0) row_store(a.d_initial_state, t.b, a.dim, d, leaving);
            s_adj[lane] = e;
            if (next < walk.tickets) s_ticket = draw();
        } else if (wave == 1) {   // the states entering the waves
            const int d = t.ct * kTileChannels + lane;
            const auto p = kernel_args<RecBwdKernelArgs>();
            const auto& a = p->a;
            float h = a.states != nullptr ? row_load(a.states, t.b * ntiles + t.tile, a.dim, d)
                                          : row_load(a.initial_state, t.b, a.dim, d);
#pragma unroll 2
            for (int w = 0; w < kWaves; ++w) {
                s_in[w][lane] = h;
                h = apply(s_P[w][lane], s_H[w][lane], h);
            }
        } else if (wave == 2) {
            add_part();
            part_row = t.b * ntiles + t.tile;
            part_channel = t.ct * kTileChannels;
        }
        lds_barrier();
        {
            constexpr int esz = Elem<T>::kBytes;
            const auto p = kernel_args<RecBwdKernelArgs>();
            const Rsrc to_x = rows_rsrc<esz>(p->a.dx, t.row_tok, t.nv, dim, dim);
            const Rsrc to_a = rows_rsrc<esz>(p->a.dgate_a, t.row_tok, t.nv, dim, dim);
            const Rsrc to_g = rows_rsrc<esz>(p->a.dgate_x, t.row_tok, t.nv, dim, dim);
            const Rsrc to_z = rows_rsrc<esz>(p->a.dz, t.row_tok, HAS_Z ? t.nv : 0, dim, dim);
            const uint32_t step = static_cast<uint32_t>(dim) * esz;
            uint32_t off = store_offset(tok + kK - 1, step, c * esz, c < dim);
            auto put = [&](auto gen) {
                constexpr bool GEN = decltype(gen)::value;
                float hp[kK][kV], e[kV], sum[kV];
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    float h = apply<GEN>(fp[j], fh[j], s_in[wave][kV * li + j]);
#pragma unroll
                    for (int k = 0; k < kK; ++k) {
                        hp[k][j] = h;
                        h = GEN && ((st >> k) & 1u) ? B[k][j] : __builtin_fmaf(A[k][j], h, B[k][j]);
                    }
                    const float2 suf = s_suf[wave][kV * li + j];
                    e[j] = apply<GEN>(rp[j], rx[j], apply(suf.x, suf.y, s_adj[kV * li + j]));
                    sum[j] = 0.0f;
                }
                static_for<kK>([&](auto kcc) {
                    constexpr int k = kK - 1 - decltype(kcc)::value;
                    float dx[kV], da[kV], dg[kV], dz[kV];
                    const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= t.nv;
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        const float G = Y[k][j] + e[j];
                        const float ah = start ? 0.0f : A[k][j] * hp[k][j];
                        dx[j] = G * W[k][j];
                        dg[j] = G * B[k][j] * O[k][j];
                        const float q = G * __builtin_fmaf(R[k][j], ah, -U[k][j]);
                        da[j] = (kLn2 * rc[j]) * (1.0f - R[k][j]) * q;   // kLn2 rate = -c softplus(a_param)
                        if constexpr (HAS_Z) dz[j] = Z[k][j] * (ah + B[k][j]);
                        sum[j] += out ? 0.0f : q;
                        e[j] = start ? 0.0f : A[k][j] * G;
                    }
                    store_vals<T, kV, ALIGNED>(to_x, off, dim - c, dx);
                    store_vals<T, kV, ALIGNED>(to_a, off, dim - c, da);
                    store_vals<T, kV, ALIGNED>(to_g, off, dim - c, dg);
                    if constexpr (HAS_Z) store_vals<T, kV, ALIGNED>(to_z, off, dim - c, dz);
                    off = next_offset(off, 0u - step);
                });
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    sum[j] += __shfl_xor(sum[j], 32);
                    s_sum[half ? kWaves : wave][kV * li + j] = sum[j];
                }
            };
            if (general) put(std::true_type{});
            else put(std::false_type{});
        }
        if (next >= walk.tickets) break;
        // Behind the staged loads this wave has issued the tile's stores at least.
        if constexpr (kStaged) wait_all_but<(HAS_Z ? 4 : 3) * kK>();
        cur = next;
        next = __builtin_amdgcn_readfirstlane(s_ticket);   // written before the last barrier
    }
    lds_barrier();
    if (wave == 2) add_part();
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

constexpr int kResident = 256;   // one workgroup of 16 waves a CU

struct BwdWs {
    size_t part, chain, states, fwd, total;
};

BwdWs bwd_ws(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
    const size_t n = static_cast<size_t>(batch * ((seqlen + kRecChunk - 1) / kRecChunk) * dim);
    BwdWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) / 256 * 256; return o; };
    w.part = take(n * 4);
    w.chain = take(recurrence_workspace_bytes(batch, seqlen, dim));
    w.states = take(have_states ? 0 : n * 4);
    w.fwd = take(have_states ? 0 : recurrence_workspace_bytes(batch, seqlen, dim));
    w.total = off;
    return w;
}

template <typename T, bool ALIGNED, bool PIN, bool HAS_Z>
hipError_t launch_bwd(const RecBwdArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const int ntiles = static_cast<int>((a.seqlen + kTileTokens - 1) / kTileTokens);
    const int64_t tiles = nct * a.batch * ntiles;
    const BwdWs w = bwd_ws(a.batch, a.seqlen, a.dim, a.states != nullptr);
    char* ws = static_cast<char*>(a.ws);
    RecBwdKernelArgs k{a, Chain{}, reinterpret_cast<float*>(ws + w.part), nct, ntiles};
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
        k.a.states = f.states;
    }
    if ((e = clear_chains(ws + w.chain, a.batch, a.dim, ntiles, a.a_param, a.c, &k.ch, a.stream)) != hipSuccess) return e;
    const int64_t grid = ntiles > 1 && tiles > kResident ? kResident : tiles;
    hipLaunchKernelGGL((rec_bwd_kernel<T, ALIGNED, PIN, HAS_Z>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                       a.stream, k);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(rec_bwd_reduce_kernel, dim3(static_cast<unsigned>((a.dim + 63) / 64)), dim3(1024), 0, a.stream,
                       k.part, a.a_param, a.da_param, a.batch * ntiles, static_cast<int>(a.dim), a.c);
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
