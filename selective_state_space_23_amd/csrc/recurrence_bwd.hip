// Backward of the gated linear recurrence (recurrence.hip), gfx950: the gradients
// of sum(dout out) + sum(d_final_state final_state).
//
// With dy = dout silu(z), v = i x and the adjoint
//     G_t = dy_t + e_{t+1},   e_t = a_t G_t  (0 at a document start),
// e after the last token being d_final_state:
//     dx = G w i,   dgate_x = G w v (1 - i),   dz = dout h silu'(z),
//     r dlog a = G a (r h_{t-1} - a r v / w),
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

// Inputs of 16 bits are staged in LDS and 4 waves share a SIMD; unaligned ones are read
// into registers, and so is float32 (too large to stage): twice the tokens in twice the
// registers of half as many waves.
template <typename T, bool ALIGNED> struct Shape {
    static constexpr bool kStaged = sizeof(T) == 2 && ALIGNED;
    static constexpr int kK = sizeof(T) == 2 ? 4 : 8;                 // tokens a lane walks
    static constexpr int kWaves = kTileTokens / (2 * kK);             // two halves of 32 lanes a wave
    static constexpr int kThreads = kWaves * 64;
};

// A gate's sigmoid r and the rest 1 - r in one register, each to its own size: the
// difference from the rounded r is 1% off at a gate of 12 and gone from 17 on.  With
// e = exp(-gate) the rest is e r; kept is r, or minus the rest where that is the smaller
// (never 0: its sign tells which), and both are s - floor(s) of it and of its negative.
// An r of 0 leaves a rest of 0 in place of 1; every term it multiplies is 0 then.
struct SplitGate {
    __device__ __forceinline__ static float pack(float gate, float e, float r) {
        const float rest = __builtin_fmaxf(e * r, 0x1p-126f);
        return gate > 0.0f ? -rest : r;
    }
    __device__ __forceinline__ static float r(float s) { return __builtin_amdgcn_fractf(s); }
    __device__ __forceinline__ static float rest(float s) { return __builtin_amdgcn_fractf(-s); }
};

struct RecBwdKernelArgs {
    RecBwdArgs a;
    Chain ch;
    float* part;       // (B * tiles, D): sum of r dlog a over a tile
    int nct, ntiles;
    int tile0;         // rows of one tile: the launch's first
};

// One pass over the data, from the row ends back.  A workgroup works off tiles as
// the forward does; what the gradients need of a token is formed before the adjoint
// entering the tile is known, as far as registers hold it: five values of a token and
// channel are kept, x, dout and z are read again from LDS and the gates' terms formed
// while the workgroup waits for that adjoint.
//
// What bounds it is the vector unit (136 issue slots an element from 8-bit inputs and
// 120 from tensors, 79% and 69% of the time; 6 of them keep 1 - r and 1 - i to their own size, which costs
// 1% and 4%), then memory: 2 rows of 32768 x 1536 from checkpoints with z take 463 us and move 1.47 GB
// (3.2 TB/s), 8 rows of 2048 x 1536 from tensors 116 us and 460 MB (4.0 TB/s; 5.2 for a copy).  One workgroup of 16 waves fills a CU's
// registers and, with two places for x, dout and z, its LDS.  A register too many costs
// more than the work it saves: with the gates' terms kept as well, their spills
// reloaded behind the loads of the next tile, the first case took 770 us.
template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, int LOOK>
__global__ __launch_bounds__((Shape<T, ALIGNED>::kThreads)) void rec_bwd_kernel(const RecBwdKernelArgs) {
    constexpr bool kStaged = Shape<T, ALIGNED>::kStaged;
    constexpr int kK = Shape<T, ALIGNED>::kK, kWaves = Shape<T, ALIGNED>::kWaves;
    __shared__ float s_rate[kTileChannels];
    // the last row of an array takes what no one reads
    __shared__ float2 s_map[kWaves + 1][kTileChannels], s_rev[kWaves + 1][kTileChannels];   // (P, H) and (P, X)
    __shared__ float s_in[kWaves][kTileChannels], s_adj[kTileChannels], s_sum[kWaves + 1][kTileChannels];
    __shared__ int s_ticket, s_second;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    using Place = LanePlace<kK>;
    const auto first = kernel_args<RecBwdKernelArgs>();
    const int dim = static_cast<int>(first->a.dim), nct = first->nct, ntiles = first->ntiles;
    Walk<PIN> walk;
    walk.init(nct, ntiles, static_cast<int>(first->a.batch));
    auto draw = [&]() { return walk.draw(kernel_args<RecBwdKernelArgs>()->ch.next); };
    auto place = [&](int ticket) { return walk.template place<true>(ticket, kernel_args<RecBwdKernelArgs>()->a.seqlen); };

    // The next tile's inputs: staged in LDS (each wave its own part) while a tile is
    // worked off; float32 (too large) and unaligned ones are loaded at its start.
    using In = LaneIn<T, ALIGNED, PIN, kK>;
    using Plain = LaneIn<T, ALIGNED, false, kK>;
    // x, dout and z are read twice, at both ends of a tile, and so have two places each.
    constexpr int kTwice = (HAS_Z ? 2 : 1) * In::kStageBytes + Plain::kStageBytes;
    constexpr int kStage = 2 * In::kStageBytes + 2 * kTwice;
    __shared__ __attribute__((aligned(16))) char s_stage[kStaged ? kWaves * kStage : 16];
    char* const stage = s_stage + (kStaged ? wave * kStage : 0);
    int twice = 2 * In::kStageBytes;   // of the tile fetched last
    In xi, ai, gi, zi;
    Plain oi;
    StartFlags fl;
    float rate[kV];
    auto fetch = [&](const Tile& t) {
        const Place l(wave);
        const int c = l.channel(t);
        const auto p = kernel_args<RecBwdKernelArgs>();
        const auto& a = p->a;
        const int64_t rows = a.batch * a.seqlen;
        if constexpr (kStaged) {
            ai.stage(stage, a.gate_a, a.in[1], t, a.ld_a, wave, dim, rows);
            gi.stage(stage + In::kStageBytes, a.gate_x, a.in[2], t, a.ld_g, wave, dim, rows);
            twice = 4 * In::kStageBytes + kTwice - twice;
            xi.stage(stage + twice, a.x, a.in[0], t, a.ld_x, wave, dim, rows);
            oi.stage(stage + twice + In::kStageBytes, a.dout, a.in[0], t, a.ld_o, wave, dim, rows);
            if constexpr (HAS_Z)
                zi.stage(stage + twice + In::kStageBytes + Plain::kStageBytes, a.z, a.in[3], t, a.ld_z, wave, dim, rows);
        } else {
            ai.load(a.gate_a, a.in[1], t, a.ld_a, l.tok, c, dim, rows);
            gi.load(a.gate_x, a.in[2], t, a.ld_g, l.tok, c, dim, rows);
            xi.load(a.x, a.in[0], t, a.ld_x, l.tok, c, dim, rows);
            oi.load(a.dout, a.in[0], t, a.ld_o, l.tok, c, dim, rows);
            if constexpr (HAS_Z) zi.load(a.z, a.in[3], t, a.ld_z, l.tok, c, dim, rows);
        }
        fl.load(a.doc_start, t.row_tok, t.nv);
        if (ntiles > 1) {
            const float2 r = *reinterpret_cast<const float2*>(p->ch.rate + c);   // padded to whole channel tiles
            rate[0] = r.x; rate[1] = r.y;
        }
    };

    int cur, next;
    if (ntiles > 1) {
        if (wave == 0) {   // both tickets are under way together
            const int t0 = draw();
            int t1 = kNone;
            if (!walk.once) t1 = draw();
            s_ticket = __builtin_amdgcn_readfirstlane(t0);
            s_second = __builtin_amdgcn_readfirstlane(t1);
        }
        lds_barrier();
        cur = __builtin_amdgcn_readfirstlane(s_ticket);
        next = __builtin_amdgcn_readfirstlane(s_second);
        if (cur >= walk.tickets) return;
        if constexpr (kStaged) fetch(place(cur));
    } else {
        cur = first->tile0 + static_cast<int>(blockIdx.x);
        next = kNone;
        const Tile t = place(cur);
        fetch(t);
        if (threadIdx.x < kTileChannels) {
            const int d = t.ct * kTileChannels + threadIdx.x;
            s_rate[threadIdx.x] = -first->a.c * kLog2e * softplus_exact(first->a.a_param[d < dim ? d : dim - 1]);
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < kV; ++j) rate[j] = s_rate[kV * Place(wave).li + j];
    }

    // A tile's part of sum r dlog a: its waves' sums added by one wave behind the
    // next barrier.
    int64_t part_row = -1;
    int part_channel = 0;
    auto add_part = [&]() {
        if (part_row < 0) return;
        const int lane = static_cast<int>(lane_now());
        float s = 0.0f;
#pragma unroll 4
        for (int w = 0; w < kWaves; ++w) s += s_sum[w][lane];
        row_store(kernel_args<RecBwdKernelArgs>()->part, part_row, dim, part_channel + lane, s);
    };

    if constexpr (kStaged) wait_all_but<0>();
    for (;;) {
        const Tile t = place(cur);
        if constexpr (!kStaged) {
            if (ntiles > 1) fetch(t);
        }
        const TileStarts starts = fl.starts();
        const bool general = starts.any() || t.nv < kTileTokens;   // the same in the whole workgroup
        const uint32_t st = starts.bits(Place(wave).tok, kK);
        const int left = t.nv - Place(wave).tok;   // of the lane's tokens, those in the row
        In xc = xi, ac = ai, gc = gi, zc = zi;
        Plain oc = oi;
        float rc[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) rc[j] = rate[j];
        const int here = twice;
        auto read_twice = [&]() {
            const Place l(wave);
            xc.read(stage + here, l.half, l.li);
            oc.read(stage + here + In::kStageBytes, l.half, l.li);
            if constexpr (HAS_Z) zc.read(stage + here + In::kStageBytes + Plain::kStageBytes, l.half, l.li);
        };
        if constexpr (kStaged) {
            const Place l(wave);
            ac.read(stage, l.half, l.li);
            gc.read(stage + In::kStageBytes, l.half, l.li);
            read_twice();
            wait_lds_reads();
        }
        if constexpr (kStaged) fetch(place(next));   // past the last ticket: a tile of no tokens, nothing is read
        // Of every token: a, r or r - 1 (SplitGate), w i, 1 - i and r v / w.
        float A[kK][kV], R[kK][kV], W[kK][kV], O[kK][kV], V[kK][kV];
        float P[kV], H[kV], X[kV];
        auto maps = [&](auto gen) {
            constexpr bool GEN = decltype(gen)::value;
            static_for<kK>([&](auto kcc) {
                constexpr int k = decltype(kcc)::value;
                float ga[kV], gx[kV], x[kV], y[kV], z[kV];
                ac.template take<k>(ga);
                gc.template take<k>(gx);
                xc.template take<k>(x);
                oc.template take<k>(y);
                if constexpr (HAS_Z) zc.template take<k>(z);
                const bool start = GEN && ((st >> k) & 1u), out = GEN && k >= left;
                // A start among the lane's tokens so far: told by its bits and not by the sign
                // of P, which a NaN decay may set or clear.
                const bool cut = GEN && (st & ((2u << k) - 1u)) != 0;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float ea = exp2_fast(-ga[j] * kLog2e), r = rcp_fast(1.0f + ea);
                    float al, om;
                    decay_terms(rc[j] * r, al, om);
                    float rw = __builtin_amdgcn_rsqf(om);
                    asm volatile("" : "+v"(rw));
                    rw = om >= 0x1p-126f ? rw : 0.0f;   // denormals count as 0
                    const float eg = exp2_fast(-gx[j] * kLog2e), ig = rcp_fast(1.0f + eg);
                    rw *= ig;
                    if constexpr (HAS_Z) y[j] *= silu_f(z[j]);
                    R[k][j] = SplitGate::pack(ga[j], ea, r);
                    W[k][j] = om * rw;
                    O[k][j] = __builtin_fminf(eg, 0x1p126f) * ig;   // 1 - ig; past the bound W is 0 or denormal
                    asm volatile("" : "+v"(R[k][j]), "+v"(O[k][j]));   // here, not where they are used
                    V[k][j] = (r * rw) * x[j];
                    float bb = W[k][j] * x[j];
                    if constexpr (GEN) {
                        al = out ? 1.0f : al;
                        bb = out ? 0.0f : bb;
                        y[j] = out ? 0.0f : y[j];
                    }
                    A[k][j] = al;
                    if constexpr (k == 0) {
                        P[j] = cut ? -0.0f : __builtin_fabsf(al);
                        H[j] = bb;
                        X[j] = cut ? 0.0f : al * y[j];
                    } else {
                        float p = __builtin_fabsf(P[j] * al), h = __builtin_fmaf(al, H[j], bb);
                        float x1 = __builtin_fmaf(p, y[j], X[j]);
                        if constexpr (GEN) asm volatile("" : "+v"(p), "+v"(h), "+v"(x1));   // selects, not a branch
                        P[j] = cut ? -0.0f : p;
                        H[j] = start ? bb : h;
                        X[j] = cut ? X[j] : x1;
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        // (Not staged: one form for both, or the compiler moves what they share, and its
        // registers, ahead of the choice.)
        if (general || !kStaged) maps(std::true_type{});
        else maps(std::false_type{});

        // what the wave's other half does before (forward) or after (adjoint), and the wave's maps
        float op[kV], oh[kV];
        {
            const Place l(wave);
            const int row = l.half ? wave : kWaves, rev = l.half ? kWaves : wave;
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float p1 = __shfl_xor(P[j], 32), h1 = __shfl_xor(H[j], 32), x1 = __shfl_xor(X[j], 32);
                const float pw = is_reset(P[j]) ? P[j] : P[j] * p1;
                s_map[row][kV * l.li + j] = make_float2(pw, apply(P[j], H[j], h1));
                s_rev[rev][kV * l.li + j] = make_float2(pw, apply(P[j], X[j], x1));
                op[j] = p1;   // the first half's map, for the second; the second half's adjoint map, for the first
                oh[j] = l.half ? h1 : x1;
            }
        }
        typename ChainWords<LOOK>::Seen seen = {};
        auto words = [&]() {
            const auto p = kernel_args<RecBwdKernelArgs>();
            return walk.template words<LOOK>(Chain{p->ch.map, p->ch.value, p->ch.next, p->ch.rate}, t);
        };
        int ticket = 0;   // wave 0's: the tile after the next one
        if (wave == 0 && ntiles > 1) {
            seen = words().peek(t.pos);
            if (next < walk.tickets) ticket = draw();
        }
        lds_barrier();
        if (wave == 0) {   // a lane per channel: the adjoint entering the tile from the right, and its waves
            const int lane = static_cast<int>(lane_now()), d = t.ct * kTileChannels + lane;
            const auto p = kernel_args<RecBwdKernelArgs>();
            const auto& a = p->a;
            const ChainWords<LOOK> chain = words();
            float e = row_load(a.d_final_state, t.b, a.dim, d);
            float2 m = s_rev[kWaves - 1][lane];
            s_rev[kWaves - 1][lane] = make_float2(1.0f, 0.0f);   // from here on of all behind a wave
            constexpr int kRows = kWaves == 16 ? 5 : 7;   // read ahead of the chain of compositions
            static_assert((kWaves - 1) % kRows == 0);
#pragma unroll 1
            for (int w = kWaves - 2; w >= 0; w -= kRows) {
                float2 v[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) v[i] = s_rev[w - i][lane];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    s_rev[w - i][lane] = m;
                    compose(v[i].x, v[i].y, m.x, m.y);
                    m = v[i];
                }
            }
            if (t.pos + 1 < ntiles) chain.publish_map(t.pos, m.x, m.y);
            e = chain.look_back(t.pos, e, seen);
            const float leaving = apply(m.x, m.y, e);
            if (t.pos + 1 < ntiles) chain.publish_value(t.pos, leaving);
            if (t.tile == 0) row_store(a.d_initial_state, t.b, a.dim, d, leaving);
            s_adj[lane] = e;
            s_ticket = __builtin_amdgcn_readfirstlane(ticket);
        } else if (wave == 1) {   // the states entering the waves
            const int lane = static_cast<int>(lane_now()), d = t.ct * kTileChannels + lane;
            const auto p = kernel_args<RecBwdKernelArgs>();
            const auto& a = p->a;
            float h = a.states != nullptr ? row_load(a.states, t.b * ntiles + t.tile, a.dim, d)
                                          : row_load(a.initial_state, t.b, a.dim, d);
#pragma unroll 1
            for (int w = 0; w < kWaves; w += 4) {
                float2 m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = s_map[w + i][lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s_in[w + i][lane] = h;
                    h = apply(m[i].x, m[i].y, h);
                }
            }
        } else if (wave == 2) {
            add_part();
            part_row = t.b * ntiles + t.tile;
            part_channel = t.ct * kTileChannels;
        }
        // Meanwhile of every token dy and dout silu'(z).
        float Y[kK][kV], Z[kK][kV];
        if constexpr (HAS_Z) {
            if constexpr (kStaged) read_twice();
            static_for<kK>([&](auto kcc) {
                constexpr int k = decltype(kcc)::value;
                float y[kV], z[kV];
                oc.template take<k>(y);
                zc.template take<k>(z);
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    // (float32: formed anew, the ones of the maps take registers that spill)
                    if constexpr (sizeof(T) == 4) asm volatile("" : "+v"(z[j]));
                    const float sg = sigmoid_f(z[j]);
                    Z[k][j] = y[j] * (sg * __builtin_fmaf(z[j], 1.0f - sg, 1.0f));
                    Y[k][j] = y[j] * (z[j] * sg);
                    asm volatile("" : "+v"(Y[k][j]), "+v"(Z[k][j]));   // here, not behind the barrier
                }
                __builtin_amdgcn_sched_barrier(0);
            });
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
            const Place l(wave);
            const int li = l.li, half = l.half, c = l.channel(t);
            uint32_t off = store_offset(l.tok + kK - 1, step, c * esz, c < dim);
            auto put = [&](auto gen) {
                constexpr bool GEN = decltype(gen)::value;
                float h[kK + 1][kV], e[kV], sum[kV];   // the states before and behind the tokens
                if constexpr (kStaged) read_twice();
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float in = s_in[wave][kV * li + j];
                    const float mid = apply<GEN>(op[j], oh[j], in);
                    h[0][j] = half ? mid : in;
                }
                static_for<kK>([&](auto kcc) {
                    constexpr int k = decltype(kcc)::value;
                    float x[kV];
                    xc.template take<k>(x);
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        const float b = W[k][j] * x[j];
                        h[k + 1][j] = GEN && ((st >> k) & 1u) ? b : __builtin_fmaf(A[k][j], h[k][j], b);
                    }
                });
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float2 suf = s_rev[wave][kV * li + j];
                    const float in = apply(suf.x, suf.y, s_adj[kV * li + j]);
                    const float mid = apply<GEN>(op[j], oh[j], in);
                    e[j] = half ? in : mid;
                    sum[j] = 0.0f;
                }
                static_for<kK>([&](auto kcc) {
                    constexpr int k = kK - 1 - decltype(kcc)::value;
                    float dx[kV], da[kV], dg[kV], dz[kV], x[kV], y[kV];
                    xc.template take<k>(x);
                    if constexpr (!HAS_Z) oc.template take<k>(y);
                    const bool start = GEN && ((st >> k) & 1u), out = GEN && k >= left;
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        const float before = start ? 0.0f : h[k][j];
                        if constexpr (HAS_Z) {
                            dz[j] = Z[k][j] * h[k + 1][j];
                            y[j] = Y[k][j];
                        }
                        if constexpr (GEN) y[j] = out ? 0.0f : y[j];
                        const float G = y[j] + e[j];
                        dx[j] = G * W[k][j];
                        dg[j] = dx[j] * x[j] * O[k][j];
                        float s = R[k][j];
                        asm volatile("" : "+v"(s));   // taken apart here, not in both parts where it is formed
                        const float q = G * (A[k][j] * __builtin_fmaf(-A[k][j], V[k][j], SplitGate::r(s) * before));
                        da[j] = (kLn2 * rc[j]) * SplitGate::rest(s) * q;   // kLn2 rate = -c softplus(a_param)
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
            if (general || !kStaged) put(std::true_type{});
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
    if (d < dim) {
#pragma unroll 8
        for (int64_t i = g; i < nparts; i += 16) s += part[i * dim + d];
    }
    red[g][o] = s;
    __syncthreads();
    if (g != 0 || d >= dim) return;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += red[k][o];
    da_param[d] = -c * t * sigmoid_f(a_param[d]);
}

constexpr int kResident = 256;   // one workgroup a CU
// A launch holds fewer than 2^32 threads: of rows of one tile, which take a workgroup
// each, a call with more tiles is launched in pieces.
constexpr int64_t kMaxGrid = int64_t(1) << 21;

struct BwdWs {
    size_t part, chain, chain_bytes, states, total;
};

BwdWs bwd_ws(int64_t batch, int64_t seqlen, int64_t dim, bool have_states) {
    const size_t n = static_cast<size_t>(batch * ((seqlen + kRecChunk - 1) / kRecChunk) * dim);
    BwdWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 255) / 256 * 256; return o; };
    w.part = take(n * 4);
    w.chain = off;   // and the recomputation's behind it
    w.chain_bytes = (recurrence_workspace_bytes(batch, seqlen, dim) + 255) / 256 * 256;
    take((have_states ? 1 : 2) * w.chain_bytes);
    w.states = take(have_states ? 0 : n * 4);
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
    RecBwdKernelArgs k{a, Chain{}, reinterpret_cast<float*>(ws + w.part), nct, ntiles, 0};
    const bool recompute = a.states == nullptr && ntiles > 1;
    Chain chains[2];
    hipError_t e = clear_chains(ws + w.chain, recompute ? 2 : 1, w.chain_bytes, a.batch, a.dim, ntiles, a.a_param, a.c,
                                chains, a.stream);
    if (e != hipSuccess) return e;
    k.ch = chains[0];
    if (recompute) {
        RecFwdArgs f{};
        f.x = a.x; f.gate_a = a.gate_a; f.gate_x = a.gate_x;
        for (int i = 0; i < 3; ++i) f.in[i] = a.in[i];
        f.a_param = a.a_param; f.doc_start = a.doc_start; f.initial_state = a.initial_state;
        f.states = reinterpret_cast<float*>(ws + w.states);
        f.chain = &chains[1];
        f.batch = a.batch; f.seqlen = a.seqlen; f.dim = a.dim;
        f.ld_x = a.ld_x; f.ld_a = a.ld_a; f.ld_g = a.ld_g;
        f.c = a.c; f.bf16 = a.bf16; f.aligned = a.aligned; f.stream = a.stream;
        if ((e = launch_recurrence_fwd(f)) != hipSuccess) return e;
        k.a.states = f.states;
    }
    const int64_t grid = ntiles > 1 && tiles > kResident ? kResident : tiles;
    // (Looking far costs the other variants registers they do not have: float32 with z,
    // 4 rows of 64 channels 125 us for 103.)
    auto kernel = rec_bwd_kernel<T, ALIGNED, PIN, HAS_Z, kLookNear>;
    if constexpr (Shape<T, ALIGNED>::kStaged) {
        if (look_far(nct * a.batch, ntiles, 8)) kernel = rec_bwd_kernel<T, ALIGNED, PIN, HAS_Z, kLookFar>;
    }
    static_assert(kMaxGrid * Shape<T, ALIGNED>::kThreads < (int64_t(1) << 32) && kMaxGrid >= kResident);
    for (int64_t first = 0; first < grid; first += kMaxGrid) {
        k.tile0 = static_cast<int>(first);
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid - first < kMaxGrid ? grid - first : kMaxGrid)),
                           dim3(Shape<T, ALIGNED>::kThreads), 0, a.stream, k);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
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
