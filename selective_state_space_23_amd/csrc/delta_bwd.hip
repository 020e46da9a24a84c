// Gated delta rule, backward: the gradient dS at every chunk's end state, the chunks of a
// row from last to first.
//
//     dU = P^T dO + exp(gamma_C - gamma) K dS,   P = scale D o Q K^T,   dX = (I + b M)^-T dU,
//     dS <- exp(gamma_C) dS + (scale exp(gamma) Q)^T dO - (exp(gamma) K)^T (beta dX).
//
// Columns do not mix here either: a wave owns 16, as in the forward (delta_fwd.hip), with dS
// in its accumulators.  Everything that sums over columns is left to delta_grads.hip,
// which works off the chunks at once from the states and gradients between them.
//
// What is not finite makes the whole of its document NaN (through the state a gradient
// reaches every token before, through the keys it came by every token after), and
// no other: its rows are taken out of every sum over tokens.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

template <typename T, int KT, int NW, bool VEC>
__global__ __launch_bounds__(NW * 64, 1) void bwd_states_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32, THREADS = NW * 64;
    constexpr bool DIRECT = VEC && N == 1;   // to LDS without registers, in two buffers
    using KQ = Tile<T, KT, THREADS, VEC>;
    constexpr int TKB = kBlocks * 3, RKB = 2, BKB = 2 * TKB + RKB;   // KB of the triangle, of P and of a record
    constexpr size_t BUF = BKB * 1024 + 2 * KQ::kBytes;
    __shared__ __align__(16) char smem[(DIRECT ? 2 : 1) * BUF];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bh = quotient(blockIdx.x, cols);
    const int col = remainder(blockIdx.x, cols);
    const int hv = remainder(bh, a.vheads), hk = quotient(hv, a.vheads / a.kheads);
    const int64_t b = quotient(bh, a.vheads);
    const int v = (col * NW + wave) * 16 + m;
    const bool v_in = v < a.vdim;
    const int n = a.nchunks;
    const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;

    // Offsets of lanes without a column, and of rows behind the last, lie behind the buffer.
    const uint32_t state_lane = v_in ? v * 4 : kPast;
    auto state_off = [&](int i, int r) { return state_lane + static_cast<uint32_t>(state_row(i, g, r) * a.vdim * 4); };
    const uint32_t value_lane = v_in ? v * ESZ : kPast;
    f32x4 S[2 * STEPS];   // dS
    {
        const Rsrc rs = rsrc(a.d_final_state + (a.d_final_state ? bh * cells : 0), a.d_final_state ? cells * 4 : 0);
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, state_off(i, r), 0, 0));
    }
    auto store_state = [&](float* to) {
        const Rsrc rs = rsrc(to, cells * 4);
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rs, state_off(i, r), 0, 0);
    };

    KQ kraw, qraw;   // not DIRECT: the next chunk in registers
    u32x4 braw[(BKB + NW - 1) / NW];
    uint32_t oraw[16];
    auto fetch = [&](int c, char* buf) {
        const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, left = a.seqlen - static_cast<int64_t>(c) * C;
        const int64_t id = bh * n + c;
        const int rows = static_cast<int>(left < C ? left : C);
        const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_k, a.kdim);
        const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_q, a.kdim);
        const Rsrc tr = rsrc(a.solve_t + id * kSolveBytes, kSolveBytes), pr = rsrc(a.pairs + id * kSolveBytes, kSolveBytes);
        const Rsrc rr = rsrc(a.chunks + id * rec_bytes, sizeof(ChunkRec));
        if constexpr (DIRECT) {
            uint16_t* Kl = reinterpret_cast<uint16_t*>(buf + BKB * 1024);
            rows_to_lds<KT, NW>(Kl, kr, a.ld_k, a.kdim, wave, lane);
            block_to_lds<RKB, NW>(buf + 2 * TKB * 1024, rr, wave, lane);
            block_to_lds<TKB, NW>(buf + TKB * 1024, pr, wave, lane);
            block_to_lds<TKB, NW>(buf, tr, wave, lane);
            rows_to_lds<KT, NW>(Kl + C * KT, qr, a.ld_q, a.kdim, wave, lane);
        } else {
            kraw.fetch(kr, a.ld_k, a.kdim, tid);
            qraw.fetch(qr, a.ld_q, a.kdim, tid);
#pragma unroll
            for (int p = 0; p < (BKB + NW - 1) / NW; ++p) {
                const int kb = p * NW + wave;
                const int at = ((kb < TKB ? kb : kb < 2 * TKB ? kb - TKB : kb - 2 * TKB) * 64 + lane) * 16;
                braw[p] = __builtin_amdgcn_raw_buffer_load_b128(kb < TKB ? tr : kb < 2 * TKB ? pr : rr, at, 0, 0);
            }
        }
        const Rsrc orr = rows_rsrc<ESZ>(a.dout, first * a.ld_o + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_o, a.vdim);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                oraw[4 * i + r] = load_one<T>(
                    orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(a.ld_o) * ESZ));
    };

    fetch(n - 1, smem + (DIRECT && ((n - 1) & 1) ? BUF : 0));
    for (int c = n - 1; c >= 0; --c) {
        char* buf = smem + (DIRECT && (c & 1) ? BUF : 0);
        const u32x4* Tl = reinterpret_cast<const u32x4*>(buf);   // [2][kBlocks][3][64]: the triangle, P
        const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buf + 2 * TKB * 1024);
        uint16_t* Kl = reinterpret_cast<uint16_t*>(buf + BKB * 1024);
        uint16_t* Ql = Kl + N * C * KT;
        if constexpr (!DIRECT) {
            kraw.land(Kl, tid);
            qraw.land(Ql, tid);
#pragma unroll
            for (int p = 0; p < (BKB + NW - 1) / NW; ++p)
                if (p * NW + wave < BKB) reinterpret_cast<u32x4*>(buf)[p * THREADS + tid] = braw[p];
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) dO[i][r] = one_value<T>(oraw[4 * i + r]);
        lds_barrier();
        if (c > 0) fetch(c - 1, smem + (DIRECT && !(c & 1) ? BUF : 0));

        const uint64_t starts = uniform(rec->starts), bad = uniform(rec->bad);
        const int first_start = starts ? __builtin_ctzll(starts) : C;
        const int last_start = starts ? 63 - __builtin_clzll(starts) : 0;
        store_state(a.dstates + (bh * n + c) * cells);

        // Rows whose gradient is not finite take no part, with the rest of their document
        uint64_t sick = 0;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) odd |= not_finite(dO[i][r]);
        if (bad != 0 || __ballot(odd) != 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sick |= uint64_t(not_finite(dO[i][r])) << (16 * i + 4 * g + r);
            sick |= __shfl_xor(sick, 16);
            sick |= __shfl_xor(sick, 32);
            sick = whole(sick | bad, starts);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) dO[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), dO[i][r]);
        }

        // K dS
        f32x4 ks[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            Frag<N> kf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) kf[i] = rows_frag<N, KT>(Kl, 16 * i + m, 4 * j + g);
            products<3, 4>(ks, kf, split(S[2 * j], S[2 * j + 1]));
        }

        // dU
        auto block = [&](int which, int i, int j) {
            Frag<3> f;
#pragma unroll
            for (int p = 0; p < 3; ++p) f.p[p] = Tl[((which * kBlocks + high_block(i, j)) * 3 + p) * 64 + lane];
            return f;
        };
        f32x4 U[4];
        {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 outof = four(rec->outof + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) U[i][r] = keep_if(16 * i + 4 * g + r >= last_start, outof[r] * ks[i][r]);
            }
            Frag<3> pf[4];
#pragma unroll
            for (int j = 1; j >= 0; --j) {
                const Frag<3> of = split(dO[2 * j], dO[2 * j + 1]);
                const int tiles = j ? 4 : 2;
#pragma unroll
                for (int i = 0; i < tiles; ++i) pf[i] = block(1, i, j);
                if constexpr (N == 1) {   // dO as stored is one piece
                    if (j) products<3, 4>(U, pf, Frag<1>{{of.p[0]}});
                    else products<3, 2>(U, pf, Frag<1>{{of.p[0]}});
                } else {
                    if (j) products<3, 4>(U, pf, of);
                    else products<3, 2>(U, pf, of);
                }
            }
        }
        odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) odd |= not_finite(U[i][r]);
        const bool any_sick = __ballot(odd || sick != 0) != 0;
        uint64_t drop = 0;   // rows out in all of the wave's columns: their keys and queries may be what is not finite
        if (any_sick) {
            uint64_t more = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) more |= uint64_t(not_finite(U[i][r])) << (16 * i + 4 * g + r);
            more |= __shfl_xor(more, 16);
            more |= __shfl_xor(more, 32);
            sick = whole(sick | more, starts);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    U[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), U[i][r]);
                    dO[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), dO[i][r]);
                }
            drop = sick;
#pragma unroll
            for (int s = 1; s < 16; s *= 2) drop &= __shfl_xor(drop, s);
            drop = uniform(drop);
        }

        // beta dX, then with what the entering state has kept; the same of dO
        f32x4 X[4];
        {
#pragma unroll
            for (int i = 0; i < 4; ++i) X[i] = f32x4{0, 0, 0, 0};
            Frag<3> tf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) tf[i] = block(0, i, 1);
            products<3, 4>(X, tf, split(U[2], U[3]));
#pragma unroll
            for (int i = 0; i < 2; ++i) tf[i] = block(0, i, 0);
            products<3, 2>(X, tf, split(U[0], U[1]));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 beta = four(rec->beta + 16 * i + 4 * g), into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool old = 16 * i + 4 * g + r < first_start;
                    X[i][r] = keep_if(old, -into[r] * (beta[r] * X[i][r]));
                    dO[i][r] = keep_if(old, a.scale * into[r] * dO[i][r]);
                }
            }
        }

        // dS
        const float keep = rec->keep;
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = keep_if(starts == 0, keep * S[i][r]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const Frag<3> xf = split(X[2 * j], X[2 * j + 1]), of = split(dO[2 * j], dO[2 * j + 1]);
#pragma unroll
            for (int i0 = 0; i0 < 2 * STEPS; i0 += 4) {
                Frag<N> kf[4], qf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kf[i] = cols_frag<N, KT>(Kl, j, g, m, state_cols4(i0 + i, m));
                    qf[i] = cols_frag<N, KT>(Ql, j, g, m, state_cols4(i0 + i, m));
                }
                if (any_sick) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        drop_rows<N>(kf[i], j, g, drop);
                        drop_rows<N>(qf[i], j, g, drop);
                    }
                }
                products<3, 4>(S + i0, qf, of);
                products<3, 4>(S + i0, kf, xf);
            }
        }
        if (any_sick) {
            const bool dead = (sick & 1) != 0 && first_start > 0;
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] = nan_if(dead, S[i][r]);
        }
        if constexpr (!DIRECT) lds_barrier();
    }
    if (a.d_initial_state) store_state(a.d_initial_state + bh * cells);
}

template <typename T, int KT, int NW, bool VEC>
hipError_t launch(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NW - 1) / (16 * NW);
    hipLaunchKernelGGL((bwd_states_kernel<T, KT, NW, VEC>), dim3(static_cast<unsigned>(a.batch * a.vheads * cols)),
                       dim3(NW * 64), 0, a.stream, a, static_cast<int64_t>(delta_chunk_bytes()), cols);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t by_width(const DeltaArgs& a) {
    return a.kdim > 64 ? launch<T, 128, 4, VEC>(a) : launch<T, 64, 4, VEC>(a);
}

}  // namespace

hipError_t launch_delta_bwd_states(const DeltaArgs& a) {
    if (a.bf16) return a.vec_k ? by_width<bf16_t, true>(a) : by_width<bf16_t, false>(a);
    return a.vec_k ? by_width<float, true>(a) : by_width<float, false>(a);
}

}  // namespace mamba
