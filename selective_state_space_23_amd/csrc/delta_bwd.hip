// Gated delta rule, backward: the gradient dS at every chunk's end state, the chunks of a
// row from last to first.
//
//     dU = P^T dO + exp(gamma_C - gamma) K dS,   P = scale D o Q K^T,   dX = (I + b M)^-T dU,
//     dS <- exp(gamma_C) dS + (scale exp(gamma) Q)^T dO - (exp(gamma) K)^T (beta dX).
//
// Columns do not mix here either: a wave owns 16, as in the forward (delta_fwd.hip), with dS
// in its accumulators.  Everything that sums over columns is left to delta_grads.hip,
// which works off the chunks at once from the states and gradients between them, and from dX as it is stored here.
//
// Bound by the chain as the forward is: 2 x 32768 tokens, 12 heads of 128 x 128, 512 chunks of 9000 cycles in 1.95 ms (3.27 ms
// with one wave for everything).
//
// What is not finite makes the whole of its document NaN (through the state a gradient
// reaches every token before, through the keys it came by every token after), and
// no other: its rows are taken out of every sum over tokens.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

// dX of 64 tokens and the 16 columns of group `group`, as the lanes hold it; NaN where the rows took no part.
__device__ __forceinline__ void store_dx(const DeltaArgs& a, int64_t id, int group, int lane, const f32x4* X, uint64_t sick) {
    const int groups = (a.vdim + 15) / 16, at = __builtin_amdgcn_readfirstlane(group);
    const Rsrc to = rsrc(a.dx + (id * groups + at) * kGroupFloats, at < groups ? kGroupFloats * 4 : 0);
    const uint64_t mine = sick >> (4 * (opaque(lane) >> 4));   // (row numbers would be kept in registers)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f32x4 x = X[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = nan_if((mine >> (16 * i + r)) & 1, x[r]);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), to, lane * 16 + i * 1024, 0, 0);
    }
}

template <typename T, int KT, int NW, bool VEC>
__global__ __launch_bounds__(NW * 64, 1) void bwd_states_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32, THREADS = NW * 64;
    using KQ = Tile<T, KT, THREADS, VEC>;
    constexpr int TKB = kBlocks * 3, RKB = 2, BKB = 2 * TKB + RKB;   // KB of the triangle, of P and of a record
    constexpr size_t BUF = BKB * 1024 + 2 * KQ::kBytes;
    __shared__ __align__(16) char buf[BUF];

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

    KQ kraw, qraw;   // the next chunk in registers
    u32x4 braw[(BKB + NW - 1) / NW];
    uint32_t oraw[16];
    auto fetch = [&](int c) {
        const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, left = a.seqlen - static_cast<int64_t>(c) * C;
        const int64_t id = bh * n + c;
        const int rows = static_cast<int>(left < C ? left : C);
        const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_k, a.kpitch);
        const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_q, a.kpitch);
        const Rsrc tr = rsrc(a.solve_t + id * kSolveBytes, kSolveBytes), pr = rsrc(a.pairs + id * kSolveBytes, kSolveBytes);
        const Rsrc rr = rsrc(a.chunks + id * rec_bytes, sizeof(ChunkRec));
        kraw.fetch(kr, a.ld_k, a.kpitch, tid);
        qraw.fetch(qr, a.ld_q, a.kpitch, tid);
#pragma unroll
        for (int p = 0; p < (BKB + NW - 1) / NW; ++p) {
            const int kb = p * NW + wave;
            const int at = ((kb < TKB ? kb : kb < 2 * TKB ? kb - TKB : kb - 2 * TKB) * 64 + lane) * 16;
            braw[p] = __builtin_amdgcn_raw_buffer_load_b128(kb < TKB ? tr : kb < 2 * TKB ? pr : rr, at, 0, 0);
        }
        const Rsrc orr = rows_rsrc<ESZ>(a.dout, first * a.ld_o + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_o, a.vdim);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                oraw[4 * i + r] = load_one<T>(
                    orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(a.ld_o) * ESZ));
    };

    fetch(n - 1);
    for (int c = n - 1; c >= 0; --c) {
        const u32x4* Tl = reinterpret_cast<const u32x4*>(buf);   // [2][kBlocks][3][64]: the triangle, P
        const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buf + 2 * TKB * 1024);
        uint16_t* Kl = reinterpret_cast<uint16_t*>(buf + BKB * 1024);
        uint16_t* Ql = Kl + N * C * KT;
        kraw.land(Kl, tid);
        qraw.land(Ql, tid);
#pragma unroll
        for (int p = 0; p < (BKB + NW - 1) / NW; ++p)
            if (p * NW + wave < BKB) reinterpret_cast<u32x4*>(buf)[p * THREADS + tid] = braw[p];
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) dO[i][r] = one_value<T>(oraw[4 * i + r]);
        lds_barrier();
        if (c > 0) fetch(c - 1);

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
            for (int i = 0; i < 4; ++i) U[i] = f32x4{0, 0, 0, 0};
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
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 outof = four(rec->outof + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    U[i][r] = starts == 0 ? __builtin_fmaf(outof[r], ks[i][r], U[i][r])
                                          : keep_if(16 * i + 4 * g + r >= last_start, outof[r] * ks[i][r]) + U[i][r];
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
            const Frag<3> uf[2] = {split(U[0], U[1]), split(U[2], U[3])};
#pragma unroll
            for (int j = 1; j >= 0; --j)   // a piece of the triangle at a time, the smallest first
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q)
#pragma unroll
                        for (int i = 0; i < 2 * j + 2; ++i) X[i] = mfma(Tl[(high_block(i, j) * 3 + p) * 64 + lane], uf[j].p[q], X[i]);
            store_dx(a, bh * n + c, v >> 4, lane, X, sick);
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
        const float keep = keep_if(starts == 0, rec->keep);
        const Frag<3> xf[2] = {split(X[0], X[1]), split(X[2], X[3])}, of[2] = {split(dO[0], dO[1]), split(dO[2], dO[3])};
#pragma unroll
        for (int i0 = 0; i0 < 2 * STEPS; i0 += 4) {
            f32x4 Z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) Z[i] = f32x4{0, 0, 0, 0};
            auto columns = [&](Frag<N>* f, const uint16_t* from, int j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = cols_frag<N, KT>(from, j, g, m, state_cols4(i0 + i, m));
                    if (any_sick) drop_rows<N>(f[i], j, g, drop);
                }
            };
            Frag<N> f[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                columns(f, Ql, j);
                products<3, 4>(Z, f, of[j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i0 + i][r] = __builtin_fmaf(keep_if(starts == 0, S[i0 + i][r]), keep, Z[i][r]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                columns(f, Kl, j);
                products<3, 4>(S + i0, f, xf[j]);
            }
        }
        if (any_sick) {
            const bool dead = (sick & 1) != 0 && first_start > 0;
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] = nan_if(dead, S[i][r]);
        }
        lds_barrier();
    }
    if (a.d_initial_state) store_state(a.d_initial_state + bh * cells);
}

// The same for bf16 in whole 16-byte pieces, two waves for every 16 columns as in the forward:
// one walks dS -> dU -> dX -> dS, the other brings what does not depend on dS, P^T dO and
// Z = (scale exp(gamma) Q)^T dO, and all loads.
//
// Chunk c:  barrier;  A: the chain forms K dS and dU;   the other forms Z of c, loads P and dO of c - 1;
//           barrier;  B: the chain forms dX, then dS;   the other forms P^T dO of c - 1, loads K, T and Q of it.
template <int KT, int NP>
constexpr int kPairsLds = 3 * C * KT * 2 + 3 * kBlocks * 3 * 1024 + 2 * 2048 + NP * (KT / 16 * 1024 + 4096 + 512);
// (LDS at the launch and two waves a SIMD: as in the forward, for sums in the lower registers)
template <int KT, int NP>
__global__ __launch_bounds__(NP * 128, 2) void bwd_pairs_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int STEPS = KT / 32;
    constexpr int TILE = C * KT * 2, TRI = kBlocks * 3 * 1024, REC = 2048;
    extern __shared__ __align__(16) char smem[];
    char* const Kb = smem;                       // [2] K
    char* const Rb = Kb + 2 * TILE;              // [2] record
    char* const Tb = Rb + 2 * REC;               // [2] triangle
    char* const Qb = Tb + 2 * TRI;                   // Q
    char* const Pb = Qb + TILE;                  // P
    char* const Zb = Pb + TRI;                   // Z
    char* const Ub = Zb + NP * 2 * STEPS * 1024; // P^T dO
    char* const Lb = Ub + NP * 4096;             // a lane's rows that take no part
    static_assert(kPairsLds<KT, NP> == 3 * TILE + 3 * TRI + 2 * REC + NP * ((2 * STEPS + 4) * 1024 + 512));

    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pair = wave & (NP - 1);
    const int64_t bh = quotient(blockIdx.x, 8 * cols) * 8 + (blockIdx.x & 7);   // a head's workgroups on one XCD
    if (bh >= a.batch * a.vheads) return;
    const int hv = remainder(bh, a.vheads), hk = quotient(hv, a.vheads / a.kheads);
    const int64_t b = quotient(bh, a.vheads);
    const int v = (remainder(blockIdx.x >> 3, cols) * NP + pair) * 16 + m;
    const bool v_in = v < a.vdim;
    const int n = a.nchunks;
    auto rows_of = [&](int c) {
        const int64_t left = a.seqlen - static_cast<int64_t>(c) * C;
        return static_cast<int>(left < C ? left : C);
    };
    auto buffer = [&](char* first, int size, int c) { return first + (c & 1) * size; };

    if (wave < NP) {
        // ---- the chain
        const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;
        const uint32_t state_lane = v_in ? static_cast<uint32_t>(v * 4 + state_row(0, g, 0) * a.vdim * 4) : kPast;
        auto state_off = [&](uint32_t from, int i, int r) {
            return from + static_cast<uint32_t>(state_row(i, 0, r) * a.vdim * 4);
        };
        auto store_state = [&](float* to, const f32x4* S) {
            const Rsrc rs = rsrc(to, cells * 4);
            const uint32_t from = opaque(state_lane);
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rs, state_off(from, i, r), 0, 0);
        };
        f32x4 S[2 * STEPS];   // dS
        {
            const Rsrc rs = rsrc(a.d_final_state + (a.d_final_state ? bh * cells : 0), a.d_final_state ? cells * 4 : 0);
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, state_off(state_lane, i, r), 0, 0));
        }
        // dS in pieces as its rows are final, between the products that do not wait for them
        Frag<3> sf[STEPS];
#pragma unroll
        for (int j = 0; j < STEPS / 2; ++j) sf[j] = split(S[2 * j], S[2 * j + 1]);
        lds_barrier();   // the other waves' first loads
        for (int c = n - 1; c >= 0; --c) {
            const uint16_t* Kl = reinterpret_cast<const uint16_t*>(buffer(Kb, TILE, c));
            const u32x4* Tl = reinterpret_cast<const u32x4*>(buffer(Tb, TRI, c));
            const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buffer(Rb, REC, c));
            lds_barrier();
            // A: dU = exp(gamma_C - gamma) K dS + P^T dO
            const uint64_t starts_ = rec->starts, bad_ = rec->bad;
            const float keep = rec->keep;
            f32x4 U[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                if (j >= STEPS / 2) sf[j] = split(S[2 * j], S[2 * j + 1]);
                Frag<1> kf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kf[i] = rows_frag<1, KT>(Kl, 16 * i + m, 4 * j + g);
                products<3, 4>(U, kf, sf[j]);
            }
            const uint64_t starts = uniform(starts_), bad = uniform(bad_);
            store_state(a.dstates + (bh * n + c) * cells, S);
            uint64_t sick = *reinterpret_cast<const uint64_t*>(Lb + (pair * 64 + lane) * 8);
            float check[2] = {0.0f, 0.0f};   // stay 0 as long as everything is finite
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 outof = four(rec->outof + 16 * i + 4 * g);
                const f32x4 part = *reinterpret_cast<const f32x4*>(Ub + ((pair * 4 + i) * 64 + lane) * 16);
                if (starts == 0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) U[i][r] = __builtin_fmaf(outof[r], U[i][r], part[r]);
                } else {
                    const int last_start = 63 - __builtin_clzll(starts);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        U[i][r] = keep_if(16 * i + 4 * g + r >= last_start, outof[r] * U[i][r]) + part[r];
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) check[i & 1] = __builtin_fmaf(U[i][r], 0.0f, check[i & 1]);
            }
            const bool any_sick = __ballot(not_finite(check[0] + check[1]) || sick != 0) != 0;
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
                    for (int r = 0; r < 4; ++r) U[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), U[i][r]);
            }
            lds_barrier();
            // B: dX, then dS.  PLAIN: one document, everything finite
            auto rest = [&](auto plain) {
                constexpr bool PLAIN = decltype(plain)::value;
                auto triangle = [&](int i, int j, int p) { return Tl[(high_block(i, j) * 3 + p) * 64 + lane]; };
                auto keys = [&](Frag<1>* kf, int i0, int j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        kf[i] = cols_frag<1, KT>(Kl, j, g, m, state_cols4(i0 + i, m));
                        if (!PLAIN) drop_rows<1>(kf[i], j, g, bad);
                    }
                };
                f32x4 X[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) X[i] = f32x4{0, 0, 0, 0};
                const Frag<3> uf1 = split(U[2], U[3]);
#pragma unroll
                for (int p = 2; p >= 0; --p) {
                    u32x4 tf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tf[i] = triangle(i, 1, p);
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) X[i] = mfma(tf[i], uf1.p[q], X[i]);
                }
                const Frag<3> uf0 = split(U[0], U[1]);
#pragma unroll
                for (int p = 2; p >= 0; --p) {
                    const u32x4 t0 = triangle(0, 0, p), t1 = triangle(1, 0, p);
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q) {
                        X[0] = mfma(t0, uf0.p[q], X[0]);
                        X[1] = mfma(t1, uf0.p[q], X[1]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                store_dx(a, bh * n + c, v >> 4, lane, X, PLAIN ? 0 : sick);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 2 * STEPS; ++i) {
                    const f32x4 z = *reinterpret_cast<const f32x4*>(Zb + ((pair * 2 * STEPS + i) * 64 + lane) * 16);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        S[i][r] = __builtin_fmaf(PLAIN ? S[i][r] : keep_if(starts == 0, S[i][r]),
                                                 PLAIN ? keep : keep_if(starts == 0, keep), z[r]);
                }
                Frag<1> kf[2][4];
                keys(kf[0], 0, 0);
                keys(kf[1], 0, 1);
                const int first_start = !PLAIN && starts != 0 ? __builtin_ctzll(starts) : C;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 beta = four(rec->beta + 16 * i + 4 * g), into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = -into[r] * (beta[r] * X[i][r]);
                        X[i][r] = PLAIN ? x : keep_if(16 * i + 4 * g + r < first_start, x);
                    }
                }
                Frag<3> xf[2];
                xf[0] = split(X[0], X[1]);
                // Products and splits that do not wait for each other, three products and a split at a time.
                auto step = [&](f32x4* acc, const Frag<1>* keyf, const Frag<3>& u, int from) {
#pragma unroll
                    for (int q = from; q < from + 3; ++q) acc[q % 4] = mfma(keyf[q % 4].p[0], u.p[2 - q / 4], acc[q % 4]);
                };
                auto cut = [&](Frag<3>& f, const f32x4& x, const f32x4& y, int k) {   // the k-th pair of eight values
                    const f32x4& z = k < 2 ? x : y;
                    uint32_t h, md, l;
                    split_pair(z[2 * (k & 1)], z[2 * (k & 1) + 1], h, md, l);
                    f.p[0][k] = h;
                    f.p[1][k] = md;
                    f.p[2][k] = l;
                };
                Frag<1> kg[2][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    __builtin_amdgcn_sched_barrier(0);
                    step(S, kf[0], xf[0], 3 * k);
                    cut(xf[1], X[2], X[3], k);
                }
                if constexpr (STEPS == 4) {
                    keys(kg[0], 4, 0);
                    keys(kg[1], 4, 1);
                }
                __builtin_amdgcn_sched_barrier(0);
                products<3, 4>(S, kf[1], xf[1]);
                const bool dead = !PLAIN && (sick & 1) != 0 && first_start > 0;
                auto end = [&](int i0) {
                    if constexpr (!PLAIN) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r) S[i0 + i][r] = nan_if(dead, S[i0 + i][r]);
                    }
                };
                end(0);
                if constexpr (STEPS == 4) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        __builtin_amdgcn_sched_barrier(0);
                        step(S + 4, kg[k / 4], xf[k / 4], 3 * (k % 4));
                        cut(sf[k / 4], S[k / 4 * 2], S[k / 4 * 2 + 1], k % 4);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    end(4);
                } else {
                    sf[0] = split(S[0], S[1]);
                }
            };
            if (any_sick || starts != 0 || bad != 0) rest(std::false_type{});
            else rest(std::true_type{});
        }
        if (a.d_initial_state) store_state(a.d_initial_state + bh * cells, S);
    } else {
        // ---- loads, P^T dO and Z
        const uint32_t value_lane = v_in ? v * 2 : kPast;
        uint32_t oraw[16];
        f32x4 dO[4];
        uint64_t sick = 0;
        bool any_sick = false;
        auto fetch_early = [&](int c) {
            const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, id = bh * n + c;
            const int rows = rows_of(c);
            const Rsrc kr = rows_rsrc<2>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_k, a.kpitch);
            rows_to_lds<KT, NP>(reinterpret_cast<uint16_t*>(buffer(Kb, TILE, c)), kr, a.ld_k, a.kpitch, pair, lane);
            const Rsrc qr = rows_rsrc<2>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_q, a.kpitch);
            rows_to_lds<KT, NP>(reinterpret_cast<uint16_t*>(Qb), qr, a.ld_q, a.kpitch, pair, lane);
            block_to_lds<kBlocks * 3, NP>(buffer(Tb, TRI, c), rsrc(a.solve_t + id * kSolveBytes, kSolveBytes), pair, lane);
        };
        auto fetch_rest = [&](int c) {   // from phase B of the chunk before on
            const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, id = bh * n + c;
            block_to_lds<2, NP>(buffer(Rb, REC, c), rsrc(a.chunks + id * rec_bytes, sizeof(ChunkRec)), pair, lane);
            block_to_lds<kBlocks * 3, NP>(Pb, rsrc(a.pairs + id * kSolveBytes, kSolveBytes), pair, lane);
            const Rsrc orr = rows_rsrc<2>(a.dout, first * a.ld_o + static_cast<int64_t>(hv) * a.vdim, rows_of(c), a.ld_o, a.vdim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    oraw[4 * i + r] = load_one<bf16_t>(
                        orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(a.ld_o) * 2));
        };
        // P^T dO of chunk c, from P and its record in LDS and dO in registers
        auto weighted = [&](int c) {
            const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buffer(Rb, REC, c));
            const uint64_t starts = uniform(rec->starts), bad = uniform(rec->bad);
            const u32x4* Pl = reinterpret_cast<const u32x4*>(Pb);
            float check = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dO[i][r] = one_value<bf16_t>(oraw[4 * i + r]);
                    check = __builtin_fmaf(dO[i][r], 0.0f, check);
                }
            sick = 0;
            any_sick = bad != 0 || __ballot(not_finite(check)) != 0;
            if (any_sick) {   // rows whose gradient is not finite take no part, with the rest of their document
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
            f32x4 U[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 1; j >= 0; --j) {
                u32x4 of;   // dO as stored is one piece
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x4& x = dO[2 * j + k / 2];
                    of[k] = __builtin_amdgcn_perm(__float_as_uint(x[2 * (k & 1) + 1]), __float_as_uint(x[2 * (k & 1)]), 0x07060302u);
                }
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int i = 0; i < (j ? 4 : 2); ++i) U[i] = mfma(Pl[(high_block(i, j) * 3 + p) * 64 + lane], of, U[i]);
            }
            float more_check = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) more_check = __builtin_fmaf(U[i][r], 0.0f, more_check);
            any_sick = any_sick || __ballot(not_finite(more_check)) != 0;
            if (any_sick) {   // queries that are not finite
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
                        dO[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), dO[i][r]);
                        U[i][r] = keep_if(!((sick >> (16 * i + 4 * g + r)) & 1), U[i][r]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(Ub + ((pair * 4 + i) * 64 + lane) * 16) = U[i];
            *reinterpret_cast<uint64_t*>(Lb + (pair * 64 + lane) * 8) = sick;
        };
        auto entering = [&](int c) {   // Z of chunk c
            const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buffer(Rb, REC, c));
            const uint64_t starts = uniform(rec->starts);
            const int first_start = starts ? __builtin_ctzll(starts) : C;
            const uint16_t* Ql = reinterpret_cast<const uint16_t*>(Qb);
            uint64_t drop = 0;   // rows out in all of the wave's columns: their queries may be what is not finite
            if (any_sick) {
                drop = sick;
#pragma unroll
                for (int s = 1; s < 16; s *= 2) drop &= __shfl_xor(drop, s);
                drop = uniform(drop);
            }
            Frag<3> of[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x4 x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const f32x4 into = four(rec->into + 32 * j + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x[i][r] = keep_if(32 * j + 16 * i + 4 * g + r < first_start, a.scale * into[r] * dO[2 * j + i][r]);
                }
                of[j] = split(x[0], x[1]);
            }
#pragma unroll
            for (int i0 = 0; i0 < 2 * STEPS; i0 += 4) {
                f32x4 Z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) Z[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    Frag<1> qf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[i] = cols_frag<1, KT>(Ql, j, g, m, state_cols4(i0 + i, m));
                    if (any_sick) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) drop_rows<1>(qf[i], j, g, drop);
                    }
                    products<3, 4>(Z, qf, of[j]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(Zb + ((pair * 2 * STEPS + i0 + i) * 64 + lane) * 16) = Z[i];
            }
        };
        auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
        // the waves of this role share what they load: a barrier of all makes it whole
        fetch_rest(n - 1);
        fetch_early(n - 1);
        landed();
        lds_barrier();
        weighted(n - 1);
        for (int c = n - 1; c >= 0; --c) {
            lds_barrier();
            // A
            if (c > 0) fetch_rest(c - 1);
            entering(c);
            landed();
            lds_barrier();
            // B
            if (c > 0) {
                fetch_early(c - 1);
                weighted(c - 1);
                landed();
            }
        }
    }
}

template <typename T, int KT, int NW, bool VEC>
hipError_t launch(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NW - 1) / (16 * NW);
    hipLaunchKernelGGL((bwd_states_kernel<T, KT, NW, VEC>), dim3(static_cast<unsigned>(a.batch * a.vheads * cols)),
                       dim3(NW * 64), 0, a.stream, a, static_cast<int64_t>(delta_chunk_bytes()), cols);
    return hipGetLastError();
}

template <int KT, int NP>
hipError_t launch_pairs(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NP - 1) / (16 * NP);
    hipLaunchKernelGGL((bwd_pairs_kernel<KT, NP>), dim3(static_cast<unsigned>((a.batch * a.vheads + 7) / 8 * 8 * cols)),
                       dim3(NP * 128), (kPairsLds<KT, NP>), a.stream, a, static_cast<int64_t>(delta_chunk_bytes()), cols);
    return hipGetLastError();
}
template <int KT>
hipError_t pairs_by_columns(const DeltaArgs& a) {
    return wide_groups(a) ? launch_pairs<KT, 4>(a) : launch_pairs<KT, 2>(a);
}

template <typename T, bool VEC>
hipError_t by_width(const DeltaArgs& a) {
    return a.kdim > 64 ? launch<T, 128, 4, VEC>(a) : launch<T, 64, 4, VEC>(a);
}

}  // namespace

hipError_t launch_delta_bwd_states(const DeltaArgs& a) {
    if (a.bf16 && a.vec_k) return a.kdim > 64 ? pairs_by_columns<128>(a) : pairs_by_columns<64>(a);
    if (a.bf16) return by_width<bf16_t, false>(a);
    return a.vec_k ? by_width<float, true>(a) : by_width<float, false>(a);
}

}  // namespace mamba
