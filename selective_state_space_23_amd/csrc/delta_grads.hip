// Gated delta rule, backward: every gradient of a chunk of 64 tokens, from the state S that
// enters it and the gradient dS at the state that leaves it (delta_bwd.hip), all chunks at
// once.  A workgroup takes one key head of a chunk and its value heads in turn, so that
// dq and dk sum over them in a fixed order.
//
//     R = V - exp(gamma) K S,  E = (I + M b)^-1 R,  U = b E,  O = scale exp(gamma) Q S + P U,
//     dU = P^T dO + exp(gamma_C - gamma) K dS,   dX = (I + b M)^-T dU,   dV = beta dX,
//     dbeta = dX . E,   dgamma = dO . O - dV . V   (row by row),
//     dq = scale exp(gamma) dO S^T + dP K,                       dP = scale D o dO U^T (s <= t),
//     dk = exp(gamma_C - gamma) U dS^T - exp(gamma) dV S^T + dP^T Q + N K,   N = G + G^T, G = -b D o dX U^T (s < t).
//
// dgamma's form follows from every decay multiplying the key and value sums alike: scaling a
// row's decay scales o . dO and v . dV by what it scales the row's query and value side, so the 64 x 64
// matrices' row and column sums cancel to these two dot products.  At the chunk's end
// <dS, S_out> = exp(gamma_C) <dS, S> + sum_t U . (exp(gamma_C - gamma) K dS) is added, and dg is the
// sum of dgamma from its token to its document's (or the chunk's) end.
//
// Phases: (1) a wave owns 16 value columns, with K, Q and the triangles in LDS; (2) the tiles of
// dP and N, contracted over the columns, with U and dX in LDS over K and Q; (3) a wave owns 16 key
// channels: the products with S and dS; (4) those with K and Q, back in LDS.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kRowV = 136, kRowP = 72;   // bf16 of a row of U and dX, of dP and N

// Sum over the 16 lanes of a DPP row, in each of them.
__device__ __forceinline__ float row_sum(float x) {
    auto moved = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                     decltype(ctrl)::value, 0xf, 0xf, false));
    };
    using I = int;
    x += moved(x, std::integral_constant<I, 0xB1>{});    // quad_perm [1, 0, 3, 2]
    x += moved(x, std::integral_constant<I, 0x4E>{});    // quad_perm [2, 3, 0, 1]
    x += moved(x, std::integral_constant<I, 0x141>{});   // row_half_mirror
    x += moved(x, std::integral_constant<I, 0x140>{});   // row_mirror
    return x;
}

// One value in N pieces, to element `at` of N planes of `plane` elements.
template <int N>
__device__ __forceinline__ void put(uint16_t* to, int plane, int at, float x) {
    if constexpr (N == 2) {
        const uint32_t h = f32_to_bf16(x);
        to[at] = static_cast<uint16_t>(h);
        to[plane + at] = f32_to_bf16(x - __uint_as_float(h << 16));
    } else {
        const uint32_t u = __float_as_uint(x);
        const float r = x - __uint_as_float(u & 0xffff0000u);
        const uint32_t w = __float_as_uint(r);
        to[at] = static_cast<uint16_t>(u >> 16);
        to[plane + at] = static_cast<uint16_t>(w >> 16);
        to[2 * plane + at] = static_cast<uint16_t>(__float_as_uint(r - __uint_as_float(w & 0xffff0000u)) >> 16);
    }
}

// Row `row` of planes [N][C][kRowP], the tokens of step j in the order of cols_frag.
template <int N>
__device__ __forceinline__ Frag<N> token_frag(const uint16_t* lds, int row, int j, int g) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint16_t* at = lds + (i * C + row) * kRowP + 32 * j + 4 * g;
        const u32x2 x = *reinterpret_cast<const u32x2*>(at), y = *reinterpret_cast<const u32x2*>(at + 16);
        f.p[i] = u32x4{x[0], x[1], y[0], y[1]};
    }
    return f;
}

// The same of column m, by transposing reads.
template <int N>
__device__ __forceinline__ Frag<N> token_cols(const uint16_t* lds, int j, int g, int m, int ch4) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        f.p[i] = transposed(lds + (i * C + 32 * j + 4 * g + m / 4) * kRowP + ch4, 16 * kRowP);
    return f;
}
// Row `row` of planes [N][C][kRowV], eight columns from `ch` on.
template <int N>
__device__ __forceinline__ Frag<N> plane_frag(const uint16_t* lds, int row, int ch) {
    Frag<N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *reinterpret_cast<const u32x4*>(lds + (i * C + row) * kRowV + ch);
    return f;
}

template <int N>
__device__ __forceinline__ void clear_if(Frag<N>& f, bool out) {
    const uint32_t on = out ? 0u : ~0u;
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] &= on;
}

constexpr size_t larger(size_t a, size_t b) { return a > b ? a : b; }

template <typename T, int KT, bool VEC>
__global__ __launch_bounds__(kThreads, 1) void grads_kernel(DeltaArgs a, int64_t rec_bytes) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32;
    constexpr int OUT = N == 1 ? 2 : 3;
    using KQ = Tile<T, KT, kThreads, VEC>;
    constexpr int PLANE_V = C * kRowV, PLANE_P = C * kRowP;
    constexpr size_t PARTS = 2 * kWaves * C * 4;
    constexpr size_t ZERO = larger(2 * KQ::kBytes, size_t(2) * OUT * PLANE_V * 2);
    constexpr size_t ONE = larger(2 * kSolveBytes + PARTS, size_t(2) * OUT * PLANE_P * 2);
    __shared__ __align__(16) char region0[ZERO];
    __shared__ __align__(16) char region1[ONE];
    __shared__ __align__(16) ChunkRec rec_;
    __shared__ float ends[kWaves];
    __shared__ uint64_t odd_rows[kWaves];
    uint16_t* Kl = reinterpret_cast<uint16_t*>(region0);
    uint16_t* Ql = Kl + N * C * KT;
    uint16_t* Ul = reinterpret_cast<uint16_t*>(region0);          // [OUT][C][kRowV]
    uint16_t* Xl = Ul + OUT * PLANE_V;
    const u32x4* Tl = reinterpret_cast<const u32x4*>(region1);
    float* parts = reinterpret_cast<float*>(region1 + 2 * kSolveBytes);   // [2][kWaves][C]
    uint16_t* Pl = reinterpret_cast<uint16_t*>(region1);          // [OUT][C][kRowP]
    uint16_t* Nl = Pl + OUT * PLANE_P;
    const ChunkRec* rec = &rec_;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int bh = quotient(blockIdx.x, a.nchunks);   // row and key head
    const int c = remainder(blockIdx.x, a.nchunks);
    const int hk = remainder(bh, a.kheads), group = quotient(a.vheads, a.kheads);
    const int64_t b = quotient(bh, a.kheads);
    const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, left = a.seqlen - static_cast<int64_t>(c) * C;
    const int rows = static_cast<int>(left < C ? left : C);
    const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;
    const int vsteps = (a.vdim + 31) / 32, vwaves = 2 * vsteps;
    const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_k, a.kdim);
    const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_q, a.kdim);

    f32x4 dq[4], dk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[i] = dk[i] = f32x4{0, 0, 0, 0};
    uint64_t sick_any = 0;

    for (int h = 0; h < group; ++h) {
        const int hv = hk * group + h;
        const int64_t id = (b * a.vheads + hv) * a.nchunks + c;
        const Rsrc vr = rows_rsrc<ESZ>(a.v, first * a.ld_v + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_v, a.vdim);
        const Rsrc orr = rows_rsrc<ESZ>(a.dout, first * a.ld_o + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_o, a.vdim);
        const Rsrc sr = rsrc(a.states + id * cells, cells * 4);
        const Rsrc dr = rsrc(a.dstates + id * cells, cells * 4);

        f32x4 U[4], X[4];
        uint64_t sick = 0, starts = 0;
        int first_start = C, last_start = 0;
        for (int pass = 0; pass < 2; ++pass) {
            const int tid = thread_now(), lane = tid & 63, g = lane >> 4, m = lane & 15;
            // (1) once more without the documents in which something is not finite, if there are any
            __syncthreads();
            {
                KQ kraw, qraw;
                kraw.fetch(kr, a.ld_k, a.kdim, tid);
                qraw.fetch(qr, a.ld_q, a.kdim, tid);
                u32x4* Tw = reinterpret_cast<u32x4*>(region1);
                const Rsrc t0 = rsrc(a.solve + id * kSolveBytes, kSolveBytes), t1 = rsrc(a.solve_t + id * kSolveBytes, kSolveBytes);
                for (int p = wave; p < 2 * kBlocks * 3; p += kWaves)
                    Tw[p * 64 + lane] = p < kBlocks * 3
                        ? __builtin_amdgcn_raw_buffer_load_b128(t0, (p * 64 + lane) * 16, 0, 0)
                        : __builtin_amdgcn_raw_buffer_load_b128(t1, ((p - kBlocks * 3) * 64 + lane) * 16, 0, 0);
                const uint32_t* from = reinterpret_cast<const uint32_t*>(a.chunks + id * rec_bytes);
                constexpr int RECW = sizeof(ChunkRec) / 4;
                static_assert(RECW <= kThreads, "one word a thread");
                reinterpret_cast<uint32_t*>(&rec_)[tid < RECW ? tid : RECW - 1] = from[tid < RECW ? tid : RECW - 1];
                odd_rows[wave] = 0;
                kraw.land_without(Kl, tid, sick);
                qraw.land_without(Ql, tid, sick);
            }
            __syncthreads();
            starts = uniform(rec->starts);
            first_start = starts ? __builtin_ctzll(starts) : C;
            last_start = starts ? 63 - __builtin_clzll(starts) : 0;
            const bool no_state = (sick & 1) != 0 && first_start > 0, no_dstate = (sick >> 63) != 0;
            if (wave < vwaves) {
                const int v = 16 * wave + m;
                const uint32_t value_lane = v < a.vdim ? v * ESZ : kPast;
                const uint32_t state_lane = v < a.vdim && !no_state ? v * 4 : kPast;
                const uint32_t dstate_lane = v < a.vdim && !no_dstate ? v * 4 : kPast;
                f32x4 V[4], dO[4];
                uint64_t odd = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        const uint32_t at = (sick >> t) & 1 ? kPast : value_lane;
                        V[i][r] = one_value<T>(load_one<T>(vr, at + static_cast<uint32_t>(t * static_cast<int>(a.ld_v) * ESZ)));
                        dO[i][r] = one_value<T>(load_one<T>(orr, at + static_cast<uint32_t>(t * static_cast<int>(a.ld_o) * ESZ)));
                        odd |= uint64_t(not_finite(dO[i][r])) << t;
                    }
                f32x4 ks[4], qs[4], kd[4];
                float inner = 0.0f;   // <dS, S> of this column, this group's channels
#pragma unroll
                for (int i = 0; i < 4; ++i) ks[i] = qs[i] = kd[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    f32x4 s0, s1, d0, d1;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t row = static_cast<uint32_t>((32 * j + 8 * g + e) * a.vdim * 4);
                        const float x = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sr, state_lane + row, 0, 0));
                        const float y = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(dr, dstate_lane + row, 0, 0));
                        (e < 4 ? s0 : s1)[e & 3] = x;
                        (e < 4 ? d0 : d1)[e & 3] = y;
                        inner = __builtin_fmaf(x, y, inner);
                    }
                    const Frag<3> sf = split(s0, s1), df = split(d0, d1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Frag<N> kf = rows_frag<N, KT>(Kl, 16 * i + m, 4 * j + g);
                        const Frag<N> qf = rows_frag<N, KT>(Ql, 16 * i + m, 4 * j + g);
                        product<3>(ks[i], kf, sf);
                        product<3>(qs[i], qf, sf);
                        product<3>(kd[i], kf, df);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // R, and what is not finite row by row (before sums over tokens mix the rows)
                f32x4 R[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        const bool old = t < first_start;
                        R[i][r] = V[i][r] - keep_if(old, into[r] * ks[i][r]);
                        const float y = keep_if(t >= last_start, kd[i][r]);
                        odd |= uint64_t(not_finite(R[i][r])) << t | uint64_t(not_finite(y)) << t;
                        qs[i][r] = keep_if(old, a.scale * into[r] * qs[i][r]);
                        odd |= uint64_t(not_finite(qs[i][r])) << t;
                    }
                }
                // E, U
                f32x4 E[4];
                {
                    const Frag<3> rf[2] = {split(R[0], R[1]), split(R[2], R[3])};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        E[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j <= i / 2; ++j) {
                            Frag<3> tf;
#pragma unroll
                            for (int p = 0; p < 3; ++p) tf.p[p] = Tl[(low_block(i, j) * 3 + p) * 64 + lane];
                            product<3>(E[i], tf, rf[j]);
                        }
                        const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) U[i][r] = beta[r] * E[i][r];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // O, a tile of rows at a time, and dO . O over this wave's columns
                float pb = 0.0f, pg = 0.0f;
                {
                    const Frag<3> uf[2] = {split(U[0], U[1]), split(U[2], U[3])};
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        __builtin_amdgcn_sched_barrier(0);
                        f32x4 P[4];   // rows s, columns t
#pragma unroll
                        for (int is = 0; is < 4; ++is) P[is] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < STEPS; ++j) {
                            const Frag<N> qf = rows_frag<N, KT>(Ql, 16 * it + m, 4 * j + g);
#pragma unroll
                            for (int is = 0; is <= it; ++is)
                                product<3>(P[is], rows_frag<N, KT>(Kl, 16 * is + m, 4 * j + g), qf);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            odd |= uint64_t(not_finite(keep_if(4 * g + r == m, P[it][r]))) << (16 * it + m);
                        const int t = 16 * it + m, from = doc_first(starts, t);
                        const float th = rec->hi[t], tl = rec->lo[t];
#pragma unroll
                        for (int is = 0; is <= it; ++is) {
                            const f32x4 sh = four(rec->hi + 16 * is + 4 * g), sl = four(rec->lo + 16 * is + 4 * g);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int s = 16 * is + 4 * g + r;
                                const float d = exp2_fast((th - sh[r]) + (tl - sl[r]));
                                P[is][r] = keep_if(s <= t && s >= from, a.scale * P[is][r] * d);
                            }
                        }
#pragma unroll
                        for (int j = 0; j <= it / 2; ++j) product<3>(qs[it], split(P[2 * j], P[2 * j + 1]), uf[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = row_sum(dO[it][r] * qs[it][r]);
                            pg = m == 4 * it + r ? y : pg;
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // dU = outof K dS + P^T dO, and dX
                {
                    f32x4 dU[4];
                    const Frag<3> of[2] = {split(dO[0], dO[1]), split(dO[2], dO[3])};
                    float end = starts == 0 ? rec->keep * inner : 0.0f;
#pragma unroll
                    for (int is = 0; is < 4; ++is) {
                        __builtin_amdgcn_sched_barrier(0);
                        const f32x4 outof = four(rec->outof + 16 * is + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            dU[is][r] = keep_if(16 * is + 4 * g + r >= last_start, outof[r] * kd[is][r]);
                            end = __builtin_fmaf(U[is][r], dU[is][r], end);
                        }
                        f32x4 P[4];   // rows t, columns s
#pragma unroll
                        for (int it = 0; it < 4; ++it) P[it] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < STEPS; ++j) {
                            const Frag<N> kf = rows_frag<N, KT>(Kl, 16 * is + m, 4 * j + g);
#pragma unroll
                            for (int it = is; it < 4; ++it)
                                product<3>(P[it], rows_frag<N, KT>(Ql, 16 * it + m, 4 * j + g), kf);
                        }
                        const int s = 16 * is + m, stop = doc_end(starts, s);
                        const float sh = rec->hi[s], sl = rec->lo[s];
#pragma unroll
                        for (int it = is; it < 4; ++it) {
                            const f32x4 th = four(rec->hi + 16 * it + 4 * g), tl = four(rec->lo + 16 * it + 4 * g);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int t = 16 * it + 4 * g + r;
                                const float d = exp2_fast((th[r] - sh) + (tl[r] - sl));
                                P[it][r] = keep_if(t >= s && t < stop, a.scale * P[it][r] * d);
                            }
                        }
#pragma unroll
                        for (int j = is / 2; j < 2; ++j) {
                            const Frag<3> pf = split(P[2 * j], P[2 * j + 1]);
                            if constexpr (N == 1) product<3>(dU[is], pf, Frag<1>{{of[j].p[0]}});   // dO as stored is one piece
                            else product<3>(dU[is], pf, of[j]);
                        }
                    }
                    end = row_sum(end);
                    end += __shfl_xor(end, 16);
                    end += __shfl_xor(end, 32);
                    ends[wave] = end;
                    __builtin_amdgcn_sched_barrier(0);
                    const Frag<3> uf[2] = {split(dU[0], dU[1]), split(dU[2], dU[3])};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        X[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                        for (int j = i / 2; j < 2; ++j) {
                            Frag<3> tf;
#pragma unroll
                            for (int p = 0; p < 3; ++p) tf.p[p] = Tl[((kBlocks + high_block(i, j)) * 3 + p) * 64 + lane];
                            product<3>(X[i], tf, uf[j]);
                        }
                    }
                }
                // dv, and the rows' other dot products over this wave's columns
                const int64_t ldv = static_cast<int64_t>(a.vheads) * a.vdim;
                const Rsrc dvr = rows_rsrc<ESZ>(a.dv, first * ldv + hv * a.vdim, rows, ldv, a.vdim);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        const float dv = beta[r] * X[i][r];
                        const float x = row_sum(X[i][r] * E[i][r]), y = row_sum(dv * V[i][r]);
                        pb = m == 4 * i + r ? x : pb;
                        pg -= m == 4 * i + r ? y : 0.0f;
                        store_one<T>(dvr, value_lane + static_cast<uint32_t>(t * static_cast<int>(ldv) * ESZ),
                                     nan_if((sick >> t) & 1, dv));
                    }
                }
                const int t = 16 * (m / 4) + 4 * g + m % 4;
                parts[wave * C + t] = pb;
                parts[(kWaves + wave) * C + t] = pg;
                if (__ballot(odd != 0) != 0) {
#pragma unroll
                    for (int s = 1; s < 64; s *= 2) odd |= __shfl_xor(odd, s);
                    odd_rows[wave] = odd;
                }
            }
            __syncthreads();
            uint64_t found = rec->bad;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) found |= odd_rows[w];
            found = whole(uniform(found), starts);
            if (pass == 1 || found == 0) break;
            sick = found;
        }
        sick_any |= sick;

        if (wave == 0) {
            const int lane = thread_now() & 63;
            float pb = 0.0f, end = 0.0f;
            double sum = 0.0;
            for (int w = 0; w < vwaves; ++w) {
                pb += parts[w * C + lane];
                sum += parts[(kWaves + w) * C + lane];
                end += ends[w];
            }
            const int stop = doc_end(starts, lane);
#pragma unroll
            for (int s = 1; s < 64; s *= 2) {
                const double other = __shfl_down(sum, s);
                sum += lane + s < stop ? other : 0.0;
            }
            if (lane >= last_start) sum += end;
            const bool nan = (sick >> lane) & 1, start = (starts >> lane) & 1;
            const Rsrc br = rows_rsrc<4>(a.dbeta, first * a.vheads + hv, rows, a.vheads, 1);
            const Rsrc gr = rows_rsrc<4>(a.dg, a.dg ? first * a.vheads + hv : 0, a.dg ? rows : 0, a.vheads, 1);
            store_one<float>(br, static_cast<uint32_t>(lane * a.vheads * 4), nan_if(nan, pb));
            store_one<float>(gr, static_cast<uint32_t>(lane * a.vheads * 4),
                             nan_if(nan, keep_if(!start, static_cast<float>(sum))));
        }
        // (2) U and dX over K and Q
        if (wave < vwaves) {
            const int lane = thread_now() & 63, g = lane >> 4, m = lane & 15;
            const int v = 16 * wave + m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = (16 * i + 4 * g + r) * kRowV + v;
                    put<OUT>(Ul, PLANE_V, at, U[i][r]);
                    put<OUT>(Xl, PLANE_V, at, X[i][r]);
                }
        }
        __syncthreads();
        const int lane = thread_now() & 63, g = lane >> 4, m = lane & 15;
        auto dout_frag = [&](int i, int j) {
            Eight<T, VEC> e;
            e.load(orr, static_cast<uint32_t>((16 * i + m) * static_cast<int>(a.ld_o) * ESZ), 32 * j + 8 * g, a.vdim);
            Frag<N> f = e.frag();
            clear_if<N>(f, (sick >> (16 * i + m)) & 1);
            return f;
        };
        for (int tile = wave; tile < 10; tile += kWaves) {
            const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, is = tile - it * (it + 1) / 2;
            f32x4 P = {0, 0, 0, 0}, G = {0, 0, 0, 0};
            for (int j = 0; j < vsteps; ++j) {
                const Frag<OUT> uf = plane_frag<OUT>(Ul, 16 * is + m, 32 * j + 8 * g);
                const Frag<OUT> xf = plane_frag<OUT>(Xl, 16 * it + m, 32 * j + 8 * g);
                product<OUT>(P, dout_frag(it, j), uf);
                product<OUT>(G, xf, uf);
            }
            const int s = 16 * is + m, stop = doc_end(starts, s);
            const float sh = rec->hi[s], sl = rec->lo[s];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * it + 4 * g + r;
                const float d = exp2_fast((rec->hi[t] - sh) + (rec->lo[t] - sl));
                const bool on = t >= s && t < stop;
                put<OUT>(Pl, PLANE_P, t * kRowP + s, keep_if(on, a.scale * d * P[r]));
                const float n = keep_if(on && t > s, -rec->beta[t] * d * G[r]);
                const int pad = t * kRowP + C;   // for the lanes above the diagonal
                put<OUT>(Nl, PLANE_P, t >= s ? t * kRowP + s : pad, n);
                put<OUT>(Nl, PLANE_P, t > s ? s * kRowP + t : pad, n);
                if (it == is + 1 && (is & 1) == 0) put<OUT>(Pl, PLANE_P, s * kRowP + t, 0.0f);   // read with the tile beside it
            }
        }

        // (3) the products with S and dS
        const bool no_state = (sick & 1) != 0 && first_start > 0, no_dstate = (sick >> 63) != 0;
        if (16 * wave < KT) {
            f32x4 os[4], xs[4], us[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) os[i] = xs[i] = us[i] = f32x4{0, 0, 0, 0};
            const uint32_t row = static_cast<uint32_t>((16 * wave + m) * a.vdim * 4);
            for (int j = 0; j < vsteps; ++j) {
                Eight<float, VEC> se, de;
                se.load(sr, row, 32 * j + 8 * g, no_state ? 0 : a.vdim);
                de.load(dr, row, 32 * j + 8 * g, no_dstate ? 0 : a.vdim);
                const Frag<OUT> sf = split_out<OUT>(__builtin_bit_cast(f32x4, se.a), __builtin_bit_cast(f32x4, se.b));
                const Frag<OUT> df = split_out<OUT>(__builtin_bit_cast(f32x4, de.a), __builtin_bit_cast(f32x4, de.b));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    product<OUT>(os[i], dout_frag(i, j), sf);
                    product<OUT>(xs[i], plane_frag<OUT>(Xl, 16 * i + m, 32 * j + 8 * g), sf);
                    product<OUT>(us[i], plane_frag<OUT>(Ul, 16 * i + m, 32 * j + 8 * g), df);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 into = four(rec->into + 16 * i + 4 * g), outof = four(rec->outof + 16 * i + 4 * g);
                const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    const bool old = t < first_start;
                    dq[i][r] += keep_if(old, a.scale * into[r] * os[i][r]);
                    dk[i][r] += keep_if(t >= last_start, outof[r] * us[i][r]) - keep_if(old, into[r] * beta[r] * xs[i][r]);
                }
            }
        }
        __syncthreads();
        // (4) the products with K and Q
        {
            const int tid = thread_now();
            KQ kraw, qraw;
            kraw.fetch(kr, a.ld_k, a.kdim, tid);
            qraw.fetch(qr, a.ld_q, a.kdim, tid);
            kraw.land_without(Kl, tid, sick);
            qraw.land_without(Ql, tid, sick);
        }
        __syncthreads();
        if (16 * wave < KT) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Frag<N> kf = cols_frag<N, KT>(Kl, j, g, m, 16 * wave + 4 * (m % 4));
                const Frag<N> qf = cols_frag<N, KT>(Ql, j, g, m, 16 * wave + 4 * (m % 4));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (j <= i / 2) product<OUT>(dq[i], token_frag<OUT>(Pl, 16 * i + m, j, g), kf);
                    if (j >= i / 2) product<OUT>(dk[i], token_cols<OUT>(Pl, j, g, m, 16 * i + 4 * (m % 4)), qf);
                    product<OUT>(dk[i], token_frag<OUT>(Nl, 16 * i + m, j, g), kf);
                }
            }
        }
    }

    const int lane = thread_now() & 63, g = lane >> 4, m = lane & 15;
    const int ch = 16 * wave + m;
    const uint32_t key_lane = ch < a.kdim ? ch * ESZ : kPast;
    const int64_t ldk = static_cast<int64_t>(a.kheads) * a.kdim;
    const Rsrc dqr = rows_rsrc<ESZ>(a.dq, first * ldk + hk * a.kdim, rows, ldk, a.kdim);
    const Rsrc dkr = rows_rsrc<ESZ>(a.dk, first * ldk + hk * a.kdim, rows, ldk, a.kdim);
    if (16 * wave < KT) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * i + 4 * g + r;
                const uint32_t off = key_lane + static_cast<uint32_t>(t * static_cast<int>(ldk) * ESZ);
                const bool nan = (sick_any >> t) & 1;
                store_one<T>(dqr, off, nan_if(nan, dq[i][r]));
                store_one<T>(dkr, off, nan_if(nan, dk[i][r]));
            }
    }
}

template <typename T, int KT, bool VEC>
hipError_t launch(const DeltaArgs& a) {
    hipLaunchKernelGGL((grads_kernel<T, KT, VEC>), dim3(static_cast<unsigned>(a.batch * a.kheads * a.nchunks)),
                       dim3(kThreads), 0, a.stream, a, static_cast<int64_t>(delta_chunk_bytes()));
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(const DeltaArgs& a) {
    if (a.vec_k && a.vec_o) return a.kdim > 64 ? launch<T, 128, true>(a) : launch<T, 64, true>(a);
    return a.kdim > 64 ? launch<T, 128, false>(a) : launch<T, 64, false>(a);
}

}  // namespace

hipError_t launch_delta_bwd_grads(const DeltaArgs& a) { return a.bf16 ? by_width<bf16_t>(a) : by_width<float>(a); }

}  // namespace mamba
