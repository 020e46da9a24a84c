// Gated delta rule, backward: every gradient of a chunk of 64 tokens, from the state S that enters it, the gradient dS at
// the state that leaves it and the dX that the chain of dS went through (delta_bwd.hip), all chunks at once.  A workgroup
// takes one key head of a chunk and its value heads in turn, so that dq and dk sum over them in a fixed order.
//
//     R = V - exp(gamma) K S,  E = (I + M b)^-1 R,  U = b E,  dX = (I + b M)^-T (P^T dO + exp(gamma_C - gamma) K dS),
//     dV = beta dX,   dbeta = dX . E,   dgamma = q . dq - dV . V   (row by row, this value head's part of dq),
//     dq = scale exp(gamma) dO S^T + dP K,                       dP = scale D o dO U^T (s <= t),
//     dk = W - exp(gamma) dV S^T + dP^T Q + N K,   W = exp(gamma_C - gamma) U dS^T,   N = G + G^T, G = -b D o dX U^T (s < t).
//
// dgamma's form follows from every decay multiplying the key and value sums alike: scaling a
// row's decay scales o . dO and v . dV by what it scales the row's query and value side, so the 64 x 64
// matrices' row and column sums cancel to these two dot products; and o . dO = q . dq, as o is linear in q.  At the chunk's
// end <dS, S_out> = exp(gamma_C) <dS, S> + sum_t k . W is added, and dg is the
// sum of dgamma from its token to its document's (or the chunk's) end.  A decay that counts as 0 ends that sum as
// a document start does, and has 0 itself: the sum across it is 0, of which rounding would leave something.
//
// Phases: (1) a wave owns 16 value columns, with K and the triangle in LDS; (2) the tiles of
// dP and N, contracted over the columns, with U and dX in LDS over K; (3) a wave owns 16 key
// channels: the products with S and dS; (4) those with K and Q, in LDS over U and dX.  dP and N lie in LDS as floats, cut
// into pieces where they are read: as pieces they leave no room for dO.
//
// Bound by memory's latency: 2 x 32768 tokens, 12 heads of 128 x 128, 1.78 ms.  A workgroup fills a CU (157 KB of LDS), a head
// of a chunk takes it 53000 cycles, of which 9000 wait for S, K, dO and the triangle, and what all read (S twice) and write,
// 4.7 GB, takes 0.92 ms.  (With P formed by every wave and o . dO from O: 2.17 ms and three times the instructions.)
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kRowV = 136, kRowP = 68;   // bf16 of a row of U and dX, floats of one of dP and N

template <int CTRL>
__device__ __forceinline__ float moved(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
// Sums over the 16 lanes of a DPP row: lane m gets that of the m-th value.  Lanes keep half of what they hold and pass
// the other half on, four times: 45 instructions in place of 80 and a selection.
__device__ __forceinline__ float row_sums(float (&x)[16], int m) {
    auto turn = [&](int n, bool high, auto ctrl) {
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float kept = high ? x[k + n] : x[k], passed = high ? x[k] : x[k + n];
            x[k] = kept + moved<decltype(ctrl)::value>(passed);
        }
    };
    using std::integral_constant;
    turn(8, (m & 8) != 0, integral_constant<int, 0x140>{});   // row_mirror: lane m with m ^ 15
    turn(4, (m & 4) != 0, integral_constant<int, 0x141>{});   // row_half_mirror: m ^ 7
    turn(2, (m & 2) != 0, integral_constant<int, 0x4E>{});    // quad_perm [2, 3, 0, 1]: m ^ 2
    turn(1, (m & 1) != 0, integral_constant<int, 0xB1>{});    // quad_perm [1, 0, 3, 2]: m ^ 1
    return x[0];
}
// Sum over a wave, in each lane.
__device__ __forceinline__ float wave_sum(float x) {
    x += moved<0xB1>(x);
    x += moved<0x4E>(x);
    x += moved<0x141>(x);
    x += moved<0x140>(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// One value in three pieces, to element `at` of planes of `plane` elements.
__device__ __forceinline__ void put(uint16_t* to, int plane, int at, float x) {
    const uint32_t u = __float_as_uint(x);
    const float r = x - __uint_as_float(u & 0xffff0000u);
    const uint32_t mid = f32_to_bf16(r);
    to[at] = static_cast<uint16_t>(u >> 16);
    to[plane + at] = static_cast<uint16_t>(mid);
    to[2 * plane + at] = static_cast<uint16_t>(__float_as_uint(r - __uint_as_float(mid << 16)) >> 16);
}

// Row `row` of [C][kRowP], the tokens of step j in the order of cols_frag ...
__device__ __forceinline__ Frag<3> token_frag(const float* lds, int row, int j, int g) {
    const float* at = lds + row * kRowP + 32 * j + 4 * g;
    return split(four(at), four(at + 16));
}
// ... and column `col`.
__device__ __forceinline__ Frag<3> token_cols(const float* lds, int col, int j, int g) {
    const float* at = lds + (32 * j + 4 * g) * kRowP + col;
    f32x4 x, y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = at[e * kRowP];
        y[e] = at[(16 + e) * kRowP];
    }
    return split(x, y);
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
    using KQ = Tile<T, KT, kThreads, VEC>;
    constexpr int PLANE_V = C * kRowV;
    constexpr size_t PARTS = 2 * kWaves * C * 4;
    constexpr size_t ZERO = larger(2 * KQ::kBytes, size_t(6) * PLANE_V * 2);
    constexpr size_t ONE = larger(kSolveBytes + PARTS, size_t(2) * C * kRowP * 4);
    __shared__ __align__(16) char region0[ZERO];
    __shared__ __align__(16) char region1[ONE];
    __shared__ __align__(16) uint16_t dout_[N == 1 ? PLANE_V : 8];   // dO [C][kRowV], where there is room for it
    __shared__ __align__(16) ChunkRec rec_;
    __shared__ float ends[kWaves];
    __shared__ float turns[kWaves][C];   // q . dq, a wave's channels
    __shared__ uint64_t odd_rows[kWaves];
    uint16_t* Kl = reinterpret_cast<uint16_t*>(region0);
    uint16_t* Ql = Kl + N * C * KT;
    uint16_t* Ul = reinterpret_cast<uint16_t*>(region0);          // [3][C][kRowV]
    uint16_t* Xl = Ul + 3 * PLANE_V;                              // the same
    const u32x4* Tl = reinterpret_cast<const u32x4*>(region1);
    float* parts = reinterpret_cast<float*>(region1 + kSolveBytes);   // [2][kWaves][C]
    float* Pl = reinterpret_cast<float*>(region1);                // [C][kRowP]
    float* Nl = Pl + C * kRowP;
    const ChunkRec* rec = &rec_;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int bh = quotient(blockIdx.x, a.nchunks);   // row and key head
    const int c = remainder(blockIdx.x, a.nchunks);
    const int hk = remainder(bh, a.kheads), group = quotient(a.vheads, a.kheads);
    const int64_t b = quotient(bh, a.kheads);
    const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, left = a.seqlen - static_cast<int64_t>(c) * C;
    const int rows = static_cast<int>(left < C ? left : C);
    const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;
    const int vsteps = (a.vdim + 31) / 32, vwaves = 2 * vsteps, groups = (a.vdim + 15) / 16;
    const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_k, a.kpitch);
    const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_q, a.kpitch);

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
        const Rsrc xr = rsrc(a.dx + (id * groups + wave) * kGroupFloats, wave < groups ? kGroupFloats * 4 : 0);

        f32x4 U[4], X[4];
        uint64_t sick = 0, starts = 0;
        int first_start = C, last_start = 0;
        for (int pass = 0; pass < 2; ++pass) {
            const int tid = thread_now(), lane = tid & 63, g = lane >> 4, m = lane & 15;
            // (1) once more without the documents in which something is not finite, if there are any
            __syncthreads();
            const bool no_state_ = pass != 0 && (sick & 1) != 0 && first_start > 0;
            const int v = 16 * wave + m;
            const uint32_t state_lane =
                v < a.vdim && !no_state_ ? static_cast<uint32_t>(v * 4 + 8 * g * a.vdim * 4) : kPast;
            f32x4 S[2 * STEPS];
            {
                KQ kraw;
                kraw.fetch(kr, a.ld_k, a.kpitch, tid);
                Eight<T, VEC> oraw[2];
                if constexpr (N == 1) {
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        oraw[p].load(orr, static_cast<uint32_t>((32 * p + tid / 16) * static_cast<int>(a.ld_o) * ESZ),
                                     tid % 16 * 8, a.vdim);
                }
                if (wave < vwaves) {
#pragma unroll
                    for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                                sr, state_lane + static_cast<uint32_t>(state_row(i, 0, r) * a.vdim * 4), 0, 0));
                }
                u32x4* Tw = reinterpret_cast<u32x4*>(region1);
                const Rsrc t0 = rsrc(a.solve + id * kSolveBytes, kSolveBytes);
                for (int p = wave; p < kBlocks * 3; p += kWaves)
                    Tw[p * 64 + lane] = __builtin_amdgcn_raw_buffer_load_b128(t0, (p * 64 + lane) * 16, 0, 0);
                const uint32_t* from = reinterpret_cast<const uint32_t*>(a.chunks + id * rec_bytes);
                constexpr int RECW = sizeof(ChunkRec) / 4;
                static_assert(RECW <= kThreads, "one word a thread");
                reinterpret_cast<uint32_t*>(&rec_)[tid < RECW ? tid : RECW - 1] = from[tid < RECW ? tid : RECW - 1];
                odd_rows[wave] = 0;
                kraw.land_without(Kl, tid, sick);
                if constexpr (N == 1) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int t = 32 * p + tid / 16;
                        Frag<N> f = oraw[p].frag();
                        clear_if<N>(f, (sick >> t) & 1);
                        *reinterpret_cast<u32x4*>(dout_ + t * kRowV + tid % 16 * 8) = f.p[0];
                    }
                }
            }
            __syncthreads();
            starts = uniform(rec->starts);
            first_start = starts ? __builtin_ctzll(starts) : C;
            last_start = starts ? 63 - __builtin_clzll(starts) : 0;
            if (wave < vwaves) {
                const uint32_t value_lane = v < a.vdim ? v * ESZ : kPast;
                f32x4 V[4];
                uint64_t odd = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    X[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, lane * 16 + i * 1024, 0, 0));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        const uint32_t at = (sick >> t) & 1 ? kPast : value_lane;
                        V[i][r] = one_value<T>(load_one<T>(vr, at + static_cast<uint32_t>(t * static_cast<int>(a.ld_v) * ESZ)));
                    }
                }
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
                // R, and what is not finite row by row (before sums over tokens mix the rows)
                f32x4 R[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        R[i][r] = V[i][r] - keep_if(t < first_start, into[r] * ks[i][r]);
                        X[i][r] = keep_if(!((sick >> t) & 1), X[i][r]);
                        odd |= uint64_t(not_finite(R[i][r])) << t | uint64_t(not_finite(X[i][r])) << t;
                    }
                }
                // E, U
                f32x4 E[4];
                {
                    const Frag<3> rf[2] = {split_values(R[0], R[1]), split_values(R[2], R[3])};
#pragma unroll
                    for (int i = 0; i < 4; ++i) E[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int p = 2; p >= 0; --p)
#pragma unroll
                            for (int q = 2 - p; q >= 0; --q)
#pragma unroll
                                for (int i = 2 * j; i < 4; ++i)
                                    E[i] = mfma(Tl[(low_block(i, j) * 3 + p) * 64 + lane], rf[j].p[q], E[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                        for (int r = 0; r < 4; ++r) U[i][r] = beta[r] * E[i][r];
                    }
                }
                float xe[16], vv[16];
                // dv, and the rows' dot products over this wave's columns
                const int64_t ldv = static_cast<int64_t>(a.vheads) * a.vdim;
                const Rsrc dvr = rows_rsrc<ESZ>(a.dv, first * ldv + hv * a.vdim, rows, ldv, a.vdim);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = 16 * i + 4 * g + r;
                        const float dv = beta[r] * X[i][r];
                        xe[4 * i + r] = X[i][r] * E[i][r];
                        vv[4 * i + r] = -dv * V[i][r];
                        store_one<T>(dvr, value_lane + static_cast<uint32_t>(t * static_cast<int>(ldv) * ESZ),
                                     nan_if((sick >> t) & 1, dv));
                    }
                }
                const int t = 16 * (m / 4) + 4 * g + m % 4;
                parts[wave * C + t] = row_sums(xe, m);
                parts[(kWaves + wave) * C + t] = row_sums(vv, m);
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

        double turn = 0.0;   // wave 0: -dV . V of token `lane`
        if (wave == 0) {
            const int lane = thread_now() & 63;
            float pb = 0.0f;
            for (int w = 0; w < vwaves; ++w) {
                pb += parts[w * C + lane];
                turn += parts[(kWaves + w) * C + lane];
            }
            const Rsrc br = rows_rsrc<4>(a.dbeta, first * a.vheads + hv, rows, a.vheads, 1);
            store_one<float>(br, static_cast<uint32_t>(lane * a.vheads * 4), nan_if((sick >> lane) & 1, pb));
            __builtin_amdgcn_raw_buffer_store_b32(static_cast<uint32_t>(lane ? sick >> 32 : sick),   // (two lanes have a place)
                                                  rsrc(a.chunks + id * rec_bytes + offsetof(ChunkRec, sick), 8), lane * 4, 0, 0);
        }
        // (2) U and dX over K
        if (wave < vwaves) {
            const int lane = thread_now() & 63, g = lane >> 4, m = lane & 15;
            const int v = 16 * wave + m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = (16 * i + 4 * g + r) * kRowV + v;
                    put(Ul, PLANE_V, at, U[i][r]);
                    put(Xl, PLANE_V, at, X[i][r]);
                }
        }
        __syncthreads();
        const int lane = thread_now() & 63, g = lane >> 4, m = lane & 15;
        auto dout_frag = [&](int i, int j) {
            if constexpr (N == 1) {
                return plane_frag<1>(dout_, 16 * i + m, 32 * j + 8 * g);
            } else {
                Eight<T, VEC> e;
                e.load(orr, static_cast<uint32_t>((16 * i + m) * static_cast<int>(a.ld_o) * ESZ), 32 * j + 8 * g, a.vdim);
                Frag<N> f = e.frag();
                clear_if<N>(f, (sick >> (16 * i + m)) & 1);
                return f;
            }
        };
        // the first rows of S and dS for (3)
        const bool no_state = (sick & 1) != 0 && first_start > 0, no_dstate = (sick >> 63) != 0;
        const uint32_t state_row_at = static_cast<uint32_t>((16 * wave + m) * a.vdim * 4);
        Eight<float, VEC> se, de;
        auto fetch_states = [&](int j) {
            se.load(sr, state_row_at, 32 * j + 8 * g, no_state ? 0 : a.vdim);
            de.load(dr, state_row_at, 32 * j + 8 * g, no_dstate ? 0 : a.vdim);
        };
        if constexpr (N == 1) fetch_states(0);   // (channels behind the last: zeros)
        for (int tile = wave; tile < 10; tile += kWaves) {
            const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, is = tile - it * (it + 1) / 2;
            f32x4 P = {0, 0, 0, 0}, G = {0, 0, 0, 0};
            for (int j = 0; j < vsteps; ++j) {
                const Frag<3> uf = plane_frag<3>(Ul, 16 * is + m, 32 * j + 8 * g);
                const Frag<3> xf = plane_frag<3>(Xl, 16 * it + m, 32 * j + 8 * g);
                const Frag<N> of = dout_frag(it, j);
                __builtin_amdgcn_sched_barrier(0);
                product<3>(P, of, uf);
                product<3>(G, xf, uf);
            }
            const int s = 16 * is + m, stop = doc_end(starts, s);
            const float sh = rec->hi[s], sl = rec->lo[s];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * it + 4 * g + r;
                const float d = exp2_fast((rec->hi[t] - sh) + (rec->lo[t] - sl));
                const bool on = t >= s && t < stop;
                Pl[t * kRowP + s] = keep_if(on, a.scale * d * P[r]);
                const float n = keep_if(on && t > s, -rec->beta[t] * d * G[r]);
                const int pad = t * kRowP + C;   // for the lanes above the diagonal
                Nl[t >= s ? t * kRowP + s : pad] = n;
                Nl[t > s ? s * kRowP + t : pad] = n;
                if (it == is + 1 && (is & 1) == 0) Pl[s * kRowP + t] = 0.0f;   // read with the tile beside it
            }
        }

        // (3) the products with S and dS
        __builtin_amdgcn_sched_barrier(0);
        f32x4 dqh[4], W[4];   // this value head's dq; what dS gives to dk
        float end = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) dqh[i] = W[i] = f32x4{0, 0, 0, 0};
        if (16 * wave < KT) {
            f32x4 xs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[i] = f32x4{0, 0, 0, 0};
            for (int j = 0; j < vsteps; ++j) {
                if constexpr (N != 1) fetch_states(j);   // (fewer registers are free)
                const f32x4 s0 = __builtin_bit_cast(f32x4, se.a), s1 = __builtin_bit_cast(f32x4, se.b);
                const f32x4 d0 = __builtin_bit_cast(f32x4, de.a), d1 = __builtin_bit_cast(f32x4, de.b);
                if (N == 1 && j + 1 < vsteps) fetch_states(j + 1);
#pragma unroll
                for (int r = 0; r < 4; ++r) end = __builtin_fmaf(s0[r], d0[r], __builtin_fmaf(s1[r], d1[r], end));
                const Frag<3> sf = split(s0, s1), df = split(d0, d1);
                if constexpr (N == 1) {
                    Frag<N> of[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) of[i] = dout_frag(i, j);
                    Frag<3> xf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) xf[i] = plane_frag<3>(Xl, 16 * i + m, 32 * j + 8 * g);
                    products<3, 4>(dqh, of, sf);
                    products<3, 4>(xs, xf, sf);
                    __builtin_amdgcn_sched_barrier(0);
                    Frag<3> uf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) uf[i] = plane_frag<3>(Ul, 16 * i + m, 32 * j + 8 * g);
                    products<3, 4>(W, uf, df);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        product<3>(dqh[i], dout_frag(i, j), sf);
                        product<3>(xs[i], plane_frag<3>(Xl, 16 * i + m, 32 * j + 8 * g), sf);
                        product<3>(W[i], plane_frag<3>(Ul, 16 * i + m, 32 * j + 8 * g), df);
                    }
                }
            }
            end = starts == 0 ? rec->keep * end : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 into = four(rec->into + 16 * i + 4 * g), outof = four(rec->outof + 16 * i + 4 * g);
                const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    const bool old = t < first_start;
                    dqh[i][r] = keep_if(old, a.scale * into[r] * dqh[i][r]);
                    W[i][r] = keep_if(t >= last_start, outof[r] * W[i][r]);
                    dk[i][r] += W[i][r] - keep_if(old, into[r] * beta[r] * xs[i][r]);
                }
            }
        }
        __syncthreads();
        // (4) the products with K and Q
        {
            const int tid = thread_now();
            KQ kraw, qraw;
            kraw.fetch(kr, a.ld_k, a.kpitch, tid);
            qraw.fetch(qr, a.ld_q, a.kpitch, tid);
            kraw.land_without(Kl, tid, sick);
            qraw.land_without(Ql, tid, sick);
        }
        __syncthreads();
        const int lane4 = thread_now() & 63;
        float dots = 0.0f;   // q . dq of row 16 (m / 4) + 4 g + m % 4
        if (16 * wave < KT) {
            const int g = lane4 >> 4, m = lane4 & 15;
            // (loads in front of what uses them: the compiler would wait for each in turn)
            auto values = [&](float (&x)[16], const uint16_t* from) {
                uint32_t raw[N][16];
#pragma unroll
                for (int p = 0; p < N; ++p)
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        raw[p][n] = from[place<KT>(16 * (n / 4) + 4 * g + n % 4, 2 * wave + m / 8) + m % 8 + p * C * KT];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    x[n] = 0.0f;
#pragma unroll
                    for (int p = N - 1; p >= 0; --p) x[n] += __uint_as_float(raw[p][n] << 16);
                }
            };
            {
                float kv[16];
                values(kv, Kl);
#pragma unroll
                for (int n = 0; n < 16; ++n) end = __builtin_fmaf(kv[n], W[n / 4][n % 4], end);
            }
            __builtin_amdgcn_sched_barrier(0);
            const Frag<N> kf[2] = {cols_frag<N, KT>(Kl, 0, g, m, 16 * wave + 4 * (m % 4)),
                                   cols_frag<N, KT>(Kl, 1, g, m, 16 * wave + 4 * (m % 4))};
            const Frag<N> qf[2] = {cols_frag<N, KT>(Ql, 0, g, m, 16 * wave + 4 * (m % 4)),
                                   cols_frag<N, KT>(Ql, 1, g, m, 16 * wave + 4 * (m % 4))};
            Frag<3> pf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pf[i] = token_frag(Pl, 16 * i + m, 0, g);
            __builtin_amdgcn_sched_barrier(0);
            products<3, 4>(dqh, pf, kf[0]);
#pragma unroll
            for (int i = 2; i < 4; ++i) pf[i] = token_frag(Pl, 16 * i + m, 1, g);
            __builtin_amdgcn_sched_barrier(0);
            products<3, 2>(dqh + 2, pf + 2, kf[1]);
            Frag<3> nf[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) nf[i] = token_frag(Nl, 16 * i + m, j, g);
                __builtin_amdgcn_sched_barrier(0);
                products<3, 4>(dk, nf, kf[j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) nf[i] = token_cols(Pl, 16 * i + m, 1, g);
            __builtin_amdgcn_sched_barrier(0);
            products<3, 4>(dk, nf, qf[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) nf[i] = token_cols(Pl, 16 * i + m, 0, g);
            __builtin_amdgcn_sched_barrier(0);
            products<3, 2>(dk, nf, qf[0]);
            __builtin_amdgcn_sched_barrier(0);
            float qv[16];
            values(qv, Ql);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    qv[4 * i + r] *= dqh[i][r];
                    dq[i][r] += dqh[i][r];
                }
            dots = row_sums(qv, m);
        }
        end = wave_sum(end);
        ends[wave] = end;
        turns[wave][16 * (m / 4) + 4 * g + m % 4] = dots;
        __syncthreads();
        if (wave == 0) {
            const int lane = thread_now() & 63;
            float end = 0.0f;
            for (int w = 0; w < KT / 16; ++w) {
                turn += turns[w][lane];
                end += ends[w];
            }
            const uint64_t walls = uniform(rec->walls);
            const int stop = doc_end(walls, lane), last_wall = walls ? 63 - __builtin_clzll(walls) : 0;
#pragma unroll
            for (int s = 1; s < 64; s *= 2) {
                const double other = __shfl_down(turn, s);
                turn += lane + s < stop ? other : 0.0;
            }
            if (lane >= last_wall) turn += end;
            const bool nan = (sick >> lane) & 1, wall = (walls >> lane) & 1;
            const Rsrc gr = rows_rsrc<4>(a.dg, a.dg ? first * a.vheads + hv : 0, a.dg ? rows : 0, a.vheads, 1);
            store_one<float>(gr, static_cast<uint32_t>(lane * a.vheads * 4),
                             nan_if(nan, keep_if(!wall, static_cast<float>(turn))));
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

// A document in which something is not finite has NaN gradients in every chunk that it lies in: a wave a row and value head
// takes what its chunks found on to the chunks behind, then back to those before.  Where none found anything, that is one
// look at their records: 5 us after a backward pass of 435 (3 x 1001 tokens, 6 heads), 7 of 4 ms (2 x 32768 tokens, 12 heads).
template <typename T>
__global__ __launch_bounds__(64) void spread_kernel(DeltaArgs a, int64_t rec_bytes) {
    constexpr int ESZ = sizeof(T);
    const int lane = threadIdx.x, n = a.nchunks;
    const int64_t bh = blockIdx.x, b = quotient(blockIdx.x, a.vheads);
    const int hv = remainder(blockIdx.x, a.vheads), hk = quotient(hv, a.vheads / a.kheads);
    auto record = [&](int c) {   // (lanes behind the last chunk: that one once more)
        return reinterpret_cast<ChunkRec*>(a.chunks + (bh * n + (c < n ? c : n - 1)) * rec_bytes);
    };
    uint64_t any = 0;
    for (int c0 = 0; c0 < n; c0 += 64) any |= record(c0 + lane)->sick;
    if (__ballot(any != 0) == 0) return;

    auto of_lane = [](uint64_t x, int i) {
        const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(x), i);
        const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), i);
        return static_cast<uint64_t>(hi) << 32 | lo;
    };
    auto count_of = [&](int c0) { return n - c0 < 64 ? n - c0 : 64; };
    bool ill = false;   // the document that the chunk before ended in
    for (int c0 = 0; c0 < n; c0 += 64) {
        const int count = count_of(c0);
        uint64_t sick = record(c0 + lane)->sick;
        const uint64_t starts = record(c0 + lane)->starts;
        for (int i = 0; i < count; ++i) {
            const uint64_t w = of_lane(starts, i), entering = w ? (w & -w) - 1 : ~0ull;
            const uint64_t m = of_lane(sick, i) | (ill ? entering : 0);
            sick = lane == i ? m : sick;
            ill = m >> 63;
        }
        const uint64_t last = of_lane(sick, count - 1);
        record(c0 + lane)->sick = lane < count ? sick : last;
    }
    ill = false;        // the document that the chunk behind goes on with
    const int64_t ldv = static_cast<int64_t>(a.vheads) * a.vdim, ldk = static_cast<int64_t>(a.kheads) * a.kdim;
    const float nan = __builtin_nanf("");
    for (int c0 = (n - 1) / 64 * 64; c0 >= 0; c0 -= 64) {
        const uint64_t sick = record(c0 + lane)->sick, starts = record(c0 + lane)->starts;
        for (int i = count_of(c0) - 1; i >= 0; --i) {
            const uint64_t w = of_lane(starts, i), leaving = w ? ~0ull << (63 - __builtin_clzll(w)) : ~0ull;
            uint64_t m = of_lane(sick, i) | (ill ? leaving : 0);
            ill = (m & 1) && !(w & 1);
            const int64_t at = static_cast<int64_t>(c0 + i) * C, first = b * a.seqlen + at;
            const int rows = static_cast<int>(a.seqlen - at < C ? a.seqlen - at : C);
            const Rsrc dv = rows_rsrc<ESZ>(a.dv, first * ldv + hv * a.vdim, rows, ldv, a.vdim);
            const Rsrc dq = rows_rsrc<ESZ>(a.dq, first * ldk + hk * a.kdim, rows, ldk, a.kdim);
            const Rsrc dk = rows_rsrc<ESZ>(a.dk, first * ldk + hk * a.kdim, rows, ldk, a.kdim);
            const Rsrc db = rows_rsrc<4>(a.dbeta, first * a.vheads + hv, rows, a.vheads, 1);
            const Rsrc dg = rows_rsrc<4>(a.dg, a.dg ? first * a.vheads + hv : 0, a.dg ? rows : 0, a.vheads, 1);
            for (; m != 0; m &= m - 1) {
                const int t = __builtin_ctzll(m);
#pragma unroll
                for (int half = 0; half < kDeltaMaxHead / 64; ++half) {
                    const int ch = half * 64 + lane;
                    const uint32_t v = ch < a.vdim ? static_cast<uint32_t>((t * static_cast<int>(ldv) + ch) * ESZ) : kPast;
                    const uint32_t k = ch < a.kdim ? static_cast<uint32_t>((t * static_cast<int>(ldk) + ch) * ESZ) : kPast;
                    store_one<T>(dv, v, nan);
                    store_one<T>(dq, k, nan);
                    store_one<T>(dk, k, nan);
                }
                const uint32_t one = lane == 0 ? static_cast<uint32_t>(t * a.vheads * 4) : kPast;
                store_one<float>(db, one, nan);
                store_one<float>(dg, one, nan);
            }
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

hipError_t launch_delta_bwd_grads(const DeltaArgs& a) {
    const hipError_t e = a.bf16 ? by_width<bf16_t>(a) : by_width<float>(a);
    if (e != hipSuccess || a.nchunks == 1) return e;
    hipLaunchKernelGGL(a.bf16 ? spread_kernel<bf16_t> : spread_kernel<float>, dim3(static_cast<unsigned>(a.batch * a.vheads)),
                       dim3(64), 0, a.stream, a, static_cast<int64_t>(delta_chunk_bytes()));
    return hipGetLastError();
}

}  // namespace mamba
