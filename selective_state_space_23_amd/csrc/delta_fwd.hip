// Gated delta rule, forward: the chunks of a row in order (delta_prepare.hip has
// solved each chunk's triangle T).
//
//     R = V - exp(gamma) K S,  U = beta T R,
//     O = scale (exp(gamma) Q S + (D o Q K^T) U),  S <- exp(gamma_C) S + (exp(gamma_C - gamma) K)^T U.
//
// The columns of V, U, O and S do not mix, so a wave owns 16 of them for the whole
// row and keeps S (K x 16) in its accumulators; R and U go from accumulator to
// operand in place. The waves of a workgroup share what has no columns: K, Q and T in LDS.
// Without an output the same walk forms the states alone, for the backward.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

template <typename T, int KT, int NW, bool VEC, bool EMIT>
__global__ __launch_bounds__(NW * 64, 1) void fwd_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32, THREADS = NW * 64;
    using KQ = Tile<T, KT, THREADS, VEC>;
    constexpr int ROW = KQ::ROW;
    constexpr int OUT = N == 1 ? 2 : 3;      // pieces that reach an output
    constexpr int RECW = sizeof(ChunkRec) / 4, RECP = (RECW + THREADS - 1) / THREADS;
    constexpr int TP = (kBlocks * 3 + NW - 1) / NW;
    __shared__ __align__(16) char smem[(EMIT ? 2 : 1) * KQ::kBytes + kSolveBytes + RECP * THREADS * 4];
    u32x4* Tl = reinterpret_cast<u32x4*>(smem);                  // [kBlocks][3][64]
    ChunkRec* rec = reinterpret_cast<ChunkRec*>(Tl + kBlocks * 3 * 64);
    uint16_t* Kl = reinterpret_cast<uint16_t*>(smem + kSolveBytes + RECP * THREADS * 4);   // [N][C][ROW]
    uint16_t* Ql = Kl + (EMIT ? N * C * ROW : 0);

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
    f32x4 S[2 * STEPS];
    {
        const Rsrc rs = rsrc(a.initial_state + (a.initial_state ? bh * cells : 0), a.initial_state ? cells * 4 : 0);
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

    KQ kraw, qraw;
    u32x4 traw[TP];
    uint32_t vraw[16], recraw[RECP];
    auto rows_of = [&](int c) {
        const int64_t left = a.seqlen - static_cast<int64_t>(c) * C;
        return static_cast<int>(left < C ? left : C);
    };
    auto fetch = [&](int c) {
        const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C;
        const int rows = rows_of(c);
        kraw.fetch(rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_k, a.kdim), a.ld_k,
                   a.kdim, tid);
        if constexpr (EMIT)
            qraw.fetch(rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_q, a.kdim),
                       a.ld_q, a.kdim, tid);
        const int64_t id = bh * n + c;
        const Rsrc tr = rsrc(a.solve + id * kSolveBytes, kSolveBytes);
#pragma unroll
        for (int p = 0; p < TP; ++p) traw[p] = __builtin_amdgcn_raw_buffer_load_b128(tr, (p * THREADS + tid) * 16, 0, 0);
        const Rsrc rr = rsrc(a.chunks + id * rec_bytes, RECW * 4);
#pragma unroll
        for (int p = 0; p < RECP; ++p) recraw[p] = __builtin_amdgcn_raw_buffer_load_b32(rr, (p * THREADS + tid) * 4, 0, 0);
        const Rsrc vr = rows_rsrc<ESZ>(a.v, first * a.ld_v + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_v, a.vdim);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                vraw[4 * i + r] = load_one<T>(
                    vr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(a.ld_v) * ESZ));
    };

    fetch(0);
    for (int c = 0; c < n; ++c) {
        kraw.land(Kl, tid);
        if constexpr (EMIT) qraw.land(Ql, tid);
#pragma unroll
        for (int p = 0; p < TP; ++p)
            if (p * NW + wave < kBlocks * 3) Tl[p * THREADS + tid] = traw[p];
#pragma unroll
        for (int p = 0; p < RECP; ++p) reinterpret_cast<uint32_t*>(rec)[p * THREADS + tid] = recraw[p];
        lds_barrier();
        float vals[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) vals[i] = one_value<T>(vraw[i]);
        if (c + 1 < n) fetch(c + 1);

        const uint64_t starts = uniform(rec->starts), bad = uniform(rec->bad);
        const int first_start = starts ? __builtin_ctzll(starts) : C;
        const int rows = rows_of(c);
        if (a.states) store_state(a.states + (bh * n + c) * cells);
        __builtin_amdgcn_sched_barrier(0);

        // K S, Q S and K Q^T: one walk over the channels
        f32x4 ks[4], qs[4], pt[4][4];   // pt[is][it]: rows (tokens s) of tile is, columns (tokens t) of tile it
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ks[i] = qs[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) pt[i][j] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            const Frag<3> sf = split(S[2 * j], S[2 * j + 1]);
            Frag<N> kf[4], qf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kf[i] = rows_frag<N, ROW>(Kl, 16 * i + m, 32 * j + 8 * g);
                if constexpr (EMIT) qf[i] = rows_frag<N, ROW>(Ql, 16 * i + m, 32 * j + 8 * g);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) product<3>(ks[i], kf[i], sf);
            if constexpr (EMIT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) product<OUT>(qs[i], qf[i], sf);
#pragma unroll
                for (int is = 0; is < 4; ++is)
#pragma unroll
                    for (int it = is; it < 4; ++it) product<OUT>(pt[is][it], kf[is], qf[it]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);

        // R
        f32x4 R[4];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool old = 16 * i + 4 * g + r < first_start;
                R[i][r] = vals[4 * i + r] - keep_if(old, into[r] * ks[i][r]);
                odd |= not_finite(R[i][r]);
            }
        }
        // Values that are not finite: the rows from there to the document's end take no part, and give NaN
        uint64_t lost = 0;
        const bool any_lost = bad != 0 || __ballot(odd) != 0;
        if (any_lost) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    lost |= uint64_t(not_finite(R[i][r])) << (16 * i + 4 * g + r);
            lost |= __shfl_xor(lost, 16);
            lost |= __shfl_xor(lost, 32);
            lost = smear(lost | bad, starts);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) R[i][r] = keep_if(!((lost >> (16 * i + 4 * g + r)) & 1), R[i][r]);
        }

        // U = beta T R
        f32x4 U[4];
        {
            const Frag<3> rf[2] = {split(R[0], R[1]), split(R[2], R[3])};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j <= i / 2; ++j) {
                    Frag<3> tf;
#pragma unroll
                    for (int p = 0; p < 3; ++p) tf.p[p] = Tl[(low_block(i, j) * 3 + p) * 64 + lane];
                    product<3>(U[i], tf, rf[j]);
                }
                const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) U[i][r] *= beta[r];
            }
        }
        __builtin_amdgcn_sched_barrier(0);

        // O
        if constexpr (EMIT) {
            f32x4 O[4], sh[4], sl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sh[i] = four(rec->hi + 16 * i + 4 * g);
                sl[i] = four(rec->lo + 16 * i + 4 * g);
            }
            const Frag<OUT> uf[2] = {split_out<OUT>(U[0], U[1]), split_out<OUT>(U[2], U[3])};
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const f32x4 into = four(rec->into + 16 * it + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    O[it][r] = keep_if(16 * it + 4 * g + r < first_start, a.scale * into[r] * qs[it][r]);
                const int t = 16 * it + m, from = doc_first(starts, t);
                const float th = rec->hi[t], tl = rec->lo[t];
                f32x4 P[4];
#pragma unroll
                for (int is = 0; is <= (it | 1); ++is)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = 16 * is + 4 * g + r;
                        const float d = exp2_fast((th - sh[is][r]) + (tl - sl[is][r]));
                        P[is][r] = is <= it ? keep_if(s <= t && s >= from, a.scale * pt[is < it ? is : it][it][r] * d) : 0.0f;
                    }
#pragma unroll
                for (int j = 0; j <= it / 2; ++j) product<OUT>(O[it], split_out<OUT>(P[2 * j], P[2 * j + 1]), uf[j]);
            }
            if (any_lost) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        O[i][r] = nan_if((lost >> (16 * i + 4 * g + r)) & 1, O[i][r]);
            }
            const int64_t ldo = static_cast<int64_t>(a.vheads) * a.vdim;
            const Rsrc orr = rows_rsrc<ESZ>(a.out, (b * a.seqlen + static_cast<int64_t>(c) * C) * ldo + hv * a.vdim, rows,
                                            ldo, a.vdim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store_one<T>(orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(ldo) * ESZ), O[i][r]);
        }
        __builtin_amdgcn_sched_barrier(0);

        // S
        const float keep = rec->keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 outof = four(rec->outof + 16 * i + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[i][r] *= outof[r];
        }
        const Frag<3> uf[2] = {split(U[0], U[1]), split(U[2], U[3])};
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = keep_if(starts == 0, keep * S[i][r]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i) {
                Frag<N> kf = cols_frag<N, ROW>(Kl, j, g, m, state_cols4(i, m));
                if (bad != 0) drop_rows<N>(kf, j, g, bad);   // keys that are not finite: their rows of U are 0
                product<3>(S[i], kf, uf[j]);
            }
        if (any_lost) {
            const bool dead = (lost >> (rows - 1)) & 1;
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] = nan_if(dead, S[i][r]);
        }
        lds_barrier();
    }
    if (a.final_state) store_state(a.final_state + bh * cells);
}

template <typename T, int KT, int NW, bool VEC>
hipError_t launch(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NW - 1) / (16 * NW);
    const dim3 grid(static_cast<unsigned>(a.batch * a.vheads * cols));
    if (a.out)
        hipLaunchKernelGGL((fwd_kernel<T, KT, NW, VEC, true>), grid, dim3(NW * 64), 0, a.stream, a,
                           static_cast<int64_t>(delta_chunk_bytes()), cols);
    else
        hipLaunchKernelGGL((fwd_kernel<T, KT, NW, VEC, false>), grid, dim3(NW * 64), 0, a.stream, a,
                           static_cast<int64_t>(delta_chunk_bytes()), cols);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t by_width(const DeltaArgs& a) {
    return a.kdim > 64 ? launch<T, 128, 4, VEC>(a) : launch<T, 64, 4, VEC>(a);
}

}  // namespace

hipError_t launch_delta_fwd(const DeltaArgs& a) {
    if (a.bf16) return a.vec_k ? by_width<bf16_t, true>(a) : by_width<bf16_t, false>(a);
    return a.vec_k ? by_width<float, true>(a) : by_width<float, false>(a);
}

}  // namespace mamba
