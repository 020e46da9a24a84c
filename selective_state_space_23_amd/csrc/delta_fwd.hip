// Gated delta rule, forward: the chunks of a row in order (delta_prepare.hip has
// solved each chunk's triangle T).
//
//     R = beta (V - exp(gamma) K S),  U = T R,
//     O = scale (exp(gamma) Q S + (D o Q K^T) U),  S <- exp(gamma_C) S + (exp(gamma_C - gamma) K)^T U.
//
// The columns of V, U, O and S do not mix, so a wave owns 16 of them for the whole
// row and keeps S (K x 16) in its accumulators; R and U go from accumulator to
// operand in place. The waves of a workgroup share what has no columns: K, Q and T in LDS.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

template <typename T, int KT, int NW, bool VEC>
__global__ __launch_bounds__(NW * 64, 1) void fwd_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32, THREADS = NW * 64;
    constexpr int ROW = KT + 8;              // bf16 of a row in LDS: 16-byte pieces of 16 rows meet no bank twice
    constexpr int OUT = N == 1 ? 2 : 3;      // pieces that reach an output
    constexpr int VECS = C * KT / 8;         // pieces of eight channels of a tile
    constexpr int PER = VECS / THREADS;
    constexpr int RECW = sizeof(ChunkRec) / 4;
    constexpr size_t LDS = size_t(2) * N * C * ROW * 2 + kSolveBytes + (RECW + THREADS - 1) / THREADS * THREADS * 4;
    __shared__ __align__(16) char smem[LDS];
    uint16_t* Kl = reinterpret_cast<uint16_t*>(smem);            // [N][C][ROW]
    uint16_t* Ql = Kl + N * C * ROW;
    u32x4* Tl = reinterpret_cast<u32x4*>(Ql + N * C * ROW);      // [kBlocks][3][64]
    ChunkRec* rec = reinterpret_cast<ChunkRec*>(Tl + kBlocks * 3 * 64);

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bh = blockIdx.x / cols;
    const int col = static_cast<int>(blockIdx.x % cols);
    const int hv = static_cast<int>(bh % a.vheads), hk = hv / (a.vheads / a.kheads);
    const int64_t b = bh / a.vheads;
    const int v = (col * NW + wave) * 16 + m;
    const bool v_in = v < a.vdim;
    const int n = a.nchunks;

    f32x4 S[2 * STEPS];   // rows 32 (i / 2) + 8 g + 4 (i % 2) + r: an operand reads 8 consecutive channels of K
    const int64_t state_at = bh * a.kdim * a.vdim;
    {
        const Rsrc rs = rsrc(a.initial_state + (a.initial_state ? state_at : 0),
                             a.initial_state ? int64_t(a.kdim) * a.vdim * 4 : 0);
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int kd = 32 * (i / 2) + 8 * g + 4 * (i % 2) + r;
                S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    rs, v_in && kd < a.kdim ? (kd * a.vdim + v) * 4 : kPast, 0, 0));
            }
    }

    Eight<T, VEC> kraw[PER], qraw[PER];
    u32x4 traw[(kBlocks * 3 + NW - 1) / NW];
    uint32_t vraw[16], recraw[(RECW + THREADS - 1) / THREADS];
    auto fetch = [&](int c) {
        const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C;
        const int rows = static_cast<int>(a.seqlen - static_cast<int64_t>(c) * C < C ? a.seqlen - static_cast<int64_t>(c) * C : C);
        const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_k, a.kdim);
        const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kdim, rows, a.ld_q, a.kdim);
        const Rsrc vr = rows_rsrc<ESZ>(a.v, first * a.ld_v + static_cast<int64_t>(hv) * a.vdim, rows, a.ld_v, a.vdim);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = p * THREADS + tid, t = x / (KT / 8), ch = x % (KT / 8) * 8;
            kraw[p].load(kr, static_cast<uint32_t>(t * a.ld_k * ESZ), ch, a.kdim);
            qraw[p].load(qr, static_cast<uint32_t>(t * a.ld_q * ESZ), ch, a.kdim);
        }
        const int64_t id = bh * n + c;
        const Rsrc tr = rsrc(a.solve + id * kSolveBytes, kSolveBytes);
#pragma unroll
        for (int p = 0; p < (kBlocks * 3 + NW - 1) / NW; ++p)
            traw[p] = __builtin_amdgcn_raw_buffer_load_b128(tr, (p * THREADS + tid) * 16, 0, 0);
        const Rsrc rr = rsrc(a.chunks + id * rec_bytes, RECW * 4);
#pragma unroll
        for (int p = 0; p < (RECW + THREADS - 1) / THREADS; ++p)
            recraw[p] = __builtin_amdgcn_raw_buffer_load_b32(rr, (p * THREADS + tid) * 4, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                vraw[4 * i + r] = load_one<T>(
                    vr, v_in ? static_cast<uint32_t>(((16 * i + 4 * g + r) * a.ld_v + v) * ESZ) : kPast);
    };
    auto land = [&]() {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = p * THREADS + tid, t = x / (KT / 8), ch = x % (KT / 8) * 8;
            const Frag<N> fk = kraw[p].frag(), fq = qraw[p].frag();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                *reinterpret_cast<u32x4*>(Kl + (i * C + t) * ROW + ch) = fk.p[i];
                *reinterpret_cast<u32x4*>(Ql + (i * C + t) * ROW + ch) = fq.p[i];
            }
        }
#pragma unroll
        for (int p = 0; p < (kBlocks * 3 + NW - 1) / NW; ++p)
            if (p * NW + wave < kBlocks * 3) Tl[p * THREADS + tid] = traw[p];
        uint32_t* rw = reinterpret_cast<uint32_t*>(rec);
#pragma unroll
        for (int p = 0; p < (RECW + THREADS - 1) / THREADS; ++p) rw[p * THREADS + tid] = recraw[p];   // room for whole waves
    };

    fetch(0);
    for (int c = 0; c < n; ++c) {
        land();
        lds_barrier();
        float vals[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) vals[i] = one_value<T>(vraw[i]);
        if (c + 1 < n) fetch(c + 1);

        const uint64_t starts = __builtin_bit_cast(uint64_t, u32x2{
            static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(rec->starts))),
            static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(rec->starts >> 32)))});
        const uint64_t bad = __builtin_bit_cast(uint64_t, u32x2{
            static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(rec->bad))),
            static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(rec->bad >> 32)))});
        const int first_start = starts ? __builtin_ctzll(starts) : C;
        const int rows = static_cast<int>(a.seqlen - static_cast<int64_t>(c) * C < C ? a.seqlen - static_cast<int64_t>(c) * C : C);

        if (a.states) {
            const Rsrc rs = rsrc(a.states + (bh * n + c) * a.kdim * a.vdim, int64_t(a.kdim) * a.vdim * 4);
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kd = 32 * (i / 2) + 8 * g + 4 * (i % 2) + r;
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rs,
                                                          v_in && kd < a.kdim ? (kd * a.vdim + v) * 4 : kPast, 0, 0);
                }
        }

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
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int p = 0; p < N; ++p) {
                    kf[i].p[p] = *reinterpret_cast<const u32x4*>(Kl + (p * C + 16 * i + m) * ROW + 32 * j + 8 * g);
                    qf[i].p[p] = *reinterpret_cast<const u32x4*>(Ql + (p * C + 16 * i + m) * ROW + 32 * j + 8 * g);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) product<3>(ks[i], kf[i], sf);
#pragma unroll
            for (int i = 0; i < 4; ++i) product<OUT>(qs[i], qf[i], sf);
#pragma unroll
            for (int is = 0; is < 4; ++is)
#pragma unroll
                for (int it = is; it < 4; ++it) product<OUT>(pt[is][it], kf[is], qf[it]);
        }

        __builtin_amdgcn_sched_barrier(0);
        // R
        f32x4 R[4];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 into = four(rec->into + 16 * i + 4 * g), beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool old = 16 * i + 4 * g + r < first_start;
                R[i][r] = beta[r] * (old ? __builtin_fmaf(-into[r], ks[i][r], vals[4 * i + r]) : vals[4 * i + r]);
                odd = odd || not_finite(R[i][r]);
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
                    lost |= not_finite(R[i][r]) ? uint64_t(1) << (16 * i + 4 * g + r) : 0;
            lost |= __shfl_xor(lost, 16);
            lost |= __shfl_xor(lost, 32);
            lost = smear(lost | bad, starts);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) R[i][r] = (lost >> (16 * i + 4 * g + r)) & 1 ? 0.0f : R[i][r];
        }

        // U = T R
        f32x4 U[4];
        {
            const Frag<3> rf[2] = {split(R[0], R[1]), split(R[2], R[3])};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j <= i / 2; ++j) {
                    const int blk = i < 2 ? i : 2 + (i - 2) * 2 + j;
                    Frag<3> tf;
#pragma unroll
                    for (int p = 0; p < 3; ++p) tf.p[p] = Tl[(blk * 3 + p) * 64 + lane];
                    product<3>(U[i], tf, rf[j]);
                }
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        // O
        f32x4 O[4];
        {
            f32x4 sh[4], sl[4];
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
                    O[it][r] = 16 * it + 4 * g + r < first_start ? a.scale * into[r] * qs[it][r] : 0.0f;
                const float th = rec->hi[16 * it + m], tl = rec->lo[16 * it + m];
                const int t = 16 * it + m;
                f32x4 P[4];
#pragma unroll
                for (int is = 0; is <= (it | 1); ++is)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = 16 * is + 4 * g + r;
                        // a start in (s, t]: bits s + 1 .. t
                        const bool on = is <= it && s <= t && ((starts >> s >> 1) & ((uint64_t(1) << (t - s)) - 1)) == 0;
                        P[is][r] = on ? a.scale * pt[is][it < is ? is : it][r] * exp2_fast((th - sh[is][r]) + (tl - sl[is][r])) : 0.0f;
                    }
#pragma unroll
                for (int j = 0; j <= it / 2; ++j) product<OUT>(O[it], split_out<OUT>(P[2 * j], P[2 * j + 1]), uf[j]);
            }
        }
        if (any_lost) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    O[i][r] = (lost >> (16 * i + 4 * g + r)) & 1 ? __builtin_nanf("") : O[i][r];
        }
        {
            const Rsrc orr = rows_rsrc<ESZ>(a.out, ((b * a.seqlen + static_cast<int64_t>(c) * C) * a.vheads + hv) * a.vdim,
                                            rows, static_cast<int64_t>(a.vheads) * a.vdim, a.vdim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store_one<T>(orr, v_in ? static_cast<uint32_t>(((16 * i + 4 * g + r) * a.vheads * a.vdim + v) * ESZ) : kPast,
                                 O[i][r]);
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
            for (int r = 0; r < 4; ++r) S[i][r] = starts != 0 ? 0.0f : keep * S[i][r];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i) {
                Frag<N> kf;
#pragma unroll
                for (int p = 0; p < N; ++p) {
                    // rows 32 j + 4 g + 0..3 and 16 further, this tile's 16 channels: lane m gets channel m
                    const uint16_t* at = Kl + (p * C + 32 * j + 4 * g + m / 4) * ROW + 32 * (i / 2) + 8 * (m % 4) + 4 * (i % 2);
                    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
                    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 16 * ROW));
                    const u32x2 xw = __builtin_bit_cast(u32x2, x), yw = __builtin_bit_cast(u32x2, y);
                    kf.p[p] = u32x4{xw[0], xw[1], yw[0], yw[1]};
                }
                if (bad != 0) {   // keys that are not finite: their rows of U are 0
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int s = 32 * j + (e < 4 ? 4 * g + e : 16 + 4 * g + e - 4);
                        const uint32_t half = e & 1 ? 0x0000ffffu : 0xffff0000u;
                        const uint32_t mask = (bad >> s) & 1 ? half : 0xffffffffu;
#pragma unroll
                        for (int p = 0; p < N; ++p) kf.p[p][e / 2] &= mask;
                    }
                }
                product<3>(S[i], kf, uf[j]);
            }
        if (any_lost) {
            const bool dead = (lost >> (rows - 1)) & 1;
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][r] = dead ? __builtin_nanf("") : S[i][r];
        }
        lds_barrier();
    }

    if (a.final_state) {
        const Rsrc rs = rsrc(a.final_state + state_at, int64_t(a.kdim) * a.vdim * 4);
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int kd = 32 * (i / 2) + 8 * g + 4 * (i % 2) + r;
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rs,
                                                      v_in && kd < a.kdim ? (kd * a.vdim + v) * 4 : kPast, 0, 0);
            }
    }
}

template <typename T, int KT, int NW, bool VEC>
hipError_t launch(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NW - 1) / (16 * NW);
    hipLaunchKernelGGL((fwd_kernel<T, KT, NW, VEC>), dim3(static_cast<unsigned>(a.batch * a.vheads * cols)),
                       dim3(NW * 64), 0, a.stream, a, static_cast<int64_t>(delta_chunk_bytes()), cols);
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
