// Gated delta rule, forward: the chunks of a row in order (delta_prepare.hip has
// solved each chunk's triangle T and formed P = scale D o Q K^T).
//
//     R = V - exp(gamma) K S,  U = beta T R,
//     O = scale exp(gamma) Q S + P U,  S <- exp(gamma_C) S + (exp(gamma_C - gamma) K)^T U.
//
// The columns of V, U, O and S do not mix, so a wave owns 16 of them for the whole
// row and keeps S (K x 16) in its accumulators; R and U go from accumulator to
// operand in place. The waves of a workgroup share what has no columns: K, Q, T and P in LDS, the next chunk's on
// their way while this one is worked off.
// Without an output the same walk forms the states alone, for the backward.
//
// A product of float32 operands, each in three bf16 pieces whose sum it is, takes the six products of pieces that reach
// 2^-22 of it; a bf16 operand is one piece.
//
// Bound by the chain of a row's chunks: 132 matrix products and some 400 vector instructions one behind the other
// in a wave, with too few rows, heads and groups of columns to fill the card.  64K tokens x 40 heads of
// 128 x 128: 2.95 ms, 1024 chunks of 7000 cycles (2.7 ms where what only reaches an output had two pieces, which is off by
// 1e-5 of the terms in the outputs of terms that cancel); reading and writing it takes 0.5 ms.
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

// float32, and bf16 that is not in whole 16-byte pieces.  (3 x 1001 tokens, 6 heads of 100 x 75 in float32: 157 us.)
template <typename T, int KT, int NW, bool VEC, bool EMIT>
__global__ __launch_bounds__(NW * 64, 1) void fwd_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int N = kPieces<T>, ESZ = sizeof(T), STEPS = KT / 32, THREADS = NW * 64;
    using KQ = Tile<T, KT, THREADS, VEC>;
    constexpr int TKB = kBlocks * 3, PKB = EMIT ? kBlocks * 3 : 0;
    constexpr int RKB = 2;                   // a record's 1304 bytes
    constexpr size_t BUF = (TKB + PKB + RKB) * 1024 + (EMIT ? 2 : 1) * KQ::kBytes;
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
    const uint32_t state_lane = v_in ? v * 4 : kPast, value_lane = v_in ? v * ESZ : kPast;
    auto state_off = [&](int i, int r) { return state_lane + static_cast<uint32_t>(state_row(i, g, r) * a.vdim * 4); };
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
    auto rows_of = [&](int c) {
        const int64_t left = a.seqlen - static_cast<int64_t>(c) * C;
        return static_cast<int>(left < C ? left : C);
    };

    KQ kraw, qraw;   // the next chunk in registers
    u32x4 braw[(TKB + PKB + RKB + NW - 1) / NW];
    uint32_t vraw[16];
    auto fetch = [&](int c) {
        const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C, id = bh * n + c;
        const int rows = rows_of(c);
        const Rsrc kr = rows_rsrc<ESZ>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_k, a.kpitch);
        const Rsrc qr = rows_rsrc<ESZ>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_q, a.kpitch);
        const Rsrc tr = rsrc(a.solve + id * kSolveBytes, kSolveBytes);
        const Rsrc pr = rsrc(a.pairs + (EMIT ? id * kSolveBytes : 0), EMIT ? kSolveBytes : 0);
        const Rsrc rr = rsrc(a.chunks + id * rec_bytes, sizeof(ChunkRec));
        kraw.fetch(kr, a.ld_k, a.kpitch, tid);
        if constexpr (EMIT) qraw.fetch(qr, a.ld_q, a.kpitch, tid);
#pragma unroll
        for (int p = 0; p < (TKB + PKB + RKB + NW - 1) / NW; ++p) {
            const int kb = p * NW + wave;
            const int at = ((kb < TKB ? kb : kb < TKB + PKB ? kb - TKB : kb - TKB - PKB) * 64 + lane) * 16;
            braw[p] = __builtin_amdgcn_raw_buffer_load_b128(kb < TKB ? tr : kb < TKB + PKB ? pr : rr, at, 0, 0);
        }
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
        const u32x4* Tl = reinterpret_cast<const u32x4*>(buf);                     // [kBlocks][3][64]
        const u32x4* Pl = Tl + TKB * 64;                                           // [kBlocks][3][64]
        const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buf + (TKB + PKB) * 1024);
        uint16_t* Kl = reinterpret_cast<uint16_t*>(buf + (TKB + PKB + RKB) * 1024);   // [N][C][KT]
        uint16_t* Ql = Kl + N * C * KT;
        kraw.land(Kl, tid);
        if constexpr (EMIT) qraw.land(Ql, tid);
#pragma unroll
        for (int p = 0; p < (TKB + PKB + RKB + NW - 1) / NW; ++p)
            if (p * NW + wave < TKB + PKB + RKB) reinterpret_cast<u32x4*>(buf)[p * THREADS + tid] = braw[p];
        float vals[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) vals[i] = one_value<T>(vraw[i]);
        lds_barrier();
        if (c + 1 < n) fetch(c + 1);

        const uint64_t starts = uniform(rec->starts), bad = uniform(rec->bad);
        const int first_start = starts ? __builtin_ctzll(starts) : C;
        const int rows = rows_of(c);
        if (a.states) store_state(a.states + (bh * n + c) * cells);

        // K S and Q S: one walk over the channels
        f32x4 ks[4], qs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = qs[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            const Frag<3> sf = split(S[2 * j], S[2 * j + 1]);
            Frag<N> kf[4], qf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kf[i] = rows_frag<N, KT>(Kl, 16 * i + m, 4 * j + g);
                if constexpr (EMIT) qf[i] = rows_frag<N, KT>(Ql, 16 * i + m, 4 * j + g);
            }
            products<3, 4>(ks, kf, sf);
            if constexpr (EMIT) products<3, 4>(qs, qf, sf);
        }

        // R
        f32x4 R[4];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 into = four(rec->into + 16 * i + 4 * g);
            if (starts == 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r) R[i][r] = __builtin_fmaf(-into[r], ks[i][r], vals[4 * i + r]);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    R[i][r] = vals[4 * i + r] - keep_if(16 * i + 4 * g + r < first_start, into[r] * ks[i][r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) odd |= not_finite(R[i][r]);
        }
        // Values that are not finite: the rows from there to the document's end take no part, and give NaN
        uint64_t lost = 0;
        bool any_lost = bad != 0 || __ballot(odd) != 0;
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

        // U = beta T R, a piece of T at a time, the smallest first
        f32x4 U[4];
        {
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] = f32x4{0, 0, 0, 0};
            const Frag<3> rf[2] = {split_values(R[0], R[1]), split_values(R[2], R[3])};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 2; p >= 0; --p)
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q)
#pragma unroll
                        for (int i = 2 * j; i < 4; ++i) U[i] = mfma(Tl[(low_block(i, j) * 3 + p) * 64 + lane], rf[j].p[q], U[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 beta = four(rec->beta + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) U[i][r] *= beta[r];
            }
        }
        // Nor has a U past float32's range: 0 times it is NaN, for other documents and earlier tokens
        float check = 0.0f;   // stays 0 as long as everything is finite
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) check = __builtin_fmaf(U[i][r], 0.0f, check);
        if (__ballot(not_finite(check)) != 0) {
            any_lost = true;
            lost = lost_with(lost, U, starts, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] = without_rows(U[i], lost, i, g);
        }

        // O
        if constexpr (EMIT) {
            f32x4 O[4];
            Frag<3> pf[4];
            auto pairs = [&](int i, int j) {
                Frag<3> f;
#pragma unroll
                for (int p = 0; p < 3; ++p) f.p[p] = Pl[(low_block(i, j) * 3 + p) * 64 + lane];
                return f;
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pf[i] = pairs(i, 0);
                const f32x4 into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    O[i][r] = keep_if(16 * i + 4 * g + r < first_start, a.scale * into[r] * qs[i][r]);
            }
            products<3, 4>(O, pf, split(U[0], U[1]));
#pragma unroll
            for (int i = 2; i < 4; ++i) pf[i] = pairs(i, 1);
            products<3, 2>(O + 2, pf + 2, split(U[2], U[3]));
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
                    store_one<T>(orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(ldo) * ESZ),
                                 O[i][r]);
        }

        // S
        const float keep = rec->keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 outof = four(rec->outof + 16 * i + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[i][r] *= outof[r];
        }
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = keep_if(starts == 0, keep * S[i][r]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const Frag<3> uf = split(U[2 * j], U[2 * j + 1]);
#pragma unroll
            for (int i0 = 0; i0 < 2 * STEPS; i0 += 4) {
                Frag<N> kf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kf[i] = cols_frag<N, KT>(Kl, j, g, m, state_cols4(i0 + i, m));
                if (bad != 0) {   // keys that are not finite: their rows of U are 0
#pragma unroll
                    for (int i = 0; i < 4; ++i) drop_rows<N>(kf[i], j, g, bad);
                }
                products<3, 4>(S + i0, kf, uf);
            }
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

// The same for bf16 in whole 16-byte pieces, two waves for every 16 columns: one walks the chain
// S -> R -> U -> S, which is what a row's time is, the other follows it by half a chunk with
// everything that does not lead back to S: the outputs, from S and U as the first leaves them in LDS,
// and all loads, straight to LDS.  (One wave doing both, four to a workgroup: more than twice as long.)
//
// Chunk c:  barrier;  A: the chain forms K S and R; the other loads K and T of c + 1 and finishes O of c - 1;
//           barrier;  B: the chain forms U, then S;   the other loads V and Q of c + 1 and P of c and forms Q S.
// NP = 4, whose LDS has no room for a second T and Q: those of c + 1 are loaded when U and Q S of c are there, behind a
// third barrier.  (Loaded in A of their own chunk, and waited for there: 8 x 2048 tokens, 12 heads of 128 x 128, a seventh more.)
//
// A workgroup has NP such pairs, for as many 16 columns of one head, a chain and a follower on a SIMD with NP = 4: a wave
// alone issues a vector instruction every 8 cycles, two together twice as many.
template <int NP> constexpr int kBuffers = NP == 2 ? 2 : 1;   // of T and Q
template <int KT, int NP, bool EMIT>
constexpr int kPairsLds = 2 * C * KT * 2 + kBuffers<NP> * kBlocks * 3 * 1024 + 2 * 2048 + NP * (2048 + 512) +
                          (EMIT ? kBuffers<NP> * C * KT * 2 + kBlocks * 3 * 1024 + NP * (KT / 32 * 2048 + 4096) : 0);
// (LDS given at the launch, and two waves a SIMD asked for: one workgroup fills a CU either way, but where the compiler
// sees that, it takes 512 registers, keeps sums in the upper 256 and moves them, 8 cycles each.)
template <int KT, int NP, bool EMIT, bool SAVE>
__global__ __launch_bounds__(NP * 128, 2) void fwd_pairs_kernel(DeltaArgs a, int64_t rec_bytes, int cols) {
    constexpr int STEPS = KT / 32;
    constexpr int TILE = C * KT * 2, TRI = kBlocks * 3 * 1024, REC = 2048;
    constexpr int BUFFERS = kBuffers<NP>;
    extern __shared__ __align__(16) char smem[];
    char* const Kb = smem;                       // [2] K
    char* const Rb = Kb + 2 * TILE;              // [2] record
    char* const Tb = Rb + 2 * REC;               // [BUFFERS] triangle
    char* const Vb = Tb + BUFFERS * TRI;                   // a lane's 16 values, packed
    char* const Lb = Vb + NP * 64 * 32;          // a lane's lost rows
    char* const Qb = Lb + NP * 64 * 8;           // [BUFFERS] Q
    char* const Pb = Qb + BUFFERS * TILE;                // P
    char* const Sb = Pb + TRI;                   // S
    char* const Ub = Sb + NP * STEPS * 2048;     // U
    static_assert(kPairsLds<KT, NP, EMIT> == 2 * (TILE + REC) + BUFFERS * TRI + NP * (64 * 32 + 64 * 8) +
                                                 (EMIT ? BUFFERS * TILE + TRI + NP * (STEPS * 2048 + 4096) : 0));

    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), pair = wave & (NP - 1);
    // workgroups of one head on one XCD (they are dealt out to the 8 in turn), which read its K, Q, T and P
    const int64_t bh = quotient(blockIdx.x, 8 * cols) * 8 + (blockIdx.x & 7);
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
    auto buffer2 = [&](char* first, int size, int c) { return BUFFERS == 2 ? first + (c & 1) * size : first; };

    if (wave < NP) {
        // ---- the chain
        const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;
        const uint32_t state_lane = v_in ? static_cast<uint32_t>(v * 4 + state_row(0, g, 0) * a.vdim * 4) : kPast;
        auto state_off = [&](uint32_t from, int i, int r) {
            return from + static_cast<uint32_t>(state_row(i, 0, r) * a.vdim * 4);
        };
        auto store_state = [&](float* to, const f32x4* S) {
            const Rsrc rs = rsrc(to, cells * 4);
            const uint32_t from = opaque(state_lane);   // 32 offsets would be kept in registers
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rs, state_off(from, i, r), 0, 0);
        };
        f32x4 S[2 * STEPS];
        {
            const Rsrc rs = rsrc(a.initial_state + (a.initial_state ? bh * cells : 0), a.initial_state ? cells * 4 : 0);
#pragma unroll
            for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, state_off(state_lane, i, r), 0, 0));
        }
        // S in pieces, step by step as its rows are final.  A matrix product takes 16 cycles, of which its issue is 4:
        // the vector instructions of the next splits go in between (sched_barrier), not behind.
        Frag<3> sf[STEPS];
#pragma unroll
        for (int j = 0; j < STEPS / 2; ++j) sf[j] = split(S[2 * j], S[2 * j + 1]);
        for (int c = 0; c < n; ++c) {
            const uint16_t* Kl = reinterpret_cast<const uint16_t*>(buffer(Kb, TILE, c));
            const u32x4* Tl = reinterpret_cast<const u32x4*>(buffer2(Tb, TRI, c));
            const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buffer(Rb, REC, c));
            lds_barrier();
            // A: K S, R = V - exp(gamma) K S
            const uint64_t starts_ = rec->starts, bad_ = rec->bad;
            const float keep = rec->keep;
            const u32x4* vals = reinterpret_cast<const u32x4*>(Vb + (pair * 64 + lane) * 32);
            const u32x4 v01 = vals[0], v23 = vals[1];
            f32x4 into[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) into[i] = four(rec->into + 16 * i + 4 * g);
            f32x4 R[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) R[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                if (j >= STEPS / 2) sf[j] = split(S[2 * j], S[2 * j + 1]);
                Frag<1> kf[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kf[i] = rows_frag<1, KT>(Kl, 16 * i + m, 4 * j + g);
                products<3, 4>(R, kf, sf[j]);
                if constexpr (EMIT) {
                    f32x4* to = reinterpret_cast<f32x4*>(Sb + (pair * STEPS + j) * 2048) + lane;
                    to[0] = S[2 * j];
                    to[64] = S[2 * j + 1];
                }
            }
            const uint64_t starts = uniform(starts_), bad = uniform(bad_);
            if constexpr (SAVE) store_state(a.states + (bh * n + c) * cells, S);
            f32x4 val[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = (i < 2 ? v01 : v23)[2 * (i & 1)], hi = (i < 2 ? v01 : v23)[2 * (i & 1) + 1];
                val[i] = f32x4{__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                               __uint_as_float(hi & 0xffff0000u)};
            }
            if (starts == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[i][r] = __builtin_fmaf(-into[i][r], R[i][r], val[i][r]);
            } else {
                const int first_start = __builtin_ctzll(starts);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        R[i][r] = val[i][r] - keep_if(16 * i + 4 * g + r < first_start, into[i][r] * R[i][r]);
            }
            float check[2] = {0.0f, 0.0f};   // stay 0 as long as everything is finite
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) check[i & 1] = __builtin_fmaf(R[i][r], 0.0f, check[i & 1]);
            // Values that are not finite: the rows from there to the document's end take no part, and give NaN
            uint64_t lost = 0;
            const bool any_lost = bad != 0 || __ballot(not_finite(check[0] + check[1])) != 0;
            if (any_lost) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) lost |= uint64_t(not_finite(R[i][r])) << (16 * i + 4 * g + r);
                lost |= __shfl_xor(lost, 16);
                lost |= __shfl_xor(lost, 32);
                lost = smear(lost | bad, starts);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) R[i][r] = keep_if(!((lost >> (16 * i + 4 * g + r)) & 1), R[i][r]);
            }
            lds_barrier();
            // B: U = beta T R, then S.  PLAIN: one document, everything finite
            auto rest = [&](auto plain) {
                constexpr bool PLAIN = decltype(plain)::value;
                const int last_start = !PLAIN && starts != 0 ? 63 - __builtin_clzll(starts) : 0;
                auto triangle = [&](int i, int j, int p) { return Tl[(low_block(i, j) * 3 + p) * 64 + lane]; };
                auto keys = [&](Frag<1>* kf, int i0, int j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        kf[i] = cols_frag<1, KT>(Kl, j, g, m, state_cols4(i0 + i, m));
                        if (!PLAIN) drop_rows<1>(kf[i], j, g, bad);   // keys that are not finite: their rows of U are 0
                    }
                };
                f32x4 U[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) U[i] = f32x4{0, 0, 0, 0};
                // a piece of T at a time, the smallest first
                const Frag<3> rf0 = split_values(R[0], R[1]);
#pragma unroll
                for (int p = 2; p >= 0; --p) {
                    u32x4 tf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tf[i] = triangle(i, 0, p);
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) U[i] = mfma(tf[i], rf0.p[q], U[i]);
                }
                const Frag<3> rf1 = split_values(R[2], R[3]);
#pragma unroll
                for (int p = 2; p >= 0; --p) {
                    const u32x4 t2 = triangle(2, 1, p), t3 = triangle(3, 1, p);
#pragma unroll
                    for (int q = 2 - p; q >= 0; --q) {
                        U[2] = mfma(t2, rf1.p[q], U[2]);
                        U[3] = mfma(t3, rf1.p[q], U[3]);
                    }
                }
                if constexpr (BUFFERS == 1) lds_barrier();   // T has been read
#pragma unroll
                for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[i][r] = PLAIN ? S[i][r] * keep : keep_if(starts == 0, S[i][r] * keep);
                Frag<1> kf[2][4];
                keys(kf[0], 0, 0);
                keys(kf[1], 0, 1);
                f32x4 beta[4], outof[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    beta[i] = four(rec->beta + 16 * i + 4 * g);
                    outof[i] = four(rec->outof + 16 * i + 4 * g);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) U[i][r] *= beta[i][r];
                    if constexpr (EMIT) *reinterpret_cast<f32x4*>(Ub + ((pair * 4 + i) * 64 + lane) * 16) = U[i];
#pragma unroll
                    for (int r = 0; r < 4; ++r)   // (0 times what has passed float32's range would be NaN)
                        U[i][r] = PLAIN ? U[i][r] * outof[i][r] : keep_if(16 * i + 4 * g + r >= last_start, U[i][r] * outof[i][r]);
                }
                Frag<3> uf[2];
                uf[0] = split(U[0], U[1]);
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
                    step(S, kf[0], uf[0], 3 * k);
                    cut(uf[1], U[2], U[3], k);
                }
                if constexpr (STEPS == 4) {
                    keys(kg[0], 4, 0);
                    keys(kg[1], 4, 1);
                }
                __builtin_amdgcn_sched_barrier(0);
                products<3, 4>(S, kf[1], uf[1]);
                const bool dead = !PLAIN && ((lost >> (rows_of(c) - 1)) & 1);
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
                        step(S + 4, kg[k / 4], uf[k / 4], 3 * (k % 4));
                        cut(sf[k / 4], S[k / 4 * 2], S[k / 4 * 2 + 1], k % 4);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    end(4);
                } else {
                    sf[0] = split(S[0], S[1]);
                }
            };
            if (any_lost || starts != 0) rest(std::false_type{});
            else rest(std::true_type{});
            if constexpr (EMIT) *reinterpret_cast<uint64_t*>(Lb + (pair * 64 + lane) * 8) = lost;
        }
        lds_barrier();
        if (a.final_state) store_state(a.final_state + bh * cells, S);
    } else {
        // ---- loads and outputs
        const uint32_t value_lane = v_in ? v * 2 : kPast;
        uint32_t vraw[16];
        auto fetch_keys = [&](int c) {
            const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C;
            const Rsrc kr = rows_rsrc<2>(a.k, first * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows_of(c), a.ld_k, a.kpitch);
            rows_to_lds<KT, NP>(reinterpret_cast<uint16_t*>(buffer(Kb, TILE, c)), kr, a.ld_k, a.kpitch, pair, lane);
        };
        auto fetch_triangle = [&](int c) {
            block_to_lds<kBlocks * 3, NP>(buffer2(Tb, TRI, c), rsrc(a.solve + (bh * n + c) * kSolveBytes, kSolveBytes), pair,
                                          lane);
        };
        auto fetch_values = [&](int c) {
            const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C;
            const Rsrc vr = rows_rsrc<2>(a.v, first * a.ld_v + static_cast<int64_t>(hv) * a.vdim, rows_of(c), a.ld_v, a.vdim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    vraw[4 * i + r] = load_one<bf16_t>(
                        vr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(a.ld_v) * 2));
            block_to_lds<2, NP>(buffer(Rb, REC, c), rsrc(a.chunks + (bh * n + c) * rec_bytes, sizeof(ChunkRec)), pair, lane);
        };
        auto queries = [&](int c) { return reinterpret_cast<uint16_t*>(buffer2(Qb, TILE, c)); };
        auto fetch_queries = [&](int c) {
            const int64_t first = b * a.seqlen + static_cast<int64_t>(c) * C;
            const Rsrc qr = rows_rsrc<2>(a.q, first * a.ld_q + static_cast<int64_t>(hk) * a.kpitch, rows_of(c), a.ld_q, a.kpitch);
            rows_to_lds<KT, NP>(queries(c), qr, a.ld_q, a.kpitch, pair, lane);
        };
        auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
        auto put_values = [&] {
            u32x4* to = reinterpret_cast<u32x4*>(Vb + (pair * 64 + lane) * 32);
            u32x4 w[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = vraw[2 * i] | (vraw[2 * i + 1] << 16);
            to[0] = w[0];
            to[1] = w[1];
        };
        fetch_values(0);
        fetch_keys(0);
        fetch_triangle(0);
        if constexpr (EMIT) fetch_queries(0);
        put_values();
        landed();
        f32x4 O[4];
        auto outputs = [&](int c) {   // from Q S in O
            const ChunkRec* rec = reinterpret_cast<const ChunkRec*>(buffer(Rb, REC, c));
            const uint64_t starts = uniform(rec->starts);
            const int first_start = starts ? __builtin_ctzll(starts) : C;
            const u32x4* Pl = reinterpret_cast<const u32x4*>(Pb);
            const f32x4* Ul = reinterpret_cast<const f32x4*>(Ub + pair * 4096);
            f32x4 qs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 into = four(rec->into + 16 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    qs[i][r] = keep_if(16 * i + 4 * g + r < first_start, a.scale * into[r] * O[i][r]);
            }
            auto weigh = [&](auto value) {
                Frag<3> pf[4];
                auto pairs = [&](int i, int j) {
                    Frag<3> f;
#pragma unroll
                    for (int p = 0; p < 3; ++p) f.p[p] = Pl[(low_block(i, j) * 3 + p) * 64 + lane];
                    return f;
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pf[i] = pairs(i, 0);
                    O[i] = qs[i];
                }
                products<3, 4>(O, pf, split(value(0), value(1)));
#pragma unroll
                for (int i = 2; i < 4; ++i) pf[i] = pairs(i, 1);
                products<3, 2>(O + 2, pf + 2, split(value(2), value(3)));
            };
            weigh([&](int i) { return Ul[i * 64 + lane]; });
            // A U past float32's range has no part in O: 0 times it is NaN, for other documents and earlier tokens, and so
            // for all tokens of the last tile, of which one tells. (All 16 of a lane's U looked at: 64K tokens, 40 heads 3.70 ms.)
            uint64_t lost = *reinterpret_cast<const uint64_t*>(Lb + (pair * 64 + lane) * 8);
            if (__ballot(not_finite(O[3][0])) != 0) {
                asm volatile("" ::: "memory");   // (loads from LDS once more, not kept for this)
                const f32x4 U[4] = {Ul[lane], Ul[64 + lane], Ul[128 + lane], Ul[192 + lane]};
                lost = lost_with(lost, U, starts, g);
                asm volatile("" ::: "memory");
                weigh([&](int i) { return without_rows(Ul[i * 64 + lane], lost, i, g); });
            }
            if (__ballot(lost != 0) != 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[i][r] = nan_if((lost >> (16 * i + 4 * g + r)) & 1, O[i][r]);
            }
            const int64_t ldo = static_cast<int64_t>(a.vheads) * a.vdim;
            const Rsrc orr = rows_rsrc<2>(a.out, (b * a.seqlen + static_cast<int64_t>(c) * C) * ldo + hv * a.vdim, rows_of(c),
                                          ldo, a.vdim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store_one<bf16_t>(orr, value_lane + static_cast<uint32_t>((16 * i + 4 * g + r) * static_cast<int>(ldo) * 2),
                                      O[i][r]);
        };
        for (int c = 0; c < n; ++c) {
            lds_barrier();
            // A
            if (c + 1 < n) {
                fetch_keys(c + 1);
                if constexpr (BUFFERS == 2) fetch_triangle(c + 1);
            }
            if constexpr (EMIT) {
                if (c > 0) outputs(c - 1);
            }
            lds_barrier();
            // B
            if (c + 1 < n) fetch_values(c + 1);
            if constexpr (EMIT) {
                if (BUFFERS == 2 && c + 1 < n) fetch_queries(c + 1);
                block_to_lds<kBlocks * 3, NP>(Pb, rsrc(a.pairs + (bh * n + c) * kSolveBytes, kSolveBytes), pair, lane);
                const uint16_t* Ql = queries(c);
#pragma unroll
                for (int i = 0; i < 4; ++i) O[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < STEPS; ++j) {
                    const f32x4* from = reinterpret_cast<const f32x4*>(Sb + (pair * STEPS + j) * 2048) + lane;
                    const Frag<3> sf = split(from[0], from[64]);
                    Frag<1> qf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[i] = rows_frag<1, KT>(Ql, 16 * i + m, 4 * j + g);
                    products<3, 4>(O, qf, sf);
                }
            }
            if constexpr (BUFFERS == 1) {
                lds_barrier();
                if (c + 1 < n) {
                    fetch_triangle(c + 1);
                    if constexpr (EMIT) fetch_queries(c + 1);
                }
            }
            if (c + 1 < n) put_values();
            landed();
        }
        lds_barrier();
        if constexpr (EMIT) outputs(n - 1);
    }
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

template <int KT, int NP, bool EMIT, bool SAVE>
hipError_t launch_pairs(const DeltaArgs& a) {
    const int cols = (a.vdim + 16 * NP - 1) / (16 * NP);
    hipLaunchKernelGGL((fwd_pairs_kernel<KT, NP, EMIT, SAVE>), dim3(static_cast<unsigned>((a.batch * a.vheads + 7) / 8 * 8 * cols)),
                       dim3(NP * 128), (kPairsLds<KT, NP, EMIT>), a.stream, a, static_cast<int64_t>(delta_chunk_bytes()), cols);
    return hipGetLastError();
}
template <int KT, int NP>
hipError_t pairs_by_outputs(const DeltaArgs& a) {
    if (!a.out) return launch_pairs<KT, NP, false, true>(a);
    return a.states ? launch_pairs<KT, NP, true, true>(a) : launch_pairs<KT, NP, true, false>(a);
}
template <int KT>
hipError_t pairs_by_columns(const DeltaArgs& a) {
    return wide_groups(a) ? pairs_by_outputs<KT, 4>(a) : pairs_by_outputs<KT, 2>(a);
}

template <typename T, bool VEC>
hipError_t by_width(const DeltaArgs& a) {
    return a.kdim > 64 ? launch<T, 128, 4, VEC>(a) : launch<T, 64, 4, VEC>(a);
}

}  // namespace

hipError_t launch_delta_fwd(const DeltaArgs& a) {
    if (a.bf16 && a.vec_k) return a.kdim > 64 ? pairs_by_columns<128>(a) : pairs_by_columns<64>(a);
    if (a.bf16) return by_width<bf16_t, false>(a);
    return a.vec_k ? by_width<float, true>(a) : by_width<float, false>(a);
}

}  // namespace mamba
