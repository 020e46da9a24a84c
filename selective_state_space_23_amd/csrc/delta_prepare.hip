// Gated delta rule, first pass: what a chunk of 64 tokens needs besides the state
// that enters it, for every chunk at once.
//
// With gamma the running sum of log decays and D[t,s] = exp(gamma_t - gamma_s) for s <= t
// of one document, the values the chunk's tokens write obey
//     u_t = beta_t (v_t - exp(gamma_t) S_in^T k_t - sum_{s<t} D[t,s] k_t.k_s u_s),
// so with M[t,s] = D[t,s] k_t.k_s (s < t), b = diag(beta) and R = V - exp(gamma) K S_in the errors are
// E = (I + M b)^-1 R and U = b E; the backward needs (I + b M)^-T besides.  Both are unit triangles
// (dbeta_t is E_t times a gradient: dividing U_t by beta_t instead fails where that is 0).
// One wave forms K K^T on the matrix cores, solves the four 16 x 16 triangles on the diagonal by substitution (lane = column; with equal keys
// and beta = 1 the powers of A that a doubling scheme adds up reach 10^17, a substitution's
// terms stay at 1) and the blocks below them as T_ij = -T_ii sum_m A_im T_mj on the fp32 matrix
// instructions, and writes the triangle in three bf16 pieces in the order in which the later
// passes' matrix instructions read it.  The weights P = scale D o Q K^T of the values in the outputs go the
// same way (formed by every wave of the later passes instead: 440 vector instructions a chunk each).
//
// Near what memory allows: 64K tokens x 40 heads of 128, 599 us for the 3.6 GB that the counters see (a quarter more with the
// loads of each 32 channels waited for in turn).
//
// gamma is summed in float64 and kept as two floats: gamma_t - gamma_s is
// then right to float32 of itself however far the sum has run.  A decay below
// exp(-200) counts as exp(-200), which is 0 in float32: -inf is such a decay.
//
// A key, gate or decay that is not finite makes its token and the rest of
// its document bad: their rows of A are taken as 0, so nothing of them reaches
// another document's or an earlier token's row, and the later passes write NaN for them.
#include "delta_rule.hpp"

namespace mamba {

size_t delta_chunk_bytes() { return (sizeof(delta::ChunkRec) + 255) / 256 * 256; }
size_t delta_solve_bytes() { return static_cast<size_t>(delta::kSolveBytes); }

namespace {

using namespace delta;

constexpr int kRowA = 68;   // floats between two rows of A in LDS (16-byte rows, 4 banks apart)
constexpr int kLds = (C * kRowA + 4 * C) * 4;   // eight workgroups of one wave a CU, as many as their registers leave room for

__device__ __forceinline__ f32x4 mfma_f32(f32x4 a, f32x4 b, f32x4 c) {   // 16 x 16 x 16: a row m, b column m
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

struct Pad {
    const void* from[2];
    void* to[2];
    int64_t ld[2];
    int64_t pieces;
    int heads, dim, pitch;
};
// One thread a piece of eight channels, of q or (second row of workgroups) of k.
template <typename T>
__global__ __launch_bounds__(256) void pad_kernel(Pad p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.pieces) return;
    const T* from = static_cast<const T*>(p.from[blockIdx.y]);
    T* to = static_cast<T*>(p.to[blockIdx.y]);
    const int heads = p.heads, dim = p.dim;
    const int64_t ld = p.ld[blockIdx.y];
    const int per = p.pitch / 8, piece = static_cast<int>(i % per);
    const int64_t head = i / per;
    const T* row = from + head / heads * ld + head % heads * dim;
    __align__(16) T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const T y = row[8 * piece + e < dim ? 8 * piece + e : 0];
        x[e] = 8 * piece + e < dim ? y : T{};
    }
#pragma unroll
    for (int n = 0; n < static_cast<int>(sizeof(x) / 16); ++n)
        reinterpret_cast<u32x4*>(to + i * 8)[n] = reinterpret_cast<const u32x4*>(x)[n];
}

template <typename T, int KT, bool VEC, bool BWD>
__global__ __launch_bounds__(64, 2) void prepare_kernel(DeltaArgs a, size_t rec_bytes) {
    // (given at the launch: where the compiler sees how few workgroups fit, it moves sums to the upper 256 registers and back)
    extern __shared__ __align__(16) float As[];
    float* const hi = As + C * kRowA;
    float* const lo = hi + C;
    float* const bet = lo + C;
    float* const kk = bet + C;
    // The solved diagonal blocks, in rows and columns of A that nothing else is in
    auto solved = [&](int block, int t) { return As + (16 * (block & 1) + t) * kRowA + 32 + 16 * (block >> 1); };
    constexpr int N = kPieces<T>, ESZ = sizeof(T);
    const int lane = threadIdx.x, g = lane >> 4, m = lane & 15;
    const int64_t id = blockIdx.x;
    const int c = remainder(blockIdx.x, a.nchunks), bh = quotient(blockIdx.x, a.nchunks);
    const int hv = remainder(bh, a.vheads), hk = quotient(hv, a.vheads / a.kheads);
    const int64_t b = quotient(bh, a.vheads), t0 = static_cast<int64_t>(c) * C;
    const int rows = static_cast<int>(a.seqlen - t0 < C ? a.seqlen - t0 : C);

    // decays
    const int64_t tok = b * a.seqlen + t0 + lane;
    const bool in = lane < rows;
    bool start = in && a.doc_start != nullptr && a.doc_start[in ? tok : 0] != 0;
    if (c == 0 && lane == 0 && a.initial_state == nullptr) start = true;
    const uint64_t starts = __ballot(start);
    float gate = in && a.g != nullptr ? a.g[tok * a.vheads + hv] : 0.0f;
    float beta = in ? a.beta[tok * a.vheads + hv] : 0.0f;
    if (start) gate = 0.0f;
    const uint64_t walls = starts | __ballot(gate < -200.0f);
    if (gate < -200.0f) gate = -200.0f;
    const bool bad_gate = not_finite(gate), bad_beta = not_finite(beta);
    if (bad_gate) gate = 0.0f;
    double sum = gate;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const double other = __shfl_up(sum, s);
        if (lane >= s) sum += other;
    }
    sum *= 1.4426950408889634;
    const double end = __shfl(sum, 63);
    const float h = static_cast<float>(sum), l = static_cast<float>(sum - h);
    const int my_seg = __popcll(starts & (~0ull >> (63 - lane)));
    const int last_seg = __popcll(starts);
    hi[lane] = h;
    lo[lane] = l;

    // K K^T, lower tiles
    const T* kp = static_cast<const T*>(a.k);
    const Rsrc kr = rows_rsrc<ESZ>(kp, (b * a.seqlen + t0) * a.ld_k + static_cast<int64_t>(hk) * a.kpitch, rows, a.ld_k,
                                   a.kpitch);
    const Rsrc qr = rows_rsrc<ESZ>(static_cast<const T*>(a.q), (b * a.seqlen + t0) * a.ld_q + static_cast<int64_t>(hk) * a.kpitch,
                                   rows, a.ld_q, a.kpitch);
    f32x4 acc[4][4], qk[4][4];   // rows t of tile i, columns s of tile j <= i
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = qk[i][j] = f32x4{0, 0, 0, 0};
    {
        // all of a tensor's rows asked for before the first is waited for (bf16; floats would take twice the registers)
        constexpr int STEPS = KT / 32, AHEAD = N == 1 ? STEPS : 1;
        Eight<T, VEC> kraw[AHEAD][4], qraw[AHEAD][4];
        auto fetch = [&](Eight<T, VEC> (*raw)[4], Rsrc rs, int64_t ld, int j) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[j % AHEAD][i].load(rs, static_cast<uint32_t>((16 * i + m) * static_cast<int>(ld) * ESZ), 32 * j + 8 * g, a.kpitch);
        };
        if constexpr (AHEAD > 1) {
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                fetch(kraw, kr, a.ld_k, j);
                if (a.pairs) fetch(qraw, qr, a.ld_q, j);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            if constexpr (AHEAD == 1) fetch(kraw, kr, a.ld_k, j);
            Frag<N> f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = kraw[j % AHEAD][i].frag();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n <= i; ++n) product<3>(acc[i][n], f[i], f[n]);
            if (a.pairs) {
                if constexpr (AHEAD == 1) fetch(qraw, qr, a.ld_q, j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Frag<N> q = qraw[j % AHEAD][i].frag();
#pragma unroll
                    for (int n = 0; n <= i; ++n) product<3>(qk[i][n], q, f[n]);
                }
            }
        }
    }
    // squared norms tell which keys are not finite
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * g + r == m) kk[16 * i + m] = acc[i][i][r];
    __syncthreads();
    const bool bad_row = bad_gate || bad_beta || not_finite(kk[lane]);
    const uint64_t bad = smear(__ballot(bad_row), starts);
    const bool is_bad = (bad >> lane) & 1;
    if (is_bad) beta = 0.0f;
    bet[lane] = beta;

    ChunkRec* rec = reinterpret_cast<ChunkRec*>(a.chunks + id * rec_bytes);
    rec->hi[lane] = h;
    rec->lo[lane] = l;
    rec->into[lane] = my_seg == 0 ? exp2_fast(h) * __builtin_fmaf(l, kLn2, 1.0f) : 0.0f;
    {
        const double d = end - sum;
        const float dh = static_cast<float>(d), dl = static_cast<float>(d - dh);
        rec->outof[lane] = my_seg == last_seg ? exp2_fast(dh) * __builtin_fmaf(dl, kLn2, 1.0f) : 0.0f;
    }
    rec->beta[lane] = beta;
    if (lane == 63) {
        rec->keep = last_seg == 0 ? exp2_fast(h) * __builtin_fmaf(l, kLn2, 1.0f) : 0.0f;
        rec->pad = 0;
        rec->starts = starts;
        rec->walls = walls;
        rec->bad = bad;
        rec->sick = 0;
    }
    __syncthreads();

    // The lower tiles in As, out in pieces in the order of an operand: rows (or, transposed, columns) in lanes
    auto emit = [&](char* to, bool transposed) {
        u32x4* out = reinterpret_cast<u32x4*>(to + id * kSolveBytes);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (transposed ? j < i / 2 : j > i / 2) continue;
                f32x4 x, y;
                if (transposed) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = As[(32 * j + 4 * g + e) * kRowA + 16 * i + m];
                        y[e] = As[(32 * j + 16 + 4 * g + e) * kRowA + 16 * i + m];
                    }
                } else {
                    x = four(As + (16 * i + m) * kRowA + 32 * j + 4 * g);
                    y = four(As + (16 * i + m) * kRowA + 32 * j + 16 + 4 * g);
                }
                const Frag<3> f = split(x, y);
                const int blk = transposed ? high_block(i, j) : low_block(i, j);
#pragma unroll
                for (int n = 0; n < 3; ++n) out[(blk * 3 + n) * 64 + lane] = f.p[n];
            }
        __syncthreads();
    };
    if (a.pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 th = four(hi + 16 * i + 4 * g), tl = four(lo + 16 * i + 4 * g);
#pragma unroll
            for (int j = 0; j <= (i | 1); ++j) {
                const int s = 16 * j + m, end = doc_end(starts, s);
                const float sh = hi[s], sl = lo[s];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    const float d = exp2_fast((th[r] - sh) + (tl[r] - sl));
                    As[t * kRowA + s] = j <= i ? keep_if(s <= t && t < end, a.scale * (d * qk[i][j <= i ? j : i][r])) : 0.0f;
                }
            }
        }
        __syncthreads();
        emit(a.pairs, BWD);
    }

#pragma unroll
    for (int which = 0; which < (BWD ? 2 : 1); ++which) {
        // A = M b, or b M, into LDS: rows 4 g + r, columns m of each lower tile
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 th = four(hi + 16 * i + 4 * g), tl = four(lo + 16 * i + 4 * g), tb = four(bet + 16 * i + 4 * g);
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                const int s = 16 * j + m;
                const float sh = hi[s], sl = lo[s], sb = bet[s];
                const int end = doc_end(starts, s);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    const float d = exp2_fast((th[r] - sh) + (tl[r] - sl));
                    const bool on = s < t && t < end && !((bad >> t) & 1);
                    As[t * kRowA + s] = keep_if(on, (which ? tb[r] : sb) * (d * acc[i][j][r]));
                }
            }
        }
        __syncthreads();

        // The diagonal triangles: group g solves block g, lane m its column m.
        {
            float x[16];
            const float* blk = As + (16 * g) * kRowA + 16 * g;
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int q = 0; q < t; q += 4) {
                    const f32x4 row = four(blk + t * kRowA + q);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (q + e < t) {
                            if (e & 1) s1 = __builtin_fmaf(row[e], x[q + e], s1);
                            else s0 = __builtin_fmaf(row[e], x[q + e], s0);
                        }
                }
                x[t] = (t == m ? 1.0f : 0.0f) - (s0 + s1);
                solved(g, t)[m] = x[t];
            }
        }
        __syncthreads();

        // The blocks below, one diagonal of blocks after the other.
        f32x4 tri[4][4], diag[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) tri[i][i][r] = solved(i, 4 * g + r)[m];
            diag[i] = four(solved(i, m) + 4 * g);
        }
#pragma unroll
        for (int d = 1; d < 4; ++d)
#pragma unroll
            for (int j = 0; j + d < 4; ++j) {
                const int i = j + d;
                f32x4 x = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k >= j && k < i) x = mfma_f32(four(As + (16 * i + m) * kRowA + 16 * k + 4 * g), tri[k][j], x);
                tri[i][j] = -mfma_f32(diag[i], x, f32x4{0, 0, 0, 0});
            }
        __syncthreads();

        // The triangle over A (zeros above the diagonal tiles and between documents), then out in pieces.
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = 16 * j + m, end = doc_end(starts, s);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    As[t * kRowA + s] = j <= i && t < end ? tri[i][j <= i ? j : i][r] : 0.0f;
                }
            }
        __syncthreads();
        emit(which ? a.solve_t : a.solve, which != 0);
    }
}

template <typename T, int KT, bool VEC>
hipError_t launch(const DeltaArgs& a, unsigned blocks) {
    if (a.solve_t)
        hipLaunchKernelGGL((prepare_kernel<T, KT, VEC, true>), dim3(blocks), dim3(64), kLds, a.stream, a,
                           delta_chunk_bytes());
    else
        hipLaunchKernelGGL((prepare_kernel<T, KT, VEC, false>), dim3(blocks), dim3(64), kLds, a.stream, a,
                           delta_chunk_bytes());
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_pad(const DeltaArgs& a, const void* q, const void* k, int64_t ld_q, int64_t ld_k) {
    const int64_t pieces = a.batch * a.seqlen * a.kheads * (a.kpitch / 8);
    const Pad p{{q, k}, {const_cast<void*>(a.q), const_cast<void*>(a.k)}, {ld_q, ld_k}, pieces, a.kheads, a.kdim, a.kpitch};
    const dim3 grid(static_cast<unsigned>((pieces + 255) / 256), 2);
    if (a.bf16) hipLaunchKernelGGL(pad_kernel<uint16_t>, grid, dim3(256), 0, a.stream, p);
    else hipLaunchKernelGGL(pad_kernel<uint32_t>, grid, dim3(256), 0, a.stream, p);
    return hipGetLastError();
}

hipError_t launch_delta_prepare(const DeltaArgs& a) {
    const unsigned blocks = static_cast<unsigned>(a.batch * a.vheads * a.nchunks);
    const bool wide = a.kdim > 64;
    if (a.bf16) {
        if (a.vec_k) return wide ? launch<bf16_t, 128, true>(a, blocks) : launch<bf16_t, 64, true>(a, blocks);
        return wide ? launch<bf16_t, 128, false>(a, blocks) : launch<bf16_t, 64, false>(a, blocks);
    }
    if (a.vec_k) return wide ? launch<float, 128, true>(a, blocks) : launch<float, 64, true>(a, blocks);
    return wide ? launch<float, 128, false>(a, blocks) : launch<float, 64, false>(a, blocks);
}

}  // namespace mamba
