// Gated linear recurrence, forward and one-token step, gfx950.
//
// With r = sigmoid(gate_a), i = sigmoid(gate_x), log a = -c softplus(a_param) r
// and w = sqrt(1 - a^2), per row and channel
//     h_t = a_t h_{t-1} + w_t i_t x_t,    out_t = h_t silu(z_t)   (h_t without z),
// where h_{t-1} is 0 at a document start.
//
// A token's map h -> a h + b composes as (P, H): h -> P h + H.  A document start
// is a map that ignores its input, marked by the sign of P (decays are never
// negative): selects on that sign, not products with zero, keep an infinite or
// NaN state of one document out of the next.
#include "recurrence.hpp"

namespace mamba {

using namespace rec;

namespace {

constexpr int kK = 8;                                // tokens a lane walks
constexpr int kWaves = kTileTokens / (2 * kK);       // two halves of 32 lanes a wave
constexpr int kThreads = kWaves * 64;
constexpr int kCus = 256;

// Workgroups of a variant that a CU holds, 2 waves a SIMD each: float32 and unaligned inputs, which
// wait in registers, leave room for two where nothing but out is written, or nothing at all.
template <typename T, bool ALIGNED, bool HAS_Z, bool SAVE, bool OUT, int LOOK>
constexpr int kPerCu = (sizeof(T) == 2 && ALIGNED) || !OUT || (!HAS_Z && !SAVE && LOOK == kLookNear) ? 2 : 1;

// One pass over the data.  A workgroup works off tiles until none is left (rows
// of one tile: one workgroup each); a tile's maps stay in registers while the value
// entering it is found by wave 0, the other waves write the checkpoints meanwhile, and
// the next tile's inputs are under way from then on.  OUT: writes out, the final state
// and the checkpoints; else the states alone (the backward's recomputation).
//
// What bounds it is memory, then the vector unit (41 issue slots an element, 34 of them
// in the maps): one row of 65536 x 5120 in
// bfloat16 without z moves 2.78 GB, of which 2.68 are inputs and outputs, in 620 to 630 us:
// 4.4 TB/s where a copy reaches 5.2, the vector unit issues for 58% of it.  8 rows of
// 2048 x 1536 with z take 76 us (3.4 TB/s): six tiles a workgroup, whose first and last are not
// hidden.  Three passes (maps, joining, outputs) read the inputs twice: 1348 us for
// the first.  A tile's 16 waves a CU, in two workgroups, fill the registers (float32 and unaligned
// inputs: kPerCu); what a workgroup waits for its neighbours (a third of its time) the
// other one's work covers.
// Staging through LDS in place of registers took the first case from 785 us to 708,
// drawing tickets one tile ahead and not two the second from 91 to 82.
struct RecFwdKernelArgs {
    RecFwdArgs a;
    Chain ch;
    int nct, ntiles;
};

template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, bool SAVE, bool OUT, int LOOK>
__global__ __launch_bounds__(kThreads, (2 * kPerCu<T, ALIGNED, HAS_Z, SAVE, OUT, LOOK>)) void rec_fwd_kernel(
    const RecFwdKernelArgs) {
    __shared__ float s_rate[kTileChannels];
    __shared__ float s_in[kTileChannels];                 // the values entering the tile
    __shared__ float2 s_agg[kWaves + 1][kTileChannels];   // the waves' maps; the last row takes what no one reads
    __shared__ float2 s_pre[kWaves][kTileChannels];       // the maps of all before a wave
    __shared__ int s_ticket, s_first;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane % kRow, half = lane / kRow;
    const auto first = kernel_args<RecFwdKernelArgs>();
    const int dim = static_cast<int>(first->a.dim), nct = first->nct, ntiles = first->ntiles;
    const int tok = (wave * 2 + half) * kK;
    Walk<false> walk;
    walk.init(nct, ntiles, static_cast<int>(first->a.batch));
    auto draw = [&]() { return walk.draw(kernel_args<RecFwdKernelArgs>()->ch.next); };
    auto place = [&](int ticket) { return walk.place<false>(ticket, kernel_args<RecFwdKernelArgs>()->a.seqlen); };

    // The next tile's inputs: in LDS (each wave its own part), or in registers where
    // these are plenty (float32, unaligned: two waves a SIMD).
    constexpr bool kStaged = sizeof(T) == 2 && ALIGNED;
    constexpr bool kZ = HAS_Z && OUT;
    using In = LaneIn<T, ALIGNED, PIN, kK>;
    using Plain = LaneIn<T, ALIGNED, false, kK>;
    constexpr int kStage = 3 * In::kStageBytes + (kZ ? Plain::kStageBytes : 0);
    __shared__ __attribute__((aligned(16))) char s_stage[kStaged ? kWaves * kStage : 16];
    char* const stage = s_stage + (kStaged ? wave * kStage : 0);
    In xi, ai, gi;
    Plain zi;
    StartFlags fl;
    float rate[kV];
    auto fetch = [&](const Tile& t) {
        const int c = t.ct * kTileChannels + kV * li;
        const auto p = kernel_args<RecFwdKernelArgs>();
        const auto& a = p->a;
        const int64_t rows = a.batch * a.seqlen;
        if constexpr (kStaged) {
            ai.stage(stage, a.gate_a, a.in[1], t, a.ld_a, wave, dim, rows);
            gi.stage(stage + In::kStageBytes, a.gate_x, a.in[2], t, a.ld_g, wave, dim, rows);
            xi.stage(stage + 2 * In::kStageBytes, a.x, a.in[0], t, a.ld_x, wave, dim, rows);
            if constexpr (kZ) zi.stage(stage + 3 * In::kStageBytes, a.z, a.in[0], t, a.ld_z, wave, dim, rows);
        } else {
            ai.load(a.gate_a, a.in[1], t, a.ld_a, tok, c, dim, rows);
            gi.load(a.gate_x, a.in[2], t, a.ld_g, tok, c, dim, rows);
            xi.load(a.x, a.in[0], t, a.ld_x, tok, c, dim, rows);
            if constexpr (kZ) zi.load(a.z, a.in[0], t, a.ld_z, tok, c, dim, rows);
        }
        fl.load(a.doc_start, t.row_tok, t.nv);
        if (ntiles > 1) {
            const float2 r = *reinterpret_cast<const float2*>(p->ch.rate + c);   // padded to whole channel tiles
            rate[0] = r.x; rate[1] = r.y;
        }
    };

    int cur;
    if (ntiles > 1) {
        if (wave == 0) s_first = __builtin_amdgcn_readfirstlane(draw());
        lds_barrier();
        cur = __builtin_amdgcn_readfirstlane(s_first);
        if (cur >= walk.tickets) return;
        fetch(place(cur));
    } else {
        cur = static_cast<int>(blockIdx.x);
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

    if constexpr (kStaged) wait_all_but<0>();
    for (;;) {
        const Tile t = place(cur);
        const int c = t.ct * kTileChannels + kV * li;
        const TileStarts starts = fl.starts();
        int ticket = kNone;   // wave 0's: the next tile
        if (wave == 0 && !walk.once) ticket = draw();
        In xc = xi, ac = ai, gc = gi;
        Plain zc = zi;
        float rc[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) rc[j] = rate[j];
        if constexpr (kStaged) {
            ac.read(stage, half, li);
            gc.read(stage + In::kStageBytes, half, li);
            xc.read(stage + 2 * In::kStageBytes, half, li);
            if constexpr (kZ) zc.read(stage + 3 * In::kStageBytes, half, li);
            wait_lds_reads();
        }
        // Maps of the lane's tokens from its first one on.  GEN: the tile has document
        // starts or ends behind the row (decided for the whole workgroup).
        float P[kK][kV], H[kK][kV];
        const bool general = starts.any() || t.nv < kTileTokens;
        auto maps = [&](auto gen) {
            constexpr bool GEN = decltype(gen)::value;
            const uint32_t st = GEN ? starts.bits(tok, kK) : 0u;
            static_for<kK>([&](auto kc) {
                constexpr int k = decltype(kc)::value;
                float ga[kV], gx[kV], x[kV];
                ac.template take<k>(ga);
                gc.template take<k>(gx);
                xc.template take<k>(x);
                const bool start = GEN && ((st >> k) & 1u), out = GEN && tok + k >= t.nv;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    float al, om;
                    decay_terms(rc[j] * sigmoid_f(ga[j]), al, om);
                    float bb = __builtin_amdgcn_sqrtf(om) * (sigmoid_f(gx[j]) * x[j]);
                    if constexpr (GEN) {
                        al = out ? 1.0f : al;
                        bb = out ? 0.0f : bb;
                    }
                    if constexpr (k == 0) {
                        P[k][j] = al;
                        H[k][j] = bb;
                    } else {
                        P[k][j] = P[k - 1][j] * al;
                        H[k][j] = __builtin_fmaf(al, H[k - 1][j], bb);
                    }
                    if constexpr (GEN) {
                        P[k][j] = start ? -0.0f : P[k][j];
                        H[k][j] = start ? bb : H[k][j];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        if (general) maps(std::true_type{});
        else maps(std::false_type{});

        // what the wave's first half does before its second, and the wave's map
        float ep[kV], eh[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            float p = P[kK - 1][j], h = H[kK - 1][j];
            const float p1 = __shfl_xor(p, 32), h1 = __shfl_xor(h, 32);
            ep[j] = half ? p1 : 1.0f;
            eh[j] = half ? h1 : 0.0f;
            compose(p, h, ep[j], eh[j]);
            s_agg[half ? wave : kWaves][kV * li + j] = make_float2(p, h);
        }
        typename ChainWords<LOOK>::Seen seen = {};
        auto words = [&]() {
            const auto p = kernel_args<RecFwdKernelArgs>();
            return walk.template words<LOOK>(Chain{p->ch.map, p->ch.value, p->ch.next, p->ch.rate}, t);
        };
        if (wave == 0) {
            if (ntiles > 1) seen = words().peek(t.pos);
            s_ticket = __builtin_amdgcn_readfirstlane(ticket);
        }
        lds_barrier();
        const int next = __builtin_amdgcn_readfirstlane(s_ticket);
        float2 m = make_float2(1.0f, 0.0f);   // wave 0's, a lane per channel: the tile's map
        if (wave == 0) {
            m = s_agg[0][lane];
            s_pre[0][lane] = make_float2(1.0f, 0.0f);
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                s_pre[w][lane] = m;
                float2 v = s_agg[w][lane];
                compose(v.x, v.y, m.x, m.y);
                m = v;
            }
            if (t.tile + 1 < ntiles) words().publish_map(t.pos, m.x, m.y);
        }
        // The next tile's inputs are on their way from here on (past the last ticket: a
        // tile of no tokens, nothing is read).
        fetch(place(next));
        if (wave == 0) {   // the value entering the tile
            const int d = t.ct * kTileChannels + lane;
            const auto p = kernel_args<RecFwdKernelArgs>();
            const auto& a = p->a;
            const ChainWords<LOOK> chain = words();
            float in = row_load(a.initial_state, t.b, a.dim, d);
            in = chain.look_back(t.pos, in, seen);
            const float leaving = apply(m.x, m.y, in);
            if (t.tile + 1 < ntiles) chain.publish_value(t.pos, leaving);
            else if (OUT) row_store(a.final_state, t.b, a.dim, d, leaving);
            row_store(a.states, t.b * ntiles + t.tile, a.dim, d, in);
            s_in[lane] = in;
        }
        if constexpr (SAVE) {   // while wave 0 waits for the value entering
            const auto p = kernel_args<RecFwdKernelArgs>();
            const auto& a = p->a;
            const int64_t rows = a.batch * a.seqlen;
            save_packed<T, ALIGNED, kK>(xc, a.save[0], t, tok, c, dim, rows);
            save_packed<T, ALIGNED, kK>(ac, a.save[1], t, tok, c, dim, rows);
            save_packed<T, ALIGNED, kK>(gc, a.save[2], t, tok, c, dim, rows);
            if constexpr (HAS_Z) save_packed<T, ALIGNED, kK>(zc, a.save[3], t, tok, c, dim, rows);
        }
        lds_barrier();
        if constexpr (OUT) {
            float e[kV];
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float2 pre = s_pre[wave][kV * li + j];
                e[j] = apply(ep[j], eh[j], apply(pre.x, pre.y, s_in[kV * li + j]));
            }
            constexpr int esz = Elem<T>::kBytes;
            const Rsrc ob = rows_rsrc<esz>(kernel_args<RecFwdKernelArgs>()->a.out, t.row_tok, t.nv, dim, dim);
            const uint32_t step = static_cast<uint32_t>(dim) * esz;
            uint32_t off = store_offset(tok, step, c * esz, c < dim);
            auto put = [&](auto gen) {
                constexpr bool GEN = decltype(gen)::value;
                static_for<kK>([&](auto kc) {
                    constexpr int k = decltype(kc)::value;
                    float o[kV];
#pragma unroll
                    for (int j = 0; j < kV; ++j) o[j] = apply<GEN>(P[k][j], H[k][j], e[j]);
                    if constexpr (HAS_Z) {
                        float z[kV];
                        zc.template take<k>(z);
#pragma unroll
                        for (int j = 0; j < kV; ++j) o[j] *= silu_f(z[j]);
                    }
                    store_vals<T, kV, ALIGNED>(ob, off, dim - c, o);
                    off = next_offset(off, step);
                });
            };
            if (general) put(std::true_type{});
            else put(std::false_type{});
        }
        if (next >= walk.tickets) return;
        // Behind the staged loads this wave has issued the tile's kK stores at least.
        if constexpr (kStaged) wait_all_but<OUT ? kK : 0>();
        cur = next;
    }
}

// Before a launch: nothing published, no ticket drawn, the channels' rates.  A
// workspace per blockIdx.y.
__global__ __launch_bounds__(256) void rec_clear_kernel(char* __restrict__ ws, size_t stride, int64_t n, int nrate,
                                                        const float* __restrict__ a_param, int dim, float c) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    uint4* words = reinterpret_cast<uint4*>(ws + blockIdx.y * stride);
    uint32_t* next = reinterpret_cast<uint32_t*>(words + n);
    float* rate = reinterpret_cast<float*>(next + 16);
    if (i < n) words[i] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
    if (i < 8) next[i] = 0;
    if (i < nrate) rate[i] = -c * kLog2e * softplus_exact(a_param[i < dim ? i : dim - 1]);
}


template <typename T, bool ALIGNED, bool PIN, bool HAS_Z, bool SAVE, bool OUT>
hipError_t launch_fwd(const RecFwdArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const int ntiles = static_cast<int>((a.seqlen + kTileTokens - 1) / kTileTokens);
    const int64_t tiles = nct * a.batch * ntiles;
    Chain ch;
    if (a.chain != nullptr) {
        ch = *a.chain;
    } else {
        const hipError_t e = clear_chains(a.ws, 1, 0, a.batch, a.dim, ntiles, a.a_param, a.c, &ch, a.stream);
        if (e != hipSuccess) return e;
    }
    auto kernel = rec_fwd_kernel<T, ALIGNED, PIN, HAS_Z, SAVE, OUT, kLookNear>;
    int64_t resident = kCus * kPerCu<T, ALIGNED, HAS_Z, SAVE, OUT, kLookNear>;
    if (look_far(nct * a.batch, ntiles, 16)) {
        kernel = rec_fwd_kernel<T, ALIGNED, PIN, HAS_Z, SAVE, OUT, kLookFar>;
        resident = kCus * kPerCu<T, ALIGNED, HAS_Z, SAVE, OUT, kLookFar>;
    }
    const int64_t grid = ntiles > 1 && tiles > resident ? resident : tiles;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, a.stream,
                       RecFwdKernelArgs{a, ch, nct, ntiles});
    return hipGetLastError();
}

template <typename T, bool ALIGNED>
hipError_t launch_fwd_typed(const RecFwdArgs& a) {
    if (a.in[0].q != nullptr) return launch_fwd<T, ALIGNED, true, false, false, false>(a);
    if (a.out == nullptr) return launch_fwd<T, ALIGNED, false, false, false, false>(a);
    if (a.save[0].q != nullptr)
        return a.z != nullptr ? launch_fwd<T, ALIGNED, false, true, true, true>(a)
                              : launch_fwd<T, ALIGNED, false, false, true, true>(a);
    return a.z != nullptr ? launch_fwd<T, ALIGNED, false, true, false, true>(a)
                          : launch_fwd<T, ALIGNED, false, false, false, true>(a);
}

// Four channels at an element offset, `left` of which exist.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void quad_load(const void* p, int64_t off, int left, float (&v)[4]) {
    if constexpr (ALIGNED) {
        VecIO<T, 4>::load(p, off, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = j < left ? Elem<T>::load(p, off + j) : 0.0f;
    }
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void quad_store(void* p, int64_t off, int left, const float (&v)[4]) {
    if constexpr (ALIGNED) {
        VecIO<T, 4>::store(p, off, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) Elem<T>::store(p, off + j, v[j]);
    }
}

// One token per row: a thread per four channels of R rows, whose decay parameters it
// turns into rates once.  2^shift threads lie along a row, `nblocks` workgroups.  Bound
// by the launch and one trip to memory: 256 rows of 5120 with z take 9.5 us (23.6 MB,
// 2.5 TB/s), two rows of 1536 3.4 us.
template <typename T, bool ALIGNED, int R>
__global__ __launch_bounds__(256) void rec_update_kernel(const RecUpdateArgs a, unsigned nblocks, int shift) {
    const int dim = static_cast<int>(a.dim);
    const int c = static_cast<int>(((blockIdx.x % nblocks << shift) + (threadIdx.x & ((1u << shift) - 1))) * 4);
    const int64_t b0 = ((static_cast<int64_t>(blockIdx.x / nblocks) << (8 - shift)) + (threadIdx.x >> shift)) * R;
    if (c >= dim || b0 >= a.batch) return;
    const int left = dim - c;
    float ga[R][4], gx[R][4], x[R][4], z[R][4], h[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t b = b0 + r < a.batch ? b0 + r : a.batch - 1;   // a row behind the last: the last one's values, not stored
        quad_load<T, ALIGNED>(a.gate_a, b * a.ld_a + c, left, ga[r]);
        quad_load<T, ALIGNED>(a.gate_x, b * a.ld_g + c, left, gx[r]);
        quad_load<T, ALIGNED>(a.x, b * a.ld_x + c, left, x[r]);
        if (a.z != nullptr) quad_load<T, ALIGNED>(a.z, b * a.ld_z + c, left, z[r]);
        quad_load<float, ALIGNED>(a.state, b * a.dim + c, left, h[r]);
    }
    float k2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k2[j] = -a.c * kLog2e * softplus_exact(a.a_param[c + j < dim ? c + j : dim - 1]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t b = b0 + r;
        if (b >= a.batch) return;
        const bool clear = a.reset != nullptr && a.reset[b] != 0;
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float al, om;
            decay_terms(k2[j] * sigmoid_f(ga[r][j]), al, om);
            const float bb = __builtin_amdgcn_sqrtf(om) * (sigmoid_f(gx[r][j]) * x[r][j]);
            h[r][j] = clear ? bb : __builtin_fmaf(al, h[r][j], bb);
            o[j] = a.z != nullptr ? h[r][j] * silu_f(z[r][j]) : h[r][j];
        }
        quad_store<float, ALIGNED>(a.state, b * a.dim + c, left, h[r]);
        quad_store<T, ALIGNED>(a.out, b * a.dim + c, left, o);
    }
}

template <typename T, bool ALIGNED, int R>
void launch_update_rows(const RecUpdateArgs& a) {
    const int64_t quads = (a.dim + 3) / 4;
    int shift = 0;
    while (shift < 8 && (1 << shift) < quads) ++shift;
    const unsigned nblocks = static_cast<unsigned>((quads + (1 << shift) - 1) >> shift);
    const int64_t rows = static_cast<int64_t>(R) << (8 - shift);   // of a workgroup
    hipLaunchKernelGGL((rec_update_kernel<T, ALIGNED, R>), dim3(static_cast<unsigned>(nblocks * ((a.batch + rows - 1) / rows))),
                       dim3(256), 0, a.stream, a, nblocks, shift);
}

template <typename T, bool ALIGNED>
void launch_update(const RecUpdateArgs& a) {
    // Four rows a thread where that still leaves a workgroup for every CU: bfloat16 with z,
    // 1024 rows of 1536 take 9.9 us (2.9 TB/s) and 12.8 with one row, 64 of 5120 take 5.6
    // and 4.8.
    if (a.batch * a.dim >= 4 * 4 * 256 * 256) launch_update_rows<T, ALIGNED, 4>(a);
    else launch_update_rows<T, ALIGNED, 1>(a);
}

}  // namespace

size_t recurrence_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    const int64_t ntiles = (seqlen + kRecChunk - 1) / kRecChunk;
    const int64_t width = (dim + kPackBlock - 1) / kPackBlock * kPackBlock;
    if (ntiles <= 1) return 0;
    return static_cast<size_t>(batch * width * ntiles) * 12 + 64 + static_cast<size_t>(width) * 4;
}

hipError_t clear_chains(void* ws, int count, size_t stride, int64_t batch, int64_t dim, int64_t ntiles,
                        const float* a_param, float c, Chain* ch, hipStream_t stream) {
    for (int i = 0; i < count; ++i) ch[i] = Chain{nullptr, nullptr, nullptr, nullptr};
    if (ntiles <= 1) return hipSuccess;
    const int64_t width = (dim + kTileChannels - 1) / kTileChannels * kTileChannels;
    const int64_t words = batch * width * ntiles;
    for (int i = 0; i < count; ++i) {
        ch[i].map = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + i * stride);
        ch[i].value = reinterpret_cast<uint32_t*>(ch[i].map + words);
        ch[i].next = ch[i].value + words;
        ch[i].rate = reinterpret_cast<float*>(ch[i].next + 16);
    }
    const int64_t n = words * 12 / 16;   // words is a multiple of 64, and 3 words at least a width: n covers the rates
    hipLaunchKernelGGL(rec_clear_kernel, dim3(static_cast<unsigned>((n + 255) / 256), static_cast<unsigned>(count)),
                       dim3(256), 0, stream, static_cast<char*>(ws), stride, n, static_cast<int>(width), a_param,
                       static_cast<int>(dim), c);
    return hipGetLastError();
}

hipError_t launch_recurrence_fwd(const RecFwdArgs& a) {
    if (a.bf16) return a.aligned ? launch_fwd_typed<bf16_t, true>(a) : launch_fwd_typed<bf16_t, false>(a);
    return a.aligned ? launch_fwd_typed<float, true>(a) : launch_fwd_typed<float, false>(a);
}

hipError_t launch_recurrence_update(const RecUpdateArgs& a) {
    if (a.bf16) {
        if (a.aligned) launch_update<bf16_t, true>(a);
        else launch_update<bf16_t, false>(a);
    } else {
        if (a.aligned) launch_update<float, true>(a);
        else launch_update<float, false>(a);
    }
    return hipGetLastError();
}

}  // namespace mamba
