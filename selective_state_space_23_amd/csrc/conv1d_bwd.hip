// Backward pass of the depthwise causal conv1d (width 4) + SiLU, gfx950.
//
// What it computes: the gradients of sum(du * u) through the forward of
// conv1d.hip ("Mamba: Selective State Spaces (S6)" section of the Mamba skill
// page; axolotl page: the conv state restarts at every document start).  With
// acc_t = bias + sum_j w[3-j] x_{t-j} over the taps inside token t's document
// and dacc_t = du_t silu'(acc_t) (du_t without SiLU):
//     dx_s      = sum_{j=0..3} dacc_{s+j} w[3-j]   over the j with s inside (s+j)'s document
//     dw[3-j]   = sum_t dacc_t x_{t-j}             over the same taps
//     dbias     = sum_t dacc_t
//
// Mapping: as the forward, each thread owns VEC consecutive channels and a
// tile of 48 tokens.  It walks the tile and the 3 tokens after it once,
// recomputing acc from a 3-token history (cleared at document starts, primed
// from the 3 tokens before the tile) and keeping the not yet complete dx of the
// last 4 tokens in a shift register: token t adds dacc_t w[3-j] to dx_{t-j} for
// the taps that stay inside its document, and dx_{t-3} is then final.  dw and
// dbias are summed over the tile's own tokens into per-tile partials, which a
// second kernel adds in a fixed order.
//
// A row that continues a given history (conv_state: the inputs of tokens -3..-1)
// treats those three as tokens of token 0's document (unless token 0 starts
// one): they feed acc of tokens 0..2, and their own dx (the gradient of the
// history, d_conv_state) comes out of the shift register of the first tile as
// tokens 0..2 complete it.
#include "device_common.hpp"
#include "launch.hpp"
#include "recurrence_launch.hpp"

namespace mamba {

// 2 channels = 4 bytes (bf16) or 8 bytes (fp32).
template <> struct VecIO<bf16_t, 2> {
    __device__ __forceinline__ static void load(const void* base, int64_t off, float (&v)[2]) {
        const uint32_t raw = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + off);
        v[0] = __uint_as_float(raw << 16);
        v[1] = __uint_as_float(raw & 0xffff0000u);
    }
    __device__ __forceinline__ static void store(void* base, int64_t off, const float (&v)[2]) {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + off) = pack_bf16x2(v[0], v[1]);
    }
};
template <> struct VecIO<float, 2> {
    __device__ __forceinline__ static void load(const void* base, int64_t off, float (&v)[2]) {
        const float2 raw = *reinterpret_cast<const float2*>(static_cast<const float*>(base) + off);
        v[0] = raw.x;
        v[1] = raw.y;
    }
    __device__ __forceinline__ static void store(void* base, int64_t off, const float (&v)[2]) {
        *reinterpret_cast<float2*>(static_cast<float*>(base) + off) = make_float2(v[0], v[1]);
    }
};

namespace {

// VEC consecutive channels of a token as stored, at element offset off + d0.  Read
// once but for the three tokens between two tiles, and so first to leave the L2 too
// (1 x 32768 x 3136 bfloat16 with the stores: 165 us to 151, from a checkpoint 154 to 149).
template <typename T, int VEC> struct VecRaw {
    using type = typename std::conditional<sizeof(T) * VEC == 8, uint2,
                                           typename std::conditional<sizeof(T) * VEC == 4, uint32_t, uint16_t>::type>::type;
    __device__ __forceinline__ static type load(const void* base, int64_t off, int d0) {
        const char* p = static_cast<const char*>(base) + off * static_cast<int64_t>(sizeof(T));
        const type* q = reinterpret_cast<const type*>(p + static_cast<uint32_t>(d0) * static_cast<uint32_t>(sizeof(T)));
        if constexpr (sizeof(type) == 4) return __builtin_nontemporal_load(q);
        else return *q;
    }
    __device__ __forceinline__ static void get(const type& r, float (&v)[VEC]) {
        if constexpr (sizeof(T) == 2) {
            v[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
            if constexpr (VEC == 2) v[1] = __uint_as_float(static_cast<uint32_t>(r) & 0xffff0000u);
        } else if constexpr (VEC == 2) {
            v[0] = __uint_as_float(r.x);
            v[1] = __uint_as_float(r.y);
        } else {
            v[0] = __uint_as_float(r);
        }
    }
};

constexpr int kTile = 48;          // tokens per thread; kTile + 6 <= 64 for one ballot
constexpr int kBlock = 256;

// The conv's input: x as stored, or its 8-bit checkpoint (codes (tokens, D), one
// scale per token and 64 channels laid out (blocks, tokens)).  The channels of a
// thread lie in one block: its scale comes with one 4-byte load per token, the
// same address in the lanes of a block.  (Scales held a token a lane and broadcast
// from there take as long; four tokens ahead in the general loop are slower, 188 us
// for 155.)  2 x 32768 x 1536 in bfloat16: 128 us from a checkpoint (590 MB, 4.6 TB/s).
template <typename T, int VEC> struct PlainX {
    using Raw = typename VecRaw<T, VEC>::type;
    const void* __restrict__ x;
    __device__ __forceinline__ Raw fetch(int64_t token, int dim, int d0) const {
        return VecRaw<T, VEC>::load(x, token * dim, d0);
    }
    __device__ __forceinline__ static void get(const Raw& r, float (&v)[VEC]) { VecRaw<T, VEC>::get(r, v); }
    __device__ __forceinline__ void load(int64_t token, int dim, int d0, float (&v)[VEC]) const {
        VecIO<T, VEC>::load(x, token * dim + d0, v);
    }
};
template <int VEC> struct PackedX {
    struct Raw { uint32_t q; float s; };
    const int8_t* __restrict__ q;
    const float* __restrict__ scale;
    int64_t tokens;
    __device__ __forceinline__ Raw fetch(int64_t token, int dim, int d0) const {
        const uint32_t d = static_cast<uint32_t>(d0);
        const int8_t* p = q + token * dim;
        const uint32_t w = VEC == 2 ? *reinterpret_cast<const uint16_t*>(p + d) : static_cast<uint8_t>(p[d]);
        return Raw{w, scale[(d0 / kPackBlock) * tokens + token]};
    }
    __device__ __forceinline__ static void get(const Raw& r, float (&v)[VEC]) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = static_cast<float>(static_cast<int8_t>(r.q >> (8 * k))) * r.s;
    }
    __device__ __forceinline__ void load(int64_t token, int dim, int d0, float (&v)[VEC]) const {
        get(fetch(token, dim, d0), v);
    }
};

// dx of a token.  LARGE: whole lines written once leave the L2 first.
template <typename T, int VEC, bool LARGE>
__device__ __forceinline__ void store_dx(void* base, int64_t off, const float (&v)[VEC]) {
    if constexpr (LARGE && sizeof(T) == 2 && VEC == 2)
        __builtin_nontemporal_store(pack_bf16x2(v[0], v[1]),
                                    reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + off));
    else
        VecIO<T, VEC>::store(base, off, v);
}

template <typename T, int VEC, bool SILU, typename X, bool LARGE>
__global__ __launch_bounds__(kBlock) void conv1d_bwd_kernel(
    const X x, const float* __restrict__ weight, const float* __restrict__ bias,
    const uint8_t* __restrict__ doc_start, const void* __restrict__ conv_state, const void* __restrict__ du,
    void* __restrict__ dx, float* __restrict__ d_conv_state, float* __restrict__ part, int64_t seqlen, int dim) {
    const int ngroups = (dim + VEC - 1) / VEC;
    const int grp = blockIdx.x * kBlock + threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int64_t b = blockIdx.z;
    const int64_t row = b * seqlen;

    // Document starts of tokens t0-3 .. t0+kTile+2: bit i <-> token t0 - 3 + i.
    const int lane = threadIdx.x & 63;
    const int64_t tl = t0 - 3 + lane;
    bool is_start = false;
    if (lane < kTile + 6 && tl >= 0 && tl < seqlen)
        is_start = (tl == 0 && conv_state == nullptr) || (doc_start != nullptr && doc_start[row + tl] != 0);
    const uint64_t starts = __ballot(is_start);
    if (grp >= ngroups) return;

    const int d0 = grp * VEC;
    float w0[VEC], w1[VEC], w2[VEC], w3[VEC], bs[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float* wr = weight + 4 * (d0 + i);
        w0[i] = wr[0]; w1[i] = wr[1]; w2[i] = wr[2]; w3[i] = wr[3];
        bs[i] = bias ? bias[d0 + i] : 0.0f;
    }

    // History x_{t-1}, x_{t-2}, x_{t-3} restricted to token t's document.
    float h1[VEC], h2[VEC], h3[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) h1[i] = h2[i] = h3[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int64_t t = t0 - 3 + k;
        float xv[VEC];
        if (t >= 0) {
            x.load(row + t, dim, d0, xv);
        } else if (conv_state != nullptr) {  // (B, D, 3): x_{-3}, x_{-2}, x_{-1} of each channel
#pragma unroll
            for (int i = 0; i < VEC; ++i) xv[i] = Elem<T>::load(conv_state, (b * dim + d0 + i) * 3 + (3 + t));
        } else {
            continue;
        }
        const bool reset = (starts >> k) & 1ull;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            h3[i] = reset ? 0.0f : h2[i];
            h2[i] = reset ? 0.0f : h1[i];
            h1[i] = xv[i];
        }
    }

    // p0..p3: the running dx of tokens t, t-1, t-2, t-3.
    float p1[VEC], p2[VEC], p3[VEC];
    float gw0[VEC], gw1[VEC], gw2[VEC], gw3[VEC], gb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        p1[i] = p2[i] = p3[i] = 0.0f;
        gw0[i] = gw1[i] = gw2[i] = gw3[i] = gb[i] = 0.0f;
    }
    // Tokens since the latest document start before t0, capped at 3 (token 0 of
    // a row without history is a start, and the history of one that has it
    // belongs to token 0's document: tiles at the row start need no special case).
    int since = 3;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if ((starts >> k) & 1ull) since = 3 - k;
    const int64_t own_end = (t0 + kTile < seqlen) ? t0 + kTile : seqlen;
    const bool all_taps = t0 >= 3 && t0 + kTile + 3 <= seqlen && (starts & ((1ull << (kTile + 6)) - 1)) == 0;
    if (LARGE && all_taps) {   // a tile whose taps all stay in the row and one document: no selects, four tokens at a time
        constexpr int kStep = 4;
        static_assert(kTile % kStep == 0);
        typename X::Raw xn[kStep];
        typename VecRaw<T, VEC>::type gn[kStep];
        auto fetch = [&](int k, int64_t t) {
            t = t < seqlen ? t : seqlen - 1;
            xn[k] = x.fetch(row + t, dim, d0);
            gn[k] = VecRaw<T, VEC>::load(du, (row + t) * dim, d0);
        };
        // Of token t, given its inputs: dx_{t-3}, complete with it, in out.
        auto taps = [&](const float (&xv)[VEC], float (&gv)[VEC], float (&out)[VEC], bool own) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float acc = __builtin_fmaf(w3[i], xv[i], bs[i]);
                acc = __builtin_fmaf(w2[i], h1[i], acc);
                acc = __builtin_fmaf(w1[i], h2[i], acc);
                acc = __builtin_fmaf(w0[i], h3[i], acc);
                float g = gv[i];
                if constexpr (SILU) {
                    const float sg = rcp_fast(1.0f + exp2_fast(-acc * kLog2e));
                    g *= sg * __builtin_fmaf(acc, 1.0f - sg, 1.0f);
                }
                if (own) {
                    gb[i] += g;
                    gw3[i] = __builtin_fmaf(g, xv[i], gw3[i]);
                    gw2[i] = __builtin_fmaf(g, h1[i], gw2[i]);
                    gw1[i] = __builtin_fmaf(g, h2[i], gw1[i]);
                    gw0[i] = __builtin_fmaf(g, h3[i], gw0[i]);
                }
                out[i] = __builtin_fmaf(g, w0[i], p3[i]);
                p3[i] = __builtin_fmaf(g, w1[i], p2[i]);
                p2[i] = __builtin_fmaf(g, w2[i], p1[i]);
                p1[i] = g * w3[i];
                h3[i] = h2[i];
                h2[i] = h1[i];
                h1[i] = xv[i];
            }
        };
#pragma unroll
        for (int k = 0; k < kStep; ++k) fetch(k, t0 + k);
#pragma unroll 1
        for (int64_t t = t0; t < t0 + kTile; t += kStep) {
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                float xv[VEC], gv[VEC], out[VEC];
                X::get(xn[k], xv);
                VecRaw<T, VEC>::get(gn[k], gv);
                fetch(k, t + kStep + k);
                taps(xv, gv, out, true);
                if (t + k >= t0 + 3) store_dx<T, VEC, LARGE>(dx, (row + t + k - 3) * dim + d0, out);
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            float xv[VEC], gv[VEC], out[VEC];
            X::get(xn[k], xv);
            VecRaw<T, VEC>::get(gn[k], gv);
            taps(xv, gv, out, false);
            store_dx<T, VEC, LARGE>(dx, (row + t0 + kTile + k - 3) * dim + d0, out);
        }
    } else {
        // x and du of the next token are fetched while the current one computes.
        auto fetch = [&](int64_t t, float (&xv)[VEC], float (&gv)[VEC]) {
            if (t < seqlen) {
                x.load(row + t, dim, d0, xv);
                VecIO<T, VEC>::load(du, (row + t) * dim + d0, gv);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) xv[i] = gv[i] = 0.0f;
            }
        };
        float xn[VEC], gn[VEC];
        fetch(t0, xn, gn);
        for (int64_t t = t0; t < own_end + 3; ++t) {
            const bool in_row = t < seqlen;
            float xv[VEC], gv[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xv[i] = xn[i];
                gv[i] = gn[i];
            }
            fetch(t + 1, xn, gn);
            if (in_row && ((starts >> (t - t0 + 3)) & 1ull)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) h1[i] = h2[i] = h3[i] = 0.0f;
                since = 0;
            }
            const bool own = t < own_end;
            float out[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float acc = __builtin_fmaf(w3[i], xv[i], bs[i]);
                acc = __builtin_fmaf(w2[i], h1[i], acc);
                acc = __builtin_fmaf(w1[i], h2[i], acc);
                acc = __builtin_fmaf(w0[i], h3[i], acc);
                float g = gv[i];
                if constexpr (SILU) {
                    const float sg = rcp_fast(1.0f + exp2_fast(-acc * kLog2e));
                    g *= sg * __builtin_fmaf(acc, 1.0f - sg, 1.0f);
                }
                if (own) {
                    gb[i] += g;
                    gw3[i] = __builtin_fmaf(g, xv[i], gw3[i]);
                    gw2[i] = __builtin_fmaf(g, h1[i], gw2[i]);
                    gw1[i] = __builtin_fmaf(g, h2[i], gw1[i]);
                    gw0[i] = __builtin_fmaf(g, h3[i], gw0[i]);
                }
                // dx_{t-3} is complete after token t's tap; shift the others along.  Taps on
                // another document are left out by selects: a NaN or an infinity in g times
                // zero would reach it.
                out[i] = since >= 3 ? __builtin_fmaf(g, w0[i], p3[i]) : p3[i];
                p3[i] = since >= 2 ? __builtin_fmaf(g, w1[i], p2[i]) : p2[i];
                p2[i] = since >= 1 ? __builtin_fmaf(g, w2[i], p1[i]) : p1[i];
                p1[i] = g * w3[i];
                h3[i] = h2[i];
                h2[i] = h1[i];
                h1[i] = xv[i];
            }
            since = since < 3 ? since + 1 : 3;
            const int64_t s = t - 3;
            if (s >= t0 && s < own_end) {
                store_dx<T, VEC, LARGE>(dx, (row + s) * dim + d0, out);
            } else if (s < 0 && d_conv_state != nullptr) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d_conv_state[(b * dim + d0 + i) * 3 + (3 + s)] = out[i];
            }
        }
    }
    // Per-tile partials: [b][tile][5][D] (dw columns 0..3, then dbias).
    const int64_t ntiles = gridDim.y;
    float* pt = part + ((b * ntiles + blockIdx.y) * 5) * dim + d0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (d0 + i >= dim) break;
        pt[i] = gw0[i];
        pt[dim + i] = gw1[i];
        pt[2 * dim + i] = gw2[i];
        pt[3 * dim + i] = gw3[i];
        pt[4 * dim + i] = gb[i];
    }
}

// dweight (D, 4) and dbias (D,): sums of the per-tile partials.  A block of 1024
// threads covers 64 consecutive outputs (coalesced 256-byte rows) with 16
// threads each; thread g adds the parts g, g + 16, ... with two accumulators,
// and the 16 sums are added in a fixed order.
__global__ __launch_bounds__(1024) void conv1d_bwd_reduce_kernel(const float* __restrict__ part, float* dweight,
                                                                 float* dbias, int64_t nparts, int dim) {
    constexpr int kGroups = 16;
    __shared__ float red[kGroups][64];
    const int64_t nout = 5 * static_cast<int64_t>(dim);
    const int o = threadIdx.x & 63;
    const int g = threadIdx.x >> 6;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 64 + o;
    float s0 = 0.0f, s1 = 0.0f;
    if (e < nout) {
        int64_t i = g;
#pragma unroll 8
        for (; i + kGroups < nparts; i += 2 * kGroups) {
            s0 += part[i * nout + e];
            s1 += part[(i + kGroups) * nout + e];
        }
        if (i < nparts) s0 += part[i * nout + e];
    }
    red[g][o] = s0 + s1;
    __syncthreads();
    if (g != 0 || e >= nout) return;
    float tot = 0.0f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) tot += red[k][o];
    const int k = static_cast<int>(e / dim);
    const int d = static_cast<int>(e % dim);
    if (k < 4) dweight[static_cast<int64_t>(d) * 4 + k] = tot;
    else if (dbias) dbias[d] = tot;
}

template <typename T, int VEC, typename X, bool LARGE>
hipError_t launch_conv_bwd_tiles(const ConvBwdArgs& a, const X& x, dim3 grid) {
    if (a.apply_silu)
        hipLaunchKernelGGL((conv1d_bwd_kernel<T, VEC, true, X, LARGE>), grid, dim3(kBlock), 0, a.stream, x, a.weight,
                           a.bias, a.doc_start, a.conv_state, a.du, a.dx, a.d_conv_state, a.ws, a.seqlen,
                           static_cast<int>(a.dim));
    else
        hipLaunchKernelGGL((conv1d_bwd_kernel<T, VEC, false, X, LARGE>), grid, dim3(kBlock), 0, a.stream, x, a.weight,
                           a.bias, a.doc_start, a.conv_state, a.du, a.dx, a.d_conv_state, a.ws, a.seqlen,
                           static_cast<int>(a.dim));
    return hipGetLastError();
}

template <typename T, int VEC, typename X>
hipError_t launch_conv_bwd_x(const ConvBwdArgs& a, const X& x) {
    const int ngroups = static_cast<int>((a.dim + VEC - 1) / VEC);
    const int64_t ntiles = (a.seqlen + kTile - 1) / kTile;
    const dim3 grid((ngroups + kBlock - 1) / kBlock, static_cast<unsigned>(ntiles), static_cast<unsigned>(a.batch));
    // The general loop alone leaves room for 8 waves a SIMD, 2048 workgroups; beside the fast
    // loop it has 6 or 7.  A grid that is there at once waits for its slowest tiles, and a
    // row's ends always take the general loop: the fast one gains nothing (8 x 2048 x 1536 in bfloat16 46
    // us alone and 53 with both; 15 x 2048 74 and 84).  Float32 gains by both from 1536 workgroups on (15 x
    // 2048 from a checkpoint 131 and 124).  What such a call writes fits the caches and stays there.
    // Above, the inner tiles' share decides: 2 x 32768 x 1536 in bfloat16 164 alone and 140 with
    // both, in documents of 30 tokens 165 and 172 (float32 301 and 279, 300 and 316).
    const bool large = static_cast<int64_t>(grid.x) * ntiles * a.batch > (sizeof(T) == 4 ? 1536 : 2048);
    const hipError_t e = large ? launch_conv_bwd_tiles<T, VEC, X, true>(a, x, grid)
                               : launch_conv_bwd_tiles<T, VEC, X, false>(a, x, grid);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(conv1d_bwd_reduce_kernel, dim3(static_cast<unsigned>((5 * a.dim + 63) / 64)), dim3(1024), 0,
                       a.stream, static_cast<const float*>(a.ws), a.dweight, a.dbias, a.batch * ntiles,
                       static_cast<int>(a.dim));
    return hipGetLastError();
}

template <typename T, int VEC>
hipError_t launch_conv_bwd_vec(const ConvBwdArgs& a, const Packed* in) {
    if (in != nullptr)
        return launch_conv_bwd_x<T, VEC>(a, PackedX<VEC>{in->q, in->scale, a.batch * a.seqlen});
    return launch_conv_bwd_x<T, VEC>(a, PlainX<T, VEC>{a.x});
}

hipError_t launch_conv_bwd(const ConvBwdArgs& a, const Packed* in) {
    constexpr int V = 2;
    if (a.bf16) return a.vectorized ? launch_conv_bwd_vec<bf16_t, V>(a, in) : launch_conv_bwd_vec<bf16_t, 1>(a, in);
    return a.vectorized ? launch_conv_bwd_vec<float, V>(a, in) : launch_conv_bwd_vec<float, 1>(a, in);
}

}  // namespace

size_t conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
    return static_cast<size_t>(batch * ((seqlen + kTile - 1) / kTile) * 5 * dim) * sizeof(float);
}

// Pairs of channels for either dtype: the history, pending-dx and gradient
// registers of 2 channels leave room for 8 waves per SIMD (6 or 7 with both loops),
// which hides the loads' latency better than 4 channels a thread at 4 waves (187 and
// 233 us on the packed 32K workload with the general loop alone, where fetching 2 or 3
// tokens ahead did not help).
hipError_t launch_causal_conv1d_bwd(const ConvBwdArgs& a) { return launch_conv_bwd(a, nullptr); }
hipError_t launch_causal_conv1d_bwd_packed(const ConvBwdArgs& a, const Packed& in) { return launch_conv_bwd(a, &in); }

}  // namespace mamba
