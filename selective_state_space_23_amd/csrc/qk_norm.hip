// Norms of queries and keys for each head with the position rotation in the same pass,
// and their gradients.
//
//     y = x r w,  r = (mean or sum of x^2 + eps)^-1/2;  pairs (a, b) of y -> (a c - b s, b c + a s)
//     dn = w rot^T(dy),   dx = r dn - x r^3 (dn . x) / n,   dw = sum rot^T(dy) x r
//
// Memory-bound: each tensor read and written once.  A lane holds the four pairs that rotate
// together of one head (4 channels of either half, or 8 in a row where pairs are interleaved),
// 4..32 lanes a head; the sums over a head are lane exchanges.  A wave takes one token's heads
// one group after the other, so the token's row of the tables is read once.  Weight
// gradients stay in registers over all a wave's tokens, then go over the workgroup through
// LDS and over the workgroups in a second launch, in a fixed order.
#include "device_common.hpp"
#include "qk_norm_launch.hpp"

namespace mamba {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
using Rsrc = __amdgpu_buffer_rsrc_t;

constexpr uint32_t kPast = 0x7fffff00u;
constexpr int kWaves = 4;
constexpr int kMaxBlocks = 1024;   // of a backward with weights: as many partial sums

// How a lane's four pairs lie in a head.
constexpr int kHalves = 0, kInterleaved = 1, kAny = 2;

__device__ __forceinline__ Rsrc rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

struct Pairs {
    f32x4 a, b;
};

// Byte offsets of channels within a head for lane l: a's and b's e-th, kPast where there is none.
struct Where {
    int l, dim, rot;
    bool interleaved;
    __device__ __forceinline__ int first(int e) const {   // kAny: channel of a[e]
        const int p = 4 * l + e, half = rot / 2;
        return p < half && !interleaved ? p : p < half ? 2 * p : rot + 2 * (p - half);
    }
    __device__ __forceinline__ int second(int e) const {
        const int p = 4 * l + e, half = rot / 2;
        return p < half && !interleaved ? p + half : first(e) + 1;
    }
    __device__ __forceinline__ int run_a() const { return 8 * l < rot ? 4 * l : 8 * l; }        // kHalves
    __device__ __forceinline__ int run_b() const { return 8 * l < rot ? 4 * l + rot / 2 : 8 * l + 4; }
    __device__ __forceinline__ bool on() const { return 8 * l < dim; }
};

__device__ __forceinline__ f32x4 wide(u32x2 w) {
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xffff0000u)};
}

// A lane's pairs of a head at byte offset `head` (kPast or more: zeros).
template <typename T, int MODE>
__device__ __forceinline__ Pairs load(Rsrc rs, uint32_t head, const Where& w) {
    constexpr int ESZ = Elem<T>::kBytes;
    Pairs p;
    if constexpr (MODE == kAny) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w.first(e), j = w.second(e);
            const uint32_t oi = i < w.dim ? head + i * ESZ : kPast, oj = j < w.dim ? head + j * ESZ : kPast;
            if constexpr (ESZ == 2) {
                p.a[e] = bf16_to_f32(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, oi, 0, 0)));
                p.b[e] = bf16_to_f32(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, oj, 0, 0)));
            } else {
                p.a[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, oi, 0, 0));
                p.b[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, oj, 0, 0));
            }
        }
    } else {
        const uint32_t at = w.on() ? head : kPast;
        const uint32_t oa = at + (MODE == kHalves ? w.run_a() : 8 * w.l) * ESZ;
        const uint32_t ob = at + (MODE == kHalves ? w.run_b() : 8 * w.l + 4) * ESZ;
        f32x4 x, y;
        if constexpr (ESZ == 2 && MODE == kInterleaved) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, oa, 0, 0);
            x = wide(u32x2{v[0], v[1]});
            y = wide(u32x2{v[2], v[3]});
        } else if constexpr (ESZ == 2) {
            x = wide(__builtin_amdgcn_raw_buffer_load_b64(rs, oa, 0, 0));
            y = wide(__builtin_amdgcn_raw_buffer_load_b64(rs, ob, 0, 0));
        } else {
            x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, oa, 0, 0));
            y = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, ob, 0, 0));
        }
        p.a = MODE == kHalves ? x : f32x4{x[0], x[2], y[0], y[2]};
        p.b = MODE == kHalves ? y : f32x4{x[1], x[3], y[1], y[3]};
    }
    return p;
}

template <typename T, int MODE>
__device__ __forceinline__ void store(Rsrc rs, uint32_t head, const Where& w, const Pairs& p) {
    constexpr int ESZ = Elem<T>::kBytes;
    if constexpr (MODE == kAny) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = w.first(e), j = w.second(e);
            const uint32_t oi = i < w.dim ? head + i * ESZ : kPast, oj = j < w.dim ? head + j * ESZ : kPast;
            if constexpr (ESZ == 2) {
                __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(p.a[e]), rs, oi, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(p.b[e]), rs, oj, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(p.a[e]), rs, oi, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(p.b[e]), rs, oj, 0, 0);
            }
        }
    } else {
        const uint32_t at = w.on() ? head : kPast;
        const uint32_t oa = at + (MODE == kHalves ? w.run_a() : 8 * w.l) * ESZ;
        const uint32_t ob = at + (MODE == kHalves ? w.run_b() : 8 * w.l + 4) * ESZ;
        const f32x4 x = MODE == kHalves ? p.a : f32x4{p.a[0], p.b[0], p.a[1], p.b[1]};
        const f32x4 y = MODE == kHalves ? p.b : f32x4{p.a[2], p.b[2], p.a[3], p.b[3]};
        if constexpr (ESZ == 2) {
            const u32x2 u = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
            const u32x2 v = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            if constexpr (MODE == kInterleaved) {
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{u[0], u[1], v[0], v[1]}, rs, oa, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b64(u, rs, oa, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b64(v, rs, ob, 0, 0);
            }
        } else {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rs, oa, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), rs, ob, 0, 0);
        }
    }
}

// A lane's four cosines or sines (1 or 0 behind the rotated channels).
template <int MODE>
__device__ __forceinline__ f32x4 angles(Rsrc rs, const Where& w, float behind, uint32_t row = 0) {
    f32x4 t;
    if constexpr (MODE == kAny) {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, row + 4 * (4 * w.l + e), 0, 0));
    } else {
        t = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, row + 16 * w.l, 0, 0));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = 4 * w.l + e < w.rot / 2 ? t[e] : behind;
    return t;
}

// The sum over LPR consecutive lanes, in each of them.
template <int LPR>
__device__ __forceinline__ float head_sum(float x) {
    auto moved = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                     decltype(ctrl)::value, 0xf, 0xf, false));
    };
    using I = int;
    x += moved(x, std::integral_constant<I, 0xB1>{});                            // quad_perm [1, 0, 3, 2]
    x += moved(x, std::integral_constant<I, 0x4E>{});                            // quad_perm [2, 3, 0, 1]
    if constexpr (LPR >= 8) x += moved(x, std::integral_constant<I, 0x141>{});   // row_half_mirror
    if constexpr (LPR >= 16) x += moved(x, std::integral_constant<I, 0x140>{});  // row_mirror
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
    return x;
}

struct Split {            // one tensor's share of a launch
    int blocks;           // workgroups
    int splits, groups;   // waves a token, groups of heads a wave
    int head_bits;        // PACKED: the lanes' groups divide into tokens of 1 << head_bits heads
};

struct Kernel {
    QkNormArgs a;
    Split s[2];
};

// One head's pairs: normed and rotated, or (BWD) their gradients from dy, with the weight's into dw.  A lane whose place
// `at` lies behind the tensor has no head: its root of 0 + eps, infinite with eps = 0, is taken out by its bits.
template <int LPR, bool BWD>
__device__ __forceinline__ Pairs normed(uint32_t at, const Pairs& x, const Pairs& dy, const Pairs& weight, f32x4 c, f32x4 s,
                                        float inv_n, float eps, Pairs& dw) {
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sq = __builtin_fmaf(x.a[e], x.a[e], sq);
        sq = __builtin_fmaf(x.b[e], x.b[e], sq);
    }
    float r = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<LPR>(sq), inv_n, eps));
    Pairs y;
    if constexpr (!BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float na = x.a[e] * r * weight.a[e], nb = x.b[e] * r * weight.b[e];
            y.a[e] = __builtin_fmaf(na, c[e], -(nb * s[e]));
            y.b[e] = __builtin_fmaf(nb, c[e], na * s[e]);
        }
    } else {
        r = __uint_as_float(__float_as_uint(r) & (at < kPast ? ~0u : 0u));
        float dot = 0.0f;
        Pairs dn;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float da = __builtin_fmaf(dy.a[e], c[e], dy.b[e] * s[e]);
            const float db = __builtin_fmaf(dy.b[e], c[e], -(dy.a[e] * s[e]));
            dw.a[e] = __builtin_fmaf(da * r, x.a[e], dw.a[e]);
            dw.b[e] = __builtin_fmaf(db * r, x.b[e], dw.b[e]);
            dn.a[e] = da * weight.a[e];
            dn.b[e] = db * weight.b[e];
            dot = __builtin_fmaf(dn.a[e], x.a[e], dot);
            dot = __builtin_fmaf(dn.b[e], x.b[e], dot);
        }
        const float k = r * r * head_sum<LPR>(dot) * inv_n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y.a[e] = r * __builtin_fmaf(-k, x.a[e], dn.a[e]);
            y.b[e] = r * __builtin_fmaf(-k, x.b[e], dn.b[e]);
        }
    }
    return y;
}

// PACKED: tokens of few heads, several to a wave.
template <typename T, int MODE, int LPR, bool BWD, bool PACKED>
__global__ __launch_bounds__(kWaves * 64) void norm_kernel(Kernel p) {
    constexpr int G = 64 / LPR, ESZ = Elem<T>::kBytes;   // G: heads of a group
    constexpr int U = 2;                                 // groups under way
    const QkNormArgs& a = p.a;
    const int which = static_cast<int>(blockIdx.x) < p.s[0].blocks ? 0 : 1;
    const int block = static_cast<int>(blockIdx.x) - (which ? p.s[0].blocks : 0);
    const int blocks = p.s[which].blocks, splits = p.s[which].splits, groups = p.s[which].groups;
    const int lane = threadIdx.x & 63, l = lane % LPR;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Where w{l, a.dim, a.rot, a.interleaved};
    const int heads = a.heads[which];
    const float inv_n = a.rms ? 1.0f / static_cast<float>(a.dim) : 1.0f;

    Pairs weight = {f32x4{1, 1, 1, 1}, f32x4{1, 1, 1, 1}};
    if (a.weight[which]) weight = load<float, MODE>(rsrc(a.weight[which], a.dim * 4), 0, w);
    Pairs dw = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};

    const uint32_t step = static_cast<uint32_t>(blocks) * kWaves;
    if constexpr (PACKED) {
        const int bits = p.s[which].head_bits, sub = (lane / LPR) >> bits, h = (lane / LPR) & ((1 << bits) - 1);
        const uint32_t per = G >> bits, tokens = static_cast<uint32_t>(a.tokens);   // tokens of U groups under way: U * per
        const uint32_t tasks = (tokens + U * per - 1) / (U * per);
        const Rsrc cr = rsrc(a.cos, a.table_rows * a.rot * 2), sr = rsrc(a.sin, a.table_rows * a.rot * 2);
        for (uint32_t task = static_cast<uint32_t>(block) * kWaves + wave; task < tasks; task += step) {
            const int64_t first = static_cast<int64_t>(task) * (U * per);
            const int64_t rows = a.tokens - first < U * per ? a.tokens - first : U * per;
            auto from = [&](const void* base, int64_t ld) {
                return rsrc(static_cast<const T*>(base) + first * ld, ((rows - 1) * ld + int64_t(heads) * a.dim) * ESZ);
            };
            const int64_t dense = int64_t(heads) * a.dim;
            const Rsrc xr = from(a.x[which], a.ld_x[which]), yr = from(a.out[which], dense);
            const Rsrc gr = BWD ? from(a.dy[which], a.ld_dy[which]) : xr;
            Pairs x[U], dy[U] = {};
            uint32_t at[U];
            f32x4 c[U], s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t row = u * per + sub;
                uint32_t head = h < heads && row < rows ? 0 : kPast;
                asm("" : "+v"(head));   // (no branch around the loads)
                head += static_cast<uint32_t>(h * a.dim * ESZ);
                at[u] = row * static_cast<uint32_t>(dense * ESZ) + head;
                x[u] = load<T, MODE>(xr, row * static_cast<uint32_t>(a.ld_x[which] * ESZ) + head, w);
                if constexpr (BWD) dy[u] = load<T, MODE>(gr, row * static_cast<uint32_t>(a.ld_dy[which] * ESZ) + head, w);
                c[u] = f32x4{1, 1, 1, 1};
                s[u] = f32x4{0, 0, 0, 0};
                if (a.cos) {
                    const uint32_t token = static_cast<uint32_t>(first) + (row < rows ? row : 0);
                    const int64_t pos = a.positions ? a.positions[token] : token % static_cast<uint32_t>(a.seqlen);
                    const bool in = pos >= 0 && pos < a.table_rows;
                    uint32_t nan = in ? 0 : 0x7fc00000;   // no row of the tables: nothing to rotate by
                    asm("" : "+v"(nan));
                    const uint32_t line = in ? static_cast<uint32_t>(pos) * static_cast<uint32_t>(a.rot * 2) : 0;
                    c[u] = angles<MODE>(cr, w, 1.0f, line);
                    s[u] = angles<MODE>(sr, w, 0.0f, line);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[u][e] = __uint_as_float(__float_as_uint(c[u][e]) | (4 * l + e < a.rot / 2 ? nan : 0));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Pairs y = normed<LPR, BWD>(at[u], x[u], dy[u], weight, c[u], s[u], inv_n, a.eps, dw);
                store<T, MODE>(yr, at[u], w, y);
            }
        }
    } else {
        const uint32_t tasks = static_cast<uint32_t>(a.tokens) * splits;
        for (uint32_t task = static_cast<uint32_t>(block) * kWaves + wave; task < tasks; task += step) {
            const uint32_t token_ = splits == 1 ? task : task / splits;   // (the vector unit's division: one value all the same)
            const int64_t token = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(token_));
            const int split = __builtin_amdgcn_readfirstlane(task - static_cast<uint32_t>(token) * splits);
            const Rsrc xr = rsrc(static_cast<const T*>(a.x[which]) + token * a.ld_x[which], int64_t(heads) * a.dim * ESZ);
            const Rsrc yr = rsrc(static_cast<T*>(a.out[which]) + token * heads * a.dim, int64_t(heads) * a.dim * ESZ);
            const Rsrc gr = rsrc(static_cast<const T*>(BWD ? a.dy[which] : a.x[which]) + (BWD ? token * a.ld_dy[which] : 0),
                                 BWD ? int64_t(heads) * a.dim * ESZ : 0);
            f32x4 c = {1, 1, 1, 1}, s = {0, 0, 0, 0};
            if (a.cos) {
                const int64_t pos = a.positions ? a.positions[token] : static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(
                    static_cast<uint32_t>(token) % static_cast<uint32_t>(a.seqlen)));
                const bool in = pos >= 0 && pos < a.table_rows;
                const int64_t row = in ? pos * (a.rot / 2) : 0;
                c = angles<MODE>(rsrc(a.cos + row, a.rot * 2), w, 1.0f);
                s = angles<MODE>(rsrc(a.sin + row, a.rot * 2), w, 0.0f);
                if (!in) {   // no row of the tables: nothing to rotate by
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = 4 * l + e < a.rot / 2 ? __builtin_nanf("") : 1.0f;
                }
            }
            const int end = (split + 1) * groups * G < heads ? (split + 1) * groups * G : heads;
            for (int h0 = split * groups * G; h0 < end; h0 += U * G) {
                Pairs x[U], dy[U] = {};
                uint32_t at[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * G + lane / LPR;
                    at[u] = h < end ? static_cast<uint32_t>(h * a.dim * ESZ) : kPast;
                    x[u] = load<T, MODE>(xr, at[u], w);
                    if constexpr (BWD) dy[u] = load<T, MODE>(gr, at[u], w);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Pairs y = normed<LPR, BWD>(at[u], x[u], dy[u], weight, c, s, inv_n, a.eps, dw);
                    store<T, MODE>(yr, at[u], w, y);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (a.dweight[which]) {
            __shared__ float sums[kWaves][kNormMaxDim];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int q = LPR; q < 64; q *= 2) {
                    dw.a[e] += __shfl_xor(dw.a[e], q);
                    dw.b[e] += __shfl_xor(dw.b[e], q);
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = MODE == kHalves ? w.run_a() + e : MODE == kInterleaved ? 8 * l + 2 * e : w.first(e);
                const int j = MODE == kHalves ? w.run_b() + e : MODE == kInterleaved ? 8 * l + 2 * e + 1 : w.second(e);
                if (lane < LPR && i < a.dim) sums[wave][i] = dw.a[e];
                if (lane < LPR && j < a.dim) sums[wave][j] = dw.b[e];
            }
            __syncthreads();
            static_assert(kNormMaxDim <= kWaves * 64, "a channel a thread");
            const int i = threadIdx.x;
            if (i < a.dim)
                a.parts[static_cast<int64_t>(blockIdx.x) * a.dim + i] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
        }
    }
}

// dweight[which][i] = the sum of its workgroups' parts: a wave a channel.
__global__ __launch_bounds__(64) void weight_sum_kernel(Kernel p) {
    const int which = blockIdx.x / p.a.dim, i = blockIdx.x % p.a.dim;
    float* to = p.a.dweight[which];
    if (to == nullptr) return;
    const int first = which ? p.s[0].blocks : 0;
    float sum = 0.0f;
    for (int b = threadIdx.x; b < p.s[which].blocks; b += 64) sum += p.a.parts[static_cast<int64_t>(first + b) * p.a.dim + i];
#pragma unroll
    for (int q = 1; q < 64; q *= 2) sum += __shfl_xor(sum, q);
    to[i] = sum;
}

int lanes_of(int dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Tokens of few heads go several to a wave where one would leave half of its lanes without a head, of q or of k (196K
// tokens of 3 + 1 heads of 26: 67 us backward, 625 one by one).
bool packed(const QkNormArgs& a) {
    for (int i = 0; i < 2; ++i)   // 32 tokens, and the tables, in 32-bit offsets
        if (a.heads[i] > 0 && (a.ld_x[i] > 1 << 23 || a.ld_dy[i] > 1 << 23)) return false;
    if (a.table_rows * a.rot * 2 >= int64_t(kPast)) return false;
    const int g = 64 / lanes_of(a.dim), most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    const int least = a.heads[0] + a.heads[1] - most > 0 ? a.heads[0] + a.heads[1] - most : most;
    return most <= g && 2 * least <= g;
}

// A token's heads are split over waves where there are few tokens: some 8192 waves fill the card.
void plan(Kernel& k, bool bwd, bool several) {
    const QkNormArgs& a = k.a;
    const int g = 64 / lanes_of(a.dim);
    for (int i = 0; i < 2; ++i) {
        Split& s = k.s[i];
        if (a.heads[i] == 0) { s = {0, 1, 1, 0}; continue; }
        const int64_t most = bwd && (a.dweight[0] || a.dweight[1]) ? kMaxBlocks : 1 << 20;
        if (several) {
            s = {0, 1, 1, 0};
            while (1 << s.head_bits < a.heads[i]) ++s.head_bits;
            const int64_t each = 2 * (g >> s.head_bits) * kWaves, blocks = (a.tokens + each - 1) / each;
            s.blocks = static_cast<int>(blocks < most ? blocks : most);
            continue;
        }
        const int groups = (a.heads[i] + g - 1) / g;
        int64_t per = a.tokens * groups / 8192;
        per = per < 1 ? 1 : per > groups ? groups : per;
        s.groups = static_cast<int>(per);
        s.splits = (groups + s.groups - 1) / s.groups;
        int64_t blocks = (a.tokens * s.splits + kWaves - 1) / kWaves;
        s.blocks = static_cast<int>(blocks < most ? blocks : most);
    }
}

template <typename T, int MODE, int LPR>
hipError_t run(const Kernel& k, bool bwd) {
    const dim3 grid(static_cast<unsigned>(k.s[0].blocks + k.s[1].blocks));
    auto start = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kWaves * 64), 0, k.a.stream, k); };
    if (packed(k.a)) bwd ? start(norm_kernel<T, MODE, LPR, true, true>) : start(norm_kernel<T, MODE, LPR, false, true>);
    else bwd ? start(norm_kernel<T, MODE, LPR, true, false>) : start(norm_kernel<T, MODE, LPR, false, false>);
    return hipGetLastError();
}

template <typename T, int MODE>
hipError_t by_lanes(const Kernel& k, bool bwd) {
    switch (lanes_of(k.a.dim)) {
        case 4: return run<T, MODE, 4>(k, bwd);
        case 8: return run<T, MODE, 8>(k, bwd);
        case 16: return run<T, MODE, 16>(k, bwd);
        default: return run<T, MODE, 32>(k, bwd);
    }
}

template <typename T>
hipError_t by_mode(const Kernel& k, bool bwd) {
    if (!k.a.vec) return by_lanes<T, kAny>(k, bwd);
    return k.a.interleaved ? by_lanes<T, kInterleaved>(k, bwd) : by_lanes<T, kHalves>(k, bwd);
}

hipError_t launch(const QkNormArgs& a, bool bwd) {
    Kernel k{a, {}};
    plan(k, bwd, packed(a));
    hipError_t e = a.bf16 ? by_mode<bf16_t>(k, bwd) : by_mode<float>(k, bwd);
    if (e != hipSuccess || !bwd || !(a.dweight[0] || a.dweight[1])) return e;
    hipLaunchKernelGGL(weight_sum_kernel, dim3(2 * a.dim), dim3(64), 0, a.stream, k);
    return hipGetLastError();
}

}  // namespace

size_t qk_norm_bwd_workspace_bytes(int64_t tokens, int q_heads, int k_heads, int dim) {
    Kernel k{};
    k.a.tokens = tokens;
    k.a.dim = dim;
    k.a.heads[0] = q_heads;
    k.a.heads[1] = k_heads;
    float any;
    k.a.dweight[0] = &any;
    plan(k, true, false);   // no fewer workgroups than with several tokens a wave
    return (static_cast<size_t>(k.s[0].blocks + k.s[1].blocks) * dim * 4 + 255) / 256 * 256;
}

hipError_t launch_qk_norm_fwd(const QkNormArgs& a) { return launch(a, false); }
hipError_t launch_qk_norm_bwd(const QkNormArgs& a) { return launch(a, true); }

}  // namespace mamba
