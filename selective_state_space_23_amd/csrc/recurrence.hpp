// Device helpers of the gated linear recurrence (recurrence.hip,
// recurrence_bwd.hip) and of the 8-bit activation checkpoints (checkpoint.hip).
//
// A tile is 128 tokens x 64 channels of one row.  16 consecutive lanes hold one
// token's 64 channels, 4 each (8 bytes of bf16, 16 of fp32), so a row of a tile
// is one contiguous span; a lane walks K consecutive tokens in registers, the
// wave's 4 groups of 16 lanes and then the workgroup's waves take the following
// ones.
#pragma once

#include "device_common.hpp"
#include "recurrence_launch.hpp"

#include <type_traits>
#include <utility>

namespace mamba {
namespace rec {

constexpr int kTileTokens = kRecChunk;   // 128: also the distance of two saved states
constexpr int kTileChannels = kPackBlock;  // 64: also the channels that share a scale

// Four consecutive channels of one token as stored.
template <typename T> struct Raw4;
template <> struct Raw4<bf16_t> { uint32_t w[2]; };
template <> struct Raw4<float> { float w[4]; };

__device__ __forceinline__ void unpack4(const Raw4<bf16_t>& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.w[0] << 16);
    v[1] = __uint_as_float(r.w[0] & 0xffff0000u);
    v[2] = __uint_as_float(r.w[1] << 16);
    v[3] = __uint_as_float(r.w[1] & 0xffff0000u);
}
__device__ __forceinline__ void unpack4(const Raw4<float>& r, float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r.w[j];
}

// Codes of four channels (bytes) times the block's scale.  A code q is decoded
// as (q + 128) s - 128 s: the flipped sign bit makes the byte unsigned, which
// the hardware converts in one instruction, and the fma rounds once.
__device__ __forceinline__ void decode4(uint32_t codes, float s, float (&v)[4]) {
    const uint32_t u = codes ^ 0x80808080u;
    const float off = -128.0f * s;
    v[0] = __builtin_fmaf(static_cast<float>(u & 0xffu), s, off);
    v[1] = __builtin_fmaf(static_cast<float>((u >> 8) & 0xffu), s, off);
    v[2] = __builtin_fmaf(static_cast<float>((u >> 16) & 0xffu), s, off);
    v[3] = __builtin_fmaf(static_cast<float>(u >> 24), s, off);
}

// Loads and stores of four channels c .. c+3 at `base` (the address of the row's
// tile, channel 0) plus a 32-bit element offset of the token.  ALIGNED: D and
// every stride are multiples of 4 and every pointer is aligned to four elements,
// so a quad is wholly inside or outside the row; `c` is then already clamped to
// a quad inside.  Otherwise each channel is read by itself, clamped to D - 1.
template <typename T, bool ALIGNED>
__device__ __forceinline__ Raw4<T> load4(const char* __restrict__ base, uint32_t tok, int c, int dim) {
    Raw4<T> r;
    constexpr uint32_t esz = Elem<T>::kBytes;
    if constexpr (ALIGNED) {
        const char* p = base + (tok + static_cast<uint32_t>(c)) * esz;
        if constexpr (esz == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            r.w[0] = v.x; r.w[1] = v.y;
        } else {
            const float4 v = *reinterpret_cast<const float4*>(p);
            r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
        }
    } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int cc = c + j < dim ? c + j : dim - 1;
            o[j] = (tok + static_cast<uint32_t>(cc)) * esz;
        }
        if constexpr (esz == 2) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = *reinterpret_cast<const uint16_t*>(base + o[j]);
            r.w[0] = h[0] | (h[1] << 16);
            r.w[1] = h[2] | (h[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[j] = *reinterpret_cast<const float*>(base + o[j]);
        }
    }
    return r;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store4(char* __restrict__ base, uint32_t tok, int c, int dim, const float (&v)[4]) {
    constexpr uint32_t esz = Elem<T>::kBytes;
    char* p = base + (tok + static_cast<uint32_t>(c)) * esz;
    if constexpr (ALIGNED) {
        if (c >= dim) return;
        if constexpr (esz == 2)
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < dim) Elem<T>::store(p, j, v[j]);
    }
}

// Four code bytes of channels c .. c+3.
template <bool ALIGNED>
__device__ __forceinline__ uint32_t load_codes(const int8_t* __restrict__ base, uint32_t tok, int c, int dim) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base);
    if constexpr (ALIGNED) return *reinterpret_cast<const uint32_t*>(p + (tok + static_cast<uint32_t>(c)));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int cc = c + j < dim ? c + j : dim - 1;
        w |= static_cast<uint32_t>(p[tok + static_cast<uint32_t>(cc)]) << (8 * j);
    }
    return w;
}

template <bool ALIGNED>
__device__ __forceinline__ void store_codes(int8_t* __restrict__ base, uint32_t tok, int c, int dim, uint32_t w) {
    uint8_t* p = reinterpret_cast<uint8_t*>(base) + (tok + static_cast<uint32_t>(c));
    if constexpr (ALIGNED) {
        if (c < dim) *reinterpret_cast<uint32_t*>(p) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < dim) p[j] = static_cast<uint8_t>(w >> (8 * j));
    }
}

// Document starts of the tile's 128 tokens (bit i: token t0 + i), the same in
// every wave.  Tokens past the row end carry no bit.
struct TileStarts {
    uint64_t lo, hi;
    __device__ __forceinline__ bool any() const { return (lo | hi) != 0; }
    // bits of the n <= 32 tokens from i on (i a multiple of n)
    __device__ __forceinline__ uint32_t bits(int i, int n) const {
        const uint64_t w = i < 64 ? lo : hi;
        return static_cast<uint32_t>(w >> (i & 63)) & (n == 32 ? 0xffffffffu : (1u << n) - 1u);
    }
};

__device__ __forceinline__ TileStarts tile_starts(const uint8_t* __restrict__ doc_start, int64_t row, int64_t t0,
                                                  int64_t seqlen) {
    TileStarts s{0, 0};
    if (doc_start == nullptr) return s;
    const int lane = threadIdx.x & 63;
    const int64_t ta = t0 + lane, tb = ta + 64;
    const bool a = ta < seqlen && doc_start[row + ta] != 0;
    const bool b = tb < seqlen && doc_start[row + tb] != 0;
    s.lo = __ballot(a);
    s.hi = __ballot(b);
    return s;
}

// softplus of the decay parameter: once per channel and workgroup, with the math
// library's own functions (its error goes into every token's decay alike).
__device__ __forceinline__ float softplus_exact(float v) {
    return __builtin_fmaxf(v, 0.0f) + log1pf(expf(-__builtin_fabsf(v)));
}

__device__ __forceinline__ float sigmoid_f(float v) { return rcp_fast(1.0f + exp2_fast(-v * kLog2e)); }

// The decay a = 2^la2 and 1 - a^2 for la2 = log2 a <= 0.  1 - a comes from the
// series of 1 - e^-t, t = -log a, where 1 - a would cancel (t < 0.35: the first
// term left out is below 2e-8 of the sum) and from a itself above.
__device__ __forceinline__ void decay_terms(float la2, float& a, float& om) {
    a = exp2_fast(la2);
    const float t = -kLn2 * la2;
    float p = __builtin_fmaf(t, 1.0f / 5040.0f, -1.0f / 720.0f);
    p = __builtin_fmaf(t, p, 1.0f / 120.0f);
    p = __builtin_fmaf(t, p, -1.0f / 24.0f);
    p = __builtin_fmaf(t, p, 1.0f / 6.0f);
    p = __builtin_fmaf(t, p, -0.5f);
    p = __builtin_fmaf(t, p, 1.0f);
    const float d = t < 0.35f ? t * p : 1.0f - a;
    om = d * (1.0f + a);
}

// Value of lane `16 * (lane / 16) + N` in every lane of the row of 16
// (row_newbcast:N).
template <int N>
__device__ __forceinline__ float row16_bcast(float x) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + N, 0xf, 0xf, false));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, false));
}

// Largest magnitude of a block as bits: comparing the bit patterns of |x| as
// integers orders NaN above infinity above every finite number.
__device__ __forceinline__ uint32_t abs_bits_max4(const float (&v)[4], uint32_t m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}

// Scale and inverse step of a block whose largest magnitude has the bits m:
// scale = m (1 / 127) and inv = (1 / m) 127, each factor and product rounded.
// A NaN or an infinity makes both NaN, so that the whole block decodes to NaN;
// blocks below 2^-100 use m = 2^-100, which keeps inv finite.
__device__ __forceinline__ void block_scale(uint32_t mbits, float& scale, float& inv) {
    float m = __uint_as_float(mbits);
    m = m < 0x1p-100f ? 0x1p-100f : m;
    scale = m * (1.0f / 127.0f);
    inv = (1.0f / m) * 127.0f;
    if (mbits >= 0x7f800000u) scale = inv = __uint_as_float(0x7fc00000u);
}

// round(v * inv) to the nearest integer, ties to even, as a byte: the product is
// rounded first, then adding 1.5 * 2^23 leaves the integer in the low bits.
__device__ __forceinline__ uint32_t encode4(const float (&v)[4], float inv) {
#pragma clang fp contract(off)
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t = v[j] * inv;
        b[j] = __float_as_uint(t + 12582912.0f) & 0xffu;
    }
    return b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
}

// Affine maps h -> P h + H of stretches of tokens.  The sign of P marks a map
// that ignores its input (a document start inside the stretch).
__device__ __forceinline__ bool is_reset(float P) { return __float_as_uint(P) >> 31; }
// (P, H) after (p, h): first the earlier tokens' map (p, h), then (P, H).
__device__ __forceinline__ void compose(float& P, float& H, float p, float h) {
    const bool cut = is_reset(P);
    H = cut ? H : __builtin_fmaf(P, h, H);
    P = cut ? P : P * p;
}
__device__ __forceinline__ float apply(float P, float H, float h) { return is_reset(P) ? H : __builtin_fmaf(P, h, H); }

template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

// A lane's K quads of one input, plain or 8-bit.
template <typename T, bool ALIGNED, bool PIN, int K> struct LaneIn {
    Raw4<T> r[K];
    __device__ __forceinline__ void load(const void* p, const Packed&, int64_t row_tok, int64_t ld, int tok, int nv,
                                         int c, int dim, int, int64_t) {
        const char* base = static_cast<const char*>(p) + row_tok * ld * Elem<T>::kBytes;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = tok + k < nv ? tok + k : nv - 1;
            r[k] = load4<T, ALIGNED>(base, static_cast<uint32_t>(t) * static_cast<uint32_t>(ld), c, dim);
        }
    }
    template <int k> __device__ __forceinline__ void get(float (&v)[4]) const { unpack4(r[k], v); }
};
template <typename T, bool ALIGNED, int K> struct LaneIn<T, ALIGNED, true, K> {
    uint32_t q[K];
    static constexpr int kPer = 16 / K;   // lanes of a row of 16 that hold one token's scale
    float s;                              // scale of token (lane % 16) / kPer of the lane's K
    __device__ __forceinline__ void load(const void*, const Packed& p, int64_t row_tok, int64_t, int tok, int nv,
                                         int c, int dim, int ct, int64_t rows) {
        const int8_t* base = p.q + row_tok * dim;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = tok + k < nv ? tok + k : nv - 1;
            q[k] = load_codes<ALIGNED>(base, static_cast<uint32_t>(t) * static_cast<uint32_t>(dim), c, dim);
        }
        const int st = tok + static_cast<int>(threadIdx.x & 15) / kPer;
        s = p.scale[ct * rows + row_tok + (st < nv ? st : nv - 1)];
    }
    template <int k> __device__ __forceinline__ void get(float (&v)[4]) const { decode4(q[k], row16_bcast<kPer * k>(s), v); }
};

// Writes the 8-bit checkpoint of a lane's K = 4 quads.  The magnitudes of the 4
// tokens are reduced over the 16 lanes by halving: at each of the first two
// steps a lane keeps half of its tokens and takes the partner's values for them
// (5 exchanges in place of 4 four-step reductions), after which lanes 4 k .. 4 k
// + 3 of the row hold token k's, do its two divisions once, and the scales of
// the wave's 16 tokens are one contiguous store.
template <typename T, bool ALIGNED, int K>
__device__ __forceinline__ void save_packed(const LaneIn<T, ALIGNED, false, K>& in, const Packed& p, int64_t row_tok,
                                            int tok, int nv, int c, int dim, int ct, int64_t rows) {
    static_assert(K == 4, "the halving below is written for four tokens");
    const int li = threadIdx.x & 15;
    uint32_t m[4];
    static_for<4>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        float v[4];
        in.template get<k>(v);
        m[k] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
            if (ALIGNED || c + j < dim) m[k] = b > m[k] ? b : m[k];
        }
        if (ALIGNED && c >= dim) m[k] = 0;
    });
    auto umax = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    const bool b3 = li & 8, b2 = li & 4;
    uint32_t m2[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        m2[k] = umax(b3 ? m[k + 2] : m[k], dpp_u32<0x128>(b3 ? m[k] : m[k + 2]));   // row_ror:8
    // row_half_mirror: lane i of a half-row reads lane 7 - i, in its other quad
    uint32_t m1 = umax(b2 ? m2[1] : m2[0], dpp_u32<0x141>(b2 ? m2[0] : m2[1]));
    m1 = umax(m1, dpp_u32<0x4E>(m1));   // quad_perm [2, 3, 0, 1]
    m1 = umax(m1, dpp_u32<0xB1>(m1));   // quad_perm [1, 0, 3, 2]
    float scale, inv;
    block_scale(m1, scale, inv);
    const int t_sc = tok + (li >> 2);
    if ((li & 3) == 0 && t_sc < nv) p.scale[ct * rows + row_tok + t_sc] = scale;
    int8_t* base = p.q + row_tok * dim;
    static_for<4>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        float v[4];
        in.template get<k>(v);
        const uint32_t w = encode4(v, row16_bcast<4 * k>(inv));
        if (tok + k < nv)
            store_codes<ALIGNED>(base, static_cast<uint32_t>(tok + k) * static_cast<uint32_t>(dim), c, dim, w);
    });
}

}  // namespace rec
}  // namespace mamba
