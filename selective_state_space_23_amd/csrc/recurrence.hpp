// Device helpers of the gated linear recurrence (recurrence.hip,
// recurrence_bwd.hip) and of the 8-bit activation checkpoints (checkpoint.hip).
//
// A tile is 128 tokens x 64 channels of one row.  In the recurrence 32
// consecutive lanes hold one token's 64 channels, 2 each (4 bytes of bf16, 8 of
// fp32), so a row of a tile is one contiguous span; a lane walks K consecutive
// tokens in registers, the wave's two halves and then the workgroup's waves take
// the following ones.  (4 channels a lane, 16 lanes a token, halve the loads but
// need three exchanges across the wave's four groups where two halves need one.)
#pragma once

#include "device_common.hpp"
#include "recurrence_launch.hpp"

#include <type_traits>
#include <utility>

namespace mamba {
namespace rec {

constexpr int kTileTokens = kRecChunk;   // 128: also the distance of two saved states
constexpr int kTileChannels = kPackBlock;  // 64: also the channels that share a scale

// V (2 or 4) consecutive channels of one token as stored.
template <typename T, int V> struct Raw {
    uint32_t w[V * Elem<T>::kBytes / 4];
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&v)[V]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = __uint_as_float(j % 2 == 0 ? r.w[j / 2] << 16 : r.w[j / 2] & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = __uint_as_float(r.w[j]);
    }
}

// Codes of V channels (bytes) times the block's scale: rounded once.
template <int V>
__device__ __forceinline__ void decode(uint32_t codes, float s, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = static_cast<float>(static_cast<int8_t>(codes >> (8 * j))) * s;
}

// A tile's rows of one tensor as a buffer: `n` tokens of `dim` channels, `ld`
// elements apart, from the tile's first token on.  Reads behind the last token
// give zero and writes there are dropped (the buffer's range check), so tokens
// past the row end need no other care.  Byte offsets in a tile fit 31 bits.
constexpr uint32_t kNoStore = 0x7fffff00u;   // a lane offset past any tile
using Rsrc = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Rsrc tile_rsrc(const void* first, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(first), 0, static_cast<int>(bytes), 0x00027000);
}
template <int ESZ>
__device__ __forceinline__ Rsrc rows_rsrc(const void* p, int64_t token, int n, int64_t ld, int dim) {
    return tile_rsrc(static_cast<const char*>(p) + token * ld * ESZ, n > 0 ? ((n - 1) * ld + dim) * ESZ : 0);
}

// Kernels that work off many tiles read their arguments anew where they need them
// (scalar loads that hit the cache): held in registers across the loop, the
// pointers and sizes of a dozen tensors overflow the scalar registers.  The
// argument struct is the kernel's only parameter, at the start of its arguments.
template <typename Args> using ArgsPtr = const __attribute__((address_space(4))) Args*;
template <typename Args>
__device__ __forceinline__ ArgsPtr<Args> kernel_args() {
    auto p = (ArgsPtr<Args>)(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    return p;
}

// The lane, formed where it is used, for the same reason.
__device__ __forceinline__ uint32_t lane_now() {
    uint32_t t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t & 63;
}

// tok * step + c for a token of a tile and a step below 2^24, and the offset one
// step on: formed where they are used, for the same reason.
__device__ __forceinline__ uint32_t next_offset(uint32_t off, uint32_t step) {
    off += step;
    asm volatile("" : "+v"(off));
    return off;
}
__device__ __forceinline__ uint32_t tile_offset(int tok, uint32_t step, int c) {
    asm volatile("" : "+v"(tok));
    return __umul24(static_cast<uint32_t>(tok), step) + static_cast<uint32_t>(c);
}

// One float of row `row` of a (rows, dim) array per lane: channels past dim, and a
// null array, read 0 and store nothing.  The loops over tiles have no divergent
// branch at all (range checks and selects in their place): the compiler has been
// seen to copy live registers at the join of such a branch before it restores the
// execution mask, which leaves the masked lanes' copies behind.
__device__ __forceinline__ Rsrc row_rsrc(const float* p, int64_t row, int64_t dim) {
    return tile_rsrc(p + row * dim, p != nullptr ? dim * 4 : 0);
}
__device__ __forceinline__ float row_load(const float* p, int64_t row, int64_t dim, int d) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_rsrc(p, row, dim), 4 * d, 0, 0));
}
__device__ __forceinline__ void row_store(float* p, int64_t row, int64_t dim, int d, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), row_rsrc(p, row, dim), 4 * d, 0, 0);
}

// The same for a store: past the buffer where the channel is past D.
__device__ __forceinline__ uint32_t store_offset(int tok, uint32_t step, int c, bool inside) {
    const uint32_t off = tile_offset(tok, step, c);
    return inside ? off : kNoStore;
}

// V consecutive channels at a byte offset.  ALIGNED: D and every stride are
// multiples of 4 and every pointer is aligned to four elements; else element by
// element.  Channels past D read what follows (another token's, or zero).
template <typename T, int V, bool ALIGNED>
__device__ __forceinline__ Raw<T, V> load_raw(Rsrc rs, uint32_t off) {
    Raw<T, V> r;
    constexpr int kWords = sizeof(r.w) / 4;
    if constexpr (ALIGNED && kWords == 1) {
        r.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
    } else if constexpr (ALIGNED && kWords == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        r.w[0] = v[0]; r.w[1] = v[1];
    } else if constexpr (ALIGNED) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = v[j];
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const uint32_t lo = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, off + 2 * j, 0, 0));
            const uint32_t hi = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, off + 2 * j + 2, 0, 0));
            r.w[j / 2] = lo | (hi << 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) r.w[j] = __builtin_amdgcn_raw_buffer_load_b32(rs, off + 4 * j, 0, 0);
    }
    return r;
}

// Cache policy of whole lines that a call reads or writes once: they leave the caches first
// (2 x 32768 x 1536 training step 796 us for 812, 8 x 2048 x 1536 backward 112 for 116,
// forward 81 for 82; only reads or only writes give half of it).  Between products that write its inputs
// and read its outputs a call gains where its tensors pass the 256 MB that the card
// caches (16 x 2048 x 1536 forward with those products 306 us for 310, backward 367 for 381) and loses
// below (forward 4 x 2048 97 for 92, 8 x 2048 165 for 157; backward 4 x 2048 117 for 110).
constexpr int kStreamed = 2;   // nt

// `off` is past the buffer where the first channel is past D; `left` of the
// channels exist (looked at only when not ALIGNED).
template <typename T, int V, bool ALIGNED>
__device__ __forceinline__ void store_vals(Rsrc rs, uint32_t off, int left, const float (&v)[V]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t o = j < left ? off + j * Elem<T>::kBytes : kNoStore;
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v[j]), rs, o, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), rs, o, 0, 0);
        }
    } else if constexpr (sizeof(T) == 2 && V == 2) {
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(v[0], v[1]), rs, off, 0, kStreamed);
    } else if constexpr (sizeof(T) == 2) {
        const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        __builtin_amdgcn_raw_buffer_store_b64(w, rs, off, 0, kStreamed);
    } else if constexpr (V == 2) {
        const u32x2 w = {__float_as_uint(v[0]), __float_as_uint(v[1])};
        __builtin_amdgcn_raw_buffer_store_b64(w, rs, off, 0, kStreamed);
    } else {
        const u32x4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        __builtin_amdgcn_raw_buffer_store_b128(w, rs, off, 0, kStreamed);
    }
}

// V code bytes.
template <int V, bool ALIGNED>
__device__ __forceinline__ uint32_t load_codes(Rsrc rs, uint32_t off) {
    if constexpr (ALIGNED && V == 4) return __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
    if constexpr (ALIGNED && V == 2) return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0));
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        w |= static_cast<uint32_t>(static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(rs, off + j, 0, 0))) << (8 * j);
    return w;
}

template <int V, bool ALIGNED>
__device__ __forceinline__ void store_codes(Rsrc rs, uint32_t off, int left, uint32_t w) {
    if constexpr (ALIGNED && V == 4) {
        __builtin_amdgcn_raw_buffer_store_b32(w, rs, off, 0, 0);
    } else if constexpr (ALIGNED) {
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(w), rs, off, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(w >> (8 * j)), rs, j < left ? off + j : kNoStore, 0, 0);
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

// The lane's two flags of a tile, loaded ahead of their use.
struct StartFlags {
    uint32_t a, b;
    __device__ __forceinline__ void load(const uint8_t* doc_start, int64_t row_tok, int nv) {
        const int lane = threadIdx.x & 63;
        const Rsrc rs = tile_rsrc(doc_start + row_tok, doc_start != nullptr ? nv : 0);
        a = static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(rs, lane, 0, 0));
        b = static_cast<uint8_t>(__builtin_amdgcn_raw_buffer_load_b8(rs, lane + 64, 0, 0));
    }
    __device__ __forceinline__ TileStarts starts() const { return TileStarts{__ballot(a != 0), __ballot(b != 0)}; }
};

// softplus of the decay parameter: once per channel and workgroup, with the math
// library's own functions (its error goes into every token's decay alike).
__device__ __forceinline__ float softplus_exact(float v) {
    return __builtin_fmaxf(v, 0.0f) + log1pf(expf(-__builtin_fabsf(v)));
}

__device__ __forceinline__ float sigmoid_f(float v) { return rcp_fast(1.0f + exp2_fast(-v * kLog2e)); }

// The decay a = 2^la2 and 1 - a^2 for la2 = log2 a <= 0.  1 - a^2 cancels where a
// is near 1: with y = -2 log a it is y p(y) there, p a degree-4 Chebyshev
// interpolant of (1 - e^-y) / y on [0, 0.35] written in la2 = -y / (2 log 2), off by
// at most 4e-8 of it.  Above 0.35 the subtraction loses at most two bits.
__device__ __forceinline__ void decay_terms(float la2, float& a, float& om) {
    a = exp2_fast(la2);
    float p = __builtin_fmaf(la2, -0.03692888095974922f, -0.1526569277048111f);
    p = __builtin_fmaf(la2, p, -0.4439232051372528f);
    p = __builtin_fmaf(la2, p, -0.9609025716781616f);
    p = __builtin_fmaf(la2, p, -1.3862943649291992f);
    float near = la2 * p, far = __builtin_fmaf(-a, a, 1.0f);
    asm volatile("" : "+v"(near), "+v"(far));   // both formed: the choice stays a select, not a branch
    om = la2 > -0.25247162580490112f ? near : far;
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

// Scale and inverse step of a block whose largest magnitude has the bits m (the
// bit patterns of |x| compared as integers order NaN above infinity above every
// finite number):
// scale = m (1 / 127) and inv = (1 / m) 127, each factor and product rounded.
// A NaN or an infinity makes both NaN, so that the whole block decodes to NaN;
// blocks below 2^-100 use m = 2^-100, which keeps inv finite.
__device__ __forceinline__ void block_scale(uint32_t mbits, float& scale, float& inv) {
    float m = __uint_as_float(mbits);
    m = m < 0x1p-100f ? 0x1p-100f : m;
    float s = m * (1.0f / 127.0f), i = (1.0f / m) * 127.0f;
    asm volatile("" : "+v"(s), "+v"(i));   // a select below, not a branch
    const bool finite = mbits < 0x7f800000u;
    scale = finite ? s : __uint_as_float(0x7fc00000u);
    inv = finite ? i : __uint_as_float(0x7fc00000u);
}

// round(v * inv) to the nearest integer, ties to even, as bytes: the product is
// rounded first, then adding 1.5 * 2^23 leaves the integer in the low bits.
template <int V>
__device__ __forceinline__ uint32_t encode(const float (&v)[V], float inv) {
#pragma clang fp contract(off)
    static_assert(V % 2 == 0);
    uint32_t w[V / 2];
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        const float lo = v[j] * inv, hi = v[j + 1] * inv;
        // byte 0 of both
        w[j / 2] = __builtin_amdgcn_perm(__float_as_uint(hi + 12582912.0f), __float_as_uint(lo + 12582912.0f), 0x0c0c0400u);
    }
    if constexpr (V == 2) return w[0];
    else return w[0] | (w[1] << 16);
}

// Affine maps h -> P h + H of stretches of tokens.  The sign of P marks a map
// that ignores its input (a document start inside the stretch); CUT false: no such
// map can occur.
__device__ __forceinline__ bool is_reset(float P) { return __float_as_uint(P) >> 31; }
template <bool CUT = true>
__device__ __forceinline__ float apply(float P, float H, float h) {
    float r = __builtin_fmaf(P, h, H);
    if constexpr (CUT) {
        asm volatile("" : "+v"(r));   // a select, not a branch
        r = is_reset(P) ? H : r;
    }
    return r;
}
// (P, H) after (p, h): first the earlier tokens' map (p, h), then (P, H).
template <bool CUT = true>
__device__ __forceinline__ void compose(float& P, float& H, float p, float h) {
    H = apply<CUT>(P, H, h);
    float r = P * p;
    if constexpr (CUT) {
        asm volatile("" : "+v"(r));
        r = is_reset(P) ? P : r;
    }
    P = r;
}

template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_impl<N>(f, std::make_integer_sequence<int, N>{});
}

// A tile's place: uniform over the workgroup.
struct Tile {
    int ct, tile, nv;      // channel tile, token tile, tokens in it (0: no such tile)
    int pos;               // position in the chain
    int64_t b, row_tok;    // row, first token counted over all rows
};

// BYTES of a tile's rows (ROW bytes each, from token `first` on, at byte `col` of the
// row) into LDS, row after row: a load moves 16 bytes a lane to lds + 16 lane, or 4 to
// lds + 4 lane where rows do not lie on 16 bytes or the wave has less than 1024.
// Issued by a whole wave; nothing waits here.  (8-bit rows are half a line, the other
// half the neighbouring tile's: POLICY 0.)
template <int ROW, int BYTES, int POLICY>
__device__ __forceinline__ void stage_rows(char* lds, Rsrc rs, uint32_t step, int first, uint32_t col, bool wide) {
    typedef __attribute__((address_space(3))) void* Lds;
    const int lane = lane_now();
    if (BYTES % 1024 == 0 && wide) {
        constexpr int kLanes = ROW / 16, kRows = 64 / kLanes;
        uint32_t off = tile_offset(first + lane / kLanes, step, col + lane % kLanes * 16);
#pragma unroll
        for (int i = 0; i < BYTES; i += 1024) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (Lds)(lds + i), 16, off, 0, 0, POLICY);
            off = next_offset(off, kRows * step);
        }
    } else {
        constexpr int kLanes = ROW / 4, kRows = 64 / kLanes;
        uint32_t off = tile_offset(first + lane / kLanes, step, col + lane % kLanes * 4);
#pragma unroll
        for (int i = 0; i < BYTES; i += 256) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (Lds)(lds + i), 4, off, 0, 0, POLICY);
            off = next_offset(off, kRows * step);
        }
    }
}
// Rows of `bytes` bytes, `step` apart, from p on: each starts and ends on 16 bytes.
__device__ __forceinline__ bool rows_of_16(const void* p, uint32_t step, uint32_t bytes) {
    return ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) | step | bytes) & 15) == 0;
}

// Waits until at most N of the wave's loads and stores are under way (they end in
// order): what was issued before the last N is done.
template <int N>
__device__ __forceinline__ void wait_all_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The wave's LDS reads are done.
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A lane's place in a tile of the recurrence's kernels.
constexpr int kV = 2;                            // channels of a lane
constexpr int kRow = kTileChannels / kV;         // lanes of a token

// The lane's channel pair and half of the wave, and its first of K tokens: formed
// where they are used, for registers.
template <int K> struct LanePlace {
    int li, half, tok;
    __device__ __forceinline__ explicit LanePlace(int wave) {
        const int lane = static_cast<int>(lane_now());
        li = lane % kRow;
        half = lane / kRow;
        tok = (wave * 2 + half) * K;
    }
    __device__ __forceinline__ int channel(const Tile& t) const { return t.ct * kTileChannels + kV * li; }
};

// A lane's K pairs of one input, plain or 8-bit: tokens tok .. tok + K - 1 of the
// tile, channels c and c + 1.  load() reads them from memory; stage() has memory
// write the wave's tokens to LDS (no registers held while in flight) and read()
// takes the lane's from there once they have landed.
template <typename T, bool ALIGNED, bool PIN, int K> struct LaneIn {
    static constexpr int kRowBytes = kTileChannels * Elem<T>::kBytes;   // one token's
    static constexpr int kStageBytes = 2 * K * kRowBytes;               // one wave's
    Raw<T, kV> r[K];
    template <typename P>
    __device__ __forceinline__ void load(const void* p, const P&, const Tile& t, int ld, int tok, int c, int dim,
                                         int64_t) {
        constexpr int esz = Elem<T>::kBytes;
        const Rsrc rs = rows_rsrc<esz>(p, t.row_tok, t.nv, ld, dim);
        const uint32_t step = static_cast<uint32_t>(ld) * esz;
        uint32_t off = tile_offset(tok, step, c * esz);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            r[k] = load_raw<T, kV, ALIGNED>(rs, off);
            off = next_offset(off, step);
        }
    }
    template <typename P>
    __device__ __forceinline__ void stage(char* lds, const void* p, const P&, const Tile& t, int ld, int wave, int dim,
                                          int64_t) {
        constexpr int esz = Elem<T>::kBytes;
        const uint32_t step = static_cast<uint32_t>(ld) * esz;
        stage_rows<kRowBytes, kStageBytes, kStreamed>(lds, rows_rsrc<esz>(p, t.row_tok, t.nv, ld, dim), step, wave * 2 * K,
                                           t.ct * kRowBytes, rows_of_16(p, step, dim * esz));
    }
    __device__ __forceinline__ void read(const char* lds, int half, int li) {
        const char* p = lds + half * K * kRowBytes + li * kV * Elem<T>::kBytes;
#pragma unroll
        for (int k = 0; k < K; ++k) __builtin_memcpy(&r[k], p + k * kRowBytes, sizeof(r[k]));
    }
    template <int k> __device__ __forceinline__ void get(float (&v)[kV]) const { unpack(r[k], v); }
    // The same, unpacked here and not where the compiler could do it for several
    // uses at once (twice the registers across everything in between).
    template <int k> __device__ __forceinline__ void take(float (&v)[kV]) {
        if constexpr (sizeof(T) == 2) {
            asm volatile("v_lshlrev_b32 %0, 16, %1" : "=v"(v[0]) : "v"(r[k].w[0]));
            asm volatile("v_and_b32 %0, 0xffff0000, %1" : "=v"(v[1]) : "v"(r[k].w[0]));
        } else {
            unpack(r[k], v);
        }
    }
};
template <typename T, bool ALIGNED, int K> struct LaneIn<T, ALIGNED, true, K> {
    static constexpr int kRowBytes = kTileChannels;
    static constexpr int kCodeBytes = 2 * K * kRowBytes;
    static constexpr int kStageBytes = kCodeBytes + 256;   // behind the codes the wave's 2 K scales
    uint32_t q[K];
    static constexpr int kPer = 16 / K;   // lanes of a DPP row of 16 that hold one token's scale
    float s;                              // scale of token (lane % 16) / kPer of the lane's K
    template <typename P>
    __device__ __forceinline__ void load(const void*, const P& p, const Tile& t, int, int tok, int c, int dim,
                                         int64_t rows) {
        const Rsrc rs = rows_rsrc<1>(p.q, t.row_tok, t.nv, dim, dim);
        uint32_t off = tile_offset(tok, dim, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            q[k] = load_codes<kV, ALIGNED>(rs, off);
            off = next_offset(off, dim);
        }
        const Rsrc ss = tile_rsrc(p.scale + t.ct * rows + t.row_tok, t.nv * 4);
        s = __uint_as_float(
            __builtin_amdgcn_raw_buffer_load_b32(ss, 4 * (tok + static_cast<int>(threadIdx.x & 15) / kPer), 0, 0));
    }
    template <typename P>
    __device__ __forceinline__ void stage(char* lds, const void*, const P& p, const Tile& t, int, int wave, int dim,
                                          int64_t rows) {
        stage_rows<kRowBytes, kCodeBytes, 0>(lds, rows_rsrc<1>(p.q, t.row_tok, t.nv, dim, dim), dim, wave * 2 * K,
                                          t.ct * kRowBytes, rows_of_16(p.q, dim, dim));
        const Rsrc ss = tile_rsrc(p.scale + t.ct * rows + t.row_tok, t.nv * 4);
        const int lane = lane_now();
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ss, (__attribute__((address_space(3))) void*)(lds + kCodeBytes), 4,
                                                 lane < 2 * K ? 4 * (wave * 2 * K + lane) : kNoStore, 0, 0, 0);
    }
    __device__ __forceinline__ void read(const char* lds, int half, int li) {
        const char* p = lds + half * K * kRowBytes + li * kV;
#pragma unroll
        for (int k = 0; k < K; ++k) q[k] = *reinterpret_cast<const uint16_t*>(p + k * kRowBytes);
        s = *reinterpret_cast<const float*>(lds + kCodeBytes + 4 * (half * K + li % 16 / kPer));
    }
    template <int k> __device__ __forceinline__ void take(float (&v)[kV]) {
        asm volatile("" : "+v"(q[k]));
        decode(q[k], row16_bcast<kPer * k>(s), v);
    }
};

// Writes the 8-bit checkpoint of a lane's K = 8 pairs.  The magnitudes of the 8
// tokens are reduced over a DPP row of 16 lanes by halving: at each of three steps
// a lane keeps half of its tokens and takes its partner's values for them (7
// exchanges in place of 8 four-step reductions); two more steps join the lanes and
// the token's other 16.  Lanes 2 k and 2 k + 1 of a row then hold token k's, do
// its division once, and the scales of the wave's 16 tokens are one contiguous
// store.
template <typename T, bool ALIGNED, int K, typename P>
__device__ __forceinline__ void save_packed(const LaneIn<T, ALIGNED, false, K>& in, const P& p, const Tile& t,
                                            int tok, int c, int dim, int64_t rows) {
    static_assert(K == 8, "the halving below is written for eight tokens");
    const int li = threadIdx.x & 15;
    // Magnitude bits of the channels that exist: bfloat16 ones as halves of a word, whose
    // maxima are taken side by side.
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    uint32_t keep[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) keep[j] = c + j < dim ? 0x7fffffffu : 0u;
    uint32_t m[8];
    static_for<8>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        if constexpr (sizeof(T) == 2) {
            m[k] = in.r[k].w[0] & ((keep[0] >> 16) | (keep[1] & 0xffff0000u));
        } else {
            const uint32_t a = in.r[k].w[0] & keep[0], b = in.r[k].w[1] & keep[1];
            m[k] = a > b ? a : b;
        }
    });
    auto umax = [](uint32_t x, uint32_t y) {
        if constexpr (sizeof(T) == 2) {
            const u16x2 a = __builtin_bit_cast(u16x2, x), b = __builtin_bit_cast(u16x2, y);
            return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
        } else {
            return x > y ? x : y;
        }
    };
    const bool b3 = li & 8, b2 = li & 4, b1 = li & 2;
    uint32_t m4[4], m2[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) m4[k] = umax(b3 ? m[k + 4] : m[k], dpp_u32<0x128>(b3 ? m[k] : m[k + 4]));   // row_ror:8
#pragma unroll
    for (int k = 0; k < 2; ++k)   // row_half_mirror: lane i of a half-row reads lane 7 - i, in its other quad
        m2[k] = umax(b2 ? m4[k + 2] : m4[k], dpp_u32<0x141>(b2 ? m4[k] : m4[k + 2]));
    uint32_t m1 = umax(b1 ? m2[1] : m2[0], dpp_u32<0x4E>(b1 ? m2[0] : m2[1]));   // quad_perm [2, 3, 0, 1]
    m1 = umax(m1, dpp_u32<0xB1>(m1));                                            // quad_perm [1, 0, 3, 2]
    m1 = umax(m1, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m1), 16)));
    if constexpr (sizeof(T) == 2) {
        const uint32_t lo = m1 << 16, hi = m1 & 0xffff0000u;
        m1 = lo > hi ? lo : hi;
    }
    float scale, inv;
    block_scale(m1, scale, inv);
    const Rsrc ss = tile_rsrc(p.scale + t.ct * rows + t.row_tok, t.nv * 4);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), ss,
                                          (threadIdx.x & 17) == 0 ? 4 * (tok + (li >> 1)) : kNoStore, 0, 0);
    const Rsrc rs = rows_rsrc<1>(p.q, t.row_tok, t.nv, dim, dim);
    uint32_t off = store_offset(tok, dim, c, c < dim);
    static_for<8>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        float v[kV];
        in.template get<k>(v);
        store_codes<kV, ALIGNED>(rs, off, dim - c, encode(v, row16_bcast<2 * k>(inv)));
        off = next_offset(off, dim);
    });
}

// Joining the tiles of a chain (one row, 64 channels) in one pass over the data.
// Tiles are taken in order (position 0, 1, ... of a chain: from the left in the
// forward, from the right in the backward).  Each publishes its composed map as
// soon as it has it, then finds the value entering it from the nearest earlier
// position whose outgoing value is published, applying the maps in between in
// order.  That is the operation sequence of the tiles' own outgoing values, so
// the result does not depend on how far a tile had to look.
//
// Every word is published by one store and read by loads at agent scope, aligned
// and so whole: a map is one 64-bit word (P, H), a value one 32-bit word.  All bits
// set (in H) means "not there yet": the launch clears the words first, and a NaN
// with that pattern is stored as the usual one.
//
// Every wait ends: workgroups draw tiles by tickets, position by position over the
// chains (so that neighbours in a row, whose lines meet, are near in time), and work on them in the order drawn.  The positions a
// workgroup waits for have lower tickets: of the tickets not yet worked off, the
// lowest is the current one of a workgroup that runs, and all that it waits for is
// published.  Against a workspace that another call overwrites meanwhile (which
// the caller has to exclude) the wait is bounded too: after kMaxPolls, 1.5 seconds,
// the value is NaN.
struct Chain {
    uint64_t* map;     // [chain][position][64]
    uint32_t* value;   // [chain][position][64]
    uint32_t* next;    // [group]: tickets drawn
    const float* rate; // [64 * channel tiles]: -c log2(e) softplus(a_param)
};

// Earlier positions looked at.  A long row's value goes from tile to tile by as many
// positions a trip: with few chains that is what a call takes (65536 x 512 in bfloat16 132
// us for 194, 32768 x 128 in float32 43 for 81).  `most` chains, of 32 tiles and more, look
// far: 16 in the forward, whatever the type (16384 tokens, far and near: bfloat16 with
// z and checkpoints 12 chains 66 and 75, 16 81 and 83; float32 9 chains 44 and 74, 16 62 and 78, 24 95 and
// 96; with z 9 chains 54 and 59, 16 74 and 74, 24 111 and 108), 8 in the backward.
constexpr int kLookNear = 2, kLookFar = 8;
inline bool look_far(int64_t chains, int64_t ntiles, int64_t most) { return chains <= most && ntiles >= 32; }
constexpr int kMaxPolls = 1 << 22;   // a third of a microsecond each

__device__ __forceinline__ uint32_t not_all_ones(float x) {
    const uint32_t b = __float_as_uint(x);
    return b == 0xffffffffu ? 0x7fc00000u : b;
}

// The words of one chain, as buffers: accesses at agent scope (the cache-policy
// bit kAgentScope), each word whole.
constexpr int kAgentScope = 16;
template <int kLook> struct ChainWords {
    Rsrc map, value;
    __device__ __forceinline__ void init(uint64_t* maps, uint32_t* values, int64_t word0, int ntiles) {
        map = tile_rsrc(maps + word0, static_cast<int64_t>(ntiles) * kTileChannels * 8);
        value = tile_rsrc(values + word0, static_cast<int64_t>(ntiles) * kTileChannels * 4);
    }
    __device__ __forceinline__ void publish_map(int pos, float P, float H) const {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 w = {__float_as_uint(P), not_all_ones(H)};
        __builtin_amdgcn_raw_buffer_store_b64(w, map, lane_now() * 8, pos * (kTileChannels * 8), kAgentScope);
    }
    __device__ __forceinline__ void publish_value(int pos, float v) const {
        __builtin_amdgcn_raw_buffer_store_b32(not_all_ones(v), value, lane_now() * 4, pos * (kTileChannels * 4),
                                              kAgentScope);
    }
    // What the kLook positions before `pos` have published so far: read ahead of
    // look_back().  Before position 0 the words read as zero (the range check).
    struct Seen {
        uint32_t v[kLook], mp[kLook - 1], mh[kLook - 1];
    };
    __device__ __forceinline__ void read_value(Seen& s, int k, int p) const {
        s.v[k] = __builtin_amdgcn_raw_buffer_load_b32(value, p * (kTileChannels * 4) + lane_now() * 4, 0,
                                                      kAgentScope);
    }
    __device__ __forceinline__ void read_map(Seen& s, int k, int p) const {
        const auto w = __builtin_amdgcn_raw_buffer_load_b64(map, p * (kTileChannels * 8) + lane_now() * 8, 0,
                                                            kAgentScope);
        s.mp[k] = w[0];
        s.mh[k] = w[1];
    }
    __device__ __forceinline__ Seen peek(int pos) const {
        Seen s;
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
            read_value(s, k, pos - 1 - k);
            if (k < kLook - 1) read_map(s, k, pos - 1 - k);
        }
        return s;
    }
    // The value entering position `pos` for the lane's channel; `first` enters
    // position 0.  All 64 lanes.
    __device__ __forceinline__ float look_back(int pos, float first, Seen s) const {
        for (int polls = 0; polls < kMaxPolls; ++polls) {
            bool ok = false;
            float c = 0.0f;
#pragma unroll
            for (int k = kLook - 1; k >= 0; --k) {
                if (k < kLook - 1) {
                    c = apply(__uint_as_float(s.mp[k]), __uint_as_float(s.mh[k]), c);
                    ok = ok && s.mh[k] != 0xffffffffu;
                }
                const bool there = s.v[k] != 0xffffffffu;
                c = there ? __uint_as_float(s.v[k]) : c;
                ok = ok || there;
                if (pos - 1 - k == -1) {
                    c = first;
                    ok = true;
                }
            }
            if (__all(ok)) return c;
            __builtin_amdgcn_s_sleep(1);
            asm volatile("" ::: "memory");   // every poll reads memory
#pragma unroll
            for (int k = 0; k < kLook; ++k) {   // read again what some lane did not get
                if (__any(s.v[k] == 0xffffffffu)) read_value(s, k, pos - 1 - k);
                if (k < kLook - 1 && __any(s.mh[k < kLook - 1 ? k : 0] == 0xffffffffu)) read_map(s, k, pos - 1 - k);
            }
        }
        return __uint_as_float(0x7fc00000u);
    }
};

constexpr int kNone = 0x7fffffff;   // a ticket behind all others

// The chains in groups of neighbours, each with tickets of its own for the workgroups
// of one blockIdx % 8 (one XCD, as they are dealt out): as many, up to 8, as divide
// the chains evenly.
__host__ __device__ inline int chain_groups(int64_t chains) {
    return chains % 8 == 0 ? 8 : chains % 4 == 0 ? 4 : chains % 2 == 0 ? 2 : 1;
}

// The tiles a workgroup draws: by tickets, position by position over the chains of its
// group.  GROUPED: chain_groups(), else one group, which lets no group run ahead of
// another.  Groups are for 8-bit inputs, whose rows of a tile are half a 128-byte line:
// with neighbours on one XCD the other half is not fetched again (the backward of
// 2 x 32768 x 1536 reads 652 MB in place of 988, training step 841 us in place of 857);
// elsewhere one group is as fast or faster (65536 x 5120 forward 647 us, grouped 678).
template <bool GROUPED> struct Walk {
    int nct, ntiles, groups, group, chains, tickets;   // chains and tickets of the group
    bool once;   // a workgroup for every tile
    __device__ __forceinline__ void init(int nct_, int ntiles_, int batch) {
        nct = nct_;
        ntiles = ntiles_;
        groups = GROUPED && ntiles > 1 ? chain_groups(nct * batch) : 1;
        group = GROUPED ? static_cast<int>(blockIdx.x) % groups : 0;
        chains = nct * batch / groups;
        tickets = chains * ntiles;
        once = static_cast<unsigned>(tickets) * groups <= gridDim.x;
    }
    // By a whole wave: lane 0 adds 1 at agent scope, the other lanes' offsets lie
    // past the counter.  The ticket is lane 0's.
    __device__ __forceinline__ int draw(uint32_t* next) const {
        const Rsrc rs = tile_rsrc(next + group, 4);
        return __builtin_amdgcn_raw_ptr_buffer_atomic_add_i32(1, rs, lane_now() == 0 ? 0u : kNoStore, 0, kAgentScope);
    }
    // The tile of a ticket, counted from the row's end with REVERSE; of no tokens
    // past the last ticket.
    template <bool REVERSE>
    __device__ __forceinline__ Tile place(int ticket, int64_t seqlen) const {
        Tile t;
        const int chain = group * chains + ticket % chains;
        t.pos = ticket / chains;
        t.tile = REVERSE ? ntiles - 1 - t.pos : t.pos;
        t.ct = chain % nct;
        t.b = chain / nct;
        const int64_t t0 = static_cast<int64_t>(t.tile) * kTileTokens;
        const int64_t left = seqlen - t0;
        t.row_tok = t.b * seqlen + t0;
        t.nv = t.pos >= ntiles || left < 0 ? 0 : left < kTileTokens ? static_cast<int>(left) : kTileTokens;
        return t;
    }
    template <int LOOK> __device__ __forceinline__ ChainWords<LOOK> words(const Chain& ch, const Tile& t) const {
        ChainWords<LOOK> w;
        w.init(ch.map, ch.value, (t.b * nct + t.ct) * ntiles * kTileChannels, ntiles);
        return w;
    }
};

}  // namespace rec

// The chains' words in `count` workspaces (recurrence_workspace_bytes each, `stride`
// bytes apart), cleared on the stream, and the rates (recurrence.hip).  Nothing for
// rows of one tile.
hipError_t clear_chains(void* ws, int count, size_t stride, int64_t batch, int64_t dim, int64_t ntiles,
                        const float* a_param, float c, rec::Chain* ch, hipStream_t stream);
}  // namespace mamba
