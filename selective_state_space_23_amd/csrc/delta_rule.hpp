// Device helpers of the gated delta rule (delta_prepare.hip, delta_fwd.hip,
// delta_bwd.hip, delta_grads.hip).
//
// Precision.  Every product of the chunked form runs on
// v_mfma_f32_16x16x32_bf16 with float32 accumulators.  A float32 operand is cut
// into three bf16 pieces of 8 bits each, x = hi + mid + lo exactly (hi by masking, which no finite
// value overflows, mid rounded, so lo is of either sign and at most 2^-16 of x, hi's remainder below 2^-7); the
// pieces of two operands are multiplied as far as they reach 2^-22 of the product: 3 products, and nothing left out,
// where one operand is bf16 as stored, 6 where both are float32, with mid lo, lo mid and lo lo left out, below 2^-22
// of the product at their largest and of either sign (2^-21 and of the product's own sign with mid cut too).  That is
// float32 arithmetic at 1/3 to 1/6 of the bf16 rate (the fp32 instructions have 1/16), and states, solved triangles
// and float32 gradients need it: they carry over thousands of tokens.
//
// Layout.  With lane l = 16 g + m of a wave, an accumulator tile holds row 4 g + r
// (r = 0..3), column m; an operand of 32 contracted values holds row (column) m and eight of them in
// lane group g.  Which eight is free as long as both operands agree.  So an accumulated
// result is an operand of the next product as it stands: two tiles give
// group g the rows 4 g + 0..3 of each, and no lane needs another's values.
#pragma once

#include "device_common.hpp"
#include "delta_launch.hpp"

namespace mamba {
namespace delta {

constexpr int C = kDeltaChunk;
constexpr int kTiles = C / 16;            // token tiles of a chunk
constexpr int kBlocks = 6;                // 16 x 32 pieces of a 64 x 64 triangle that are not all zero
constexpr uint32_t kPast = 0x7fffff00u;   // a byte offset behind any buffer
constexpr int64_t kSolveBytes = kBlocks * 3 * 1024;   // a chunk's solved triangle, or P, in three pieces

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
using Rsrc = __amdgpu_buffer_rsrc_t;

// An eighth of a row of 32 contracted values in N pieces.
template <int N> struct Frag {
    u32x4 p[N];
};

// Per-chunk record of the first pass: what the tokens' decays come to.
struct ChunkRec {
    float hi[C], lo[C];   // sum of log2 decays from the chunk's start (document starts count 0), as hi + lo
    float into[C];        // exp2 of it where no document start lies before: what the entering state has kept
    float outof[C];       // from the token to the chunk's end, 0 where a later document starts
    float beta[C];
    float keep;           // the entering state's part of the leaving one (0 with a start inside)
    uint32_t pad;
    uint64_t starts;      // bit t: token t starts a document
    uint64_t walls;       // bit t: it does, or its decay counts as 0: nothing reaches it from before
    uint64_t bad;         // bit t: a key, gate or decay of token t or before it in its document is not finite
    uint64_t sick;        // (backward) bit t: something in token t's document, as far as the chunk holds it, is not finite
};

__device__ __forceinline__ Rsrc rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// acc += a b with the products of pieces i, j with i + j < ORDER, the smallest first.
template <int ORDER, int NA, int NB>
__device__ __forceinline__ void product(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = ORDER - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) acc = mfma(a.p[i], b.p[s - i], acc);
}

// The same for M accumulators in turn, so that none waits for its own last product (44 cycles against 16).
template <int ORDER, int M, int NA, int NB>
__device__ __forceinline__ void products(f32x4* acc, const Frag<NA>* a, const Frag<NB>& b) {
#pragma unroll
    for (int s = ORDER - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) {
#pragma unroll
                for (int k = 0; k < M; ++k) acc[k] = mfma(a[k].p[i], b.p[s - i], acc[k]);
            }
}

// What is left of two floats without their bf16 pieces h = {x0's, x1's}: v_dot2_f32_bf16 is exact here, as its sum has
// no more than 24 bits, and takes both a piece out of its pair and the difference (two instructions of 8 cycles each to a
// lone wave, against four).  An infinity or NaN in one of the two makes both NaN: pairs lie along what is summed over.
// (The multipliers are hidden from the compiler, which took {0, -1} for the constant -1.0f, read here as {-1, 0}.)
__device__ __forceinline__ void without_pieces(uint32_t h, float& x0, float& x1) {
    uint32_t first = 0x0000bf80u, second = 0xbf800000u;   // {-1, 0} and {0, -1}
    asm("" : "+s"(first));
    asm("" : "+s"(second));
    x0 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, h), __builtin_bit_cast(bf16x2_t, first), x0, false);
    x1 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, h), __builtin_bit_cast(bf16x2_t, second), x1, false);
}

// A value that the compiler does not know: what is computed from it stays where it is used.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Whether a workgroup of the chains takes 64 columns of a head rather than 32.  One fills a CU either way, and a chunk of
// 64 columns takes a third longer: 32 as long as all have a CU at once (2048 tokens, 64 heads of 128 columns: 107 us
// forward, 145 with 64 columns), 64 when that saves a turn (72 heads: 146, 201 with 32 columns).
inline bool wide_groups(const DeltaArgs& a) {
    return a.vdim > 32 && a.batch * a.vheads * ((a.vdim + 31) / 32) > 256;
}

// The bf16 pieces of pairs of floats: the highest 8 significant bits, the rest rounded (CUT: cut) to as many, and what is left.
template <bool CUT = false>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
    without_pieces(hi, x0, x1);
    mid = CUT ? __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u) : pack_bf16x2(x0, x1);
    without_pieces(mid, x0, x1);
    lo = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302u);
}

// Eight floats in three pieces: slots 0..3 from a, 4..7 from b.
template <bool CUT = false>
__device__ __forceinline__ Frag<3> split(f32x4 a, f32x4 b) {
    Frag<3> f;
    uint32_t h, m, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 x = i < 2 ? a : b;
        split_pair<CUT>(x[2 * (i & 1)], x[2 * (i & 1) + 1], h, m, l);
        f.p[0][i] = h;
        f.p[1][i] = m;
        f.p[2][i] = l;
    }
    return f;
}

// Eight of the differences R = v - ..., which are v itself where no state and no other token has a part: the lowest float,
// at tokens that count for nothing with beta = 0, has to come out of T R as it went in.  The matrix instruction cuts sums
// towards minus infinity, and with a rounded second piece, -2^120 here, anything else in the sum makes it -2^128; with
// cut pieces what lies below 2^96 does not reach it.  (What T R leaves out is up to 1.5 x 2^-22 of a product.)
__device__ __forceinline__ Frag<3> split_values(f32x4 a, f32x4 b) { return split<true>(a, b); }

// The rows of one chunk of one tensor as a buffer: reads behind the last token
// give zero, writes there are dropped.
template <int ESZ>
__device__ __forceinline__ Rsrc rows_rsrc(const void* p, int64_t first, int rows, int64_t ld, int width) {
    return rsrc(static_cast<const char*>(p) + first * ESZ, rows > 0 ? ((rows - 1) * ld + width) * ESZ : 0);
}

// Eight consecutive channels c .. c + 7 of a row, as stored, zeros past `width`.  VEC: in 16-byte pieces
// (width and strides multiples of 8, pointers aligned), else one by one.
template <typename T, bool VEC> struct Eight;
template <bool VEC> struct Eight<bf16_t, VEC> {
    u32x4 w;
    __device__ __forceinline__ void load(Rsrc rs, uint32_t row_off, int c, int width) {
        if constexpr (VEC) {
            w = __builtin_amdgcn_raw_buffer_load_b128(rs, c < width ? row_off + 2 * c : kPast, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t o = row_off + 2 * (c + 2 * i);
                const uint32_t x = static_cast<uint16_t>(
                    __builtin_amdgcn_raw_buffer_load_b16(rs, c + 2 * i < width ? o : kPast, 0, 0));
                const uint32_t y = static_cast<uint16_t>(
                    __builtin_amdgcn_raw_buffer_load_b16(rs, c + 2 * i + 1 < width ? o + 2 : kPast, 0, 0));
                w[i] = x | (y << 16);
            }
        }
    }
    __device__ __forceinline__ Frag<1> frag() const { return Frag<1>{{w}}; }
};
template <bool VEC> struct Eight<float, VEC> {
    u32x4 a, b;
    __device__ __forceinline__ void load(Rsrc rs, uint32_t row_off, int c, int width) {
        if constexpr (VEC) {
            const uint32_t o = c < width ? row_off + 4 * c : kPast;
            a = __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0);
            b = __builtin_amdgcn_raw_buffer_load_b128(rs, o + (c < width ? 16 : 0), 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, c + i < width ? row_off + 4 * (c + i) : kPast, 0, 0);
                b[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, c + 4 + i < width ? row_off + 4 * (c + 4 + i) : kPast,
                                                            0, 0);
            }
        }
    }
    __device__ __forceinline__ Frag<3> frag() const {
        return split(__builtin_bit_cast(f32x4, a), __builtin_bit_cast(f32x4, b));
    }
};

// Pieces of an operand as stored.
template <typename T> constexpr int kPieces = sizeof(T) == 2 ? 1 : 3;

// One element of T at a byte offset of a buffer.
template <typename T>
__device__ __forceinline__ uint32_t load_one(Rsrc rs, uint32_t off) {
    if constexpr (sizeof(T) == 2)
        return static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0));
    else
        return __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
}
template <typename T>
__device__ __forceinline__ float one_value(uint32_t raw) {
    return sizeof(T) == 2 ? __uint_as_float(raw << 16) : __uint_as_float(raw);
}
template <typename T>
__device__ __forceinline__ void store_one(Rsrc rs, uint32_t off, float v) {
    if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), rs, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rs, off, 0, 0);
}

// A chunk of q or k in LDS: [pieces][C][KT] bf16, rows of KT / 8 pieces of 16 bytes, piece q of row r
// at place q ^ swizzle(r).  Then neither 16 rows' pieces of one number (operands with the rows
// in lanes) nor the 4 x 4 half pieces that 16 lanes read to transpose lie on a bank twice, and a row is as long as
// what goes to LDS straight from memory, 1 KB a wave.  (That is for 16 lanes of one group g; what lanes of several groups
// do together the counters tell: 27 % of the LDS cycles of the forward's chains are conflicts, 25 % of the backward's.)
template <int KT> __device__ __forceinline__ int swizzle(int r) {
    return KT == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r & 2) << 1) | ((r >> 2) & 3);
}
template <int KT> __device__ __forceinline__ int place(int r, int q) { return r * KT + ((q ^ swizzle<KT>(r)) << 3); }

typedef __attribute__((address_space(3))) void* Lds;

// Straight from memory, by the NW waves of a workgroup: bf16 rows of whole 16-byte pieces.
template <int KT, int NW>
__device__ __forceinline__ void rows_to_lds(uint16_t* lds, Rsrc rs, int64_t ld, int width, int wave, int lane) {
    constexpr int PIECES = KT / 8, ROWS = 64 / PIECES;
#pragma unroll
    for (int n = 0; n < C / ROWS / NW; ++n) {
        const int first = (n * NW + wave) * ROWS, r = first + lane / PIECES;
        const int q = (lane % PIECES) ^ swizzle<KT>(r);
        const uint32_t off = q * 8 < width ? static_cast<uint32_t>(r * static_cast<int>(ld) * 2 + q * 16) : kPast;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (Lds)(lds + first * KT), 16, off, 0, 0, 0);
    }
}
// KB of consecutive memory, piece p by wave p % NW; what lies behind `rs` reads as zeros.
template <int KB, int NW>
__device__ __forceinline__ void block_to_lds(char* lds, Rsrc rs, int wave, int lane) {
#pragma unroll
    for (int p = 0; p < (KB + NW - 1) / NW; ++p)
        if (p * NW + wave < KB)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (Lds)(lds + (p * NW + wave) * 1024), 16,
                                                     ((p * NW + wave) * 64 + lane) * 16, 0, 0, 0);
}

// Through registers: any type and alignment.
template <typename T, int KT, int THREADS, bool VEC> struct Tile {
    static constexpr int N = kPieces<T>, PER = C * KT / 8 / THREADS;
    static constexpr size_t kBytes = size_t(N) * C * KT * 2;
    Eight<T, VEC> raw[PER];
    __device__ __forceinline__ void fetch(Rsrc rs, int64_t ld, int width, int tid) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = p * THREADS + tid, t = x / (KT / 8), ch = x % (KT / 8) * 8;
            raw[p].load(rs, static_cast<uint32_t>(t * static_cast<int>(ld) * static_cast<int>(sizeof(T))), ch, width);
        }
    }
    __device__ __forceinline__ void land(uint16_t* lds, int tid) const { land_without(lds, tid, 0); }
    // With the rows of `out` as zeros.
    __device__ __forceinline__ void land_without(uint16_t* lds, int tid, uint64_t out) const {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int x = p * THREADS + tid, t = x / (KT / 8), q = x % (KT / 8);
            const Frag<N> f = raw[p].frag();
            const uint32_t on = (out >> t) & 1 ? 0u : ~0u;
#pragma unroll
            for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(lds + i * C * KT + place<KT>(t, q)) = f.p[i] & on;
        }
    }
};

// Operands from such a tile: row `row`, its q-th eight channels ...
template <int N, int KT>
__device__ __forceinline__ Frag<N> rows_frag(const uint16_t* lds, int row, int q) {
    Frag<N> f;
    const uint16_t* at = lds + place<KT>(row, q);
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = *reinterpret_cast<const u32x4*>(at + i * C * KT);
    return f;
}
// ... or a column of rows 32 j + 4 g + 0..3 and 16 further, by transposing reads: 16 lanes read four rows
// of 16 columns, lane m giving the address of row m / 4, channels `ch4`.. + 3, and getting the m-th of the 16
// columns.
__device__ __forceinline__ u32x4 transposed(const uint16_t* at, int rows16) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + rows16));
    const u32x2 xw = __builtin_bit_cast(u32x2, x), yw = __builtin_bit_cast(u32x2, y);
    return u32x4{xw[0], xw[1], yw[0], yw[1]};
}
template <int N, int KT>
__device__ __forceinline__ Frag<N> cols_frag(const uint16_t* lds, int j, int g, int m, int ch4) {
    Frag<N> f;
    const uint16_t* at = lds + place<KT>(32 * j + 4 * g + m / 4, ch4 >> 3) + (ch4 & 4);
#pragma unroll
    for (int i = 0; i < N; ++i) f.p[i] = transposed(at + i * C * KT, 16 * KT);
    return f;
}
// Zeros in the slots of the rows of `out`.
template <int N>
__device__ __forceinline__ void drop_rows(Frag<N>& f, int j, int g, uint64_t out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int s = 32 * j + (e < 4 ? 4 * g + e : 12 + 4 * g + e);
        const uint32_t mask = (out >> s) & 1 ? (e & 1 ? 0x0000ffffu : 0xffff0000u) : 0xffffffffu;
#pragma unroll
        for (int i = 0; i < N; ++i) f.p[i][e / 2] &= mask;
    }
}

// The channel of a state that row 4 g + r of tile i stands for: with it an operand of 32
// contracted channels reads 8 consecutive ones of a row of q or k.
__device__ __forceinline__ int state_row(int i, int g, int r) { return 32 * (i / 2) + 8 * g + 4 * (i % 2) + r; }
__device__ __forceinline__ int state_cols4(int i, int m) { return 32 * (i / 2) + 8 * (m % 4) + 4 * (i % 2); }

// The 6 pieces of a triangle's operand order: rows of tile i, columns 32 j .. 32 j + 31
__device__ __forceinline__ constexpr int low_block(int i, int j) { return i < 2 ? i : 2 + (i - 2) * 2 + j; }
__device__ __forceinline__ constexpr int high_block(int i, int j) { return i < 2 ? i * 2 + j : i + 2; }   // of its transpose

// The thread, formed where it is used: offsets of every phase held across the loops around them
// overflow the registers.
__device__ __forceinline__ int thread_now() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// a / b and a % b of values that all lanes share, in scalar registers (the division itself runs
// on the vector unit, and a buffer's address that comes from there costs a loop at every access).
__device__ __forceinline__ int quotient(uint32_t a, uint32_t b) { return __builtin_amdgcn_readfirstlane(a / b); }
__device__ __forceinline__ int remainder(uint32_t a, uint32_t b) { return __builtin_amdgcn_readfirstlane(a % b); }

__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// The first token of t's document, as far as the chunk holds it, and the end of s's.
__device__ __forceinline__ int doc_first(uint64_t starts, int t) {
    const uint64_t at = starts & (~0ull >> (63 - t));
    return at ? 63 - __builtin_clzll(at) : 0;
}
__device__ __forceinline__ int doc_end(uint64_t starts, int s) {
    const uint64_t at = starts >> s >> 1;
    return at ? s + 1 + __builtin_ctzll(at) : C;
}

// Bits from each set bit of `m` up to the end of its document (next bit of `starts`).
__device__ __forceinline__ uint64_t smear(uint64_t m, uint64_t starts) {
    uint64_t walls = starts;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        m |= (m << s) & ~walls;
        walls |= walls << s;
    }
    return m;
}

// Bits of the whole documents that a set bit of `m` lies in.
__device__ __forceinline__ uint64_t whole(uint64_t m, uint64_t starts) {
    m = smear(m, starts);
    uint64_t walls = starts >> 1;   // a start at t + 1 ends the document of t
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        m |= (m >> s) & ~walls;
        walls |= walls >> s;
    }
    return m;
}

// x or 0, whatever x is, by its bits: a select of a costly x becomes a divergent branch, which is slower here and
// not safe in a loop with this many registers (the compiler has been seen to copy live registers at the join
// before it restores the execution mask).
__device__ __forceinline__ float keep_if(bool on, float x) { return __uint_as_float(__float_as_uint(x) & (on ? ~0u : 0u)); }

// x, or a NaN.
__device__ __forceinline__ float nan_if(bool on, float x) { return __uint_as_float(__float_as_uint(x) | (on ? 0x7fc00000u : 0u)); }

__device__ __forceinline__ bool not_finite(float x) { return __builtin_isfpclass(x, 0x207); }   // nan, +-inf

// `lost`, rows of a chunk for a lane's column, with those whose value x (rows 16 i + 4 g + r) is not finite and the rest of
// their documents.
__device__ __forceinline__ uint64_t lost_with(uint64_t lost, const f32x4 (&x)[4], uint64_t starts, int g) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) lost |= uint64_t(not_finite(x[i][r])) << (16 * i + 4 * g + r);
    lost |= __shfl_xor(lost, 16);
    lost |= __shfl_xor(lost, 32);
    return smear(lost, starts);
}
// x of tile i without the rows of `lost`.
__device__ __forceinline__ f32x4 without_rows(f32x4 x, uint64_t lost, int i, int g) {
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = keep_if(!((lost >> (16 * i + 4 * g + r)) & 1), x[r]);
    return x;
}

// Four consecutive token values of a record.
__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

}  // namespace delta
}  // namespace mamba
