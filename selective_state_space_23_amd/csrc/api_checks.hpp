// Argument checks shared by the C-ABI files (host only).
#pragma once

#include <cstddef>
#include <cstdint>

namespace mamba {
namespace api {

constexpr int64_t kMaxDim = int64_t(1) << 24;        // channels per row
constexpr int64_t kMaxElems = int64_t(1) << 40;      // elements per tensor
constexpr int64_t kMaxSeqlen = 3000000;              // grid.y limits of the kernels

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [p, p + bytes) and [q, q + qbytes) overlap (null or empty ranges never do).
inline bool overlap(const void* p, size_t bytes, const void* q, size_t qbytes) {
    if (!p || !q || bytes == 0 || qbytes == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qbytes && b < a + bytes;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t c, int64_t* out) {
    if (a < 0 || b < 0 || c < 0) return false;
    __int128 r = static_cast<__int128>(a) * b * c;
    if (r > kMaxElems) return false;
    *out = static_cast<int64_t>(r);
    return true;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Span {
    const void* p;
    size_t bytes;
};

// No output overlaps an input, another output or the workspace, nor the
// workspace an input.
template <size_t NI, size_t NO>
bool disjoint(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (size_t o = 0; o < NO; ++o) {
        for (const Span& i : ins)
            if (overlap(outs[o].p, outs[o].bytes, i.p, i.bytes)) return false;
        for (size_t k = o + 1; k < NO; ++k)
            if (overlap(outs[o].p, outs[o].bytes, outs[k].p, outs[k].bytes)) return false;
    }
    return true;
}

// Bytes from the first to behind the last element of `rows` strided rows.
inline size_t span(int64_t rows, int64_t dim, int64_t ld, size_t esz) {
    return static_cast<size_t>((rows - 1) * ld + dim) * esz;
}

}  // namespace api
}  // namespace mamba
