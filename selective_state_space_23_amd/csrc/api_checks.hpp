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

}  // namespace api
}  // namespace mamba
