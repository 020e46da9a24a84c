// 8-bit activation checkpoints, gfx950: x (rows, D) as int8 codes (rows, D) and
// one float32 scale per row and 64 channels, stored (ceil(D / 64), rows).
//
//     m = max |x| over the block (at least 2^-100),  scale = m (1 / 127),
//     code = round(x ((1 / m) 127)), ties to even,   value = code * scale,
// |value - x| <= scale / 2 up to 32-bit rounding.  A block with a NaN or an
// infinity gets a NaN scale: all of it decodes to NaN.
//
// 16 lanes hold a block's 64 channels, 4 each; a lane takes kRows consecutive
// rows so that their loads are in flight together.  Bound by memory: 65536 x 1536 in
// bfloat16 are packed in 60 us and unpacked in 58 (308 MB each, 5.2 and 5.3 TB/s).
#include "recurrence.hpp"

namespace mamba {

namespace {

using namespace rec;

constexpr int kRows = 4;            // rows a lane takes
constexpr int kTileRows = 64;       // 16 groups of 16 lanes

template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void pack_kernel(const PackArgs a, int nct) {
    const int li = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int dim = static_cast<int>(a.dim);
    const int ct = static_cast<int>(blockIdx.x % static_cast<unsigned>(nct));
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(nct)) * kTileRows;
    const int nv = a.rows - r0 < kTileRows ? static_cast<int>(a.rows - r0) : kTileRows;
    const int c = ct * kTileChannels + 4 * li;
    constexpr int esz = Elem<T>::kBytes;
    const Rsrc xs = rows_rsrc<esz>(a.x, r0, nv, a.ld, dim);
    const Rsrc qs = rows_rsrc<1>(a.p.q, r0, nv, dim, dim);
    const Rsrc ss = tile_rsrc(a.p.scale + ct * a.rows + r0, nv * 4);
    const uint32_t step = static_cast<uint32_t>(a.ld) * esz, row = grp * kRows;
    Raw<T, 4> raw[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) raw[k] = load_raw<T, 4, ALIGNED>(xs, (row + k) * step + static_cast<uint32_t>(c) * esz);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        float v[4];
        unpack(raw[k], v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = c + j < dim ? __float_as_uint(v[j]) & 0x7fffffffu : 0u;
            m = b > m ? b : m;
        }
        auto umax = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
        m = umax(m, dpp_u32<0xB1>(m));
        m = umax(m, dpp_u32<0x4E>(m));
        m = umax(m, dpp_u32<0x141>(m));
        m = umax(m, dpp_u32<0x128>(m));
        float scale, inv;
        block_scale(m, scale, inv);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), ss, li == 0 ? 4 * (row + k) : kNoStore, 0, 0);
        store_codes<4, ALIGNED>(qs, c < dim ? (row + k) * static_cast<uint32_t>(dim) + c : kNoStore, dim - c, encode(v, inv));
    }
}

template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void unpack_kernel(const PackArgs a, int nct) {
    const int li = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int dim = static_cast<int>(a.dim);
    const int ct = static_cast<int>(blockIdx.x % static_cast<unsigned>(nct));
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(nct)) * kTileRows;
    const int nv = a.rows - r0 < kTileRows ? static_cast<int>(a.rows - r0) : kTileRows;
    const int c = ct * kTileChannels + 4 * li;
    constexpr int esz = Elem<T>::kBytes;
    const Rsrc qs = rows_rsrc<1>(a.p.q, r0, nv, dim, dim);
    const Rsrc ss = tile_rsrc(a.p.scale + ct * a.rows + r0, nv * 4);
    const Rsrc os = rows_rsrc<esz>(a.out, r0, nv, dim, dim);
    const uint32_t row = grp * kRows;
    uint32_t q[kRows];
    float s[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        q[k] = load_codes<4, ALIGNED>(qs, (row + k) * static_cast<uint32_t>(dim) + c);
        s[k] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ss, 4 * (row + k), 0, 0));
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        float v[4];
        decode(q[k], s[k], v);
        store_vals<T, 4, ALIGNED>(os, c < dim ? ((row + k) * static_cast<uint32_t>(dim) + c) * esz : kNoStore, dim - c, v);
    }
}

}  // namespace

hipError_t launch_pack(const PackArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const dim3 grid(static_cast<unsigned>(((a.rows + kTileRows - 1) / kTileRows) * nct));
    if (a.bf16) {
        if (a.aligned) hipLaunchKernelGGL((pack_kernel<bf16_t, true>), grid, dim3(256), 0, a.stream, a, nct);
        else hipLaunchKernelGGL((pack_kernel<bf16_t, false>), grid, dim3(256), 0, a.stream, a, nct);
    } else {
        if (a.aligned) hipLaunchKernelGGL((pack_kernel<float, true>), grid, dim3(256), 0, a.stream, a, nct);
        else hipLaunchKernelGGL((pack_kernel<float, false>), grid, dim3(256), 0, a.stream, a, nct);
    }
    return hipGetLastError();
}

hipError_t launch_unpack(const PackArgs& a) {
    const int nct = static_cast<int>((a.dim + kTileChannels - 1) / kTileChannels);
    const dim3 grid(static_cast<unsigned>(((a.rows + kTileRows - 1) / kTileRows) * nct));
    if (a.bf16) {
        if (a.aligned) hipLaunchKernelGGL((unpack_kernel<bf16_t, true>), grid, dim3(256), 0, a.stream, a, nct);
        else hipLaunchKernelGGL((unpack_kernel<bf16_t, false>), grid, dim3(256), 0, a.stream, a, nct);
    } else {
        if (a.aligned) hipLaunchKernelGGL((unpack_kernel<float, true>), grid, dim3(256), 0, a.stream, a, nct);
        else hipLaunchKernelGGL((unpack_kernel<float, false>), grid, dim3(256), 0, a.stream, a, nct);
    }
    return hipGetLastError();
}

}  // namespace mamba
