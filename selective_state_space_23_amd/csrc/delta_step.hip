// Gated delta rule: the step of one token.
//
// A workgroup keeps the K x (4 COLS) part of one head's state in registers, four
// consecutive columns and K COLS / 256 consecutive rows a thread:
//     S' = a S;  u = beta (v - S'^T k);  S = S' + k u^T;  out = scale S^T q,
// the sums over rows by lane exchanges, then over the four waves through LDS.  Bound by memory
// (the state read and written once: 128 rows of 40 heads of 128 x 128, 675 MB, in 134 us over six states in turn, the time of a
// copy as large; 113 us with one state again and again, part of which the last cache keeps); the columns
// of one head are split over workgroups where there are few heads, whose time is a trip to memory (two rows of 12: 3.9 us).
#include "delta_rule.hpp"

namespace mamba {

namespace {

using namespace delta;

// The sum over the workgroup's row groups of four columns, in every thread.
template <int COLS>
__device__ __forceinline__ f32x4 over_rows(f32x4 x, f32x4 (*red)[COLS], int wave, int lane) {
#pragma unroll
    for (int s = COLS; s < 64; s *= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += __shfl_xor(x[e], s);
    const int c = lane % COLS;
    red[wave][c] = x;   // the same from all lanes of a column
    __syncthreads();
    return (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
}

template <typename T, int KT, int COLS, bool VEC>
__global__ __launch_bounds__(256) void step_kernel(DeltaUpdateArgs a, int cols) {
    constexpr int R = KT * COLS / 256;   // rows a thread
    __shared__ __align__(16) float kv[128], qv[128];
    __shared__ __align__(16) f32x4 red[2][4][COLS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bh = quotient(blockIdx.x, cols);
    const int hv = remainder(bh, a.vheads), hk = quotient(hv, a.vheads / a.kheads);
    const int64_t b = quotient(bh, a.vheads);
    const int v0 = (remainder(blockIdx.x, cols) * COLS + lane % COLS) * 4;
    const int row0 = (wave * (64 / COLS) + lane / COLS) * R;
    const int64_t cells = static_cast<int64_t>(a.kdim) * a.vdim;

    // Offsets of columns behind the last lie behind the buffer, as those of rows do.
    uint32_t lane_off[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) lane_off[e] = v0 + e < a.vdim ? (v0 + e) * 4 : kPast;
    f32x4 S[R];
    {
        const Rsrc rs = rsrc(a.state + bh * cells, cells * 4);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t row = static_cast<uint32_t>((row0 + i) * a.vdim * 4);
            if constexpr (VEC) {
                S[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, lane_off[0] + row, 0, 0));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S[i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, lane_off[e] + row, 0, 0));
            }
        }
    }
    const bool start = a.reset != nullptr && a.reset[b] != 0;
    float gate = a.g != nullptr ? a.g[b * a.vheads + hv] : 0.0f;
    if (gate < -200.0f) gate = -200.0f;
    const float decay = exp2_fast(gate * kLog2e), beta = a.beta[b * a.vheads + hv];
    f32x4 vals;
    {
        const Rsrc vr = rsrc(static_cast<const T*>(a.v) + b * a.ld_v + static_cast<int64_t>(hv) * a.vdim,
                             a.vdim * static_cast<int>(sizeof(T)));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            vals[e] = one_value<T>(load_one<T>(vr, static_cast<uint32_t>((v0 + e) * sizeof(T))));
    }
    {   // k by the first two waves, q by the others
        const bool key = wave < 2;
        const int ch = tid & 127;
        const Rsrc r = key ? rsrc(static_cast<const T*>(a.k) + b * a.ld_k + static_cast<int64_t>(hk) * a.kdim,
                                  a.kdim * static_cast<int>(sizeof(T)))
                           : rsrc(static_cast<const T*>(a.q) + b * a.ld_q + static_cast<int64_t>(hk) * a.kdim,
                                  a.kdim * static_cast<int>(sizeof(T)));
        (key ? kv : qv)[ch] = one_value<T>(load_one<T>(r, static_cast<uint32_t>(ch * sizeof(T))));
    }
    __syncthreads();
    float kr[R], qr[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        kr[i] = kv[row0 + i];
        qr[i] = qv[row0 + i];
    }
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = start ? 0.0f : S[i][e] * decay;
            sum[e] = __builtin_fmaf(S[i][e], kr[i], sum[e]);
        }
    sum = over_rows<COLS>(sum, red[0], wave, lane);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float u = beta * (vals[e] - sum[e]);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            S[i][e] = __builtin_fmaf(kr[i], u, S[i][e]);
            o[e] = __builtin_fmaf(S[i][e], qr[i], o[e]);
        }
    }
    o = over_rows<COLS>(o, red[1], wave, lane);
    const Rsrc orr = rsrc(static_cast<T*>(a.out) + (b * a.vheads + hv) * a.vdim, a.vdim * static_cast<int>(sizeof(T)));
#pragma unroll
    for (int e = 0; e < 4; ++e)
        store_one<T>(orr, tid < COLS ? static_cast<uint32_t>((v0 + e) * sizeof(T)) : kPast, a.scale * o[e]);
    {
        const Rsrc rs = rsrc(a.state + bh * cells, cells * 4);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t row = static_cast<uint32_t>((row0 + i) * a.vdim * 4);
            if constexpr (VEC) {
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[i]), rs, lane_off[0] + row, 0, 0);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][e]), rs, lane_off[e] + row, 0, 0);
            }
        }
    }
}

template <typename T, int KT, int COLS>
hipError_t launch(const DeltaUpdateArgs& a) {
    const int cols = (a.vdim + 4 * COLS - 1) / (4 * COLS);
    const dim3 grid(static_cast<unsigned>(a.batch * a.vheads * cols));
    if (a.vec) hipLaunchKernelGGL((step_kernel<T, KT, COLS, true>), grid, dim3(256), 0, a.stream, a, cols);
    else hipLaunchKernelGGL((step_kernel<T, KT, COLS, false>), grid, dim3(256), 0, a.stream, a, cols);
    return hipGetLastError();
}

// Few heads: 32 columns a workgroup, more of them, where these are whole lines of memory (128 heads of 128 x 128, over states that
// no cache holds: 6.5 us, 7.4 with 128 columns; 256: 9.7 and 10.1; 512: 16.2 and 17.2; 8192: 214 and 214).  Parts of lines cost
// more than they gain: 128 heads of 128 x 100 9.8 us, 6.6 with whole rows; 240 heads of 64 x 36 5.7 and 4.6.
template <typename T>
hipError_t by_size(const DeltaUpdateArgs& a) {
    const bool few = a.batch * a.vheads < 256 && (a.vdim <= 32 || a.vdim % 32 == 0);
    if (a.kdim > 64) return few ? launch<T, 128, 8>(a) : launch<T, 128, 32>(a);
    return few ? launch<T, 64, 8>(a) : launch<T, 64, 32>(a);
}

}  // namespace

hipError_t launch_delta_update(const DeltaUpdateArgs& a) { return a.bf16 ? by_size<bf16_t>(a) : by_size<float>(a); }

}  // namespace mamba
