// Sums over the lanes of a wave, the same value in every lane that took part (a
// fixed tree, so the same bits on every call).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kq {

// The value of v in the lane that differs: DPP patterns within 16 lanes.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// v + its value 16 (then 32) lanes away, by the swaps of rows and half waves.
__device__ __forceinline__ float sum_across_rows(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t s = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(s, s, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
__device__ __forceinline__ double sum_across_rows(double v) {
    auto join = [](uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo); };
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    const auto pl = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto ph = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    u = __builtin_bit_cast(uint64_t, join(pl[0], ph[0]) + join(pl[1], ph[1]));
    const auto ql = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto qh = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    return join(ql[0], qh[0]) + join(ql[1], qh[1]);
}
// Sum over a wave, the same value in every lane (a fixed tree).
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
    v += moved<0xB1>(v);   // quad_perm [1,0,3,2]
    v += moved<0x4E>(v);   // quad_perm [2,3,0,1]
    v += moved<0x141>(v);  // mirrored within 8 lanes
    v += moved<0x140>(v);  // mirrored within 16 lanes
    return sum_across_rows(v);
}

// Sum over the lanes of a wave at the same place of every group of LG: LG = 4, 8, 16 or 32. (By __shfl_xor, through LDS, the
// gradients of the heads' two weights took 2.5 us more: one token of 24 x 64 8.5 instead of 6.0.)
template <int LG>
__device__ __forceinline__ float slots_sum(float v) {
    if (LG <= 32) {
        const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    if (LG <= 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (LG <= 8) v += moved<0x128>(v);  // 8 lanes on in a ring of 16
    if (LG <= 4) v += moved<0x124>(v);  // and 4
    return v;
}

}  // namespace kq
