// Elements of bf16 (as bit patterns) or fp32 rows, one by one and in chunks of
// eight neighbours, for the kernels that take either type.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.hpp"

namespace kq {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Buffer over `bytes` bytes: loads past them read zeros, stores are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}

// One element through a buffer.
template <bool NT = false>
__device__ __forceinline__ uint32_t load_raw1(__amdgpu_buffer_rsrc_t r, uint32_t i, const uint16_t *) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, 2 * i, 0, NT ? 2 : 0);
}
template <bool NT = false>
__device__ __forceinline__ uint32_t load_raw1(__amdgpu_buffer_rsrc_t r, uint32_t i, const float *) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, 4 * i, 0, NT ? 2 : 0);
}
template <bool NT = false>
__device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t i, float v, const uint16_t *) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, 2 * i, 0, NT ? 2 : 0);
}
template <bool NT = false>
__device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t i, float v, const float *) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, 4 * i, 0, NT ? 2 : 0);
}

// How a wave's lanes share the 512 channels of a piece. VEC: lane l has the 8 neighbours from
// 8 l on, in one or two 16-byte accesses (rows of whole 16-byte pieces). Otherwise lane l has
// the channels l, 64 + l, 128 + l .., element by element, at any width and alignment; an access
// of the wave is one run of a row either way.
template <bool VEC>
struct Lanes {
    static constexpr uint32_t kStep = VEC ? 1 : 64;  // from a lane's element to its next
    static __device__ __forceinline__ uint32_t first(uint32_t piece, int lane) {
        return 512u * piece + (VEC ? 8u : 1u) * (uint32_t)lane;
    }
};

// A lane's eight channels as they are loaded; NT: non-temporal (streamed_once below).
template <class T, bool VEC = true>
struct Chunk;
template <>
struct Chunk<uint16_t, true> {
    u32x4_t q;
    template <bool NT = false>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t ch) {
        q = __builtin_amdgcn_raw_buffer_load_b128(r, 2 * ch, 0, NT ? 2 : 0);
    }
    __device__ __forceinline__ void widen(float x[8]) const { widen8(make_uint4(q[0], q[1], q[2], q[3]), x); }
};
template <>
struct Chunk<float, true> {
    u32x4_t a, b;
    template <bool NT = false>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t ch) {
        a = __builtin_amdgcn_raw_buffer_load_b128(r, 4 * ch, 0, NT ? 2 : 0);
        b = __builtin_amdgcn_raw_buffer_load_b128(r, 4 * ch + 16, 0, NT ? 2 : 0);
    }
    __device__ __forceinline__ void widen(float x[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = __uint_as_float(a[e]);
            x[4 + e] = __uint_as_float(b[e]);
        }
    }
};
template <class T>
struct Chunk<T, false> {
    uint32_t q[8];
    template <bool NT = false>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t ch) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = load_raw1<NT>(r, ch + 64 * e, (const T *)nullptr);
    }
    __device__ __forceinline__ void widen(float x[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(sizeof(T) == 2 ? q[e] << 16 : q[e]);
    }
};
template <bool NT = false, bool VEC = true>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t ch, const float y[8], const uint16_t *type) {
    if (!VEC) {
#pragma unroll
        for (int e = 0; e < 8; ++e) store1<NT>(r, ch + 64 * e, y[e], type);
        return;
    }
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                   pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])},
                                           r, 2 * ch, 0, NT ? 2 : 0);
}
template <bool NT = false, bool VEC = true>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t ch, const float y[8], const float *type) {
    if (!VEC) {
#pragma unroll
        for (int e = 0; e < 8; ++e) store1<NT>(r, ch + 64 * e, y[e], type);
        return;
    }
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{__float_as_uint(y[0]), __float_as_uint(y[1]),
                                                   __float_as_uint(y[2]), __float_as_uint(y[3])},
                                           r, 4 * ch, 0, NT ? 2 : 0);
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{__float_as_uint(y[4]), __float_as_uint(y[5]),
                                                   __float_as_uint(y[6]), __float_as_uint(y[7])},
                                           r, 4 * ch + 16, 0, NT ? 2 : 0);
}

// Whether a call that moves `bytes` marks its accesses non-temporal: from half of the 256 MiB
// Infinity Cache on. What it reads is then not there from before (us: norm 16384 x 8192 bf16
// 92.6 -> 87.2, 8192 x 4608 30.5 -> 27.1; its gradients 16384 x 8192 152 -> 133 with the loads
// marked, 138 with the stores too; linear's gradient 8192 x 16384 158 -> 131; below, input that the
// cache holds is lost: norm 8192 x 1152 8.4 -> 9.9, 2048 x 4096 7.8 -> 8.7).
inline bool streamed_once(int64_t bytes) { return bytes >= (int64_t)128 << 20; }

}  // namespace kq
