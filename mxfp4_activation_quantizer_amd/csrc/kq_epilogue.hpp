// The epilogue of kq_mxfp4_linear on fp32 sums,
//   z = sum + bias,  O = act(z) + residual,
// applied by every product kernel where a lane holds neighbouring columns of a
// row, so that each access is one piece of 8 or 16 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_act.hpp"
#include "kq_chunk.hpp"
#include "kq_device.hpp"

namespace kq {

struct Epi {
    const float *bias;     // [n] or NULL
    const void *residual;  // [m][ldr] of O's type, or NULL
    void *O;               // [m][ldo], bf16 bits or fp32
    void *Z;               // [m][ldz] of O's type, or NULL: receives z
    int64_t m, n, ldr, ldo, ldz;
    int act;
    int align;  // every row of O, Z and the residual starts at a multiple of this many bytes (16, 8 or less)
    // whether the residual is read non-temporally: from 256 MiB on, where the Infinity Cache cannot
    // have it (us, fp32 8192 x 16384 x 4096: 410, 480 without; 8192 x 4096 x 4096: 105, 92 without)
    int stream;
};

// N neighbouring elements in one piece. Non-temporal stores: outputs are not read again
// here, so they should not push the operand lines that other workgroups still read.
template <int N>
__device__ __forceinline__ void load_piece(const float *p, float (&v)[N]) {
    static_assert(N % 4 == 0, "pieces of 16 bytes");
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const floatx4_t q = *reinterpret_cast<const floatx4_t *>(p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i + e] = q[e];
    }
}
template <int N>
__device__ __forceinline__ void load_piece(const uint16_t *p, float (&v)[N]) {
    typedef uint32_t piece_t __attribute__((ext_vector_type(N / 2)));
    const piece_t q = *reinterpret_cast<const piece_t *>(p);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        v[2 * e] = bf16_lo(q[e]);
        v[2 * e + 1] = bf16_hi(q[e]);
    }
}
template <int N>
__device__ __forceinline__ void store_piece(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
        __builtin_nontemporal_store(floatx4_t{v[i], v[i + 1], v[i + 2], v[i + 3]}, reinterpret_cast<floatx4_t *>(p + i));
}
template <int N>
__device__ __forceinline__ void store_piece(uint16_t *p, const float (&v)[N]) {
    typedef uint32_t piece_t __attribute__((ext_vector_type(N / 2)));
    piece_t q;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) q[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    __builtin_nontemporal_store(q, reinterpret_cast<piece_t *>(p));
}

// The lane's columns j .. j + N - 1 of the bias (0 past n).
template <int N>
__device__ __forceinline__ void load_bias(const Epi &ep, int64_t j, float (&b)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) b[e] = ep.bias && j + e < ep.n ? ep.bias[j + e] : 0.f;
}

// The residual of row i, columns j .. j + N - 1 (0 without one); they are inside n, in one
// aligned piece. Apart from finish(), so that a lane has its rows' loads in flight together:
// behind a store the compiler would keep each in its place.
template <class T, int N>
__device__ __forceinline__ void load_residual(const Epi &ep, int64_t i, int64_t j, float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.f;
    if (ep.residual) load_piece(static_cast<const T *>(ep.residual) + i * ep.ldr + j, v);
}

// Those columns from z (the bias added) and the residual.
template <class T, int N>
__device__ __forceinline__ void finish(float (&v)[N], const float (&add)[N], const Epi &ep, int64_t i, int64_t j) {
    if (ep.Z) store_piece(static_cast<T *>(ep.Z) + i * ep.ldz + j, v);
    activate<T>(v, ep.act);
    if (ep.residual) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += add[e];
    }
    store_piece(static_cast<T *>(ep.O) + i * ep.ldo + j, v);
}

// The same for one element: rows without alignment, and the columns of a last partial tile.
template <class T>
__device__ __forceinline__ float load_residual1(const Epi &ep, int64_t i, int64_t j) {
    return ep.residual ? load1(static_cast<const T *>(ep.residual) + i * ep.ldr + j) : 0.f;
}
template <class T>
__device__ __forceinline__ void finish1(float z, float add, const Epi &ep, int64_t i, int64_t j) {
    float v[1] = {z};
    if (ep.Z) store1(static_cast<T *>(ep.Z) + i * ep.ldz + j, z);
    activate<T>(v, ep.act);
    store1(static_cast<T *>(ep.O) + i * ep.ldo + j, ep.residual ? v[0] + add : v[0]);
}

// How a wave takes a staged block of ROWS x COLS sums where a lane moves whole 16-byte pieces of
// O's rows: lane l has columns EC (l % kLanes) .. of the rows l / kLanes + kRows i, i < N, U of
// them at a time.
template <class T, int ROWS, int COLS>
struct Staged {
    static constexpr int EC = 16 / (int)sizeof(T), kLanes = COLS / EC, kRows = 64 / kLanes, N = ROWS / kRows;
    static constexpr int U = N < 4 ? N : N < 16 ? 4 : 8;
};

// The bias of a lane's columns in such a block (0 past n).
template <class T, int ROWS, int COLS>
struct Bias {
    typedef Staged<T, ROWS, COLS> S;
    u32x4_t q[S::EC / 4];
    __device__ __forceinline__ void load(const Epi &ep, int64_t j0) {
        const int64_t left = ep.n - j0;
        const auto rb = row_rsrc(ep.bias + j0, ep.bias && left > 0 ? 4 * (left < COLS ? left : COLS) : 0);
        const uint32_t c = S::EC * ((threadIdx.x & 63) % S::kLanes);
#pragma unroll
        for (int i = 0; i < S::EC / 4; ++i) q[i] = __builtin_amdgcn_raw_buffer_load_b128(rb, 4 * c + 16 * i, 0, 0);
    }
    __device__ __forceinline__ float operator[](int e) const { return __uint_as_float(q[e >> 2][e & 3]); }
};

// Buffer over `cols` columns from j0 on of the rows i0 .. i0 + rows - 1: loads of the rows behind
// them read zeros and stores are dropped (a row's pitch is no less than its columns).
template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t block_rsrc(const void *p, int64_t ld, int64_t i0, int rows,
                                                             int64_t j0, int cols) {
    return row_rsrc(static_cast<const T *>(p) + i0 * ld + j0, ((rows - 1) * ld + cols) * (int)sizeof(T));
}

// The residual's pieces of the rows i .. i + U - 1 of that block, as they are in memory.
template <class T, int ROWS, int COLS>
struct Residual {
    typedef Staged<T, ROWS, COLS> S;
    u32x4_t q[S::U];
    __device__ __forceinline__ void load(const Epi &ep, int64_t i0, int rows, int64_t j0, int i) {
        if (!ep.residual || ep.align < 16 || j0 + COLS > ep.n || rows <= 0 || i >= S::N) return;
        const auto rs = block_rsrc<T>(ep.residual, ep.ldr, i0, rows, j0, COLS);
        const int lane = threadIdx.x & 63;
        const uint32_t pitch = (uint32_t)ep.ldr * (uint32_t)sizeof(T);
        const uint32_t at = (uint32_t)(lane / S::kLanes) * pitch + 16u * (uint32_t)(lane % S::kLanes);
        if (ep.stream) {
#pragma unroll
            for (int u = 0; u < S::U; ++u)
                q[u] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (uint32_t)(S::kRows * (i + u)) * pitch, 0, 2);
        } else {
#pragma unroll
            for (int u = 0; u < S::U; ++u)
                q[u] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (uint32_t)(S::kRows * (i + u)) * pitch, 0, 0);
        }
    }
    __device__ __forceinline__ void add_to(float (&v)[S::U * S::EC]) const {
#pragma unroll
        for (int u = 0; u < S::U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (sizeof(T) == 2) {
                    v[S::EC * u + 2 * e] += bf16_lo(q[u][e]);
                    v[S::EC * u + 2 * e + 1] += bf16_hi(q[u][e]);
                } else {
                    v[S::EC * u + e] += __uint_as_float(q[u][e]);
                }
            }
    }
};

__device__ __forceinline__ u32x4_t piece_of(const float *v, const uint16_t *) {
    return u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ u32x4_t piece_of(const float *v, const float *) {
    return u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}

// Rows [0, ROWS) x columns [0, COLS) of a wave's fp32 sums, staged in LDS at reg in rows of COLS
// with 16-byte chunk c at c ^ (row % (COLS / 4)), to O's rows i0 .. (those < rows) and columns
// j0 ..: a lane takes 16 bytes of a row of O, or, where those are not aligned or not all inside
// n, the wave takes a row's elements side by side. `bias` and `first`, the first rows' residual,
// were asked for before the sums were staged; each next batch's is in flight while one is finished.
//
// In batches, since a large tile has one wave per SIMD and nothing else to hide a row's latency:
// with every row's bias, z, activation and residual on its own, 8192 x 16384 x 4096 took 427 us
// instead of 346 (fp32, gelu by a shorter formula; 396 with the present one) and 470 instead of 323
// (bf16, residual), 4096 x 4001 x 2048 with a residual 137 instead of 41.
template <class T, int ROWS, int COLS>
__device__ __forceinline__ void finish_staged(const uint8_t *reg, const Epi &ep, int64_t i0, int rows, int64_t j0,
                                              const Bias<T, ROWS, COLS> &bias,
                                              const Residual<T, ROWS, COLS> &first) {
    constexpr int CH = COLS / 4;
    const int lane = threadIdx.x & 63;
    auto at = [&](int row, int chunk) { return reg + row * (COLS * 4) + 16 * (chunk ^ (row & (CH - 1))); };
    if (rows <= 0 || j0 >= ep.n) return;
    const T *type = nullptr;
    const int cols = (int)(ep.n - j0 < COLS ? ep.n - j0 : COLS);
    const auto ro = block_rsrc<T>(ep.O, ep.ldo, i0, rows, j0, cols);
    const auto rz = block_rsrc<T>(ep.Z, ep.ldz, i0, rows, j0, cols);
    const uint32_t po = (uint32_t)ep.ldo * (uint32_t)sizeof(T), pz = (uint32_t)ep.ldz * (uint32_t)sizeof(T);
    if (ep.align >= 16 && cols == COLS) {
        typedef Staged<T, ROWS, COLS> S;
        constexpr int EC = S::EC, U = S::U;
        const int c = lane % S::kLanes, r0 = lane / S::kLanes;
        Residual<T, ROWS, COLS> now = first, next;
        for (int i = 0; i < S::N; i += U) {
            next.load(ep, i0, rows, j0, i + U);
            float v[U * EC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e4 = 0; e4 < EC / 4; ++e4) {
                    const floatx4_t f =
                        *reinterpret_cast<const floatx4_t *>(at(S::kRows * (i + u) + r0, (EC / 4) * c + e4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[EC * u + 4 * e4 + e] = f[e] + bias[4 * e4 + e];
                }
            // non-temporal: not read again here, so they should not push the operands' lines
            auto store = [&](__amdgpu_buffer_rsrc_t r, uint32_t pitch) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    __builtin_amdgcn_raw_buffer_store_b128(piece_of(v + EC * u, type), r,
                                                           (uint32_t)(S::kRows * (i + u) + r0) * pitch + 16u * c, 0, 2);
            };
            if (ep.Z) store(rz, pz);
            activate<T>(v, ep.act);
            if (ep.residual) now.add_to(v);
            store(ro, po);
            now = next;
        }
        return;
    }
    // kRows rows side by side, U such at a time, the next ones' residual in flight
    constexpr int kRows = 64 / COLS, N = ROWS / kRows, U = 16;
    static_assert(N % U == 0, "whole batches");
    const int c = lane % COLS, r0 = lane / COLS;
    if (c >= cols) return;
    const float bias1 = ep.bias ? ep.bias[j0 + c] : 0.f;
    const auto ra = block_rsrc<T>(ep.residual, ep.ldr, i0, rows, j0, cols);
    uint32_t now[U], next[U];
    auto fetch = [&](int i) {
        if (!ep.residual || i >= N) return;
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = load_raw1(ra, (uint32_t)(kRows * (i + u) + r0) * (uint32_t)ep.ldr + c, type);
    };
    fetch(0);
    for (int i = 0; i < N; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        fetch(i + U);
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = *reinterpret_cast<const float *>(at(kRows * (i + u) + r0, c >> 2) + 4 * (c & 3)) + bias1;
        auto store = [&](__amdgpu_buffer_rsrc_t r, uint32_t ld) {
#pragma unroll
            for (int u = 0; u < U; ++u) store1(r, (uint32_t)(kRows * (i + u) + r0) * ld + c, v[u], type);
        };
        if (ep.Z) store(rz, (uint32_t)ep.ldz);
        activate<T>(v, ep.act);
        if (ep.residual) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] += __uint_as_float(sizeof(T) == 2 ? now[u] << 16 : now[u]);
        }
        store(ro, (uint32_t)ep.ldo);
    }
}

}  // namespace kq
