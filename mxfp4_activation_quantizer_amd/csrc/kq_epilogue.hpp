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
    activate(v, ep.act);
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
    activate(v, ep.act);
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

// The residual's pieces of the rows i .. i + U - 1 of that block, as they are in memory; rows past
// the last take row 0's, and without a residual nothing is read.
template <class T, int ROWS, int COLS>
struct Residual {
    typedef Staged<T, ROWS, COLS> S;
    u32x4_t q[S::U];
    __device__ __forceinline__ void load(const Epi &ep, int64_t i0, int rows, int64_t j0, int i) {
        if (!ep.residual || ep.align < 16 || j0 + COLS > ep.n || rows <= 0 || i >= S::N) return;
        const int lane = threadIdx.x & 63, r0 = lane / S::kLanes;
        const int64_t j = j0 + S::EC * (lane % S::kLanes);
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
            const int row = S::kRows * (i + u) + r0;
            q[u] = *reinterpret_cast<const u32x4_t *>(static_cast<const T *>(ep.residual) +
                                                      (i0 + (row < rows ? row : 0)) * ep.ldr + j);
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

// Rows [0, ROWS) x columns [0, COLS) of a wave's fp32 sums, staged in LDS at reg in rows of COLS
// with 16-byte chunk c at c ^ (row % (COLS / 4)), to O's rows i0 .. (those < rows) and columns
// j0 ..: a lane takes 16 bytes of a row of O, or, where those are not aligned or not all inside
// n, the wave takes a row's elements side by side. `first` holds the first rows' residual
// (asked for before the sums were staged); each next batch's is in flight while one is finished.
template <class T, int ROWS, int COLS>
__device__ __forceinline__ void finish_staged(const uint8_t *reg, const Epi &ep, int64_t i0, int rows, int64_t j0,
                                              const Residual<T, ROWS, COLS> &first) {
    constexpr int CH = COLS / 4;
    const int lane = threadIdx.x & 63;
    auto at = [&](int row, int chunk) { return reg + row * (COLS * 4) + 16 * (chunk ^ (row & (CH - 1))); };
    if (rows <= 0) return;
    if (ep.align >= 16 && j0 + COLS <= ep.n) {
        typedef Staged<T, ROWS, COLS> S;
        constexpr int EC = S::EC, U = S::U;
        const int c = lane % S::kLanes, r0 = lane / S::kLanes;
        const int64_t j = j0 + EC * c;
        float bias[EC];
        load_bias(ep, j, bias);
        Residual<T, ROWS, COLS> now = first, next;
        for (int i = 0; i < S::N; i += U) {
            auto row_of = [&](int u) { return S::kRows * (i + u) + r0; };
            next.load(ep, i0, rows, j0, i + U);
            float v[U * EC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e4 = 0; e4 < EC / 4; ++e4) {
                    const floatx4_t f = *reinterpret_cast<const floatx4_t *>(at(row_of(u), (EC / 4) * c + e4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[EC * u + 4 * e4 + e] = f[e] + bias[4 * e4 + e];
                }
            auto store = [&](void *to, int64_t ld) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[EC];
#pragma unroll
                    for (int e = 0; e < EC; ++e) x[e] = v[EC * u + e];
                    if (row_of(u) < rows) store_piece(static_cast<T *>(to) + (i0 + row_of(u)) * ld + j, x);
                }
            };
            if (ep.Z) store(ep.Z, ep.ldz);
            activate(v, ep.act);
            if (ep.residual) now.add_to(v);
            store(ep.O, ep.ldo);
            now = next;
        }
        return;
    }
    constexpr int kRows = 64 / COLS, N = ROWS / kRows, U = 8;  // kRows rows side by side
    const int c = lane % COLS, r0 = lane / COLS;
    const int64_t j = j0 + c;
    if (j >= ep.n) return;
    const float bias = ep.bias ? ep.bias[j] : 0.f;
    for (int i = 0; i < N; i += U) {
        float add[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = kRows * (i + u) + r0;
            add[u] = load_residual1<T>(ep, i0 + (row < rows ? row : 0), j);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = kRows * (i + u) + r0;
            const float z = *reinterpret_cast<const float *>(at(row, c >> 2) + 4 * (c & 3)) + bias;
            if (row < rows) finish1<T>(z, add[u], ep, i0 + row, j);
        }
    }
}

}  // namespace kq
