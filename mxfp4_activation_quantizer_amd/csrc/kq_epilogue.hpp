// The epilogue of kq_mxfp4_linear on fp32 sums,
//   z = sum + bias,  O = act(z) + residual,
// applied by every product kernel where a lane holds neighbouring columns of a
// row, so that each access is one piece of 8 or 16 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_act.hpp"
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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

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

// Row i (< m), columns j .. j + N - 1 (from z, the bias added). `whole`: all of them inside
// n and in one aligned piece.
template <class T, int N>
__device__ __forceinline__ void finish(float (&v)[N], const Epi &ep, int64_t i, int64_t j, bool whole) {
    T *o = static_cast<T *>(ep.O) + i * ep.ldo + j;
    T *z = static_cast<T *>(ep.Z) + i * ep.ldz + j;
    const T *r = static_cast<const T *>(ep.residual) + i * ep.ldr + j;
    if (whole) {
        float add[N];
        if (ep.residual) load_piece(r, add);
        if (ep.Z) store_piece(z, v);
        activate(v, ep.act);
        if (ep.residual) {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += add[e];
        }
        store_piece(o, v);
        return;
    }
    if (ep.Z) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (j + e < ep.n) store1(z + e, v[e]);
    }
    activate(v, ep.act);
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (j + e < ep.n) store1(o + e, ep.residual ? v[e] + load1(r + e) : v[e]);
}

}  // namespace kq
