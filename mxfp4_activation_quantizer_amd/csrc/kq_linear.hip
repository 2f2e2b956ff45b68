// The W4A4 product with a linear layer's epilogue, for few rows or few tiles,
//   z = deq(A) deq(W)^T + bias,  O = act(z) + residual
// (KroQuant, arXiv 2607.21446v1, Sec. 1 Eq. 2 for the product), and the
// gradients of that epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq.h"
#include "kq_act.hpp"
#include "kq_device.hpp"
#include "kq_host.hpp"

namespace kq {
namespace linear {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Geom {
    int64_t m, n, ldr, ldo, ldz;
    int kbytes, kblocks;  // k / 2, k / 32
    int stages;           // ceil(k / 256)
    int tiles_n;
    int act;
    int vec;  // rows of O, Z and the residual in whole aligned groups of four
};

template <class T>
__device__ __forceinline__ void load4(const T *p, float v[4]);
template <>
__device__ __forceinline__ void load4<float>(const float *p, float v[4]) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
template <>
__device__ __forceinline__ void load4<uint16_t>(const uint16_t *p, float v[4]) {
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void store4(float *p, const float v[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t *p, const float v[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Four neighbouring elements of row i from column j: bias, activation, residual, stores.
template <class T>
__device__ __forceinline__ void finish4(float (&v)[4], const Geom &g, int64_t i, int64_t j, const float *bias,
                                        const T *res, T *O, T *Z) {
    if (g.vec) {
        if (bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += bias[j + e];
        }
        if (Z) store4(Z + i * g.ldz + j, v);
        activate(v, g.act);
        if (res) {
            float r[4];
            load4(res + i * g.ldr + j, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += r[e];
        }
        store4(O + i * g.ldo + j, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (bias && j + e < g.n) v[e] += bias[j + e];
    if (Z) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < g.n) store1(Z + i * g.ldz + j + e, v[e]);
    }
    activate(v, g.act);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < g.n) store1(O + i * g.ldo + j + e, res ? v[e] + load1(res + i * g.ldr + j + e) : v[e]);
}

// A workgroup of WK waves computes 16 MF rows x 16 NF columns of O, each wave every
// WK-th 256-k stage of the whole tile on v_mfma_scale_f32_16x16x128_f8f6f4, operands
// straight from memory into registers (a stage of a row is 128 code bytes, one cache
// line), and the waves' sums meet in LDS in wave order. The instruction's A operand is
// a W fragment and its B operand an A fragment: lane l supplies row l % 16 of each and
// k group l / 16 (one MX block: 16 code bytes, one scale byte), and receives O row
// l % 16, columns 4 (l / 16) + 0..3 of the fragment. Rows past m or n and k groups
// past k are past a record count (or pushed past it) and read zero codes.
template <class T, bool PACKED, int MF, int NF, int WK>
__global__ __launch_bounds__(64 * WK) void product_kernel(const uint8_t *__restrict__ ca,
                                                          const uint8_t *__restrict__ sa,
                                                          const uint8_t *__restrict__ cw,
                                                          const uint8_t *__restrict__ sw, Geom g,
                                                          const float *__restrict__ bias, const T *__restrict__ res,
                                                          T *__restrict__ O, T *__restrict__ Z) {
    __shared__ float4 red[WK][MF * NF][64];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tn = (int)(blockIdx.x % (unsigned)g.tiles_n), tm = (int)(blockIdx.x / (unsigned)g.tiles_n);
    const int64_t m0 = (int64_t)tm * (16 * MF), n0 = (int64_t)tn * (16 * NF);
    const int rows_a = (int)(g.m - m0 < 16 * MF ? g.m - m0 : 16 * MF);
    const int rows_w = (int)(g.n - n0 < 16 * NF ? g.n - n0 : 16 * NF);
    const int row = lane & 15, grp = lane >> 4;

    auto rsrc = [](const uint8_t *p, int64_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), (short)0, (int)bytes, 0x00020000);
    };
    const auto rca = rsrc(ca + m0 * g.kbytes, (int64_t)rows_a * g.kbytes);
    const auto rcw = rsrc(cw + n0 * g.kbytes, (int64_t)rows_w * g.kbytes);
    // packed: a padding row reads a neighbour's or a later stage's byte, or zero past the
    // array; its codes are zero and its outputs are not stored
    const auto rsa = PACKED ? rsrc(sa + 8 * m0, (int64_t)g.stages * 8 * g.m - 8 * m0)
                            : rsrc(sa + m0 * g.kblocks, (int64_t)rows_a * g.kblocks);
    const auto rsw = PACKED ? rsrc(sw + 8 * n0, (int64_t)g.stages * 8 * g.n - 8 * n0)
                            : rsrc(sw + n0 * g.kblocks, (int64_t)rows_w * g.kblocks);
    constexpr uint32_t kNone = 0x80000000u;

    floatx4_t acc[NF][MF];
#pragma unroll
    for (int b = 0; b < NF; ++b)
#pragma unroll
        for (int a = 0; a < MF; ++a) acc[b][a] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    auto codes = [&](__amdgpu_buffer_rsrc_t r, int f, int kb) {  // block kb of row 16 f + lane % 16
        const uint32_t off = kb < g.kblocks ? (uint32_t)((16 * f + row) * g.kbytes + 16 * kb) : kNone;
        const u32x4_t q = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
        return i32x8_t{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
    };
    auto scale = [&](__amdgpu_buffer_rsrc_t r, int64_t rows, int f, int kb) {
        uint32_t off;
        if (PACKED) off = (uint32_t)((kb >> 3) * 8 * rows) + 8 * (16 * f + row) + 4 * (kb & 1) + ((kb & 7) >> 1);
        else off = (uint32_t)((16 * f + row) * g.kblocks + kb);
        return (int)__builtin_amdgcn_raw_buffer_load_b8(r, kb < g.kblocks ? off : kNone, 0, 0);
    };
    for (int s = wave; s < g.stages; s += WK) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kb = 8 * s + 4 * h + grp;
            i32x8_t fa[MF], fw[NF];
            int xa[MF], xw[NF];
#pragma unroll
            for (int a = 0; a < MF; ++a) {
                fa[a] = codes(rca, a, kb);
                xa[a] = scale(rsa, g.m, a, kb);
            }
#pragma unroll
            for (int b = 0; b < NF; ++b) {
                fw[b] = codes(rcw, b, kb);
                xw[b] = scale(rsw, g.n, b, kb);
            }
#pragma unroll
            for (int b = 0; b < NF; ++b)
#pragma unroll
                for (int a = 0; a < MF; ++a)
                    acc[b][a] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[b], fa[a], acc[b][a], 4, 4, 0,
                                                                                  xw[b], 0, xa[a]);
        }
    }
#pragma unroll
    for (int b = 0; b < NF; ++b)
#pragma unroll
        for (int a = 0; a < MF; ++a)
            red[wave][b * MF + a][lane] = make_float4(acc[b][a][0], acc[b][a][1], acc[b][a][2], acc[b][a][3]);
    __syncthreads();
    // group q of four columns: row q / (4 NF) of the tile, columns 4 (q % (4 NF)) ..
    for (int q = t; q < 64 * MF * NF; q += 64 * WK) {
        const int r = q / (4 * NF), c4 = q % (4 * NF);
        const int f = (c4 >> 2) * MF + (r >> 4), l = (c4 & 3) * 16 + (r & 15);
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float4 v = red[w][f][l];
            z[0] += v.x; z[1] += v.y; z[2] += v.z; z[3] += v.w;
        }
        if (r < rows_a && 4 * c4 < rows_w) finish4<T>(z, g, m0 + r, n0 + 4 * c4, bias, res, O, Z);
    }
}

// Backward of the epilogue, any layout: workgroup (x, p) takes 256 columns of the rows
// p, p + parts, ...
template <class T>
__global__ __launch_bounds__(256) void backward_any_kernel(const T *__restrict__ dO, int64_t lddo,
                                                           const T *__restrict__ Z, int64_t ldz, int64_t m, int64_t n,
                                                           int act, T *__restrict__ dZ, int64_t lddz, int parts,
                                                           float *__restrict__ part) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    const int p = (int)blockIdx.y;
    float s = 0.f;
    for (int64_t i = p; i < m; i += parts) {
        float d[1] = {load1(dO + i * lddo + c)}, z[1] = {0.f};
        if (act != KQ_ACT_NONE) z[0] = load1(Z + i * ldz + c);
        activate_grad(d, z, act);
        if (dZ) store1(dZ + i * lddz + c, d[0]);
        s += d[0];
    }
    if (part) part[p * n + c] = s;
}

}  // namespace linear
}  // namespace kq

// ===========================================================================
// Host side
// ===========================================================================
namespace kqhost {
kq_status gemm256_linear(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_w,
                         const uint8_t *scales_w, int packed, int64_t m, int64_t n, int64_t k, const float *bias,
                         int act, int type, const void *residual, int64_t ldr, void *O, int64_t ldo, void *Z,
                         int64_t ldz, kq_stream_t stream);  // kq_gemm256.hip
}

namespace {

using kqhost::aligned;
using kqhost::launched;
using kqhost::sizes_fit;

bool good_type(int type) { return type == KQ_F32 || type == KQ_BF16; }
bool good_act(int act) { return act >= KQ_ACT_NONE && act <= KQ_ACT_GELU_TANH; }

template <class T, bool PACKED>
kq_status launch_product(const uint8_t *ca, const uint8_t *sa, const uint8_t *cw, const uint8_t *sw,
                         kq::linear::Geom g, const float *bias, const void *res, void *O, void *Z,
                         kq_stream_t stream) {
    constexpr int MF = 2, NF = 2, WK = 4;
    const int64_t tiles_m = (g.m + 16 * MF - 1) / (16 * MF), tiles_n = (g.n + 16 * NF - 1) / (16 * NF);
    g.tiles_n = (int)tiles_n;
    // the launch's work-items are counted in 32 bits
    if (tiles_m * tiles_n > (int64_t)0xFFFFFFFF / (64 * WK)) return KQ_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((kq::linear::product_kernel<T, PACKED, MF, NF, WK>), dim3((unsigned)(tiles_m * tiles_n)),
                       dim3(64 * WK), 0, (hipStream_t)stream, ca, sa, cw, sw, g, bias, (const T *)res, (T *)O, (T *)Z);
    return launched();
}

}  // namespace

extern "C" {

kq_status kq_mxfp4_linear(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_w,
                          const uint8_t *scales_w, int packed, int64_t m, int64_t n, int64_t k, const float *bias,
                          int act, int type, const void *residual, int64_t ldr, void *O, int64_t ldo, void *Z,
                          int64_t ldz, kq_stream_t stream) {
    if (m < 0 || n < 0 || k < 0 || k % 32 != 0 || (packed && k % 256 != 0) || ldo < n || (residual && ldr < n) ||
        (Z && ldz < n))
        return KQ_ERR_SHAPE;
    if (!residual) ldr = 0;
    if (!Z) ldz = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, k, ldr, ldo, ldz})) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return KQ_OK;
    if (!O || (k > 0 && (!codes_a || !scales_a || !codes_w || !scales_w))) return KQ_ERR_NULL;
    const int es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(codes_a, 16) || !aligned(codes_w, 16) || (packed && (!aligned(scales_a, 8) || !aligned(scales_w, 8))) ||
        !aligned(bias, 4) || !aligned(residual, es) || !aligned(O, es) || !aligned(Z, es))
        return KQ_ERR_ALIGN;
    // buffer record counts and offsets are 32-bit
    const int64_t lim = (int64_t)1 << 31;
    if (256 * (k / 2) >= lim || m * (k / 32) >= lim || n * (k / 32) >= lim || (255 * ldo + n) * es >= lim ||
        (255 * ldr + n) * es >= lim || (255 * ldz + n) * es >= lim)
        return KQ_ERR_UNSUPPORTED;
    const bool big = packed ? aligned(scales_a, 16) && aligned(scales_w, 16)
                            : k % 128 == 0 && aligned(scales_a, 4) && aligned(scales_w, 4);
    if (big && ((m + 255) / 256) * ((n + 255) / 256) >= 64)
        return kqhost::gemm256_linear(codes_a, scales_a, codes_w, scales_w, packed, m, n, k, bias, act, type, residual,
                                      ldr, O, ldo, Z, ldz, stream);
    kq::linear::Geom g;
    g.m = m;
    g.n = n;
    g.ldr = ldr;
    g.ldo = ldo;
    g.ldz = ldz;
    g.kbytes = (int)(k / 2);
    g.kblocks = (int)(k / 32);
    g.stages = (int)((k + 255) / 256);
    g.act = act;
    g.vec = n % 4 == 0 && ldo % 4 == 0 && ldr % 4 == 0 && ldz % 4 == 0 && aligned(O, 4 * es) &&
            aligned(residual, 4 * es) && aligned(Z, 4 * es);
    if (type == KQ_BF16)
        return packed ? launch_product<uint16_t, true>(codes_a, scales_a, codes_w, scales_w, g, bias, residual, O, Z,
                                                       stream)
                      : launch_product<uint16_t, false>(codes_a, scales_a, codes_w, scales_w, g, bias, residual, O, Z,
                                                        stream);
    return packed
               ? launch_product<float, true>(codes_a, scales_a, codes_w, scales_w, g, bias, residual, O, Z, stream)
               : launch_product<float, false>(codes_a, scales_a, codes_w, scales_w, g, bias, residual, O, Z, stream);
}

kq_status kq_mxfp4_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || n < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, n})) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = kqhost::row_parts(m);
    if (parts > 1) *bytes = parts * n * 4;
    return KQ_OK;
}

kq_status kq_mxfp4_linear_backward(const void *dO, int64_t lddo, const void *Z, int64_t ldz, int type, int64_t m,
                                   int64_t n, int act, void *dZ, int64_t lddz, float *dbias, void *workspace,
                                   int64_t workspace_bytes, kq_stream_t stream) {
    const bool reads_z = act != KQ_ACT_NONE;
    if (m < 0 || n < 0 || lddo < n || (reads_z && ldz < n) || (dZ && lddz < n)) return KQ_ERR_SHAPE;
    if (!reads_z) ldz = 0;
    if (!dZ) lddz = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, lddo, ldz, lddz})) return KQ_ERR_UNSUPPORTED;
    if (n == 0) return KQ_OK;
    if (!aligned(dbias, 4)) return KQ_ERR_ALIGN;
    if (m == 0) return dbias ? kqhost::reduce_parts(nullptr, nullptr, 0, n, dbias, nullptr, stream) : KQ_OK;
    if (!dO || (reads_z && !Z) || (!dZ && !dbias)) return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(dO, es) || (reads_z && !aligned(Z, es)) || !aligned(dZ, es)) return KQ_ERR_ALIGN;
    const int64_t parts = kqhost::row_parts(m);
    float *part = dbias;
    if (dbias && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * n * 4) return KQ_ERR_SHAPE;
        part = static_cast<float *>(workspace);
    }
    const dim3 grid((unsigned)((n + 255) / 256), (unsigned)parts);
    if (type == KQ_BF16)
        hipLaunchKernelGGL((kq::linear::backward_any_kernel<uint16_t>), grid, dim3(256), 0, (hipStream_t)stream,
                           (const uint16_t *)dO, lddo, (const uint16_t *)Z, ldz, m, n, act, (uint16_t *)dZ, lddz,
                           (int)parts, part);
    else
        hipLaunchKernelGGL((kq::linear::backward_any_kernel<float>), grid, dim3(256), 0, (hipStream_t)stream,
                           (const float *)dO, lddo, (const float *)Z, ldz, m, n, act, (float *)dZ, lddz, (int)parts,
                           part);
    if (dbias && parts > 1) return kqhost::reduce_parts(part, nullptr, parts, n, dbias, nullptr, stream);
    return launched();
}

}  // extern "C"
