// Layer norm in front of the quantized layers: forward, backward with the
// reduction of its parameters' gradients, and forward straight into the
// Kronecker transform and MXFP4 quantizer (KroQuant, arXiv 2607.21446v1,
// Sec. 1 Eq. 1, Sec. 3.1-3.2).
//
// Per row x of d values, in fp32:
//   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
//   y = (x - mean) rstd w + b.
// The mean is summed in 64 bits: a mean near zero is what is left of values
// that cancel, and 32 bits would leave it with the rounding of the largest. It
// is kept as c + off (c its fp32 rounding, off the rest), and values are
// centred as (x - c) - off, so that the rounding of the mean itself (2^-24
// |mean|, 1000 times the rest for a mean of 3000 beside a deviation of 1) never
// enters y. The squares are summed around it, with nothing large to cancel.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kq.h"
#include "kq_device.hpp"
#include "kq_host.hpp"

namespace kq {
namespace norm {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Sum over a wave, the same value in every lane (xor tree: a fixed order).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
    return v;
}

// Sum over a workgroup of 4 waves, in every thread.
template <class V>
__device__ __forceinline__ V block_sum(V v) {
    __shared__ V red[kThreads / 64];
    v = wave_sum(v);
    __syncthreads();  // the previous call's values have been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// A row's statistics.
struct Stats {
    float c, off, rstd;
    __device__ __forceinline__ float centred(float x) const { return (x - c) - off; }
    __device__ __forceinline__ void set_mean(double sum, int64_t d) {
        const double mean = sum / (double)d;
        c = (float)mean;
        off = (float)(mean - c);
    }
    __device__ __forceinline__ void set_rstd(float squares, int64_t d, float eps) {
        rstd = 1.0f / sqrtf(squares / (float)d + eps);
    }
};

// Statistics of a row by a workgroup that reads it element by element.
template <class T>
__device__ __forceinline__ Stats row_stats(const T *x, int64_t d, float eps) {
    Stats st;
    double s = 0.0;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) s += (double)load1(x + c);
    st.set_mean(block_sum(s), d);
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) {
        const float v = st.centred(load1(x + c));
        q = fmaf(v, v, q);
    }
    st.set_rstd(block_sum(q), d, eps);
    return st;
}

// General forward: any width, stride and alignment; one workgroup per row.
template <class T>
__global__ __launch_bounds__(kThreads) void forward_any_kernel(const T *__restrict__ X, int64_t m, int64_t d,
                                                               int64_t ldx, const float *__restrict__ w,
                                                               const float *__restrict__ b, float eps,
                                                               T *__restrict__ Y, int64_t ldy,
                                                               float *__restrict__ mean, float *__restrict__ rstd) {
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const T *x = X + i * ldx;
        const Stats st = row_stats(x, d, eps);
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float h = st.centred(load1(x + c)) * st.rstd;
            store1(Y + i * ldy + c, fmaf(h, w ? w[c] : 1.0f, b ? b[c] : 0.0f));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = st.c;
            if (rstd) rstd[i] = st.rstd;
        }
    }
}

// General backward, dx: one workgroup per row.
template <class T>
__global__ __launch_bounds__(kThreads) void backward_dx_any_kernel(const T *__restrict__ dY, int64_t lddy,
                                                                   const T *__restrict__ X, int64_t ldx, int64_t m,
                                                                   int64_t d, const float *__restrict__ w,
                                                                   const float *__restrict__ mean,
                                                                   const float *__restrict__ rstd,
                                                                   T *__restrict__ dX, int64_t lddx) {
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const float mu = mean[i], rs = rstd[i], inv = 1.0f / (float)d;
        float a = 0.f, b = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = load1(dY + i * lddy + c) * (w ? w[c] : 1.0f);
            const float h = (load1(X + i * ldx + c) - mu) * rs;
            a += g;
            b = fmaf(g, h, b);
        }
        a = block_sum(a) * inv;
        b = block_sum(b) * inv;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = load1(dY + i * lddy + c) * (w ? w[c] : 1.0f);
            const float h = (load1(X + i * ldx + c) - mu) * rs;
            store1(dX + i * lddx + c, rs * (fmaf(-h, b, g - a)));
        }
    }
}

// General backward, the parameters' gradients: workgroup (x, p) sums 256 columns over
// the rows p, p + parts, ... into row p of the partial sums.
template <class T>
__global__ __launch_bounds__(kThreads) void backward_params_any_kernel(
    const T *__restrict__ dY, int64_t lddy, const T *__restrict__ X, int64_t ldx, int64_t m, int64_t d,
    const float *__restrict__ mean, const float *__restrict__ rstd, int parts, float *__restrict__ pw,
    float *__restrict__ pb) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= d) return;
    const int p = (int)blockIdx.y;
    float sw = 0.f, sb = 0.f;
    for (int64_t i = p; i < m; i += parts) {
        const float dy = load1(dY + i * lddy + c);
        sw = fmaf(dy, (load1(X + i * ldx + c) - mean[i]) * rstd[i], sw);
        sb += dy;
    }
    if (pw) pw[p * d + c] = sw;
    if (pb) pb[p * d + c] = sb;
}

// out[c] = sum over p of part[p][c], p ascending in four interleaved chains (one per
// wave of the workgroup), then the chains: 64 columns per workgroup, y = 0 for the first
// output, 1 for the second.
__global__ __launch_bounds__(kThreads) void reduce_parts_kernel(const float *__restrict__ part0,
                                                                const float *__restrict__ part1, int parts, int64_t d,
                                                                float *__restrict__ out0, float *__restrict__ out1) {
    __shared__ float red[4][64];
    const float *part = blockIdx.y ? part1 : part0;
    float *out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < d; c0 += (int64_t)gridDim.x * 64) {
        const int64_t c = c0 + lane;
        float s = 0.f;
        if (c < d)
            for (int p = w; p < parts; p += 4) s += part[p * d + c];
        red[w][lane] = s;
        __syncthreads();
        if (w == 0 && c < d) out[c] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
        __syncthreads();
    }
}

// Layer norm, transform and quantizer: one workgroup per row, a quad of lanes per
// 32-channel block (8 channels per lane).
template <class T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T *__restrict__ X, int64_t m, int64_t d,
                                                            int64_t ldx, const float *__restrict__ w,
                                                            const float *__restrict__ b, float eps,
                                                            const float *__restrict__ factors,
                                                            uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales, int packed,
                                                            float *__restrict__ y_debug, float *__restrict__ mean,
                                                            float *__restrict__ rstd) {
    const int sub = threadIdx.x & 3;
    const int nblk = (int)(d / 32);
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const T *x = X + i * ldx;
        const Stats st = row_stats(x, d, eps);
        for (int j = threadIdx.x >> 2; j < nblk; j += kThreads / 4) {
            const int c = 32 * j + 8 * sub;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = st.centred(load1(x + c + e)) * st.rstd;
                y[e] = fmaf(h, w ? w[c + e] : 1.0f, b ? b[c + e] : 0.0f);
            }
            if (factors) {
                KronLane L;
                kron_lane_setup(factors + (int64_t)j * 20, sub, L);
                kron_apply8(y, L);
            }
            uint32_t sbyte;
            const uint32_t q = quantize_quad_f32(y, sbyte);
            *reinterpret_cast<uint32_t *>(codes + i * (d / 2) + c / 2) = q;
            if (sub == 0) {
                if (packed) scales[((int64_t)(j >> 3) * m + i) * 8 + 4 * (j & 1) + ((j & 7) >> 1)] = (uint8_t)sbyte;
                else scales[i * nblk + j] = (uint8_t)sbyte;
            }
            if (y_debug) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y_debug[i * d + c + e] = y[e];
            }
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = st.c;
            if (rstd) rstd[i] = st.rstd;
        }
    }
}

}  // namespace norm
}  // namespace kq

// ===========================================================================
// Host side
// ===========================================================================
namespace {

using kqhost::aligned;
using kqhost::launched;
using kqhost::sizes_fit;

bool good_eps(float eps) { return eps >= 0.f && eps <= 3.4e38f; }
bool good_type(int type) { return type == KQ_F32 || type == KQ_BF16; }
uintptr_t size_of(int type) { return type == KQ_BF16 ? 2 : 4; }

// Workgroups that walk m rows: enough to fill the chip, the rest by stride.
unsigned row_grid(int64_t m) { return (unsigned)(m < 65536 ? m : 65536); }

}  // namespace

namespace kqhost {

kq_status reduce_parts(const float *part0, const float *part1, int64_t parts, int64_t d, float *out0, float *out1,
                       kq_stream_t stream) {
    const int64_t groups = (d + 63) / 64;
    hipLaunchKernelGGL(kq::norm::reduce_parts_kernel, dim3((unsigned)(groups < 65536 ? groups : 65536), out1 ? 2 : 1),
                       dim3(kq::norm::kThreads), 0, (hipStream_t)stream, part0, part1, (int)parts, d, out0, out1);
    return launched();
}

}  // namespace kqhost

extern "C" {

kq_status kq_layernorm(const void *X, int type, int64_t m, int64_t d, int64_t ldx, const float *weight,
                       const float *bias, float eps, void *Y, int64_t ldy, float *mean, float *rstd,
                       kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || ldy < d || !good_eps(eps)) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx, ldy})) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || d == 0) return KQ_OK;
    if (!X || !Y) return KQ_ERR_NULL;
    const uintptr_t es = size_of(type);
    if (!aligned(X, es) || !aligned(Y, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    if (type == KQ_BF16)
        hipLaunchKernelGGL((kq::norm::forward_any_kernel<uint16_t>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const uint16_t *)X, m, d, ldx, weight, bias, eps, (uint16_t *)Y, ldy,
                           mean, rstd);
    else
        hipLaunchKernelGGL((kq::norm::forward_any_kernel<float>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const float *)X, m, d, ldx, weight, bias, eps, (float *)Y, ldy, mean,
                           rstd);
    return launched();
}

kq_status kq_layernorm_backward_workspace_bytes(int64_t m, int64_t d, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || d < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, d})) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = kqhost::row_parts(m);
    if (parts > 1) *bytes = parts * 2 * d * 4;
    return KQ_OK;
}

kq_status kq_layernorm_backward(const void *dY, int64_t lddy, const void *X, int64_t ldx, int type, int64_t m,
                                int64_t d, const float *weight, const float *mean, const float *rstd, void *dX,
                                int64_t lddx, float *dweight, float *dbias, void *workspace, int64_t workspace_bytes,
                                kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || lddy < d || lddx < d) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx, lddy, lddx})) return KQ_ERR_UNSUPPORTED;
    if (d == 0) return KQ_OK;
    if (!aligned(dweight, 4) || !aligned(dbias, 4)) return KQ_ERR_ALIGN;
    const bool params = dweight || dbias;
    if (m == 0) return params ? kqhost::reduce_parts(nullptr, nullptr, 0, d, dweight, dbias, stream) : KQ_OK;
    if (!dY || !X || !mean || !rstd || !dX) return KQ_ERR_NULL;
    const uintptr_t es = size_of(type);
    if (!aligned(dY, es) || !aligned(X, es) || !aligned(dX, es) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    const int64_t parts = kqhost::row_parts(m);
    float *pw = dweight, *pb = dbias;
    if (params && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * 2 * d * 4) return KQ_ERR_SHAPE;
        pw = static_cast<float *>(workspace);
        pb = pw + parts * d;
    }
    const dim3 pgrid((unsigned)((d + 255) / 256), (unsigned)parts);
    if (type == KQ_BF16) {
        hipLaunchKernelGGL((kq::norm::backward_dx_any_kernel<uint16_t>), dim3(row_grid(m)), dim3(kq::norm::kThreads),
                           0, (hipStream_t)stream, (const uint16_t *)dY, lddy, (const uint16_t *)X, ldx, m, d, weight,
                           mean, rstd, (uint16_t *)dX, lddx);
        if (params)
            hipLaunchKernelGGL((kq::norm::backward_params_any_kernel<uint16_t>), pgrid, dim3(kq::norm::kThreads), 0,
                               (hipStream_t)stream, (const uint16_t *)dY, lddy, (const uint16_t *)X, ldx, m, d, mean,
                               rstd, (int)parts, pw, pb);
    } else {
        hipLaunchKernelGGL((kq::norm::backward_dx_any_kernel<float>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const float *)dY, lddy, (const float *)X, ldx, m, d, weight, mean,
                           rstd, (float *)dX, lddx);
        if (params)
            hipLaunchKernelGGL((kq::norm::backward_params_any_kernel<float>), pgrid, dim3(kq::norm::kThreads), 0,
                               (hipStream_t)stream, (const float *)dY, lddy, (const float *)X, ldx, m, d, mean, rstd,
                               (int)parts, pw, pb);
    }
    if (params && parts > 1) return kqhost::reduce_parts(pw, pb, parts, d, dweight, dbias, stream);
    return launched();
}

kq_status kq_layernorm_quantize_mxfp4(const void *X, int type, int64_t m, int64_t d, int64_t ldx, const float *weight,
                                      const float *bias, float eps, const float *factors, uint8_t *codes,
                                      uint8_t *scales, int packed, float *y_debug, float *mean, float *rstd,
                                      kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || d % 32 != 0 || (packed && d % 256 != 0) || !good_eps(eps)) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx}) || d > 32768) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || d == 0) return KQ_OK;
    if (packed && m > (((int64_t)1 << 31) - 16) / (d / 32)) return KQ_ERR_UNSUPPORTED;
    if (!X || !codes || !scales) return KQ_ERR_NULL;
    if (!aligned(X, 16) || ldx % (type == KQ_BF16 ? 8 : 4) != 0 || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(factors, 16) || !aligned(codes, 16) || !aligned(y_debug, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    if (type == KQ_BF16)
        hipLaunchKernelGGL((kq::norm::quantize_kernel<uint16_t>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const uint16_t *)X, m, d, ldx, weight, bias, eps, factors, codes,
                           scales, packed, y_debug, mean, rstd);
    else
        hipLaunchKernelGGL((kq::norm::quantize_kernel<float>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const float *)X, m, d, ldx, weight, bias, eps, factors, codes, scales,
                           packed, y_debug, mean, rstd);
    return launched();
}

}  // extern "C"
