// Activation functions of the W4A4 product's epilogue and their slopes, in
// fp32 on the hardware's exp2 and reciprocal (each good to 1 ulp).
//
//   relu       max(z, 0); slope 1 for z > 0, else 0
//   silu       z s(z), s(z) = 1 / (1 + exp(-z)); slope s + z s (1 - s)
//   gelu       z P(z), P(z) = (1 + erf(z / sqrt 2)) / 2; slope P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z (1 + tanh u) / 2 = z s(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
//
// (1 + tanh u) / 2 is written as the logistic function s(2 u): one exponential
// and no cancellation for negative z. P takes Abramowitz and Stegun's
// approximation 7.1.26 of erf (|error| <= 1.5e-7, so P to 0.75e-7) for |z|,
// mirrored for negative z; its exponential is the one the slope needs. Error:
// a few 2^-24 relative in s, at most |z| 1.5e-7 absolute in gelu.
#pragma once

#include <hip/hip_runtime.h>

#include "kq.h"

namespace kq {

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + 2^x): 0 for x = inf, 1 for x = -inf
__device__ __forceinline__ float logistic2(float x) { return rcp_hw(1.0f + exp2_hw(x)); }

// -2 sqrt(2 / pi) log2(e) (z + 0.044715 z^3), the exponent of gelu_tanh's logistic
__device__ __forceinline__ float gelu_tanh_exponent(float z, float z2) {
    constexpr float a = -2.30220819813864f, b = a * 0.044715f;
    return z * fmaf(b, z2, a);
}

// P(z) = (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = rcp_hw(fmaf(0.3275911f, x, 1.0f));
    e = exp2_hw(-(x * x) * kLog2e);
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    const float tail = 0.5f * (p * t) * e;
    return z < 0.f ? tail : 1.0f - tail;
}

template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
    switch (act) {
        case KQ_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];
            break;
        case KQ_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] * logistic2(-kLog2e * z[i]);
            break;
        case KQ_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float e;
                z[i] = z[i] * normal_cdf(z[i], e);
            }
            break;
        case KQ_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] * logistic2(gelu_tanh_exponent(z[i], z[i] * z[i]));
            break;
        default: break;
    }
}

// d[i] *= slope of the activation at z[i]
template <int N>
__device__ __forceinline__ void activate_grad(float (&d)[N], const float (&z)[N], int act) {
    switch (act) {
        case KQ_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = z[i] > 0.f ? d[i] : 0.f;
            break;
        case KQ_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = logistic2(-kLog2e * z[i]);
                d[i] = d[i] * fmaf(z[i] * s, 1.0f - s, s);
            }
            break;
        case KQ_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float e;
                const float p = normal_cdf(z[i], e);
                d[i] = d[i] * fmaf(z[i] * 0.39894228040143268f, e, p);
            }
            break;
        case KQ_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // z^2 kept finite: where it would overflow, s (1 - s) is 0
                const float z2 = fminf(z[i] * z[i], 0x1p96f);
                const float s = logistic2(gelu_tanh_exponent(z[i], z2));
                constexpr float c = 1.59576912160573f;  // 2 sqrt(2 / pi)
                d[i] = d[i] * fmaf(z[i] * s * (1.0f - s), fmaf(3.0f * 0.044715f * c, z2, c), s);
            }
            break;
        default: break;
    }
}

}  // namespace kq
