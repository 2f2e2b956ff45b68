// Activation functions of the W4A4 product's epilogue and their slopes, in
// fp32 on the hardware's exp2 and reciprocal (each good to 1 ulp).
//
//   relu       max(z, 0); slope 1 for z > 0, else 0
//   silu       z s(z), s(z) = 1 / (1 + exp(-z)); slope s + z s (1 - s)
//   gelu       z P(z), P(z) = (1 + erf(z / sqrt 2)) / 2; slope P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z (1 + tanh u) / 2 = z s(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
//
// (1 + tanh u) / 2 is written as the logistic function s(2 u): one exponential
// and no cancellation for negative z. Error of s for negative z, relative: the exponent's roundings
// are multiplied by the exponent, so (1.3 |z| + 5) 2^-24 in silu and (6 w + 5) 2^-24 in gelu_tanh,
// w = 2 |u| (20 2^-24 for silu at z = -12 and 300 for gelu_tanh at -8, where s is 6e-6 and 4e-22);
// 6 2^-24 and less for positive z. Absolute, at most 8 2^-24 |z| of the value.
//
// P, the normal distribution function, is 1 - tail(|z|) or, for negative z, tail(|z|) itself:
//   tail(a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) R(a),
// where R falls smoothly from 1/2 to 1 / (a sqrt(2 pi)): t times a polynomial in
// t = 1 / (1 + 0.35 a), fitted to the least largest relative error on 0 <= a <= 14.5.
// For fp32 outputs and all gradients: degree 8 (3.2e-8), and the rounding of a^2 and of the
// exponent, which would grow with a^2, is carried along: P is good to 13 2^-24 of itself for
// z >= -13, where it is 6e-39 (t 2 of them times 2.3 for R's slope, the exponential 4, the rest
// the polynomial and its products). For bf16 outputs: degree 6 (1.7e-6) without that, good to
// (45 + 1.2 z^2) 2^-24, at most 1.5e-5 of itself, a hundredth of the output's own half step
// (bf16 8192 x 16384 x 4096 with gelu 343 us, 383 with the longer form; fp32 396). The exponential is
// the one the slope needs.
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
template <bool FULL>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float a = fminf(fabsf(z), 16.0f);  // exp(-a^2 / 2) is 0 in fp32 from 14 on
    const float den = fmaf(0.35f, a, 1.0f), q = a * a;
    constexpr float c = 0.7213475f, c_low = 9.629815e-09f;  // log2(e) / 2
    const float x = -(q * c);
    e = exp2_hw(x);
    float t = rcp_hw(den), p;
    if (FULL) {
        t = fmaf(t, fmaf(-den, t, 1.0f), t);
        // x + d = -a^2 log2(e) / 2: the products' roundings and the constant's own in d
        const float d = fmaf(fmaf(a, a, -q), -c, fmaf(q, -c_low, fmaf(-q, c, -x)));
        e = fmaf(e, d * 0.69314718f, e);
        p = fmaf(t, -0.029157827f, 0.14403063f);
        p = fmaf(t, p, -0.25583842f);
        p = fmaf(t, p, 0.15931903f);
        p = fmaf(t, p, -0.023211906f);
        p = fmaf(t, p, 0.105552316f);
        p = fmaf(t, p, 0.11982133f);
        p = fmaf(t, p, 0.1398635f);
        p = fmaf(t, p, 0.1396213f);
    } else {
        p = fmaf(t, 0.042030837f, -0.17598428f);
        p = fmaf(t, p, 0.20035155f);
        p = fmaf(t, p, 0.015617063f);
        p = fmaf(t, p, 0.14103363f);
        p = fmaf(t, p, 0.13719165f);
        p = fmaf(t, p, 0.13975868f);
    }
    const float tail = (p * t) * e;
    return z < 0.f ? tail : 1.0f - tail;
}

// z[i] = act(z[i]), for outputs of type T
template <class T, int N>
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
                z[i] = z[i] * normal_cdf<sizeof(T) == 4>(z[i], e);
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
                const float p = normal_cdf<true>(z[i], e);
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

// The gradients of act(z) u for the gradient d of it: d[i] = d[i] u[i] act'(z[i]), u[i] = d[i] act(z[i]), with
// activate's value in its long form and activate_grad's slope.
template <int N>
__device__ __forceinline__ void activate_gated_grad(float (&d)[N], float (&u)[N], const float (&z)[N], int act) {
    auto put = [&](int i, float value, float slope) {
        const float t = d[i];
        d[i] = t * slope * u[i];
        u[i] = t * value;
    };
    switch (act) {
        case KQ_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) put(i, z[i] < 0.f ? 0.f : z[i], z[i] > 0.f ? 1.f : 0.f);
            break;
        case KQ_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = logistic2(-kLog2e * z[i]), v = z[i] * s;
                put(i, v, fmaf(v, 1.0f - s, s));
            }
            break;
        case KQ_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float e;
                const float p = normal_cdf<true>(z[i], e);
                put(i, z[i] * p, fmaf(z[i] * 0.39894228040143268f, e, p));
            }
            break;
        case KQ_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float z2 = fminf(z[i] * z[i], 0x1p96f);
                const float s = logistic2(gelu_tanh_exponent(z[i], z2));
                constexpr float c = 1.59576912160573f;  // 2 sqrt(2 / pi)
                const float v = z[i] * s;
                put(i, v, fmaf(v * (1.0f - s), fmaf(3.0f * 0.044715f * c, z2, c), s));
            }
            break;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) put(i, z[i], 1.f);
            break;
    }
}

}  // namespace kq
