// Sine and cosine of the position rotation.
#pragma once

#include <hip/hip_runtime.h>

namespace kq {

// cos and sin of a quarter turn times f, |f| <= 1/2: the angle x = pi f / 2 is made in 64 bits and rounded once, then
// the series in x to x^10 and x^9 (what follows is below 2^-32.5 and 2^-28.5 of them), Horner's rule in x^2. Over f as
// it is given, 1.5 units in the last place at most (1.47 for the sine, 1.22 for the cosine, on the CPU over 10^7
// values); with f rounded to 32 bits first and multiplied there 2.63 and 1.61.
__host__ __device__ __forceinline__ float2 quarter_turn(double f) {
    const float x = (float)(f * 1.5707963267948966), x2 = x * x;
    float c = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f), s = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
    c = fmaf(x2, c, -1.38888889e-3f);
    s = fmaf(x2, s, 8.33333333e-3f);
    c = fmaf(x2, c, 4.16666667e-2f);
    s = fmaf(x2, s, -1.66666667e-1f);
    c = fmaf(x2, c, -0.5f);
    s = s * x2;
    return make_float2(fmaf(x2, c, 1.0f), fmaf(x, s, x));
}

}  // namespace kq
