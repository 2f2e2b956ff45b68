// Host-only: the largest errors of kq_turn.hpp's quarter_turn, in units in the last place of the result and over an even
// grid, random fractions of all sizes and both signs, against the C library in 80 bits. Prints "sine cosine".
#include <cmath>
#include <cstdio>
#include <random>

#include "kq_turn.hpp"

typedef long double real;

static real ulps(float got, real want) {
    int e;
    std::frexp(want, &e);
    return std::fabs((real)got - want) / std::ldexp((real)1, e - 24);
}

int main() {
    const real half_pi = 1.57079632679489661923132169163975144L;
    real sine = 0, cosine = 0;
    auto one = [&](double f) {
        const float2 v = kq::quarter_turn(f);
        const real s = std::sin(half_pi * f), c = std::cos(half_pi * f);
        if (f != 0) sine = std::fmax(sine, ulps(v.y, s));
        cosine = std::fmax(cosine, ulps(v.x, c));
    };
    for (long i = -(1 << 21); i <= 1 << 21; ++i) one(0.5 * i / (1 << 21));
    std::mt19937_64 r(1);
    for (int i = 0; i < 3000000; ++i) {
        const double f = (double)(r() >> 11) * 0x1p-54;
        one(i % 3 ? f : -std::ldexp(f, -(i % 100)));
    }
    const float2 none = kq::quarter_turn(0.0);
    if (none.x != 1.0f || none.y != 0.0f) return 1;
    std::printf("%.3Lf %.3Lf\n", sine, cosine);
    return 0;
}
