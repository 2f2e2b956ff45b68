// The choice of kq_mxfp4_linear's kernel. Plain C++, so that a host-only build can say which kernel
// a product runs on (the tests' shapes have to reach every one).
#pragma once

#include <math.h>
#include <stdint.h>

namespace kq {
namespace linear {

// Which kernel a product of m x n outputs over `stages` 256-k stages runs on: the least of
// seven estimates, in us, fitted to 535 measured products (profiles/linear_products_by_kernel.md: m = 1
// .. 8192, n = 512 .. 11008, k = 256 .. 8192; the choice is 1.0% slower than the fastest on average, 35% at
// worst): a launch, and per round of tiles a tile's own time and that of its stages. Up to 16 rows only the kernel that
// splits k is considered (16384 x 8192, W from HBM: one row 19.2 us, 20.5 with 64 x 64 tiles, 16 rows
// 19.8 and 20.9).
// Measured at k = 4096, n = 4096, in the order of the list:
//      16 rows  5.7   6.4   6.8   8.2  10.5  14.1
//      64      12.9   9.9   7.6   8.1  10.7  14.4
//     128      22.5  16.3  12.1   8.2  10.6  14.8  19.0
//     512                  39.1  15.6  12.7  16.0  21.3
//    1024                        27.0  22.9  16.9  22.0
//    4096                        94.2  71.4  52.6  38.2
enum Kernel { kProduct11, kProduct12, kProduct22, kTile64Deep, kTile64, kTile128, kTile256 };

// can256: the scales' alignment and k allow the 256 x 256 kernel; cus: compute units.
inline Kernel choose_kernel(int64_t m, int64_t n, int stages, bool packed, bool can256, int cus) {
    const double st = stages;
    auto tiles = [&](int64_t tm, int64_t tn) {  // per compute unit
        return (double)((m + tm - 1) / tm) * (double)((n + tn - 1) / tn) / cus;
    };
    Kernel best = kProduct11;
    double least = 2.8 + ceil(tiles(16, 16)) * (0.148 * st + 0.14);
    auto consider = [&](Kernel k, double us) {
        if (us < least) best = k, least = us;
    };
    consider(kProduct12, 2.6 + ceil(tiles(16, 32)) * (0.21 * st + 0.13));
    if (m <= 16) return best;
    consider(kProduct22, 2.6 + ceil(tiles(32, 32)) * (0.277 * st + 0.27));
    consider(kTile64Deep, 2.5 + ceil(tiles(64, 64)) * (0.296 * st + 2.69));
    // four at a time per compute unit, a stage's latency each while there are fewer
    consider(kTile64, 2.8 + fmax(0.63 * st, 0.25 * st + tiles(64, 64) * (0.2 * st + 0.89)));
    consider(kTile128, 2.9 + ceil(tiles(128, 128)) * (0.65 * st + 2.65));
    if (can256) {
        // whole rounds, and a last one of at most half the compute units in half tiles
        const double full = packed ? 13.55 + 1.41 * st : 2.1 + 2.33 * st, half = packed ? 6.07 + 1.05 * st : 3.16 + 1.48 * st;
        const double t256 = tiles(256, 256), rem = t256 - floor(t256);
        consider(kTile256, 1.65 + floor(t256) * full + (rem == 0 ? 0 : rem <= 0.5 ? half : full));
    }
    return best;
}

// The same for kq_mxfp4_gated_linear, whose tiles hold as many columns of both weights (`n` is the output's): tiles of
// 16 x 16 and 32 x 16 outputs with k split over four waves, 64 x 64 four stages deep and two, 128 x 64, and 256 x 128 on
// persistent workgroups. Six estimates for each layout of the scales, fitted to 1043 measured products
// (profiles/gated_products_by_kernel.md: m = 1 .. 8192, n = 512 .. 11008, k = 256 .. 8192; the choice is 0.6%
// slower than the fastest on average, 25% at worst). The split of k wins while its tiles are few for the compute units;
// one token of n = 11008, k = 4096 takes 11.4 us on either the first kernel or the third. What counts of the tiles is mostly
// the rounds they make: 258 tiles of 128 x 64 (768 x 2752) take longer than 256 by more than their number. The large kernel's
// first round starts from cold, the next ones behind another tile's loads. (With estimates linear in the tiles 42 products
// lost more than 10%, 50% at worst; 11 do now. On 1920 others drawn at random, ragged ones among them, the choice is 1.2%
// slower on average and 33% at worst; 1.7% and 71% before.)
// Measured at n = 11008, k = 4096, packed scales, in the order of the list (us):
//       1 row   11.4         11.4  13.2
//      64              29.7  12.1  13.7  15.8
//     256              99.6  32.2  26.6  28.8  24.7
//    1024                   108.7  83.5  76.3  52.2
//    8192                   785.7 610.0 514.2 343.1
enum GatedKernel { kGatedProduct1, kGatedProduct2, kGatedTile64Deep, kGatedTile64, kGatedTile128, kGatedTile256 };

// can256: the scales' alignment and k allow the 256 x 128 kernel.
inline GatedKernel choose_gated_kernel(int64_t m, int64_t n, int stages, bool packed, bool can256, int cus) {
    // t: tiles per compute unit, or, by the last number of a list (0: as they are, 1: whole rounds), between
    struct Estimate {
        double split1[5], split2[5];   // a + b stages + t (c stages + d)
        double deep[3];                // a + rounds (b stages + c)
        double tile64[6], tile128[6];  // a + the larger of b stages and c stages + t (d stages + e)
        double big[10];                // a + the first round (b + c stages; in half tiles d + e stages) + each later one (f +
                                       // g stages; a last one in half tiles h + i stages) + j (below)
    };
    static const Estimate layouts[2] = {
        {{2.73, 0.0308, 0.229, 0.0854, 0.697}, {2.85, 0.0451, 0.305, 0.149, 0.87}, {1.3, 0.453, 3.48},
         {3.06, 0.577, 0.266, 0.343, 1.79, 0.58}, {3.06, 0.345, 0.0598, 0.675, 2.85, 0.791},
         {1.75, 7.2, 1.81, 4.04, 1.46, 4.91, 1.83, 3.48, 1.57, 5.79}},  // MX layout
        {{2.82, 0.00257, 0.216, 0.0894, 0.662}, {2.98, 0.000877, 0.27, 0.194, 0.869}, {0.81, 0.452, 3.2},
         {2.65, 0.577, 0.235, 0.35, 1.3, 0.61}, {2.98, 0.224, 0.0471, 0.713, 1.73, 0.775},
         {0.0112, 9.42, 1.4, 6.72, 0.92, 5.22, 1.59, 4.05, 1.12, 5.83}}};  // packed
    const Estimate &e = layouts[packed ? 1 : 0];
    const double st = stages;
    auto tiles = [&](int64_t tm, int64_t tn) {  // per compute unit
        return (double)((m + tm - 1) / tm) * (double)((n + tn - 1) / tn) / cus;
    };
    auto between = [](double t, double whole) { return t + whole * (ceil(t) - t); };
    GatedKernel best = kGatedProduct1;
    double least = HUGE_VAL;
    auto consider = [&](GatedKernel k, double us) {
        if (us < least) best = k, least = us;
    };
    auto split = [&](const double (&x)[5], double t) { return x[0] + x[1] * st + between(t, x[4]) * (x[2] * st + x[3]); };
    auto shared = [&](const double (&x)[6], double t) {
        return x[0] + fmax(x[1] * st, x[2] * st + between(t, x[5]) * (x[3] * st + x[4]));
    };
    if (m <= 16) consider(kGatedProduct1, split(e.split1, tiles(16, 16)));
    else if (m <= 256) consider(kGatedProduct2, split(e.split2, tiles(32, 16)));  // measured up to there
    consider(kGatedTile64Deep, e.deep[0] + ceil(tiles(64, 64)) * (e.deep[1] * st + e.deep[2]));
    consider(kGatedTile64, shared(e.tile64, tiles(64, 64)));
    consider(kGatedTile128, shared(e.tile128, tiles(128, 64)));
    if (can256) {
        const double t = tiles(256, 128), rounds = floor(t), rem = t - rounds, later = e.big[5] + e.big[6] * st;
        const bool halves = rem > 0 && rem <= 0.5;
        double us = e.big[0] + (rounds > 0 || !halves ? e.big[1] + e.big[2] * st : e.big[3] + e.big[4] * st);
        if (rounds > 0) us += (rounds - 1) * later + (rem == 0 ? 0 : halves ? e.big[7] + e.big[8] * st : later);
        // a wave's 64 columns that n cuts short leave element by element: at the end of a single round nothing hides that (4096 x
        // 1376 x 512 18.1 us, 2048 x 2752 x 512, as many tiles, 12.1)
        if (t <= 1 && !halves && n % 64 != 0) us += e.big[9];
        consider(kGatedTile256, us);
    }
    return best;
}

}  // namespace linear
}  // namespace kq
