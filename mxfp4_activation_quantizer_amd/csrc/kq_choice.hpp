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

}  // namespace linear
}  // namespace kq
