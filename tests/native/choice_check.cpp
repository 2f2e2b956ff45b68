// Host-only: for every line "m n stages packed can256 cus" of the standard input, the kernel that
// kq_mxfp4_linear runs such a product on (kq_choice.hpp, in its enum's order), and for the 256 x 256 one how
// many tiles are computed whole and how many as two halves (kq_tileorder.hpp).
#include <cstdio>

#include "kq_choice.hpp"
#include "kq_tileorder.hpp"

int main() {
    long long m, n;
    int stages, packed, can256, cus;
    while (std::scanf("%lld %lld %d %d %d %d", &m, &n, &stages, &packed, &can256, &cus) == 6) {
        const int k = kq::linear::choose_kernel(m, n, stages, packed != 0, can256 != 0, cus);
        const auto o = kq::g256::make_tile_order((int)((m + 255) / 256 * ((n + 255) / 256)), cus);
        std::printf("%d %d %d\n", k, o.nwg - o.split, o.split);
    }
}
