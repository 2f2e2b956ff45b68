// Host-only: for every line "m n stages packed can256 cus" of the standard input, the kernel that
// kq_mxfp4_gated_linear runs such a product on (kq_choice.hpp, in its enum's order), and for the 256 x 128 one how
// many tiles are computed whole, how many as two halves, how many of them follow another one on their workgroup with
// its operands on their way, and how often a workgroup goes from whole tiles to halves or back (kq_tileorder.hpp).
#include <cstdio>

#include "kq_choice.hpp"
#include "kq_tileorder.hpp"

int main() {
    long long m, n;
    int stages, packed, can256, cus;
    while (std::scanf("%lld %lld %d %d %d %d", &m, &n, &stages, &packed, &can256, &cus) == 6) {
        const int k = kq::linear::choose_gated_kernel(m, n, stages, packed != 0, can256 != 0, cus);
        const auto o = kq::g256::make_tile_order((int)((m + 255) / 256 * ((n + 127) / 128)), cus);
        const int works = kq::g256::tile_order_groups(o), grid = works < cus ? works : cus;
        int warm = 0, turns = 0;
        for (int i = grid; i < works; ++i) {
            const bool half = kq::g256::tile_work(i, o).half >= 0, before = kq::g256::tile_work(i - grid, o).half >= 0;
            ++(half == before ? warm : turns);
        }
        std::printf("%d %d %d %d %d\n", k, o.nwg - o.split, o.split, warm, turns);
    }
}
