// Host-only: what the workgroups of the gated product's 256 x 128 kernel work on and load (kq_tileorder.hpp), for every
// line "m n k packed can256 cus" of the standard input. Each workgroup takes every cus-th work, passes over halves that
// have no column inside n, and asks for stages 0 and 1 of the work that follows beside its own last stage and epilogue
// (of none at all behind the last of a kind). Checked:
//  1. every row tile's columns 0 .. n - 1 are covered once;
//  2. every span of codes lies inside its operand, and no stage's scalar offset passes the span's bytes.
// Prints "kernel works empty passed" for each line (the kernel that the product runs on, in its enum's order; halves
// without a column, and those of them on a workgroup that has other works); the first failure is printed and exits 1.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kq_choice.hpp"
#include "kq_tileorder.hpp"

using namespace kq::g256;

static long long m, n, k;
static int cus;

static void fail(const char *what, long long x) {
    std::printf("FAIL %s m=%lld n=%lld k=%lld cus=%d: %lld\n", what, m, n, k, cus, x);
    std::exit(1);
}

// the loads of stages 0 .. stages - 1 of `rows` rows from row0 on, of an operand of `all` rows
static void check_span(int64_t row0, int rows, int64_t all, int stages) {
    const int kbytes = (int)(k / 2);
    const CodeSpan s = code_span(row0, rows, kbytes);
    if (s.first < 0 || s.first + (int64_t)s.bytes > all * kbytes) fail("outside the operand", s.first);
    for (int i = 0; i < stages; ++i)
        if ((uint64_t)s.step * i > s.bytes) fail("offset past the count", (long long)s.step * i);
    if (rows > 0 && (s.bytes != (uint64_t)rows * kbytes || (uint64_t)s.step * (stages - 1) >= (uint64_t)kbytes)) fail("not all of it", s.bytes);
}

int main() {
    int packed, can256;
    while (std::scanf("%lld %lld %lld %d %d %d", &m, &n, &k, &packed, &can256, &cus) == 6) {
        const int stages = (int)((k + 255) / 256), tiles_m = (int)((m + 255) / 256), tiles_n = (int)((n + 127) / 128);
        const int kernel = kq::linear::choose_gated_kernel(m, n, stages, packed != 0, can256 != 0, cus);
        const TileOrder o = make_tile_order(tiles_m * tiles_n, cus);
        const int works = tile_order_groups(o), grid = works < cus ? works : cus;
        std::vector<std::vector<int>> covered(tiles_m, std::vector<int>(n, 0));
        int empty = 0, passed = 0;
        for (int b = 0; b < grid; ++b) {
            int done = 0, none = 0;
            for (int i = b; i < works; i += grid) {
                const TileWork w = tile_work(i, o);
                const int tm = w.tile % tiles_m, tn = w.tile / tiles_m;  // any numbering of the tiles covers them
                const GatedCols c = gated_cols(tn, w.half, n);
                if (c.count < 0 || c.count > (w.half < 0 ? 128 : 64)) fail("columns", c.count);
                if (c.count == 0) {
                    ++none;
                    continue;
                }
                ++done;
                for (int64_t j = c.first; j < c.first + c.count; ++j)
                    if (j < 0 || j >= n || covered[tm][j]++) fail("column", j);
                const int64_t m0 = (int64_t)tm * 256;
                check_span(m0, (int)(m - m0 < 256 ? m - m0 : 256), m, stages);
                check_span(c.first, c.count, n, stages);
            }
            // behind the last one: nothing
            check_span(0, 0, m, 2);
            check_span(0, 0, n, 2);
            empty += none;
            if (done) passed += none;
        }
        for (const auto &row : covered)
            for (const int x : row)
                if (x != 1) fail("covered", x);
        std::printf("%d %d %d %d\n", kernel, works, empty, passed);
    }
}
