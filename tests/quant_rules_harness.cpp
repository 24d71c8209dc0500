// Host checks of the rules that spread the int8 products over the chip
// (tw_quant_rules.hpp), over many sizes; prints RULES_OK.
#include <cstdio>
#include <initializer_list>

#include "tw_quant_rules.hpp"

namespace {

int g_fail = 0;

void expect(bool ok, const char *what, int M, int N) {
    if (ok || ++g_fail > 20) return;
    std::printf("FAIL %s: M=%d N=%d\n", what, M, N);
}

// Blocks of 16 token rows: where 16 weight rows a workgroup fit the chip, the
// share that is launched does too, and a share is at most a block.
void few() {
    using namespace tw;
    for (int M = 1; M <= 4200; M += M < 200 ? 1 : 37)
        for (int N = 1; N <= 9000; N += N < 300 ? 1 : 61)
            for (int NC = 1; NC <= 2; ++NC)
                for (int fused = 0; fused <= (M <= 4); ++fused) {
                    if (!few_fits(M, N, 1, NC)) continue;
                    const int R = few_rows(M, N, NC, fused);
                    expect(R >= (fused ? 8 : 4) && R <= 16 * NC && R % 2 == 0, "share", M, N);
                    expect(few_blocks(M, 16) * few_blocks(N, R) <= kFewGrid, "grid of shares", M, N);
                    // no larger than it has to be: the next smaller even share would not fit
                    expect(R <= (fused ? 8 : 4) || few_blocks(M, 16) * few_blocks(N, R - 2) > kFewGrid ||
                               few_blocks(N, R - 2) > kFewGrid / few_blocks(M, 16),
                           "even share", M, N);
                }
    expect(few_rows(1, 1 << 24, 2, false) == 32 && few_rows(1 << 24, 5, 1, false) == 5 + 1, "extremes", 0, 0);
}

// Row regions of the large tiles: 2, 4 or 8; a split that divides the grid
// wherever one does, and no other such split with fewer operand copies.
void regions() {
    using namespace tw;
    auto divides = [](int m, int n, int r) { return m % r == 0 && n % (8 / r) == 0; };
    auto copies = [](int m, int n, int r) { return m * (8 / r) + n * r; };
    for (int m = 1; m <= 200; ++m)
        for (int n = 1; n <= 200; ++n) {
            const int got = wide_row_regions(m, n);
            expect(got == 2 || got == 4 || got == 8, "regions", m, n);
            for (int r : {2, 4, 8}) {
                if (!divides(m, n, r)) continue;
                expect(divides(m, n, got), "a split that divides", m, n);
                expect(copies(m, n, got) <= copies(m, n, r), "fewest copies", m, n);
            }
        }
    expect(wide_row_regions(64, 8) == 8 && wide_row_regions(64, 16) == 4 && wide_row_regions(16, 16) == 2 &&
               wide_row_regions(8, 7) == 8 && wide_row_regions(8, 34) == 4 && wide_row_regions(20, 17) == 2,
           "regions by hand", 0, 0);
}

}  // namespace

int main() {
    few();
    regions();
    if (g_fail) return 1;
    std::printf("RULES_OK\n");
    return 0;
}
