// Host checks of the rules that spread the int8 products over the chip
// (tw_quant_rules.hpp), over many sizes; prints RULES_OK.
#include <cstdio>

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

}  // namespace

int main() {
    few();
    if (g_fail) return 1;
    std::printf("RULES_OK\n");
    return 0;
}
