// tw_quant_rules.hpp -- how the int8 products are spread over the chip: plain
// host arithmetic on sizes, apart from the kernels.
#pragma once

#include <stdint.h>

namespace tw {

// ---- a few rows: blocks of 16 MB token rows by 16 NC weight rows ------------
// A CU runs one workgroup of these well; a second one on the same CU, or a
// second round, costs about as much as the first.  So the block grows (which
// also has the token rows read by fewer workgroups) until the grid is at most
// one workgroup a CU.
constexpr int kFewGrid = 256;
constexpr int64_t few_blocks(int rows, int block) { return ((int64_t)rows + block - 1) / block; }
constexpr bool few_fits(int M, int N, int MB, int NC) {
    return few_blocks(M, 16 * MB) * few_blocks(N, 16 * NC) <= kFewGrid;
}

// Weight rows a workgroup of one block of 16 token rows takes: an even share of
// N over the workgroups that each of the M / 16 row blocks has of the grid, so
// that every CU streams as much (the other rows of its last block of 16 repeat
// the last one's and are not stored).  At least 8 where each workgroup also
// quantises the rows.  Measured (us, 16 NC against this): one row, linear 5632 x
// 2048 6.1, 5.3; gateup 5632 x 2048 10.6, 8.9, 2048 x 5632 8.0, 7.6; 32 rows,
// 2048 x 1001 4.1, 3.9, gateup 5.2, 4.7 (shares of 1 / 256 of N each, so a grid of
// 502 workgroups: 5.0, 6.0).
constexpr int few_rows(int M, int N, int NC, bool fused) {
    const int64_t row_blocks = few_blocks(M, 16);
    const int64_t groups = row_blocks < kFewGrid ? kFewGrid / row_blocks : 1;
    const int64_t share = (N + groups - 1) / groups, least = fused ? 8 : 4;
    const int64_t R = share < least ? least : (share + 1) / 2 * 2;
    return (int)(R < 16 * NC ? R : 16 * NC);
}

// ---- large tiles: row regions of the 8 XCDs ---------------------------------
// With r row regions (and 8 / r column regions) a token row comes into 8 / r of
// the L2s and a weight row into r: the fewest such copies of the splits into 2,
// 4 and 8 row regions that divide the grid of nbm x nbn tiles.  2 where none
// does: the grid is then walked without regions.  Measured (us): on zeros,
// 16384 x 8192 x 2048, 8 regions 172, 2 regions 178, gateup 16384 x 2048 x 8192
// 411 and 380; on normal values, 4 regions against the undivided walk, gateup 4096
// x 1024 x 4352 43.2, 46.2, linear 2048 x 5632 x 5632 59.3, 60.9.
constexpr int wide_row_regions(int64_t nbm, int64_t nbn) {
    int best = 0;
    int64_t copies = 0;
    for (int r = 2; r <= 8; r *= 2) {
        if (nbm % r || nbn % (8 / r)) continue;
        const int64_t c = nbm * (8 / r) + nbn * r;
        if (best && c >= copies) continue;
        best = r;
        copies = c;
    }
    return best ? best : 2;
}

}  // namespace tw
