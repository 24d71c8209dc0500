// tw_few.hpp -- products of few token rows (up to 64) with a weight matrix that is
// streamed once from memory: the rows of a decoded batch.
//
// Weight fragments come straight from memory into registers (no other wave reads
// them), the tokens' from the L2, and 16 weight rows meet 16 token rows in one
// matrix instruction of 32 reduction elements; token rows past the last
// repeat it.  What bounds these products is the stream of weights, so a wave keeps
// two batches of loads: one in flight while the other is multiplied.
#pragma once

#include "tw_rows.hpp"

namespace tw {

constexpr int kFewRowsMax = 64;  // of the FFN's products

// Blocks of 16 token rows that M rows take, rounded up to a power of 2.
constexpr int few_blocks_of(int M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

// acc[b][m] += weight rows of block b times token rows of block m, over the steps
// [s0, s1) of 32 reduction elements.  wp[b]: the lane's weight row (l % 16 of each
// 16) and xp[m]: its token row, both at reduction element 8 (l / 16); a piece past K
// is zero on both sides.  A lane of acc[b][m] holds token l % 16, weight rows 4 (l /
// 16) + r.
template <int NBLK, int MB, int U>
__device__ __forceinline__ void few_product(const uint16_t *const (&wp)[NBLK],
                                            const uint16_t *const (&xp)[MB], int K, int s0, int s1,
                                            f32x4 (&acc)[NBLK][MB]) {
    const int lane8 = 8 * ((threadIdx.x & 63) >> 4);
    struct Batch {
        u32x4 w[U][NBLK], x[U][MB];
    };
    auto load = [&](Batch &b, int s) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            // past the slice or the row: read the row's first piece, use zeros
            const int k = 32 * (s + i);
            const bool in = s + i < s1 && k + lane8 < K;
            const int at = in ? k : -lane8;
#pragma unroll
            for (int m = 0; m < MB; ++m) b.x[i][m] = ld16(xp[m] + at);
#pragma unroll
            for (int n = 0; n < NBLK; ++n) b.w[i][n] = ld16(wp[n] + at);
        }
    };
    auto multiply = [&](Batch &b, int s) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool in = s + i < s1 && 32 * (s + i) + lane8 < K;
            u32x4 x[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) x[m] = in ? b.x[i][m] : u32x4{};
#pragma unroll
            for (int n = 0; n < NBLK; ++n) {
                const u32x4 w = in ? b.w[i][n] : u32x4{};
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x[m]), acc[n][m],
                        0, 0, 0);
            }
        }
    };
    if (s0 >= s1) return;
    Batch a, b;
    load(a, s0);
    for (int s = s0; s < s1; s += 2 * U) {
        if (s + U < s1) load(b, s + U);
        multiply(a, s);
        if (s + U >= s1) break;
        if (s + 2 * U < s1) load(a, s + 2 * U);
        multiply(b, s + U);
    }
}

}  // namespace tw
