// tw_few.hpp -- products of few token rows (up to 64) with a weight matrix that is
// streamed once from memory: the rows of a decoded batch.
//
// few_product takes weight rows of reduction elements, few_down_kernel weight rows that
// are the reduction's own.  Weight fragments come straight from memory into registers
// (no other wave reads them), the tokens' from the L2, and 16 weight rows or columns
// meet 16 token rows in one matrix instruction of 32 reduction elements; token rows past
// the last repeat it.  What bounds these products is the stream of weights, so a wave keeps
// two batches of loads: one in flight while the other is multiplied.
#pragma once

#include "tw_rows.hpp"
#include "tw_tiles.hpp"

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

// ------------------ rows times a matrix of reduction rows --------------------
// part[split][m][k] = sum over n of the split of h[m][n] w[n][k], for up to 64 token
// rows (of ldh elements, zeros from N to the next multiple of 8); with a second pair of h
// and w its splits behind the first one's.  A wave reads 32 rows of w, 128 columns wide,
// 16 bytes a lane: lane l has the 8 rows from 8 (l / 16) on of the 8 columns from 8 (l %
// 16) on.  A matrix instruction wants one column's 8 rows in a lane, so pairs of rows are
// interleaved (one permute a register) and instruction j of 8 takes every lane's column j.
// Bound by the stream of w (2048 x 5632, with the sum of the parts: 10.7 us for one row,
// 11.1 for 16, 16.8 for 64; in tiles 17, 18 and 20; the FFN's dx, two pairs, 14, 15, 21 and
// 20, 21, 23.  Products on the vector units took 32 us for 16).
constexpr int kFewDownMax = 64;  // token rows
constexpr int kDownGrid = 256;   // (512: 64 rows 22 us)
template <int MB>
constexpr int kDownWaves = MB == 4 ? 4 : 8;  // (their sums are 8 MB KB of LDS each)

template <int MB>
__global__ __launch_bounds__(64 * kDownWaves<MB>) void few_down_kernel(
    const uint16_t *__restrict__ h0, const uint16_t *__restrict__ w0,
    const uint16_t *__restrict__ h1, const uint16_t *__restrict__ w1, int64_t ldh, int M, int K,
    int N, int per, float *__restrict__ part) {
    const uint16_t *const h = blockIdx.z ? h1 : h0, *const w = blockIdx.z ? w1 : w0;
    constexpr int NW = kDownWaves<MB>;
    extern __shared__ __attribute__((aligned(16))) char smem[];  // [NW][8 MB][64] f32x4
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, r8 = 8 * (lane >> 4);
    const int at = min(blockIdx.x * 128 + 8 * l16, K - 8);  // (past K: the last columns again)
    const int n0 = blockIdx.y * per, n1 = min(n0 + per, N);
    const uint16_t *hp[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) hp[m] = h + min(16 * m + l16, M - 1) * ldh;
    struct Step {
        u32x4 w[8], h[MB];
    };
    // Rows past the split (a multiple of 8, or the end): the first ones again, used as
    // zeros.  Past the end within a group of 8, the last row again, which meets h's zeros.
    auto load = [&](Step &s, int n) {
        const int row = n + r8 < n1 ? n + r8 : n0;
#pragma unroll
        for (int m = 0; m < MB; ++m) s.h[m] = ld16(hp[m] + row);
#pragma unroll
        for (int r = 0; r < 8; ++r) s.w[r] = ld16(w + (int64_t)min(row + r, N - 1) * K + at);
    };
    f32x4 acc[8][MB] = {};
    auto multiply = [&](Step &s, int n) {
        if (n + r8 >= n1) {
#pragma unroll
            for (int r = 0; r < 8; ++r) s.w[r] = u32x4{};
#pragma unroll
            for (int m = 0; m < MB; ++m) s.h[m] = u32x4{};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u32x4 v;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = __builtin_amdgcn_perm(s.w[2 * p + 1][j >> 1], s.w[2 * p][j >> 1],
                                             j & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int m = 0; m < MB; ++m)
                acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, s.h[m]), acc[j][m],
                    0, 0, 0);
        }
    };
    constexpr int kStep = 32 * NW;
    int n = n0 + 32 * wave;
    if (n < n1) {
        Step a, b;
        load(a, n);
        for (;; n += 2 * kStep) {
            if (n + kStep < n1) load(b, n + kStep);
            multiply(a, n);
            if (n + kStep >= n1) break;
            if (n + 2 * kStep < n1) load(a, n + 2 * kStep);
            multiply(b, n + kStep);
            if (n + 2 * kStep >= n1) break;
        }
    }
    // The waves' sums meet in LDS.  Lane l of acc[j][m] holds token l % 16, columns 8 (4
    // (l / 16) + e) + j; a thread then adds the 8 columns of one token.
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int m = 0; m < MB; ++m) sums[((wave * 8 + j) * MB + m) * kWave + lane] = acc[j][m];
    __syncthreads();
    const float *f = reinterpret_cast<const float *>(smem);
    for (int t = threadIdx.x; t < 256 * MB; t += 64 * NW) {
        const int mb = t >> 8, m = 16 * mb + (t & 15), i = t >> 4 & 15;
        const int col = blockIdx.x * 128 + 8 * i;
        if (m >= M || col >= K) continue;
        float s[8] = {};
#pragma unroll
        for (int q = 0; q < NW; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] += f[(((q * 8 + j) * MB + mb) * kWave + (i >> 2) * 16 + (m & 15)) * 4 +
                          (i & 3)];
        const int64_t split = blockIdx.z * gridDim.y + blockIdx.y;
        f32x4 *out = reinterpret_cast<f32x4 *>(part + (split * M + m) * K + col);
        out[0] = f32x4{s[0], s[1], s[2], s[3]};
        out[1] = f32x4{s[4], s[5], s[6], s[7]};
    }
}

// Parts of N: about kDownGrid workgroups, each with as many steps of 32 rows for every
// one of its waves.
struct DownSplit {
    int splits, per;
};
inline DownSplit few_down_split(int pairs, int M, int K, int N) {
    const int rows = 32 * (M <= 32 ? kDownWaves<1> : kDownWaves<4>);
    const int cols = (K + 127) / 128, rounds = (N + rows - 1) / rows;
    const int most = kDownGrid / (pairs * cols) > 1 ? kDownGrid / (pairs * cols) : 1;
    const int each = (rounds + most - 1) / most;
    return {(rounds + each - 1) / each, rows * each};
}

template <int MB>
hipError_t few_down_as(const uint16_t *const (&h)[2], const uint16_t *const (&w)[2], int pairs,
                       int64_t ldh, int M, int K, int N, float *part, hipStream_t s) {
    constexpr auto kernel = &few_down_kernel<MB>;
    constexpr int lds = kDownWaves<MB> * 8 * MB * kWave * 16;
    const hipError_t e = lds_limit_once<kernel>(lds);
    if (e != hipSuccess) return e;
    const DownSplit d = few_down_split(pairs, M, K, N);
    const dim3 grid((K + 127) / 128, d.splits, pairs);
    kernel<<<grid, 64 * kDownWaves<MB>, lds, s>>>(h[0], w[0], h[1], w[1], ldh, M, K, N,
                                                d.per, part);
    return hipGetLastError();
}

inline hipError_t few_down(const uint16_t *const (&h)[2], const uint16_t *const (&w)[2], int pairs,
                           int64_t ldh, int M, int K, int N, float *part, void *out, int type,
                           hipStream_t s) {
    const int mb = few_blocks_of(M);
    const hipError_t e = mb == 1   ? few_down_as<1>(h, w, pairs, ldh, M, K, N, part, s)
                         : mb == 2 ? few_down_as<2>(h, w, pairs, ldh, M, K, N, part, s)
                                   : few_down_as<4>(h, w, pairs, ldh, M, K, N, part, s);
    if (e != hipSuccess) return e;
    const int splits = pairs * few_down_split(pairs, M, K, N).splits;
    return launch_sum_parts(part, splits, (int64_t)M * K, out, type, s);
}

}  // namespace tw
