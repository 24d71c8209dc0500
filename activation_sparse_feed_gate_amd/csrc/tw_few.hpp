// tw_few.hpp -- products of up to 64 token rows with a weight matrix that is
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

constexpr int kFewRowsMax = 64;   // of the products that stream weight rows
constexpr int kFewDownMax = 16;   // of few_down_kernel

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
// part[split][m][k] = sum over n of the split of h[m][n] w[n][k]: w rows are read
// whole, 128 columns a workgroup (16 lanes of 16 bytes, 4 rows a wave), the products
// on the vector units (a matrix instruction would need w transposed), h from LDS.
constexpr int kDownThreads = 512, kDownRows = 256;  // reduction rows between two barriers

template <int MT>
__global__ __launch_bounds__(kDownThreads) void few_down_kernel(const uint16_t *__restrict__ h,
                                                                const uint16_t *__restrict__ w,
                                                                int M, int K, int N, int per,
                                                                float *__restrict__ part) {
    constexpr int NW = kDownThreads / kWave, STEPS = kDownRows / (4 * NW);
    __shared__ float hs[MT][kDownRows];
    __shared__ __attribute__((aligned(16))) float sums[NW / 2][MT][128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.x * 128 + 8 * (lane & 15);
    const int at = col < K ? col : K - 8;  // (columns past K repeat the last ones)
    const int n0 = blockIdx.y * per, n1 = min(n0 + per, N);
    const int r0 = 4 * wave + (lane >> 4);
    float acc[MT][8] = {};
    for (int c = n0; c < n1; c += kDownRows) {
        u32x4 v[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int n = c + 4 * NW * i + r0;
            v[i] = ld16(w + (int64_t)min(n, n1 - 1) * K + at);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < MT * kDownRows; i += kDownThreads) {
            const int m = i / kDownRows, n = c + i % kDownRows;
            hs[m][i % kDownRows] =
                m < M && n < n1 ? bf_lo((uint32_t)h[(int64_t)m * N + n]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int r = 4 * NW * i + r0;
            // (rows past the split repeat its last one, which must not enter: 0 times
            // an infinity is NaN)
            const bool in = c + r < n1;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = in ? (e & 1 ? bf_hi(v[i][e >> 1]) : bf_lo(v[i][e >> 1])) : 0.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float hv = hs[m][r];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m][e] = fmaf(hv, f[e], acc[m][e]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[m][e] += __shfl_xor(acc[m][e], 16);
            acc[m][e] += __shfl_xor(acc[m][e], 32);
        }
    // the waves' sums, halves of them at a time
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (wave >= half && wave < 2 * half && lane < 16)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[wave - half][m][8 * lane + e] = acc[m][e];
        __syncthreads();
        if (wave < half && lane < 16)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[m][e] += sums[wave][m][8 * lane + e];
    }
    if (wave || lane >= 16 || col >= K) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m >= M) continue;
        float *p = part + ((int64_t)blockIdx.y * M + m) * K + col;
        *reinterpret_cast<f32x4 *>(p) = f32x4{acc[m][0], acc[m][1], acc[m][2], acc[m][3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{acc[m][4], acc[m][5], acc[m][6], acc[m][7]};
    }
}

// Splits of N that give every CU a workgroup, none of fewer than 32 rows.
inline int few_down_splits(int K, int N) {
    const int cols = (K + 127) / 128, most = (N + 31) / 32;
    const int want = (256 + cols - 1) / cols;
    return want < most ? want : most;
}

inline hipError_t launch_few_down(const uint16_t *h, const uint16_t *w, int M, int K, int N,
                                  float *part, hipStream_t s) {
    const int splits = few_down_splits(K, N);
    const int per = (N + splits - 1) / splits;
    const dim3 grid((K + 127) / 128, splits);
    if (M == 1) few_down_kernel<1><<<grid, kDownThreads, 0, s>>>(h, w, M, K, N, per, part);
    else if (M == 2) few_down_kernel<2><<<grid, kDownThreads, 0, s>>>(h, w, M, K, N, per, part);
    else if (M <= 4) few_down_kernel<4><<<grid, kDownThreads, 0, s>>>(h, w, M, K, N, per, part);
    else if (M <= 8) few_down_kernel<8><<<grid, kDownThreads, 0, s>>>(h, w, M, K, N, per, part);
    else few_down_kernel<16><<<grid, kDownThreads, 0, s>>>(h, w, M, K, N, per, part);
    return hipGetLastError();
}

}  // namespace tw
