// linear_ce.hip -- softmax cross entropy of an output projection over a large
// vocabulary, without the logits in memory, and its gradient.
//
// With l = x w^T (one row a token, V columns) and a row's target t:
//   lse = log sum_v exp(l_v),  loss = lse - l_t,
//   D_v = dloss (exp(l_v - lse) - [v = t]),  dx = D w,  dw = D^T x.
// Forward: the product's tiles stay in registers; each leaves, for every row
// of it, the largest logit and the sum of the exponentials below it, and a
// second kernel joins a row's column blocks and takes the target's logit as
// one more dot product.  Backward: the logits are computed again, a piece of the
// vocabulary at a time; a piece's D (bf16: it feeds the matrix cores) is the
// operand of both products.
//
// A row whose target is outside [0, V) is left out: its loss and its row of D
// are 0.
//
// D's rounding to bf16 is up to 2^-8 of a term: a gradient in bf16 is off by 0.0024 of its
// norm, 0.0017 with D in fp32.
//
// What bounds it (bf16, normal operands, calls in a row): 4096 x 1024 x 32768 forward 206
// to 225 us, 1220 to 1330 TFLOP/s, the chip's power (tw_tiles.hpp); backward 4096 x 1024
// x 49999 1123 to 1179 us for three products of 419 GFLOP, D's exponentials (3 us a tile,
// while the matrix cores wait) and its 410 MB written and read twice.  4 rows 1024 x
// 32768: 16.6 to 17 us for 67 MB.
#include <algorithm>

#include "tw_few.hpp"
#include "tw_tiles.hpp"
#include "tw_train.hpp"

namespace tw {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ int64_t target(Targets t, int m) {
    return t.wide ? static_cast<const int64_t *>(t.p)[m]
                  : (int64_t) static_cast<const int32_t *>(t.p)[m];
}

// Largest logit and sum of exponentials of a set of columns, in units of
// log 2: the sum is of 2^(l log2e - top).  The rounding of `top` does not
// matter, as the same number is added back.
struct Soft {
    float top, sum;
};
__device__ __forceinline__ Soft join_soft(Soft a, Soft b) {
    const float top = fmaxf(a.top, b.top);
    const float at = top == -INFINITY ? 0.0f : top;  // nothing yet: sums stay 0
    return {top, a.sum * __builtin_amdgcn_exp2f(a.top - at) +
                     b.sum * __builtin_amdgcn_exp2f(b.top - at)};
}

struct EpiSoft {
    static constexpr bool kStats = true;
    static constexpr int kWalk = 8;
    Soft *part;  // [column blocks][M]
    int M, N;
    typedef NoRaw Raw;
    struct Row {
        float most = -INFINITY, top = 0.0f, sum = 0.0f;
        __device__ Row(const EpiSoft &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ int stores(const Place &) const { return 0; }
    template <int W, bool ALL>
    __device__ __forceinline__ void most(Row &r, int n, const float (&v)[W]) const {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (ALL || n + e < N) r.most = fmaxf(r.most, v[e]);
    }
    template <int W, bool ALL>
    __device__ __forceinline__ void add(Row &r, int n, const float (&v)[W]) const {
        r.top = r.most == -INFINITY ? 0.0f : r.most * kLog2e;
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (ALL || n + e < N) r.sum += __builtin_amdgcn_exp2f(fmaf(v[e], kLog2e, -r.top));
    }
    template <int L>
    __device__ __forceinline__ void join(Row &r) const {
        const Soft a{r.most == -INFINITY ? -INFINITY : r.top, r.sum};
        const Soft b{__shfl_xor(a.top, L), __shfl_xor(a.sum, L)};
        const Soft j = join_soft(a, b);
        r.most = r.top = j.top;
        r.sum = j.sum;
    }
    __device__ __forceinline__ void put(const Row &r, int m, int cb) const {
        part[(int64_t)cb * M + m] = {r.top, r.sum};
    }
};

// Up to 32 token rows (16 MB): a wave takes 32 words and all of K, a workgroup of 4
// waves the 128 of a column block.  (16 words a wave: the tokens' fragments, read anew
// by each, cost more than the shorter waves gain; 16 rows 1024 x 32768 26 us for 22.
// Batches of 9 loads: 20 us, of 18 22.)
constexpr int kSoftBlocks = 2, kFewSoftThreads = 512 / kSoftBlocks;
template <int MB>
__global__ __launch_bounds__(kFewSoftThreads) void few_soft_kernel(
    const uint16_t *__restrict__ x, int64_t x_stride, const uint16_t *__restrict__ w, int M, int K,
    int V, Soft *__restrict__ part) {
    __shared__ Soft all[kFewSoftThreads / kWave][16 * MB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int v0 = blockIdx.x * 128 + 16 * kSoftBlocks * wave;
    const int k8 = 8 * (lane >> 4);
    const uint16_t *wp[kSoftBlocks], *xp[MB];
#pragma unroll
    for (int b = 0; b < kSoftBlocks; ++b)
        wp[b] = w + (int64_t)min(v0 + 16 * b + (lane & 15), V - 1) * K + k8;
#pragma unroll
    for (int m = 0; m < MB; ++m) xp[m] = x + min(16 * m + (lane & 15), M - 1) * x_stride + k8;
    f32x4 acc[kSoftBlocks][MB] = {};
    few_product<kSoftBlocks, MB, 9 / (kSoftBlocks + MB)>(wp, xp, K, 0, (K + 31) / 32, acc);
    const EpiSoft epi{part, M, V};
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        EpiSoft::Row row(epi, {});
        float l[kSoftBlocks][4];
#pragma unroll
        for (int b = 0; b < kSoftBlocks; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) l[b][e] = acc[b][m][e];
#pragma unroll
        for (int b = 0; b < kSoftBlocks; ++b)
            epi.most<4, false>(row, v0 + 16 * b + 4 * (lane >> 4), l[b]);
#pragma unroll
        for (int b = 0; b < kSoftBlocks; ++b)
            epi.add<4, false>(row, v0 + 16 * b + 4 * (lane >> 4), l[b]);
        epi.join<16>(row);
        epi.join<32>(row);
        if (lane < 16) all[wave][16 * m + lane] = {row.top, row.sum};
    }
    __syncthreads();
    if (threadIdx.x >= M) return;
    Soft j = all[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kFewSoftThreads / kWave; ++i) j = join_soft(j, all[i][threadIdx.x]);
    part[(int64_t)blockIdx.x * M + threadIdx.x] = j;
}

// Whether few_soft_kernel takes a product.  A wave of it reads the token rows from the L2
// for its own 32 words, which from 17 rows on costs more than tiles save, unless these
// (256 words wide) would leave half of the CUs idle.  Measured (us, this kernel and
// tiles): 16 rows, 1024 x 32768 20, 30; 2048 x 49999 52, 48 (from memory 87, 93); 32
// rows 24, 30 and 66, 49; 64 rows 32, 31.
bool streams_words(int M, int V) {
    return M <= 16 || (M <= 32 && V <= kWideCols * kWideGrid / 2);
}

// Joins the column blocks of a row and takes the target's logit.  TPR threads a row:
// 16 where rows are many (16 neighbouring rows of a block are then read together),
// a workgroup where they are few.  Bound by latency.  Measured (us with the products, a
// workgroup and 16 threads a row): 4 rows 20.4, 22.6; 300 37.4, 38.9; 512 39.6, 41.0;
// 1024 66.6, 65.5; 4096 238, 225.
template <int TPR>
__global__ __launch_bounds__(256) void ce_rows_kernel(const Soft *__restrict__ part, int blocks,
                                                      const uint16_t *__restrict__ x,
                                                      int64_t x_stride,
                                                      const uint16_t *__restrict__ w, Targets t,
                                                      int M, int K, int V,
                                                      float *__restrict__ loss,
                                                      float *__restrict__ lse) {
    constexpr int ROWS = 256 / TPR;
    __shared__ Soft all[TPR][ROWS + 1];
    __shared__ float dots[TPR][ROWS + 1];
    // thread i of row r; the parts with the rows next to each other, the dot product with
    // a row's threads next to each other
    const int r = threadIdx.x % ROWS, i = threadIdx.x / ROWS;
    const int dr = threadIdx.x / TPR, di = threadIdx.x % TPR;
    const int m = blockIdx.x * ROWS + r, dm = blockIdx.x * ROWS + dr;
    Soft s{-INFINITY, 0.0f};
    if (m < M) {
#pragma unroll 4
        for (int b = i; b < blocks; b += TPR) s = join_soft(s, part[(int64_t)b * M + m]);
    }
    all[i][r] = s;
    const int64_t tgt = dm < M ? target(t, dm) : -1;
    float d = 0.0f;
    if (tgt >= 0 && tgt < V) {
        const uint16_t *xr = x + dm * x_stride, *wr = w + tgt * K;
#pragma unroll 2
        for (int k = 8 * di; k < K; k += 8 * TPR) {
            const u32x4 a = ld16(xr + k), b = ld16(wr + k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d += bf_lo(a[e]) * bf_lo(b[e]) + bf_hi(a[e]) * bf_hi(b[e]);
        }
    }
    dots[di][dr] = d;
    // halves of the threads join pairs, in a fixed order
    for (int half = TPR / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (i < half) {
            all[i][r] = join_soft(all[i][r], all[i + half][r]);
            dots[i][r] += dots[i + half][r];
        }
    }
    if (i || m >= M) return;
    s = all[0][r];
    const float l = kLn2 * (s.top + __builtin_amdgcn_logf(s.sum));
    lse[m] = l;
    // a loss is never negative; the two sums may cross by a rounding
    const float v = l - dots[0][r];
    const int64_t tm = target(t, m);
    loss[m] = tm < 0 || tm >= V || v < 0.0f ? 0.0f : v;
}

// D of a piece of the vocabulary, columns first .. first + N - 1 of V.
struct EpiD {
    static constexpr bool kStats = false;
    static constexpr int kWalk = 4;
    static constexpr int kOuts = 1;
    const float *lse, *dloss;
    Targets t;
    uint16_t *d;
    int64_t ldd;  // N rounded up to 8; the columns past N are written as zeros
    int N, first, V;
    struct Raw {
        float lse, dloss;
        uint32_t lo, hi;  // the target
        __device__ __forceinline__ Raw of(int l) const {
            return {__shfl(lse, l), __shfl(dloss, l), (uint32_t)__shfl((int)lo, l),
                    (uint32_t)__shfl((int)hi, l)};
        }
    };
    // A row without a target has scale 0 and an infinite top, below which every
    // exponential is 0.  A row of scale 0 has a D of 0 also where its logits are NaN or
    // infinite.
    struct Row {
        float top, scale;
        int t;  // the target's column of the piece, or -1
        __device__ __forceinline__ Row(const EpiD &e, const Raw &r) {
            const int64_t v = (int64_t)((uint64_t)r.hi << 32 | r.lo);
            const bool live = v >= 0 && v < e.V;
            top = live ? r.lse * kLog2e : INFINITY;
            scale = live ? r.dloss : 0.0f;
            t = v >= e.first && v < (int64_t)e.first + e.N ? (int)(v - e.first) : -1;
        }
    };
    __device__ __forceinline__ Raw raw(int m) const {
        if (t.wide) {
            const u32x2 v = static_cast<const u32x2 *>(t.p)[m];
            return {lse[m], dloss[m], v[0], v[1]};
        }
        const int32_t v = static_cast<const int32_t *>(t.p)[m];
        return {lse[m], dloss[m], (uint32_t)v, (uint32_t)(v >> 31)};
    }
    __device__ __forceinline__ Dest dest(int, const Place &) const {
        return {d, TW_T_BF16, ldd, (int)ldd, false};
    }
    __device__ int stores(const Place &) const { return 16; }
    typedef NoFetch Fetched;
    __device__ Fetched fetch(int, int) const { return {}; }
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &r, const Fetched &, int n, const float (&v)[W],
                                           const float (&)[W], float (&o)[kOuts][W]) const {
        float p[W];
#pragma unroll
        for (int e = 0; e < W; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(v[e], kLog2e, -r.top));
        const unsigned at = (unsigned)(r.t - n);  // (few lanes have the target: a branch)
        if (at < W) {
#pragma unroll
            for (int e = 0; e < W; ++e) p[e] -= at == (unsigned)e ? 1.0f : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < W; ++e) o[0][e] = ALL || n + e < N ? p[e] * r.scale : 0.0f;
        if (r.scale == 0.0f) {
#pragma unroll
            for (int e = 0; e < W; ++e) o[0][e] = 0.0f;
        }
    }
};

constexpr size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The backward pass's pieces of the vocabulary: columns of D in at most 512 MB (or 256
// of them), and at most kTileStrideMost where tiles read D's rows; dx's sums in parts
// that every piece adds to, a piece's dw.
struct Pieces {
    int width;
    bool few;  // dx in one piece by the kernel of few rows
    SplitPlan dx;
    size_t d_bytes, dx_bytes, part_bytes;
};
SplitPlan dw_plan(int M, int K, int width) {
    return split_plan<1>(TileArgs{{}, {}, 0, 0, width, K, M}, false);
}
Pieces pieces_of(int M, int K, int V) {
    Pieces p;
    int64_t most = (int64_t)(512 << 20) / 2 / (M > 0 ? M : 1) / 256 * 256;
    // Measured (us of D and dx; few rows' kernel, tiles): 1 row 1024 x 32768 33, 40; 64 rows
    // 45, 46; 4 rows 2048 x 49999 69, 72.
    p.few = M <= kFewDownMax && most >= V;
    if (!p.few) most = std::min(most, kTileStrideMost);
    p.width = (int)(most < 256 ? 256 : most < V ? most : V);
    p.d_bytes = up256((size_t)M * ((p.width + 7) / 8 * 8) * 2);
    p.dx = split_plan<1>(TileArgs{{}, {}, 0, 0, M, K, p.width}, p.width < V);
    // the weight gradient's parts behind them, since dx's stay
    size_t dw = dw_plan(M, K, p.width).bytes;
    if (V % p.width) dw = std::max(dw, dw_plan(M, K, V % p.width).bytes);
    p.dx_bytes = up256(p.few ? (size_t)few_down_split(1, M, K, V).splits * M * K * 4 : p.dx.bytes);
    p.part_bytes = p.dx_bytes + up256(dw);
    return p;
}

}  // namespace

size_t ce_fwd_bytes(int M, int, int V) {
    return up256((size_t)M * (((size_t)V + 127) / 128) * sizeof(Soft));
}

hipError_t launch_ce_fwd(const uint16_t *x, int64_t x_stride, const uint16_t *w, Targets t, int M,
                         int K, int V, float *loss, float *lse, void *ws, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const TileArgs p{{x}, {w}, x_stride, K, M, V, K};
    Soft *part = static_cast<Soft *>(ws);
    hipError_t e;
    if (streams_words(M, V)) {
        const int grid = (V + 127) / 128;
        if (few_blocks_of(M) == 1)
            few_soft_kernel<1><<<grid, kFewSoftThreads, 0, s>>>(x, x_stride, w, M, K, V, part);
        else
            few_soft_kernel<2><<<grid, kFewSoftThreads, 0, s>>>(x, x_stride, w, M, K, V, part);
        e = hipGetLastError();
    } else {
        e = launch_tiles<kRows, kRows, 1, 1>(p, EpiSoft{part, M, V}, s);
    }
    if (e != hipSuccess) return e;
    const int blocks = (V + 127) / 128;
    if (M <= 512)
        ce_rows_kernel<256><<<M, 256, 0, s>>>(part, blocks, x, x_stride, w, t, M, K, V, loss, lse);
    else
        ce_rows_kernel<16><<<(M + 15) / 16, 256, 0, s>>>(part, blocks, x, x_stride, w, t, M, K, V,
                                                         loss, lse);
    return hipGetLastError();
}

size_t ce_bwd_bytes(int M, int K, int V) {
    const Pieces p = pieces_of(M, K, V);
    return p.d_bytes + p.part_bytes;
}

hipError_t launch_ce_bwd(const float *dloss, const uint16_t *x, int64_t x_stride,
                         const uint16_t *w, Targets t, const float *lse, int M, int K, int V,
                         void *dx, int dx_type, void *dw, int dw_type, void *ws, hipStream_t s) {
    const Pieces pc = pieces_of(M, K, V);
    uint16_t *d = static_cast<uint16_t *>(ws);
    float *parts = reinterpret_cast<float *>(static_cast<char *>(ws) + pc.d_bytes);
    float *dw_parts = parts + pc.dx_bytes / 4;
    hipError_t e = hipSuccess;
    for (int first = 0; first < V && e == hipSuccess; first += pc.width) {
        const int N = V - first < pc.width ? V - first : pc.width;
        const int64_t ldd = (N + 7) / 8 * 8;
        const uint16_t *wp = w + (int64_t)first * K;
        if (M > 0)
            e = launch_tiles<kRows, kRows, 1, 1>(TileArgs{{x}, {wp}, x_stride, K, M, N, K},
                                                 EpiD{lse, dloss, t, d, ldd, N, first, V}, s);
        if (e == hipSuccess && dx && M > 0 && pc.few)
            e = few_down({d, nullptr}, {wp, nullptr}, 1, ldd, M, K, N, parts, dx, dx_type, s);
        else if (e == hipSuccess && dx && M > 0)
            e = launch_split<kRows, kCols, 1>(
                TileArgs{{d}, {wp}, ldd, K, M, K, N}, pc.dx,
                EpiStore{{dx}, dx_type, K, parts, first > 0}, first + N == V, s);
        if (e == hipSuccess && dw) {
            char *out =
                static_cast<char *>(dw) + (int64_t)first * K * (dw_type == TW_T_F32 ? 4 : 2);
            e = launch_split<kCols, kCols, 1>(TileArgs{{d}, {x}, ldd, x_stride, N, K, M},
                                                 dw_plan(M, K, N),
                                                 EpiStore{{out}, dw_type, K, dw_parts}, true, s);
        }
    }
    return e;
}

}  // namespace tw
