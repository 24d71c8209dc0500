// quant_gemm.hip -- the dense projections of the gated FFN on int8 operands:
// token rows with one scale each, weights [N][K] with one scale per output
// channel, products summed exactly in 32-bit integers on the matrix cores.
//
//   linear:  y[m][n] = (sum_k q[m][k] w[n][k]) x_scale[m] w_scale[n] (+ bias[n])
//   gateup:  h = ReLU(gate) * up, gate and up both such products of one x
//
// |sum| <= 127^2 K stays below 2^31 for K <= 131072, and the integer sum does
// not depend on its order, so every split of K gives the same bits.
//
// Two kernels: a few rows stream the weights (every weight byte is read once
// and K is split over the waves of a workgroup); more rows are tiled over
// the direct-to-LDS ring of tw_gemm.hpp, whose 64-byte stage rows hold 64
// int8 elements: the 16 bytes a lane feeds to v_mfma_i32_32x32x32_i8 lie
// where v_mfma_f32_32x32x16_bf16 has its 8 bf16.
#include "tw_gemm.hpp"
#include "tw_internal.hpp"
#include "tw_rows.hpp"

namespace tw {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x16 mfma32_i8(u32x4 a, u32x4 b, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
// D[16x16] += A[16x64] B[64x16]: lane l holds row (column) l % 16 at k =
// 16 (l / 16) ..+15; result register i is D[4 (l / 16) + i][l % 16].
__device__ __forceinline__ i32x4 mfma16_i8(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// One product's weights.
struct QW {
    const int8_t *w;
    const float *scale;
};
struct QArgs {
    const int8_t *q;
    const float *x_scale;
    QW w[2];            // w[1]: the up projection (gateup)
    const float *bias;  // linear only, or null
    int M, K, N;
    char *y;
    int y_type;
};

// The value of one output element from its integer sums.
template <int NB>
__device__ __forceinline__ float finish(int s0, int s1, float xs, float ws0, float ws1, float b) {
    const float v = (float)s0 * xs * ws0;
    if constexpr (NB == 1) return v + b;
    // a NaN gate stays NaN
    return (v < 0.0f ? 0.0f : v) * ((float)s1 * xs * ws1);
}

__device__ __forceinline__ void put(char *y, int type, size_t o, float v) {
    if (type == TW_T_F32) reinterpret_cast<float *>(y)[o] = v;
    else reinterpret_cast<uint16_t *>(y)[o] = (uint16_t)pack_bf16(v, v);
}

// ------------------------------- a few rows --------------------------------
constexpr int kFewWaves = 8;

// 16 weight rows a workgroup, MB blocks of 16 token rows; wave w takes the
// 64-element steps w, w + 8, ... of K.
template <int MB, int NB>
__global__ __launch_bounds__(kFewWaves *kWave) void quant_few_kernel(QArgs a) {
    __shared__ __attribute__((aligned(16))) i32x4 part[NB][kFewWaves][MB][kWave];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int l16 = lane & 15, kc = (lane >> 4) * 16;
    const int8_t *wr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wr[b] = a.w[b].w + (size_t)min(n0 + l16, a.N - 1) * a.K;
    const int8_t *xr[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) xr[i] = a.q + (size_t)min(i * 16 + l16, a.M - 1) * a.K;
    i32x4 acc[NB][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[b][i] = i32x4{};
    const int steps = (a.K + 63) / 64;
#pragma unroll 2
    for (int s = wave; s < steps; s += kFewWaves) {
        const int k = s * 64 + kc;
        const bool in = k < a.K;  // K is a multiple of 16: a chunk is in or out
        const int kk = in ? k : 0;
        u32x4 wf[NB], xf[MB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wf[b] = ld16(wr[b] + kk);
#pragma unroll
        for (int i = 0; i < MB; ++i) xf[i] = ld16(xr[i] + kk);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (!in) wf[b] = u32x4{};
#pragma unroll
            for (int i = 0; i < MB; ++i) acc[b][i] = mfma16_i8(wf[b], xf[i], acc[b][i]);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MB; ++i) part[b][wave][i][lane] = acc[b][i];
    __syncthreads();
    // one lane position of one row block per thread: 4 outputs of one row
    for (int i = wave; i < MB; i += kFewWaves) {
        i32x4 s[2] = {};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) s[b] += part[b][w][i][lane];
        const int m = i * 16 + l16;
        if (m >= a.M) continue;
        const float xs = a.x_scale[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 4 * (lane >> 4) + j;
            if (n >= a.N) continue;
            put(a.y, a.y_type, (size_t)m * a.N + n,
                finish<NB>(s[0][j], s[1][j], xs, a.w[0].scale[n], NB == 2 ? a.w[1].scale[n] : 0.0f,
                           NB == 1 && a.bias ? a.bias[n] : 0.0f));
        }
    }
}

// ------------------------------- many rows ---------------------------------
template <int BM_, int BN_, int WM, int WN, int S_, int NB_>
struct QG {
    static constexpr int BM = BM_, BN = BN_, S = S_, NB = NB_;
    static constexpr int NW = WM * WN, NTH = NW * 64;
    static constexpr int TM = BM / WM, TN = BN / WN;  // wave tile
    static constexpr int FA = TM / 32, FB = TN / 32;
    static constexpr int SR = BM + NB * BN;           // stage rows: x, then the weights
    static constexpr int NI = SR / (16 * NW);         // direct loads per wave and stage
    static constexpr int STAGE = SR * kPRow;
    static constexpr int LDS = S * STAGE;
    static_assert(TM % 32 == 0 && TN % 32 == 0, "wave tile");
    static_assert(BM % 16 == 0 && BN % 16 == 0 && SR % (16 * NW) == 0, "load slices");
};

// A byte offset past every tile's descriptor (a tile spans at most 256 rows
// of 131072 bytes), where a lane reads zeros.
constexpr uint32_t kOutside = 1u << 30;

template <int BM, int BN, int WM, int WN, int S, int NB>
__global__ __launch_bounds__(WM * WN * 64) void quant_gemm_kernel(QArgs a) {
    using P = QG<BM, BN, WM, WN, S, NB>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int l32 = lane & 31;
    const int KT = (a.K + kPRow - 1) / kPRow;
    int rb, cb;
    xcd_tile(blockIdx.x, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, rb, cb);
    const int m0 = rb * BM, n0 = cb * BN;
    const int mr = min(BM, a.M - m0), nr = min(BN, a.N - n0);  // rows in this tile
    settle_scalars(a.x_scale, a.w[0].scale, a.w[1].scale, a.bias, a.y, a.y_type, a.M, a.N);

    // Load j of a wave fetches stage rows [16 (j NW + wave), +16), all in one
    // operand.  Rows past the matrix read its last one (their results are not
    // stored).
    uint32_t voff[P::NI];
    int chunk[P::NI];  // the lane's 16-byte chunk of a stage row
#pragma unroll
    for (int j = 0; j < P::NI; ++j) {
        const int row0 = (j * P::NW + wave) * 16;
        const int sr = row0 + (lane >> 2);
        int r;
        if (row0 < BM) r = min(sr, mr - 1);
        else if (NB == 1 || row0 < BM + BN) r = min(sr - BM, nr - 1);
        else r = min(sr - BM - BN, nr - 1);
        voff[j] = rows16_voff((uint32_t)r * a.K, lane, row0);
        chunk[j] = (lane & 3) ^ swz(sr);
    }
    const rsrc_t rx = make_rsrc(a.q + (size_t)m0 * a.K, (uint64_t)mr * a.K);
    const rsrc_t r0 = make_rsrc(a.w[0].w + (size_t)n0 * a.K, (uint64_t)nr * a.K);
    const rsrc_t r1 = NB == 2 ? make_rsrc(a.w[1].w + (size_t)n0 * a.K, (uint64_t)nr * a.K) : r0;
    auto issue = [&](int kt, char *st) {
        const uint32_t soff = kt * kPRow;
        const bool last = (kt + 1) * kPRow > a.K;
#pragma unroll
        for (int j = 0; j < P::NI; ++j) {
            const int row0 = (j * P::NW + wave) * 16;
            char *dst = st + row0 * kPRow;
            // chunks past a row's end read zeros in x, so what the weights'
            // chunks hold there does not matter
            if (row0 < BM)
                dma16(rx, last && kt * kPRow + chunk[j] * 16 >= a.K ? kOutside : voff[j], soff, dst);
            else if (NB == 1 || row0 < BM + BN) dma16(r0, voff[j], soff, dst);
            else dma16(r1, voff[j], soff, dst);
        }
    };
    i32x16 acc[NB][P::FA][P::FB];
#pragma unroll
    for (int o = 0; o < NB; ++o)
#pragma unroll
        for (int i = 0; i < P::FA; ++i)
#pragma unroll
            for (int j = 0; j < P::FB; ++j) acc[o][i][j] = i32x16{};
    u32x4 fa[2][P::FA], fb[2][NB][P::FB];  // [register set][...]
    auto load = [&](const char *st, int s, int buf) {
#pragma unroll
        for (int i = 0; i < P::FA; ++i) fa[buf][i] = frag(st, wm * P::TM + i * 32, s, lane);
#pragma unroll
        for (int o = 0; o < NB; ++o)
#pragma unroll
            for (int j = 0; j < P::FB; ++j)
                fb[buf][o][j] = frag(st, BM + o * BN + wn * P::TN + j * 32, s, lane);
    };
    auto mma = [&](int buf) {
#pragma unroll
        for (int i = 0; i < P::FA; ++i)
#pragma unroll
            for (int j = 0; j < P::FB; ++j)
#pragma unroll
                for (int o = 0; o < NB; ++o)
                    acc[o][i][j] = mfma32_i8(fa[buf][i], fb[buf][o][j], acc[o][i][j]);
    };
    kloop_pipelined<S, P::NI>(0, KT, smem, P::STAGE, issue, load, mma);

    float ws[2][P::FB], bias[P::FB];
    int n[P::FB];
#pragma unroll
    for (int j = 0; j < P::FB; ++j) {
        n[j] = n0 + wn * P::TN + j * 32 + l32;
        const int nn = min(n[j], a.N - 1);
        ws[0][j] = a.w[0].scale[nn];
        ws[1][j] = NB == 2 ? a.w[1].scale[nn] : 0.0f;
        bias[j] = NB == 1 && a.bias ? a.bias[nn] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < P::FA; ++i) {
        float xs[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
            xs[r] = a.x_scale[min(m0 + wm * P::TM + i * 32 + mfma32_row(r, lane), a.M - 1)];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int m = m0 + wm * P::TM + i * 32 + mfma32_row(r, lane);
            if (m >= a.M) continue;
#pragma unroll
            for (int j = 0; j < P::FB; ++j) {
                if (n[j] >= a.N) continue;
                put(a.y, a.y_type, (size_t)m * a.N + n[j],
                    finish<NB>(acc[0][i][j][r], acc[NB - 1][i][j][r], xs[r], ws[0][j], ws[1][j],
                               bias[j]));
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, int S, int NB>
hipError_t launch_tiles(const QArgs &a, hipStream_t s) {
    using P = QG<BM, BN, WM, WN, S, NB>;
    constexpr auto kernel = &quant_gemm_kernel<BM, BN, WM, WN, S, NB>;
    const hipError_t e = lds_limit_once<kernel>(P::LDS);
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)(((int64_t)a.M + BM - 1) / BM * (((int64_t)a.N + BN - 1) / BN));
    kernel<<<grid, P::NTH, P::LDS, s>>>(a);
    return hipGetLastError();
}

template <int NB>
hipError_t launch_product(const QArgs &a, hipStream_t s) {
    if (a.M == 0) return hipSuccess;
    const int few = (a.N + 15) / 16;
    if (a.M <= 16) {
        quant_few_kernel<1, NB><<<few, kFewWaves * kWave, 0, s>>>(a);
        return hipGetLastError();
    }
    if (a.M <= 32) {
        quant_few_kernel<2, NB><<<few, kFewWaves * kWave, 0, s>>>(a);
        return hipGetLastError();
    }
    auto tiles = [&](int bm, int bn) {
        return ((int64_t)a.M + bm - 1) / bm * (((int64_t)a.N + bn - 1) / bn);
    };
    if constexpr (NB == 1) {
        if (tiles(256, 256) >= 192) return launch_tiles<256, 256, 4, 2, 4, 1>(a, s);
        if (tiles(128, 128) >= 192) return launch_tiles<128, 128, 2, 4, 4, 1>(a, s);
        return launch_tiles<64, 64, 2, 2, 4, 1>(a, s);
    } else {
        if (tiles(256, 128) >= 192) return launch_tiles<256, 128, 4, 2, 4, 2>(a, s);
        if (tiles(128, 64) >= 192) return launch_tiles<128, 64, 4, 2, 4, 2>(a, s);
        return launch_tiles<64, 64, 2, 2, 4, 2>(a, s);
    }
}

}  // namespace

hipError_t launch_quant_linear(const int8_t *q, const float *x_scale, const int8_t *w,
                               const float *w_scale, const float *bias, int M, int K, int N,
                               void *y, int y_type, hipStream_t s) {
    return launch_product<1>(
        QArgs{q, x_scale, {{w, w_scale}, {w, w_scale}}, bias, M, K, N, (char *)y, y_type}, s);
}

hipError_t launch_quant_gateup(const int8_t *q, const float *x_scale, const int8_t *wg,
                               const float *g_scale, const int8_t *wu, const float *u_scale, int M,
                               int K, int N, void *h, int h_type, hipStream_t s) {
    return launch_product<2>(
        QArgs{q, x_scale, {{wg, g_scale}, {wu, u_scale}}, nullptr, M, K, N, (char *)h, h_type}, s);
}

}  // namespace tw
