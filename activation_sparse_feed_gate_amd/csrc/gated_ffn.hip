// gated_ffn.hip -- the dense gated FFN of a trained model, y = (act(x W_g) *
// (x W_u)) W_d, and its gradient.
//
// Forward: one kernel computes both projections, the activation and the
// product (h, and on request the projections g and u for the backward pass,
// each rounded once to bf16 from the fp32 sums); a second one h W_d.
// Backward, from g and u:
//   dh = dy W_d^T,  du = dh act(g),  dz = dh u act'(g),  h = act(g) u  (one kernel)
//   dx = dz W_g^T + du W_u^T                          (one sum over both terms)
//   dW_g^T = dz^T x,  dW_u^T = du^T x,  dW_d = h^T dy           (one launch)
// dz, du and h feed the matrix cores, so they are rounded to bf16 (half a unit
// of 2^-8 a term, averaged out over the sums they enter); every sum is fp32.
//
// Activations of the form g s(a(g)) with the logistic function s: SiLU has
// a = g, the tanh form of GELU a = 2 sqrt(2 / pi) (g + 0.044715 g^3), since
// (1 + tanh(v)) / 2 = s(2 v).  Their derivative is s + g s (1 - s) a'.
#include "tw_few.hpp"
#include "tw_tiles.hpp"
#include "tw_train.hpp"

namespace tw {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// s(a) = 1 / (1 + e^-a); e^-a past the fp32 range gives 0.
__device__ __forceinline__ float logistic(float a) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * a));
}

constexpr float kGelu = 1.59576912160573071176f;  // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == TW_A_RELU) return g <= 0.0f ? 0.0f : g;  // NaN stays NaN
    else if constexpr (ACT == TW_A_SILU) return g * logistic(g);
    else return g * logistic(kGelu * g * (1.0f + kGelu3 * g * g));
}

struct Slope {
    float value, slope;
};
template <int ACT>
__device__ __forceinline__ Slope activate_slope(float g) {
    if constexpr (ACT == TW_A_RELU) return {g <= 0.0f ? 0.0f : g, g <= 0.0f ? 0.0f : 1.0f};
    const bool silu = ACT == TW_A_SILU;
    const float s = logistic(silu ? g : kGelu * g * (1.0f + kGelu3 * g * g));
    const float da = silu ? 1.0f : kGelu * (1.0f + 3.0f * kGelu3 * g * g);
    const float t = s * (1.0f - s);
    // t = 0 far from 0, where g da may be infinite
    return {g * s, s + (t == 0.0f ? 0.0f : g * t * da)};
}

// Gate and up projections -> h (and g, u).
template <int ACT>
struct EpiGlu {
    static constexpr bool kStats = false;
    static constexpr int kOuts = 3;
    uint16_t *h, *g, *u;  // g, u or null
    int N;
    typedef NoRaw Raw;
    struct Row {
        __device__ Row(const EpiGlu &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ int stores(const Place &) const { return 8 * (1 + (g != nullptr) + (u != nullptr)); }
    __device__ __forceinline__ Dest dest(int o, const Place &) const {
        return {o == 0 ? h : o == 1 ? g : u, TW_T_BF16, N, N, false};
    }
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &, int, int, const float (&v)[W],
                                           const float (&w)[W], float (&o)[kOuts][W]) const {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            o[0][e] = activate<ACT>(v[e]) * w[e];
            o[1][e] = v[e];
            o[2][e] = w[e];
        }
    }
};

// dh -> dz, du, h.
template <int ACT>
struct EpiDh {
    static constexpr bool kStats = false;
    static constexpr int kOuts = 3;
    const uint16_t *g, *u;
    uint16_t *dz, *du, *h;
    int N;
    typedef NoRaw Raw;
    struct Row {
        __device__ Row(const EpiDh &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ int stores(const Place &) const { return 48; }
    __device__ __forceinline__ Dest dest(int o, const Place &) const {
        return {o == 0 ? dz : o == 1 ? du : h, TW_T_BF16, N, N, false};
    }
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &, int m, int n, const float (&v)[W],
                                           const float (&)[W], float (&o)[kOuts][W]) const {
        float gv[W], uv[W];
        load_bf16<W>(g + (int64_t)m * N + n, gv);
        load_bf16<W>(u + (int64_t)m * N + n, uv);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const Slope a = activate_slope<ACT>(gv[e]);
            o[0][e] = v[e] * uv[e] * a.slope;
            o[1][e] = v[e] * a.value;
            o[2][e] = a.value * uv[e];
        }
    }
};

// Up to 64 token rows (16 MB): a workgroup takes up to 16 C hidden neurons of both
// matrices, its 8 waves a slice of K each; their sums meet in LDS.
constexpr int kFewUpThreads = 512;
template <int ACT, int C, int MB>
__global__ __launch_bounds__(kFewUpThreads) void few_up_kernel(
    const uint16_t *__restrict__ x, int64_t x_stride, const uint16_t *__restrict__ wg_t,
    const uint16_t *__restrict__ wu_t, int M, int K, int N, int share, uint16_t *__restrict__ g,
    uint16_t *__restrict__ u, uint16_t *__restrict__ h) {
    constexpr int NW = kFewUpThreads / kWave;
    extern __shared__ __attribute__((aligned(16))) char smem[];  // [NW][2 C MB][64] f32x4
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * share, n1 = min(n0 + share, N);
    const int k8 = 8 * (lane >> 4);
    const uint16_t *wp[2 * C], *xp[MB];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t row = min(n0 + 16 * c + (lane & 15), n1 - 1);
        wp[2 * c] = wg_t + row * K + k8;
        wp[2 * c + 1] = wu_t + row * K + k8;
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) xp[m] = x + min(16 * m + (lane & 15), M - 1) * x_stride + k8;
    const int steps = (K + 31) / 32, per = (steps + NW - 1) / NW;
    f32x4 acc[2 * C][MB] = {};
    constexpr int U = 10 / (2 * C + MB) < 1 ? 1 : 10 / (2 * C + MB);  // loads in flight
    few_product<2 * C, MB, U>(wp, xp, K, wave * per, min(wave * per + per, steps), acc);
#pragma unroll
    for (int b = 0; b < 2 * C; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            sums[((wave * 2 * C + b) * MB + m) * kWave + lane] = acc[b][m];
    __syncthreads();
    for (int i = wave; i < C * MB; i += NW) {  // block i / MB of neurons, i % MB of rows
        f32x4 v{}, w{};
#pragma unroll
        for (int q = 0; q < NW; ++q) {
            v += sums[((q * 2 * C + 2 * (i / MB)) * MB + i % MB) * kWave + lane];
            w += sums[((q * 2 * C + 2 * (i / MB) + 1) * MB + i % MB) * kWave + lane];
        }
        const int m = 16 * (i % MB) + (lane & 15);
        if (m >= M) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + 16 * (i / MB) + 4 * (lane >> 4) + e;
            if (n >= n1) continue;
            const int64_t at = (int64_t)m * N + n;
            h[at] = (uint16_t)pack_bf16(activate<ACT>(v[e]) * w[e], 0.0f);
            if (g) g[at] = (uint16_t)pack_bf16(v[e], 0.0f);
            if (u) u[at] = (uint16_t)pack_bf16(w[e], 0.0f);
        }
    }
}

template <int ACT, int C, int MB>
hipError_t few_up_as(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                     const uint16_t *wu_t, int M, int K, int N, int share, uint16_t *g,
                     uint16_t *u, uint16_t *h, hipStream_t s) {
    constexpr auto kernel = &few_up_kernel<ACT, C, MB>;
    constexpr int lds = kFewUpThreads / kWave * 2 * C * MB * kWave * 16;
    const hipError_t e = lds_limit_once<kernel>(lds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)((N + share - 1) / share), kFewUpThreads, lds, s>>>(
        x, x_stride, wg_t, wu_t, M, K, N, share, g, u, h);
    return hipGetLastError();
}

template <int ACT>
hipError_t few_up(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t, const uint16_t *wu_t,
                  int M, int K, int N, uint16_t *g, uint16_t *u, uint16_t *h, hipStream_t s) {
    // an even share of the neurons for each of 256 workgroups, at most 32
    int share = (N + 255) / 256;
    share = share < 4 ? 4 : share > 32 ? 32 : share;
    auto go = [&](auto c, auto mb) {
        return few_up_as<ACT, decltype(c)::value, decltype(mb)::value>(
            x, x_stride, wg_t, wu_t, M, K, N, share, g, u, h, s);
    };
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, 4> four{};
    const int mb = few_blocks_of(M);
    if (share <= 16) return mb == 1 ? go(one, one) : mb == 2 ? go(one, two) : go(one, four);
    return mb == 1 ? go(two, one) : mb == 2 ? go(two, two) : go(two, four);
}

template <int ACT>
hipError_t ffn_up(const TileArgs &p, uint16_t *g, uint16_t *u, uint16_t *h, hipStream_t s) {
    return launch_tiles<kRows, kRows, 2, 1>(p, EpiGlu<ACT>{h, g, u, p.N}, s);
}
template <int ACT>
hipError_t ffn_dh(const TileArgs &p, const uint16_t *g, const uint16_t *u, uint16_t *dz,
                  uint16_t *du, uint16_t *h, hipStream_t s) {
    return launch_tiles<kRows, kRows, 1, 1>(p, EpiDh<ACT>{g, u, dz, du, h, p.N}, s);
}

}  // namespace

static SplitPlan down_plan(int M, int K, int N) {
    return split_plan<1, 1>(TileArgs{{}, {}, N, K, M, K, N}, false);
}
static SplitPlan dx_plan(int M, int K, int N) {
    return split_plan<1, 2>(TileArgs{{}, {}, N, K, M, K, N}, false);
}
static SplitPlan dw_plan(int M, int K, int N) {
    TileArgs p{{}, {}, N, K, N, K, M};
    p.groups = 3;
    return split_plan<1, 1>(p, false);
}

size_t ffn_fwd_part_bytes(int M, int K, int N) {
    if (M <= kFewDownMax) return (size_t)few_down_splits(K, N) * M * K * 4;
    return down_plan(M, K, N).bytes;
}
size_t ffn_bwd_part_bytes(int M, int K, int N) {
    const size_t a = dx_plan(M, K, N).bytes, b = dw_plan(M, K, N).bytes;
    return a > b ? a : b;
}

hipError_t launch_ffn_up(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                         const uint16_t *wu_t, int act, int M, int K, int N, uint16_t *g,
                         uint16_t *u, uint16_t *h, hipStream_t s) {
    if (M <= kFewRowsMax) {
        if (act == TW_A_RELU)
            return few_up<TW_A_RELU>(x, x_stride, wg_t, wu_t, M, K, N, g, u, h, s);
        if (act == TW_A_SILU)
            return few_up<TW_A_SILU>(x, x_stride, wg_t, wu_t, M, K, N, g, u, h, s);
        return few_up<TW_A_GELU>(x, x_stride, wg_t, wu_t, M, K, N, g, u, h, s);
    }
    const TileArgs p{{x}, {wg_t, wu_t}, x_stride, K, M, N, K};
    if (act == TW_A_RELU) return ffn_up<TW_A_RELU>(p, g, u, h, s);
    if (act == TW_A_SILU) return ffn_up<TW_A_SILU>(p, g, u, h, s);
    return ffn_up<TW_A_GELU>(p, g, u, h, s);
}

hipError_t launch_ffn_down(const uint16_t *h, const uint16_t *wd, int M, int K, int N, void *y,
                           int y_type, float *part, hipStream_t s) {
    if (M <= kFewDownMax) {
        const hipError_t e = launch_few_down(h, wd, M, K, N, part, s);
        if (e != hipSuccess) return e;
        return launch_sum_parts(part, few_down_splits(K, N), (int64_t)M * K, y, y_type, s);
    }
    return launch_split<kRows, kCols, 1, 1>(TileArgs{{h}, {wd}, N, K, M, K, N},
                                            down_plan(M, K, N), EpiStore{{y}, y_type, K, part},
                                            true, s);
}

hipError_t launch_ffn_dh(const uint16_t *dy, const uint16_t *wd, int act, const uint16_t *g,
                         const uint16_t *u, int M, int K, int N, uint16_t *dz, uint16_t *du,
                         uint16_t *h, hipStream_t s) {
    const TileArgs p{{dy}, {wd}, K, K, M, N, K};
    if (act == TW_A_RELU) return ffn_dh<TW_A_RELU>(p, g, u, dz, du, h, s);
    if (act == TW_A_SILU) return ffn_dh<TW_A_SILU>(p, g, u, dz, du, h, s);
    return ffn_dh<TW_A_GELU>(p, g, u, dz, du, h, s);
}

hipError_t launch_ffn_dx(const uint16_t *dz, const uint16_t *du, const uint16_t *wg_t,
                         const uint16_t *wu_t, int M, int K, int N, void *dx, int dx_type,
                         float *part, hipStream_t s) {
    return launch_split<kRows, kCols, 1, 2>(TileArgs{{dz, du}, {wg_t, wu_t}, N, K, M, K, N},
                                            dx_plan(M, K, N), EpiStore{{dx}, dx_type, K, part},
                                            true, s);
}

hipError_t launch_ffn_dw(const uint16_t *dz, const uint16_t *du, const uint16_t *h,
                         const uint16_t *x, int64_t x_stride, const uint16_t *dy, int M, int K,
                         int N, void *dwg_t, void *dwu_t, void *dwd, int dw_type, float *part,
                         hipStream_t s) {
    TileArgs p{{dz, du, h}, {x, x, dy}, N, x_stride, N, K, M};
    p.groups = 3;
    p.ldb_last = K;
    return launch_split<kCols, kCols, 1, 1>(
        p, dw_plan(M, K, N), EpiStore{{dwg_t, dwu_t, dwd}, dw_type, K, part}, true, s);
}

}  // namespace tw
