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
// h, dz and du feed the matrix cores, so they are rounded to bf16 between the products
// (up to 2^-8 of a term, averaged out over the sums they enter); every sum is fp32.  An
// output in bf16 is then off by 0.0023 of its norm, 0.0017 with these values in fp32:
// its own rounding and as much again.
//
// What bounds them (bf16, normal operands, calls in a row): 16384 x 2048 x 8192 forward
// 1254 to 1336 us, 1235 to 1315 TFLOP/s, the chip's power (tw_tiles.hpp); backward 4096 x
// 1024 x 4096 224 to 239 us, of 224 dh 56 (one round of tiles, whose 170 MB of g, u, dz,
// du and h pass only after it: 23 us of products, 36 us of memory), dx 73 (128 tiles,
// each in two parts, and their sum) and the weight gradients 95 (192 whole tiles on 256
// CUs).  One row, 2048 x 5632: 17.5 to 18 us for 69 MB of weights, 3.9 TB/s.  65 to about
// 1000 rows: gate and up and dh take every tile's whole reduction, so few workgroups walk
// a long one (4096 x 1024: 128 rows on 8 and 4 workgroups, 47 and 52 us, as much as 1024
// rows take).
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

// g s(a) with s = s(a(g)): below -128, where s is 0 for every activation here, g is
// taken at -128, so that minus infinity gives the limit and not infinity times 0.  (s of a
// NaN is NaN.)
__device__ __forceinline__ float gated(float g, float s) { return fmaxf(g, -128.0f) * s; }

template <int ACT>
__device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == TW_A_RELU) return g <= 0.0f ? 0.0f : g;  // NaN stays NaN
    else if constexpr (ACT == TW_A_SILU) return gated(g, logistic(g));
    else return gated(g, logistic(kGelu * g * (1.0f + kGelu3 * g * g)));
}

struct Slope {
    float value, slope;
};
template <int ACT>
__device__ __forceinline__ Slope activate_slope(float g) {
    if constexpr (ACT == TW_A_RELU) return {g <= 0.0f ? 0.0f : g, g <= 0.0f ? 0.0f : 1.0f};
    // s (1 + g a' (1 - s)), with g a' taken at a bound past which s is 0 or 1 - s is: 0
    // times an infinity would be NaN.  For SiLU that holds from |g| = 128 on; GELU's g a'
    // grows as g^3, but its s is 0 or 1 long before |g| = 16.
    const bool silu = ACT == TW_A_SILU;
    const float most = silu ? 128.0f : 16.0f;
    const float s = logistic(silu ? g : kGelu * g * (1.0f + kGelu3 * g * g));
    const float c = fminf(fmaxf(g, -most), most);
    const float d = silu ? c : kGelu * c * (1.0f + 3.0f * kGelu3 * c * c);
    return {gated(g, s), s * fmaf(d, 1.0f - s, 1.0f)};
}

// Gate and up projections -> h (and g, u).
template <int ACT>
struct EpiGlu {
    static constexpr bool kStats = false;
    static constexpr int kWalk = 4;
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
    typedef NoFetch Fetched;
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &, const Fetched &, int, const float (&v)[W],
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
    static constexpr int kWalk = 4;
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
    struct Fetched {
        u32x4 g, u;
    };
    __device__ __forceinline__ Fetched fetch(int m, int n) const {
        const int64_t at = (int64_t)m * N + n;
        return {ld16(g + at), ld16(u + at)};
    }
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &, const Fetched &f, int, const float (&v)[W],
                                           const float (&)[W], float (&o)[kOuts][W]) const {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const uint32_t gp = f.g[e >> 1], up = f.u[e >> 1];
            const float uv = e & 1 ? bf_hi(up) : bf_lo(up);
            const Slope a = activate_slope<ACT>(e & 1 ? bf_hi(gp) : bf_lo(gp));
            o[0][e] = v[e] * uv * a.slope;
            o[1][e] = v[e] * a.value;
            o[2][e] = a.value * uv;
        }
    }
};

// Up to 64 token rows (16 MB): a workgroup takes up to 16 C hidden neurons of NM
// matrices, its 8 waves a slice of K each; their sums meet in LDS.  Bound by the stream
// of weights.  Measured (us, these kernels and tiles): gate and up, 1 row 1024 x 4096
// 7.6, 17.8, 64 rows 11.9, 18.1; 64 rows 2048 x 5632 20, 28; dh of 64 rows 21, 35.  The
// limit of 64 is not where tiles begin to win but what the waves' sums leave of the LDS
// (128 KB): by kernel, 64 and 65 rows of 2048 x 5632 take 17, 26 (gate and up) and 18, 31
// (dh), of 4096 x 1024 21, 45 and 20, 50.
template <int ACT>
struct FewUp {
    static constexpr int NM = 2;
    uint16_t *g, *u, *h;
    __device__ __forceinline__ void put(int64_t at, float v, float w) const {
        h[at] = (uint16_t)pack_bf16(activate<ACT>(v) * w, 0.0f);
        if (g) g[at] = (uint16_t)pack_bf16(v, 0.0f);
        if (u) u[at] = (uint16_t)pack_bf16(w, 0.0f);
    }
};
template <int ACT>
struct FewDh {
    static constexpr int NM = 1;
    const uint16_t *g, *u;
    uint16_t *dz, *du, *h;
    __device__ __forceinline__ void put(int64_t at, float v, float) const {
        const Slope a = activate_slope<ACT>(bf_lo((uint32_t)g[at]));
        const float uv = bf_lo((uint32_t)u[at]);
        dz[at] = (uint16_t)pack_bf16(v * uv * a.slope, 0.0f);
        du[at] = (uint16_t)pack_bf16(v * a.value, 0.0f);
        h[at] = (uint16_t)pack_bf16(a.value * uv, 0.0f);
    }
};

constexpr int kFewThreads = 512;
template <int C, int MB, class Put>
__global__ __launch_bounds__(kFewThreads) void few_hidden_kernel(
    const uint16_t *__restrict__ x, int64_t x_stride, const uint16_t *__restrict__ w0,
    const uint16_t *__restrict__ w1, int M, int K, int N, int share, Put put) {
    constexpr int NW = kFewThreads / kWave, NM = Put::NM;
    extern __shared__ __attribute__((aligned(16))) char smem[];  // [NW][NM C MB][64] f32x4
    f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * share, n1 = min(n0 + share, N);
    const int k8 = 8 * (lane >> 4);
    const uint16_t *wp[NM * C], *xp[MB];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t row = min(n0 + 16 * c + (lane & 15), n1 - 1);
        wp[NM * c] = w0 + row * K + k8;
        if constexpr (NM == 2) wp[2 * c + 1] = w1 + row * K + k8;
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) xp[m] = x + min(16 * m + (lane & 15), M - 1) * x_stride + k8;
    const int steps = (K + 31) / 32, per = (steps + NW - 1) / NW;
    f32x4 acc[NM * C][MB] = {};
    // Steps in a batch of loads: few, as 8 waves have one each on its way (2 x 1024 x 4096:
    // 7.6 us with 6 loads in a batch, 8.8 with 10, 8.6 with 20).
    constexpr int U = 6 / (NM * C + MB) < 1 ? 1 : 6 / (NM * C + MB);
    few_product<NM * C, MB, U>(wp, xp, K, wave * per, min(wave * per + per, steps), acc);
#pragma unroll
    for (int b = 0; b < NM * C; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            sums[((wave * NM * C + b) * MB + m) * kWave + lane] = acc[b][m];
    __syncthreads();
    for (int i = wave; i < C * MB; i += NW) {  // block i / MB of neurons, i % MB of rows
        f32x4 s[2] = {};
#pragma unroll
        for (int q = 0; q < NW; ++q)
#pragma unroll
            for (int o = 0; o < NM; ++o)
                s[o] += sums[((q * NM * C + NM * (i / MB) + o) * MB + i % MB) * kWave + lane];
        const int m = 16 * (i % MB) + (lane & 15);
        if (m >= M) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + 16 * (i / MB) + 4 * (lane >> 4) + e;
            if (n < n1) put.put((int64_t)m * N + n, s[0][e], s[1][e]);
        }
    }
}

template <int C, int MB, class Put>
hipError_t few_hidden_as(const uint16_t *x, int64_t x_stride, const uint16_t *w0,
                         const uint16_t *w1, int M, int K, int N, int share, const Put &put,
                         hipStream_t s) {
    constexpr auto kernel = &few_hidden_kernel<C, MB, Put>;
    constexpr int lds = kFewThreads / kWave * Put::NM * C * MB * kWave * 16;
    const hipError_t e = lds_limit_once<kernel>(lds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)((N + share - 1) / share), kFewThreads, lds, s>>>(x, x_stride, w0, w1, M, K,
                                                                        N, share, put);
    return hipGetLastError();
}

template <class Put>
hipError_t few_hidden(const uint16_t *x, int64_t x_stride, const uint16_t *w0, const uint16_t *w1,
                      int M, int K, int N, const Put &put, hipStream_t s) {
    // An even share of the neurons for each of 256 workgroups, at most 32.  (512: 1024 x
    // 4096 10.0 us for 8.8; 16 at most: 2048 x 5632 16.1 for 12.8.)
    int share = (N + 255) / 256;
    share = share < 4 ? 4 : share > 32 ? 32 : share;
    auto go = [&](auto c, auto mb) {
        return few_hidden_as<decltype(c)::value, decltype(mb)::value>(x, x_stride, w0, w1, M, K, N,
                                                                      share, put, s);
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
    if (p.M <= kFewRowsMax)
        return few_hidden(p.a[0], p.lda, p.b[0], p.b[1], p.M, p.R, p.N, FewUp<ACT>{g, u, h}, s);
    return launch_tiles<kRows, kRows, 2, 1>(p, EpiGlu<ACT>{h, g, u, p.N}, s);
}
template <int ACT>
hipError_t ffn_dh(const TileArgs &p, const uint16_t *g, const uint16_t *u, uint16_t *dz,
                  uint16_t *du, uint16_t *h, hipStream_t s) {
    if (p.M <= kFewRowsMax)
        return few_hidden(p.a[0], p.lda, p.b[0], p.b[0], p.M, p.R, p.N,
                          FewDh<ACT>{g, u, dz, du, h}, s);
    return launch_tiles<kRows, kRows, 1, 1>(p, EpiDh<ACT>{g, u, dz, du, h, p.N}, s);
}

}  // namespace

static SplitPlan down_plan(int M, int K, int N) {
    return split_plan<1>(TileArgs{{}, {}, N, K, M, K, N}, false);
}
static SplitPlan dx_plan(int M, int K, int N) {
    return split_plan<2>(TileArgs{{}, {}, N, K, M, K, N}, false);
}
static SplitPlan dw_plan(int M, int K, int N) {
    TileArgs p{{}, {}, N, K, N, K, M};
    p.groups = 3;
    return split_plan<1>(p, false);
}

size_t ffn_fwd_part_bytes(int M, int K, int N) {
    if (M <= kFewDownMax) return (size_t)few_down_split(1, M, K, N).splits * M * K * 4;
    return down_plan(M, K, N).bytes;
}
size_t ffn_bwd_part_bytes(int M, int K, int N) {
    const size_t a = M <= kFewDownMax ? (size_t)2 * few_down_split(2, M, K, N).splits * M * K * 4
                                      : dx_plan(M, K, N).bytes;
    const size_t b = dw_plan(M, K, N).bytes;
    return a > b ? a : b;
}

hipError_t launch_ffn_up(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                         const uint16_t *wu_t, int act, int M, int K, int N, uint16_t *g,
                         uint16_t *u, uint16_t *h, hipStream_t s) {
    const TileArgs p{{x}, {wg_t, wu_t}, x_stride, K, M, N, K};
    if (act == TW_A_RELU) return ffn_up<TW_A_RELU>(p, g, u, h, s);
    if (act == TW_A_SILU) return ffn_up<TW_A_SILU>(p, g, u, h, s);
    return ffn_up<TW_A_GELU>(p, g, u, h, s);
}

hipError_t launch_ffn_down(const uint16_t *h, const uint16_t *wd, int M, int K, int N, void *y,
                           int y_type, float *part, hipStream_t s) {
    if (M <= kFewDownMax) {
        return few_down({h, nullptr}, {wd, nullptr}, 1, N, M, K, N, part, y, y_type, s);
    }
    return launch_split<kRows, kCols, 1>(TileArgs{{h}, {wd}, N, K, M, K, N},
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
    if (M <= kFewDownMax)
        return few_down({dz, du}, {wg_t, wu_t}, 2, N, M, K, N, part, dx, dx_type, s);
    return launch_split<kRows, kCols, 2>(TileArgs{{dz, du}, {wg_t, wu_t}, N, K, M, K, N},
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
    return launch_split<kCols, kCols, 1>(
        p, dw_plan(M, K, N), EpiStore{{dwg_t, dwu_t, dwd}, dw_type, K, part}, true, s);
}

}  // namespace tw
