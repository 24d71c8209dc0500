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
    struct Raw {};
    struct Row {
        __device__ Row(const EpiGlu &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ __forceinline__ Dest dest(int o, int, int) const {
        return {o == 0 ? h : o == 1 ? g : u, TW_T_BF16, N, N, false};
    }
    __device__ __forceinline__ void values(Row &, int, int, f32x4 v, f32x4 w, f32x4 *o) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][e] = activate<ACT>(v[e]) * w[e];
        o[1] = v;
        o[2] = w;
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
    struct Raw {};
    struct Row {
        __device__ Row(const EpiDh &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ __forceinline__ Dest dest(int o, int, int) const {
        return {o == 0 ? dz : o == 1 ? du : h, TW_T_BF16, N, N, false};
    }
    __device__ __forceinline__ void values(Row &, int m, int n, f32x4 v, f32x4, f32x4 *o) const {
        const int64_t at = (int64_t)m * N + min(n, N - 4);
        const f32x4 gv = load4_bf16(g, at), uv = load4_bf16(u, at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Slope a = activate_slope<ACT>(gv[e]);
            o[0][e] = v[e] * uv[e] * a.slope;
            o[1][e] = v[e] * a.value;
            o[2][e] = a.value * uv[e];
        }
    }
};

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

size_t ffn_fwd_part_bytes(int, int, int) { return 0; }
size_t ffn_bwd_part_bytes(int, int, int) { return 0; }

hipError_t launch_ffn_up(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                         const uint16_t *wu_t, int act, int M, int K, int N, uint16_t *g,
                         uint16_t *u, uint16_t *h, float *, hipStream_t s) {
    const TileArgs p{{x}, {wg_t, wu_t}, x_stride, K, M, N, K};
    if (act == TW_A_RELU) return ffn_up<TW_A_RELU>(p, g, u, h, s);
    if (act == TW_A_SILU) return ffn_up<TW_A_SILU>(p, g, u, h, s);
    return ffn_up<TW_A_GELU>(p, g, u, h, s);
}

hipError_t launch_ffn_down(const uint16_t *h, const uint16_t *wd, int M, int K, int N, void *y,
                           int y_type, float *, hipStream_t s) {
    const TileArgs p{{h}, {wd}, N, K, M, K, N};
    return launch_tiles<kRows, kCols, 1, 1>(p, EpiStore{{y}, y_type, nullptr, 0, M, K}, s);
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
                         float *, hipStream_t s) {
    const TileArgs p{{dz, du}, {wg_t, wu_t}, N, K, M, K, N};
    return launch_tiles<kRows, kCols, 1, 2>(p, EpiStore{{dx}, dx_type, nullptr, 0, M, K}, s);
}

hipError_t launch_ffn_dw(const uint16_t *dz, const uint16_t *du, const uint16_t *h,
                         const uint16_t *x, int64_t x_stride, const uint16_t *dy, int M, int K,
                         int N, void *dwg_t, void *dwu_t, void *dwd, int dw_type, float *,
                         hipStream_t s) {
    // W_g and W_u share x; dy, of another stride, is W_d's
    const TileArgs p{{dz, du}, {x, x}, N, x_stride, N, K, M, 1, 2};
    hipError_t e = launch_tiles<kCols, kCols, 1, 1>(
        p, EpiStore{{dwg_t, dwu_t}, dw_type, nullptr, 0, N, K}, s);
    if (e != hipSuccess) return e;
    const TileArgs q{{h}, {dy}, N, K, N, K, M};
    return launch_tiles<kCols, kCols, 1, 1>(q, EpiStore{{dwd}, dw_type, nullptr, 0, N, K}, s);
}

}  // namespace tw
