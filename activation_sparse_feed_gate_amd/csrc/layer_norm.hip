// layer_norm.hip -- the layer norm of a pre-norm block over token rows, with
// the residual addition in front of it and the int8 quantisation behind it,
// and its gradient.
//
// Forward, a row z = x (+ add) of K elements:
//   mean = sum(z) / K,  d = z - mean,  rstd = 1 / sqrt(sum(d^2) / K + eps),
//   y = d rstd gamma (+ beta).
// The row stays in registers between its steps, so memory is read once and
// the variance is the sum over centred values (no cancellation for rows far
// from zero).  Everything is fp32 until the one rounding of each output; the
// stored sum z is rounded to x's type after it was used.
//
// Backward, with n = (z - mean) rstd and t = dy gamma:
//   dx = rstd (t - sum(t) / K - n sum(t n) / K) (+ dres),
//   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy.
// Each wave (or workgroup) walks rows and keeps its share of dgamma and dbeta
// in registers; the workgroups' shares go to the workspace and a second
// kernel adds them in a fixed order (no atomics: results do not depend on
// timing).
#include "tw_rows.hpp"

namespace tw {
namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
    const char *x, *add;
    int64_t x_stride;  // elements between rows of x (add is contiguous)
    const float *gamma, *beta;
    float eps;
    int M, K;
    char *sum, *y;  // sum in x's type, or null
    int y_type;
    float *mean, *rstd;  // or null
    int8_t *q;
    float *scale;
};

// What becomes of a row: its norm, the norm quantised to int8, or the row
// itself quantised.
enum { kNorm = 0, kNormQuant = 1, kQuant = 2 };

// TPR threads hold a row, VPT vectors of 8 elements each (vector v of thread
// t starts at element 8 (v TPR + t): every load of a wave is contiguous).
template <int TX, int TA, int MODE, int TPR, int VPT>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) void norm_rows_kernel(
    NormArgs a) {
    constexpr int RPB = TPR >= kNormThreads ? 1 : kNormThreads / TPR;  // rows per workgroup
    __shared__ float red[2 * (TPR / kWave)];
    RowReduce<TPR> rr(red);
    const int t = threadIdx.x % TPR;
    // no barrier when a row is one wave, so waves may leave at different rows
    for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < a.M;
         m += (int64_t)gridDim.x * RPB) {
        const char *xr = a.x + m * a.x_stride * type_bytes(TX);
        Vec8<TX> xv[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) xv[v] = load8<TX>(xr, 8 * (v * TPR + t), a.K);
        float z[VPT][8];
        if constexpr (TA >= 0) {
            const char *ar = a.add + m * a.K * type_bytes(TA);
            Vec8<TA> av[VPT];
#pragma unroll
            for (int v = 0; v < VPT; ++v) av[v] = load8<TA>(ar, 8 * (v * TPR + t), a.K);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float f[8];
                unpack8<TX>(xv[v], z[v]);
                unpack8<TA>(av[v], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[v][i] += f[i];
            }
            if (a.sum) {
#pragma unroll
                for (int v = 0; v < VPT; ++v)
                    store8<TX>(a.sum + m * a.K * type_bytes(TX), 8 * (v * TPR + t), a.K, z[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v) unpack8<TX>(xv[v], z[v]);
        }

        if constexpr (MODE != kQuant) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += z[v][i];  // zeros past the end
            const float mean = rr.sum(s) / a.K;
            s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[v][i] = 8 * (v * TPR + t) + i < a.K ? z[v][i] - mean : 0.0f;
                    s += z[v][i] * z[v][i];
                }
            const float rstd = 1.0f / sqrtf(rr.sum(s) / a.K + a.eps);
            if (t == 0) {
                if (a.mean) a.mean[m] = mean;
                if (a.rstd) a.rstd[m] = rstd;
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int e = 8 * (v * TPR + t);
                float g[8], b[8];
                unpack8<TW_T_F32>(load8<TW_T_F32>((const char *)a.gamma, e, a.K), g);
                if (a.beta) unpack8<TW_T_F32>(load8<TW_T_F32>((const char *)a.beta, e, a.K), b);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[v][i] = z[v][i] * rstd * g[i] + (a.beta ? b[i] : 0.0f);
            }
        }
        if constexpr (MODE == kNorm) {
            char *yr = a.y + m * a.K * (a.y_type == TW_T_F32 ? 4 : 2);
#pragma unroll
            for (int v = 0; v < VPT; ++v) store8_as(a.y_type, yr, 8 * (v * TPR + t), a.K, z[v]);
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(z[v][i]) & 0x7fffffffu);
            const RowScale rs = row_scale(rr.max_u32(top));
            if (t == 0) a.scale[m] = rs.scale;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                store_q8(a.q + m * a.K, 8 * (v * TPR + t), a.K, quant8(z[v], rs.inv));
        }
    }
}

template <int TX, int TA, int MODE>
hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
    // Rows of up to 4096 elements are one wave's (4 rows per workgroup, no
    // barrier); longer ones a workgroup's.
    auto go = [&](auto kernel, int tpr) {
        const int rpb = tpr >= kNormThreads ? 1 : kNormThreads / tpr;
        const int64_t blocks = ((int64_t)a.M + rpb - 1) / rpb;
        kernel<<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)),
                 tpr > kNormThreads ? tpr : kNormThreads, 0, s>>>(a);
        return hipGetLastError();
    };
    if (a.M == 0) return hipSuccess;
    if (a.K <= 512) return go(norm_rows_kernel<TX, TA, MODE, 64, 1>, 64);
    if (a.K <= 1024) return go(norm_rows_kernel<TX, TA, MODE, 64, 2>, 64);
    if (a.K <= 2048) return go(norm_rows_kernel<TX, TA, MODE, 64, 4>, 64);
    if (a.K <= 4096) return go(norm_rows_kernel<TX, TA, MODE, 64, 8>, 64);
    if (a.K <= 16384) return go(norm_rows_kernel<TX, TA, MODE, 256, 8>, 256);
    return go(norm_rows_kernel<TX, TA, MODE, 1024, 8>, 1024);
}

template <int MODE>
hipError_t launch_norm(const NormArgs &a, int x_type, int add_type, hipStream_t s) {
    if (x_type == TW_T_F32) {
        if (!a.add) return launch_rows<TW_T_F32, -1, MODE>(a, s);
        if (add_type == TW_T_F32) return launch_rows<TW_T_F32, TW_T_F32, MODE>(a, s);
        return launch_rows<TW_T_F32, TW_T_BF16, MODE>(a, s);
    }
    if (!a.add) return launch_rows<TW_T_BF16, -1, MODE>(a, s);
    if (add_type == TW_T_F32) return launch_rows<TW_T_BF16, TW_T_F32, MODE>(a, s);
    return launch_rows<TW_T_BF16, TW_T_BF16, MODE>(a, s);
}

// --------------------------------- backward --------------------------------
struct NormBwdArgs {
    const char *dy, *x, *dres;  // dres: dx's type, or null
    int64_t x_stride;
    const float *gamma, *mean, *rstd;
    int M, K;
    char *dx;
    int dx_type;
    float *part;  // [gridDim.x][2][K] shares of dgamma and dbeta, or null
};

template <int TD, int TX, int TPR, int VPT>
__global__ __launch_bounds__(kNormThreads) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int RPB = kNormThreads / TPR;
    extern __shared__ __attribute__((aligned(16))) float share[];  // 2 K floats (TPR == 64)
    __shared__ float red[2 * (TPR / kWave)];
    RowReduce<TPR> rr(red);
    const int t = threadIdx.x % TPR;
    float dg[VPT][8], db[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] = db[v][i] = 0.0f;

    for (int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; m < a.M;
         m += (int64_t)gridDim.x * RPB) {
        const char *dr = a.dy + m * a.K * type_bytes(TD);
        const char *xr = a.x + m * a.x_stride * type_bytes(TX);
        Vec8<TD> dv[VPT];
        Vec8<TX> xv[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) dv[v] = load8<TD>(dr, 8 * (v * TPR + t), a.K);
#pragma unroll
        for (int v = 0; v < VPT; ++v) xv[v] = load8<TX>(xr, 8 * (v * TPR + t), a.K);
        const float mean = a.mean[m], rstd = a.rstd[m];
        float n[VPT][8], g[VPT][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = 8 * (v * TPR + t);
            float gm[8];
            unpack8<TW_T_F32>(load8<TW_T_F32>((const char *)a.gamma, e, a.K), gm);
            unpack8<TD>(dv[v], g[v]);
            unpack8<TX>(xv[v], n[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // past the end dy = gamma = 0: only n has to be cleared (it
                // may be infinite where mean is)
                n[v][i] = e + i < a.K ? (n[v][i] - mean) * rstd : 0.0f;
                dg[v][i] += g[v][i] * n[v][i];
                db[v][i] += g[v][i];
                g[v][i] *= gm[i];
                s1 += g[v][i];
                s2 += g[v][i] * n[v][i];
            }
        }
        const float c1 = rr.sum(s1) / a.K, c2 = rr.sum(s2) / a.K;
        const int ds = a.dx_type == TW_T_F32 ? 4 : 2;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int e = 8 * (v * TPR + t);
            float r[8];
            if (a.dres) {
                const char *rrow = a.dres + m * a.K * ds;
                if (a.dx_type == TW_T_F32) unpack8<TW_T_F32>(load8<TW_T_F32>(rrow, e, a.K), r);
                else unpack8<TW_T_BF16>(load8<TW_T_BF16>(rrow, e, a.K), r);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[v][i] = rstd * (g[v][i] - c1 - n[v][i] * c2) + (a.dres ? r[i] : 0.0f);
            store8_as(a.dx_type, a.dx + m * a.K * ds, e, a.K, g[v]);
        }
    }
    if (!a.part) return;

    // the workgroup's share: its waves add theirs in wave order
    float *pg = a.part + (size_t)blockIdx.x * 2 * a.K, *pb = pg + a.K;
    if constexpr (TPR == kWave) {
        const int wave = threadIdx.x / kWave;
        for (int w = 0; w < RPB; ++w) {
            if (wave == w) {
#pragma unroll
                for (int v = 0; v < VPT; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = 8 * (v * TPR + t) + i;
                        if (e >= a.K) continue;
                        share[e] = w ? share[e] + dg[v][i] : dg[v][i];
                        share[a.K + e] = w ? share[a.K + e] + db[v][i] : db[v][i];
                    }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < 2 * a.K; e += kNormThreads) pg[e] = share[e];
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            store8<TW_T_F32>((char *)pg, 8 * (v * TPR + t), a.K, dg[v]);
            store8<TW_T_F32>((char *)pb, 8 * (v * TPR + t), a.K, db[v]);
        }
    }
}

// dgamma and dbeta from the workgroups' shares: 32 columns a workgroup, 32
// threads a column, each adding every 32nd share; then their sums in order.
constexpr int kColsPerBlock = 32, kColThreads = 32;
__global__ __launch_bounds__(kColsPerBlock *kColThreads) void norm_cols_kernel(
    const float *__restrict__ part, int G, int K, float *__restrict__ dgamma,
    float *__restrict__ dbeta) {
    __shared__ float s[kColThreads][kColsPerBlock + 1];
    const int c = threadIdx.x % kColsPerBlock, r = threadIdx.x / kColsPerBlock;
    const int64_t col = (int64_t)blockIdx.x * kColsPerBlock + c;
    float v = 0.0f;
    if (col < 2 * (int64_t)K)
#pragma unroll 4
        for (int g = r; g < G; g += kColThreads) v += part[(size_t)g * 2 * K + col];
    s[r][c] = v;
    __syncthreads();
    if (r == 0 && col < 2 * (int64_t)K) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kColThreads; ++i) v += s[i][c];
        float *out = col < K ? dgamma : dbeta;
        if (out) out[col < K ? col : col - K] = v;
    }
}

template <int TD, int TX>
hipError_t launch_bwd(const NormBwdArgs &a, int grid, hipStream_t s) {
    const size_t lds = a.part && a.K <= 2048 ? (size_t)a.K * 8 : 0;
    auto go = [&](auto kernel) {
        kernel<<<grid, kNormThreads, lds, s>>>(a);
        return hipGetLastError();
    };
    if (a.K <= 512) return go(norm_bwd_kernel<TD, TX, 64, 1>);
    if (a.K <= 1024) return go(norm_bwd_kernel<TD, TX, 64, 2>);
    if (a.K <= 2048) return go(norm_bwd_kernel<TD, TX, 64, 4>);
    if (a.K <= 4096) return go(norm_bwd_kernel<TD, TX, 256, 2>);
    if (a.K <= 8192) return go(norm_bwd_kernel<TD, TX, 256, 4>);
    return go(norm_bwd_kernel<TD, TX, 256, 8>);
}

}  // namespace

hipError_t launch_layernorm(const void *x, int x_type, int64_t x_stride, const void *add,
                            int add_type, const float *gamma, const float *beta, float eps, int M,
                            int K, void *sum, void *y, int y_type, float *mean, float *rstd,
                            hipStream_t s) {
    NormArgs a{(const char *)x, (const char *)add, x_stride, gamma, beta, eps, M, K,
               (char *)sum, (char *)y, y_type, mean, rstd, nullptr, nullptr};
    return launch_norm<kNorm>(a, x_type, add_type, s);
}

hipError_t launch_layernorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                                  int add_type, const float *gamma, const float *beta, float eps,
                                  int M, int K, void *sum, int8_t *q, float *scale,
                                  hipStream_t s) {
    NormArgs a{(const char *)x, (const char *)add, x_stride, gamma, beta, eps, M, K,
               (char *)sum, nullptr, 0, nullptr, nullptr, q, scale};
    return launch_norm<kNormQuant>(a, x_type, add_type, s);
}

hipError_t launch_quant_rows(const void *x, int x_type, int64_t x_stride, int M, int K, int8_t *q,
                             float *scale, hipStream_t s) {
    NormArgs a{(const char *)x, nullptr, x_stride, nullptr, nullptr, 0.0f, M, K,
               nullptr, nullptr, 0, nullptr, nullptr, q, scale};
    if (x_type == TW_T_F32) return launch_rows<TW_T_F32, -1, kQuant>(a, s);
    return launch_rows<TW_T_BF16, -1, kQuant>(a, s);
}

int layernorm_bwd_groups(int M, int K) {
    const int rpb = K <= 2048 ? kNormThreads / kWave : 1;
    const int64_t need = ((int64_t)M + rpb - 1) / rpb;
    return (int)(need < 1 ? 1 : need < 512 ? need : 512);
}

hipError_t launch_layernorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                                int64_t x_stride, const float *gamma, const float *mean,
                                const float *rstd, const void *dres, int M, int K, void *dx,
                                int dx_type, float *dgamma, float *dbeta, float *part,
                                hipStream_t s, hipEvent_t ev_rows) {
    const int grid = layernorm_bwd_groups(M, K);
    NormBwdArgs a{(const char *)dy, (const char *)x, (const char *)dres, x_stride, gamma, mean,
                  rstd, M, K, (char *)dx, dx_type, dgamma || dbeta ? part : nullptr};
    hipError_t e = hipSuccess;
    if (M > 0 || a.part)
        e = dy_type == TW_T_F32
                ? (x_type == TW_T_F32 ? launch_bwd<TW_T_F32, TW_T_F32>(a, grid, s)
                                      : launch_bwd<TW_T_F32, TW_T_BF16>(a, grid, s))
                : (x_type == TW_T_F32 ? launch_bwd<TW_T_BF16, TW_T_F32>(a, grid, s)
                                      : launch_bwd<TW_T_BF16, TW_T_BF16>(a, grid, s));
    if (e == hipSuccess && ev_rows) e = hipEventRecord(ev_rows, s);
    if (e != hipSuccess || !a.part) return e;
    const int blocks = (2 * K + kColsPerBlock - 1) / kColsPerBlock;
    norm_cols_kernel<<<blocks, kColsPerBlock * kColThreads, 0, s>>>(part, grid, K, dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace tw
