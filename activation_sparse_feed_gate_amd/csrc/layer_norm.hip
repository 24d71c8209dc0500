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
#include <type_traits>

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
// WHOLE: K is a multiple of 8, and the loads need no branch (4096 x 1024 bf16
// 5.1 us against 5.8).  A
// workgroup walks rows with gamma and beta in registers (read per row from
// the L2 they would cost as much as the row) and the next row's loads in
// flight.  Memory bounds it: 16384 x 2048 fp32 with add takes 88 us (5.3
// TB/s, the rate of a copy), 16384 x 4096 bf16 with add 105, 8192 x 8192 bf16
// 51.
template <int TX, int TA, int MODE, int TPR, int VPT, bool WHOLE>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) void norm_rows_kernel(
    NormArgs a) {
    constexpr int RPB = TPR >= kNormThreads ? 1 : kNormThreads / TPR;  // rows per workgroup
    constexpr bool kNorms = MODE != kQuant, kAdds = TA >= 0;
    constexpr bool kAhead = VPT <= 4;  // registers for the next row
    __shared__ float red[2 * (TPR / kWave)];
    RowReduce<TPR> rr(red);
    const int t = threadIdx.x % TPR;
    auto at = [&](int v) { return 8 * (v * TPR + t); };
    float gamma[kNorms ? VPT : 1][8], beta[kNorms ? VPT : 1][8];
    if constexpr (kNorms) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack8<TW_T_F32>(load8_of<WHOLE, TW_T_F32>((const char *)a.gamma, at(v), a.K),
                              gamma[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) beta[v][i] = 0.0f;
            // none past the end, where z stays 0 and the row's maximum must not
            // see another vector's
            if (a.beta && (!WHOLE || at(v) < a.K))
                unpack8<TW_T_F32>(load8_of<WHOLE, TW_T_F32>((const char *)a.beta, at(v), a.K),
                                  beta[v]);
        }
    }
    Vec8<TX> xv[VPT];
    Vec8<kAdds ? TA : TX> av[kAdds ? VPT : 1];
    auto fetch = [&](int64_t m) {
        const char *xr = a.x + m * a.x_stride * type_bytes(TX);
#pragma unroll
        for (int v = 0; v < VPT; ++v) xv[v] = load8_of<WHOLE, TX>(xr, at(v), a.K);
        if constexpr (kAdds) {
            const char *ar = a.add + m * a.K * type_bytes(TA);
#pragma unroll
            for (int v = 0; v < VPT; ++v) av[v] = load8_of<WHOLE, TA>(ar, at(v), a.K);
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (kAhead && m < a.M) fetch(m);
    // no barrier when a row is one wave, so waves may leave at different rows
    for (; m < a.M; m += step) {
        if (!kAhead) fetch(m);
        float z[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack8<TX>(xv[v], z[v]);
            if constexpr (kAdds) {
                float f[8];
                unpack8<TA>(av[v], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[v][i] += f[i];
            }
            if (WHOLE && at(v) >= a.K) {  // the others read zeros past the end
#pragma unroll
                for (int i = 0; i < 8; ++i) z[v][i] = 0.0f;
            }
        }
        // a stored sum may be x or add itself: every element is read here by
        // the thread that writes it, and the next row's are other elements
        if (kAhead && m + step < a.M) fetch(m + step);
        if constexpr (kAdds) {
            if (a.sum) {
#pragma unroll
                for (int v = 0; v < VPT; ++v)
                    store8<TX>(a.sum + m * a.K * type_bytes(TX), at(v), a.K, z[v]);
            }
        }
        if constexpr (kNorms) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += z[v][i];  // zeros past the end
            const float mean = rr.sum(s) / a.K;
            s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (at(v) + 8 <= a.K) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[v][i] -= mean;
                } else {  // past the end stays zero
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[v][i] = at(v) + i < a.K ? z[v][i] - mean : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) s += z[v][i] * z[v][i];
            }
            const float rstd = 1.0f / sqrtf(rr.sum(s) / a.K + a.eps);
            if (t == 0) {
                if (a.mean) a.mean[m] = mean;
                if (a.rstd) a.rstd[m] = rstd;
            }
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[v][i] = z[v][i] * rstd * gamma[v][i] + beta[v][i];
        }
        if constexpr (MODE == kNorm) {
            char *yr = a.y + m * a.K * (a.y_type == TW_T_F32 ? 4 : 2);
#pragma unroll
            for (int v = 0; v < VPT; ++v) store8_as(a.y_type, yr, at(v), a.K, z[v]);
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(z[v][i]) & 0x7fffffffu);
            const RowScale rs = row_scale(rr.max_u32(top));
            if (t == 0) a.scale[m] = rs.scale;
#pragma unroll
            for (int v = 0; v < VPT; ++v) store_q8(a.q + m * a.K, at(v), a.K, quant8(z[v], rs.inv));
        }
    }
}

template <int TX, int TA, int MODE, int TPR, int VPT>
hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
    constexpr int threads = TPR > kNormThreads ? TPR : kNormThreads;
    constexpr int rpb = threads / TPR;
    const int64_t need = ((int64_t)a.M + rpb - 1) / rpb;
    // Norms: the workgroups the chip holds at once (2048 threads a CU, 1024
    // with the registers an add takes), so that gamma is read once per
    // workgroup; the quantiser has nothing to keep and takes a row each.
    // Measured (us at 1024, 2048, no limit): 8192 x 8192 bf16 51, 51, 66; 16384 x
    // 2048 bf16 30, 28, 35, fp32 with add 88, 92, 88; int8 16384 x 8192 71, 75, 70.
    const int64_t most = MODE == kQuant ? 1 << 20 : 256 * (TA >= 0 ? 1024 : 2048) / threads;
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (a.K % 8 == 0) norm_rows_kernel<TX, TA, MODE, TPR, VPT, true><<<grid, threads, 0, s>>>(a);
    else norm_rows_kernel<TX, TA, MODE, TPR, VPT, false><<<grid, threads, 0, s>>>(a);
    return hipGetLastError();
}

// A wave a row up to 1024 elements, then a workgroup a row of as few vectors
// a thread as its 256 to 1024 threads allow.  Measured (us): 16384 x 2048 fp32
// with add, a workgroup of 256 a row 88, a wave a row 98; 8 rows of 2048, 2.9
// and 4.3; 4096 x 1024 bf16, a wave a row 5.6, a workgroup 8.1.
template <int TX, int TA, int MODE>
hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
    if (a.M == 0) return hipSuccess;
    if (a.K <= 512) return launch_rows<TX, TA, MODE, 64, 1>(a, s);
    if (a.K <= 1024) return launch_rows<TX, TA, MODE, 64, 2>(a, s);
    if (a.K <= 2048) return launch_rows<TX, TA, MODE, 256, 1>(a, s);
    if (a.K <= 4096) return launch_rows<TX, TA, MODE, 256, 2>(a, s);
    if (a.K <= 8192) return launch_rows<TX, TA, MODE, 512, 2>(a, s);
    if constexpr (MODE == kQuant)
        if (a.K > kNormMaxK) return launch_rows<TX, TA, MODE, 1024, 8>(a, s);
    return launch_rows<TX, TA, MODE, 1024, 2>(a, s);
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
    float *part;  // [gridDim.x][2][KP] shares of dgamma and dbeta, or null
};

// Columns of a share: K rounded up to what the threads of a row hold, so that
// shares are stored and summed without regard to where K ends.
// Measured: a wave a row up to K = 1024 (16384 x 1024 bf16: 35 us); at 2048 a
// workgroup a row takes 103 us for 16384 fp32 rows with dres (5.2 TB/s), a
// wave a row 150 (its registers hold too little besides the sums).
constexpr int norm_bwd_tpr(int K) { return K <= 1024 ? 64 : K <= 4096 ? 256 : 512; }
constexpr int norm_bwd_vpt(int K) {
    return K <= 512 ? 1 : K <= 1024 ? 2 : K <= 2048 ? 1 : K <= 8192 ? 2 : 4;
}
constexpr int norm_bwd_threads(int K) {
    return norm_bwd_tpr(K) > kNormThreads ? norm_bwd_tpr(K) : kNormThreads;
}
constexpr int norm_bwd_cols(int K) { return norm_bwd_tpr(K) * norm_bwd_vpt(K) * 8; }

// The next row's loads are issued before this row is reduced, since the column
// sums leave room for few waves, too few to hide the loads behind each other
// (rows of more than 8192 elements fill the registers without).  They are not
// in flight over the reductions, though: gamma, read anew for every row behind
// them, waits for them too, as loads complete in order.  Up to K = 1024, where a
// wave walks few rows, that latency bounds the kernel (4096 x 1024, fp32 dy: 12
// us for 42 MB); from 2048 on it runs at the rate of a copy.
template <int TD, int TX, int TPR, int VPT>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads, 2)
void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int RPB = TPR > kNormThreads ? 1 : kNormThreads / TPR;
    constexpr int KP = TPR * VPT * 8;
    constexpr bool kAhead = VPT < 4;
    extern __shared__ __attribute__((aligned(16))) float share[];  // [RPB][2][KP] (TPR == 64)
    __shared__ float red[2 * (TPR / kWave)];
    RowReduce<TPR> rr(red);
    const int t = threadIdx.x % TPR;
    float dg[VPT][8], db[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[v][i] = db[v][i] = 0.0f;

    Vec8<TD> dv[VPT];
    Vec8<TX> xv[VPT];
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](int64_t m) {
        const char *dr = a.dy + m * a.K * type_bytes(TD);
        const char *xr = a.x + m * a.x_stride * type_bytes(TX);
        mean = a.mean[m];
        rstd = a.rstd[m];
#pragma unroll
        for (int v = 0; v < VPT; ++v) dv[v] = load8<TD>(dr, 8 * (v * TPR + t), a.K);
#pragma unroll
        for (int v = 0; v < VPT; ++v) xv[v] = load8<TX>(xr, 8 * (v * TPR + t), a.K);
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t m = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (kAhead && m < a.M) fetch(m);
    for (; m < a.M; m += step) {
        if (!kAhead) fetch(m);
        const float r = rstd;
        float n[VPT][8], g[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            unpack8<TD>(dv[v], g[v]);
            unpack8<TX>(xv[v], n[v]);
            const int left = a.K - 8 * (v * TPR + t);
            if (left >= 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) n[v][i] = (n[v][i] - mean) * r;
            } else {  // past the end zero: -mean r may be infinite, and 0 inf is NaN
#pragma unroll
                for (int i = 0; i < 8; ++i) n[v][i] = i < left ? (n[v][i] - mean) * r : 0.0f;
            }
        }
        if (kAhead && m + step < a.M) fetch(m + step);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float gm[8];
            unpack8<TW_T_F32>(load8<TW_T_F32>((const char *)a.gamma, 8 * (v * TPR + t), a.K), gm);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
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
            float d[8];
            if (a.dres) {
                const char *rrow = a.dres + m * a.K * ds;
                if (a.dx_type == TW_T_F32) unpack8<TW_T_F32>(load8<TW_T_F32>(rrow, e, a.K), d);
                else unpack8<TW_T_BF16>(load8<TW_T_BF16>(rrow, e, a.K), d);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[v][i] = r * (g[v][i] - c1 - n[v][i] * c2) + (a.dres ? d[i] : 0.0f);
            store8_as(a.dx_type, a.dx + m * a.K * ds, e, a.K, g[v]);
        }
    }
    if (!a.part) return;

    // the workgroup's share: its waves' column sums, added in wave order
    float *pg = a.part + (size_t)blockIdx.x * 2 * KP;
    if constexpr (TPR == kWave) {
        float *mine = share + (threadIdx.x / kWave) * 2 * KP;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            store8<TW_T_F32>((char *)mine, 8 * (v * TPR + t), KP, dg[v]);
            store8<TW_T_F32>((char *)(mine + KP), 8 * (v * TPR + t), KP, db[v]);
        }
        __syncthreads();
        for (int e = 4 * threadIdx.x; e < 2 * KP; e += 4 * kNormThreads) {
            f32x4 s = *reinterpret_cast<const f32x4 *>(share + e);
#pragma unroll
            for (int w = 1; w < RPB; ++w)
                s += *reinterpret_cast<const f32x4 *>(share + w * 2 * KP + e);
            *reinterpret_cast<f32x4 *>(pg + e) = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            store8<TW_T_F32>((char *)pg, 8 * (v * TPR + t), KP, dg[v]);
            store8<TW_T_F32>((char *)(pg + KP), 8 * (v * TPR + t), KP, db[v]);
        }
    }
}

// dgamma (blockIdx.y 0) and dbeta (1) from the workgroups' shares: 32 columns
// a workgroup, 32 threads a column, each adding every 32nd share; then their
// sums in order.
constexpr int kColsPerBlock = 32, kColThreads = 32;
__global__ __launch_bounds__(kColsPerBlock *kColThreads) void norm_cols_kernel(
    const float *__restrict__ part, int G, int K, int KP, float *__restrict__ dgamma,
    float *__restrict__ dbeta) {
    float *out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    __shared__ float s[kColThreads][kColsPerBlock + 1];
    const int c = threadIdx.x % kColsPerBlock, r = threadIdx.x / kColsPerBlock;
    const int col = blockIdx.x * kColsPerBlock + c;  // below KP, a multiple of 32
    const float *p = part + (size_t)blockIdx.y * KP + col;
    float v = 0.0f;
#pragma unroll 8
    for (int g = r; g < G; g += kColThreads) v += p[(size_t)g * 2 * KP];
    s[r][c] = v;
    __syncthreads();
    if (r == 0 && col < K) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kColThreads; ++i) v += s[i][c];
        out[col] = v;
    }
}

template <int TD, int TX, int TPR, int VPT>
hipError_t launch_bwd(const NormBwdArgs &a, int grid, hipStream_t s) {
    constexpr int lds = TPR == kWave ? kNormThreads / TPR * 2 * TPR * VPT * 8 * 4 : 0;
    constexpr int threads = TPR > kNormThreads ? TPR : kNormThreads;
    norm_bwd_kernel<TD, TX, TPR, VPT><<<grid, threads, a.part ? lds : 0, s>>>(a);
    return hipGetLastError();
}

template <int TD, int TX>
hipError_t launch_bwd(const NormBwdArgs &a, int grid, hipStream_t s) {
    auto go = [&](auto k) {
        constexpr int K = decltype(k)::value;
        return launch_bwd<TD, TX, norm_bwd_tpr(K), norm_bwd_vpt(K)>(a, grid, s);
    };
    if (a.K <= 512) return go(std::integral_constant<int, 512>{});
    if (a.K <= 1024) return go(std::integral_constant<int, 1024>{});
    if (a.K <= 2048) return go(std::integral_constant<int, 2048>{});
    if (a.K <= 4096) return go(std::integral_constant<int, 4096>{});
    if (a.K <= 8192) return go(std::integral_constant<int, 8192>{});
    return go(std::integral_constant<int, 16384>{});
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

// Workgroups of the row kernel.  Each writes a share of 2 KP floats that the
// column sums read again, so their number is kept to what fills the chip: 2 a
// CU, 1 of 512 threads, 3 where every one still walks 16 rows or more.
// Measured (us at 256, 512, 768, 1024): 16384 x 2048 fp32 139, 103, 104, 108;
// the same bf16 91, 55, 48, 48; 4096 x 2048 25.9, 22.4, 24.5, 26.6; 4096 x 8192
// bf16 57, 64, 72, 79.
static int norm_bwd_groups(int M, int K) {
    const int rpb = norm_bwd_threads(K) / norm_bwd_tpr(K);
    const int64_t need = ((int64_t)M + rpb - 1) / rpb;
    const int most = norm_bwd_threads(K) > kNormThreads ? 256 : M >= 16 * 768 ? 768 : 512;
    return (int)(need < 1 ? 1 : need < most ? need : most);
}

size_t layernorm_bwd_bytes(int M, int K) {
    return (size_t)norm_bwd_groups(M, K) * 2 * norm_bwd_cols(K) * 4;
}

hipError_t launch_layernorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                                int64_t x_stride, const float *gamma, const float *mean,
                                const float *rstd, const void *dres, int M, int K, void *dx,
                                int dx_type, float *dgamma, float *dbeta, float *part,
                                hipStream_t s, hipEvent_t ev_rows) {
    const int grid = norm_bwd_groups(M, K);
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
    const dim3 blocks((K + kColsPerBlock - 1) / kColsPerBlock, 2);
    norm_cols_kernel<<<blocks, kColsPerBlock * kColThreads, 0, s>>>(part, grid, K,
                                                                    norm_bwd_cols(K), dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace tw
