// tw_norm_quant.hpp -- launchers of the layer-norm and int8 kernels behind the
// C ABI (the others are in tw_internal.hpp).  Every launcher only enqueues work
// on `s` and returns the launch status; the C ABI layer validates all
// arguments before calling them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tw {

// Element types of rows (the values of tw_type in the C ABI).
enum { TW_T_BF16 = 0, TW_T_F32 = 1, TW_T_INT8 = 2 };

// Layer norm over rows (layer_norm.hip): z = x (+ add), rows of x x_stride
// elements apart, add contiguous; y = norm(z) gamma (+ beta).  sum (z in x's
// type), mean and rstd are optional outputs.
constexpr int kNormMaxK = 16384;
constexpr int kQuantMaxK = 65536;
hipError_t launch_layernorm(const void *x, int x_type, int64_t x_stride, const void *add,
                            int add_type, const float *gamma, const float *beta, float eps, int M,
                            int K, void *sum, void *y, int y_type, float *mean, float *rstd,
                            hipStream_t s);
// The same norm quantised to int8 with one scale per row.
hipError_t launch_layernorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                                  int add_type, const float *gamma, const float *beta, float eps,
                                  int M, int K, void *sum, int8_t *q, float *scale,
                                  hipStream_t s);
hipError_t launch_quant_rows(const void *x, int x_type, int64_t x_stride, int M, int K, int8_t *q,
                             float *scale, hipStream_t s);
// Gradient of the layer norm.  part: layernorm_bwd_bytes(M, K) bytes (unused
// when dgamma and dbeta are both null).
size_t layernorm_bwd_bytes(int M, int K);
hipError_t launch_layernorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                                int64_t x_stride, const float *gamma, const float *mean,
                                const float *rstd, const void *dres, int M, int K, void *dx,
                                int dx_type, float *dgamma, float *dbeta, float *part,
                                hipStream_t s, hipEvent_t ev_rows);

// int8 products (quant_gemm.hip): y = (q w^T) x_scale w_scale (+ bias), and
// h = ReLU(gate) * up of two such products.  The input is either int8 rows q
// with x_scale, or, for a few rows (quant_fused), float rows that the same
// kernel norms (gamma not null) and quantises; q and x_scale are then unused.
struct QuantRows {
    const void *x;
    int x_type;
    int64_t x_stride;
    const float *gamma, *beta;
    float eps;
};
bool quant_fused(int M, int K);
hipError_t launch_quant_linear(const int8_t *q, const float *x_scale, const QuantRows *rows,
                               const int8_t *w, const float *w_scale, const float *bias, int M,
                               int K, int N, void *y, int y_type, hipStream_t s);
hipError_t launch_quant_gateup(const int8_t *q, const float *x_scale, const QuantRows *rows,
                               const int8_t *wg, const float *g_scale, const int8_t *wu,
                               const float *u_scale, int M, int K, int N, void *h, int h_type,
                               hipStream_t s);

}  // namespace tw
