// tw_train.hpp -- launchers of the dense training step's kernels behind the C
// ABI: the RMS norm, the gated FFN with its gradient, the cross entropy of the
// output projection, gradient clipping.  Every launcher only enqueues work on
// `s` and returns the launch status; the C ABI layer validates all arguments
// before calling them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tw_norm_quant.hpp"

namespace tw {

// RMS norm over rows (layer_norm.hip), arguments as launch_layernorm's.
hipError_t launch_rmsnorm(const void *x, int x_type, int64_t x_stride, const void *add,
                          int add_type, const float *gamma, float eps, int M, int K, void *sum,
                          void *y, int y_type, float *rstd, hipStream_t s);
hipError_t launch_rmsnorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                                int add_type, const float *gamma, float eps, int M, int K,
                                void *sum, int8_t *q, float *scale, hipStream_t s);
// part: layernorm_bwd_bytes(M, K) bytes (unused when dgamma is null).
hipError_t launch_rmsnorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                              int64_t x_stride, const float *gamma, const float *rstd,
                              const void *dres, int M, int K, void *dx, int dx_type, float *dgamma,
                              float *part, hipStream_t s, hipEvent_t ev_rows);

// Elements of a row that the tile kernels take, and between rows (tw_tiles.hpp).
constexpr int kTileRowMost = 1 << 20;

// Activations of the gated FFN (the values of tw_act in the C ABI).
enum { TW_A_RELU = 0, TW_A_SILU = 1, TW_A_GELU = 2 };

// The gated FFN (gated_ffn.hip).  h: [M][N] bf16 scratch, part: scratch of
// ffn_fwd_part_bytes (down) or ffn_bwd_part_bytes (dx, dw).  g and u (the
// projections before the activation) are optional outputs.
size_t ffn_fwd_part_bytes(int M, int K, int N);
size_t ffn_bwd_part_bytes(int M, int K, int N);
hipError_t launch_ffn_up(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                         const uint16_t *wu_t, int act, int M, int K, int N, uint16_t *g,
                         uint16_t *u, uint16_t *h, hipStream_t s);
hipError_t launch_ffn_down(const uint16_t *h, const uint16_t *wd, int M, int K, int N, void *y,
                           int y_type, float *part, hipStream_t s);
// dz, du, h: [M][N] bf16 each.
hipError_t launch_ffn_dh(const uint16_t *dy, const uint16_t *wd, int act, const uint16_t *g,
                         const uint16_t *u, int M, int K, int N, uint16_t *dz, uint16_t *du,
                         uint16_t *h, hipStream_t s);
hipError_t launch_ffn_dx(const uint16_t *dz, const uint16_t *du, const uint16_t *wg_t,
                         const uint16_t *wu_t, int M, int K, int N, void *dx, int dx_type,
                         float *part, hipStream_t s);
hipError_t launch_ffn_dw(const uint16_t *dz, const uint16_t *du, const uint16_t *h,
                         const uint16_t *x, int64_t x_stride, const uint16_t *dy, int M, int K,
                         int N, void *dwg_t, void *dwu_t, void *dwd, int dw_type, float *part,
                         hipStream_t s);

// Cross entropy of x w^T (linear_ce.hip).  Targets are 32- or 64-bit integers;
// one outside [0, V) leaves its row out.
struct Targets {
    const void *p;
    int wide;  // 64 bits
};
size_t ce_fwd_bytes(int M, int K, int V);
hipError_t launch_ce_fwd(const uint16_t *x, int64_t x_stride, const uint16_t *w, Targets t, int M,
                         int K, int V, float *loss, float *lse, void *ws, hipStream_t s);
size_t ce_bwd_bytes(int M, int K, int V);
hipError_t launch_ce_bwd(const float *dloss, const uint16_t *x, int64_t x_stride,
                         const uint16_t *w, Targets t, const float *lse, int M, int K, int V,
                         void *dx, int dx_type, void *dw, int dw_type, void *ws, hipStream_t s);

// Gradient clipping (grad_clip.hip) over `count` buffers of n[i] elements each, at
// most kClipMost; part: grad_norm_bytes.
constexpr int64_t kClipMost = int64_t(1) << 34;
size_t grad_norm_bytes(int count, const int64_t *n);
hipError_t launch_grad_norm(int count, const void *const *g, const int64_t *n, const int *g_type,
                            float *norm, float *part, hipStream_t s);
hipError_t launch_grad_clip(int count, const void *const *g, const int64_t *n, const int *g_type,
                            void *const *out, const int *out_type, float max_norm, float eps,
                            float *norm, float *part, hipStream_t s, hipEvent_t ev_norm);

}  // namespace tw
