// tw_api.cpp -- the C ABI declared in include/tw.h: argument validation,
// workspace carving, kernel launches on the caller's stream.
#include "tw.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "tw_internal.hpp"
#include "tw_norm_quant.hpp"

namespace {

thread_local char g_err[512] = "";

tw_status fail(tw_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Shape checks shared by the TwELL entry points.
#define TW_TRY_SHAPE(expr)                \
    do {                                  \
        tw_status st_ = (expr);           \
        if (st_ != TW_OK) return st_;     \
    } while (0)

tw_status check_shape(int M, int K, int N, int T, int C, int R_max) {
    if (M < 0 || K <= 0 || N <= 0) return fail(TW_EINVAL, "M=%d K=%d N=%d: need M >= 0, K, N > 0", M, K, N);
    if (T != 128 && T != 256) return fail(TW_EUNSUPPORTED, "tile width T=%d: supported 128, 256", T);
    if (N % T) return fail(TW_EINVAL, "N=%d is not a multiple of T=%d", N, T);
    if (N / T > 256) return fail(TW_EUNSUPPORTED, "N/T=%d tiles per row: at most 256", N / T);
    if (C < 1 || C > T) return fail(TW_EINVAL, "capacity C=%d outside [1, T=%d]", C, T);
    if (K % 128) return fail(TW_EUNSUPPORTED, "K=%d: must be a multiple of 128", K);
    if (K > 4096) return fail(TW_EUNSUPPORTED, "K=%d: at most 4096", K);
    if (R_max < 0 || R_max > M) return fail(TW_EINVAL, "R_max=%d outside [0, M=%d]", R_max, M);
    if ((int64_t)M * K >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "M*K=%lld: x must stay under 4 GiB", (long long)M * K);
    return TW_OK;
}

// Shape checks of the hybrid entry points: the TwELL limits, the dense
// kernels' (N a multiple of 128, each weight matrix and the backup rows
// under 4 GiB) and the sparse row capacity.
tw_status check_hybrid(int M, int K, int N, int T, int C, int P, int R_max) {
    TW_TRY_SHAPE(check_shape(M, K, N, T, C, R_max));
    if (N % 128) return fail(TW_EUNSUPPORTED, "N=%d: must be a multiple of 128", N);
    if ((int64_t)N * K >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "N*K=%lld: weights must stay under 4 GiB", (long long)N * K);
    if ((int64_t)R_max * N >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "R_max*N=%lld: backup rows must stay under 4 GiB",
                    (long long)R_max * N);
    if (P < 1 || P > N) return fail(TW_EINVAL, "sparse row capacity P=%d outside [1, N=%d]", P, N);
    // the kernels name a stored slot by the 32-bit id m * P + s
    if ((int64_t)M * P >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "M*P = %lld stored slots: at most 2^31 - 1",
                    (long long)M * P);
    return TW_OK;
}

// row-overflow bits: at most N / 128 column blocks (the small-batch gate
// kernel with T = 128) by ceil(M / 32) words
size_t pack_ws(int M, int N) {
    return round_up(((size_t)N + 127) / 128 * (((size_t)M + 31) / 32) * 4, 256);
}
// tw_pack_gate: the overflow bits, then the small-batch gate's partial gates
size_t gate_ws(int M, int K, int N) {
    return pack_ws(M, N) + round_up(tw::gate_part_bytes(M, K, N), 256);
}
// overflow path: h rows [R_max][N] bf16, then the split partial tiles;
// then the sparse kernel's partial rows (small batches)
size_t overflow_ws(int R_max, int N) {
    if (R_max == 0) return 0;
    return round_up((size_t)R_max * N * 2, 256) + tw::split_partial_bytes();
}
// the sparse step's workspace: the overflow rows' h and split partials, the
// sparse kernel's partial rows (small batches), the heaviest-first row order
size_t sparse_ws(int M, int K, int R_max, int N) {
    return overflow_ws(R_max, N) + round_up(tw::sparse_rowpart_bytes(M, K), 256) +
           round_up(tw::row_order_bytes(M), 256);
}

tw_status record(void *const *events, int i, hipStream_t s) {
    if (!events) return TW_OK;
    hipError_t e = hipEventRecord(static_cast<hipEvent_t>(events[i]), s);
    if (e != hipSuccess) return fail(TW_EHIP, "hipEventRecord(events[%d]): %s", i, hipGetErrorString(e));
    return TW_OK;
}

tw_status launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(TW_EHIP, "%s: %s", what, hipGetErrorString(e));
    return TW_OK;
}

#define TW_TRY(expr)                      \
    do {                                  \
        tw_status st_ = (expr);           \
        if (st_ != TW_OK) return st_;     \
    } while (0)

#define TW_NEED(p)                                                                   \
    do {                                                                             \
        if (!(p)) return fail(TW_EINVAL, "%s is NULL", #p);                          \
        if (!aligned16(p)) return fail(TW_EINVAL, "%s is not 16-byte aligned", #p);  \
    } while (0)

// Buffers sized by M may be NULL when M == 0.
#define TW_NEED_M(p)                                                                 \
    do {                                                                             \
        if (M > 0 || (p)) TW_NEED(p);                                                \
    } while (0)


// Argument checks of tw_pack_gate and tw_pack_gate_noalloc (all but the
// workspace).
tw_status check_pack_args(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N, int T,
                          int C, float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                          int32_t *ovf_rows, int32_t *ovf_count, int R_max, float *z_debug) {
    TW_TRY(check_shape(M, K, N, T, C, R_max));
    TW_NEED_M(x);
    TW_NEED(wg_t);
    TW_NEED_M(tw_val);
    TW_NEED_M(tw_idx);
    TW_NEED_M(tw_cnt);
    // both NULL: no overflow list is built (callers that route rows from
    // tw_cnt themselves)
    if (!ovf_rows != !ovf_count)
        return fail(TW_EINVAL, "ovf_rows and ovf_count must both be given or both be NULL");
    if (ovf_rows) {
        TW_NEED(ovf_rows);
        TW_NEED(ovf_count);
    }
    if (z_debug && !aligned16(z_debug)) return fail(TW_EINVAL, "z_debug is not 16-byte aligned");
    return TW_OK;
}

// The gate kernel and the compaction on a workspace of at least
// gate_ws(M, K, N) bytes: row-overflow bits, then the small-batch gate's
// partial gates.  Every word of it that a kernel reads is written earlier in
// the same call, so it needs no clearing.
tw_status pack_gate_launch(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N, int T,
                           int C, float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                           int32_t *ovf_rows, int32_t *ovf_count, int R_max, float *z_debug,
                           void *ws, void *stream, void *const *events) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint32_t *oflag = static_cast<uint32_t *>(ws);
    float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + pack_ws(M, N));
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_gate_twell(x, wg_t, M, K, N, T, C, tw_val, tw_idx, tw_cnt, oflag,
                                          z_debug, part, s),
                    "gate_twell launch"));
    TW_TRY(record(events, 1, s));
    if (ovf_rows)
        TW_TRY(launched(tw::launch_ovf_compact(oflag, tw::gate_flag_blocks(M, N, T),
                                               tw::row_words(M), R_max, ovf_rows, ovf_count, s),
                        "ovf_compact launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

// ---- scratch of the entry point that allocates nothing --------------------
// tw_pack_gate_noalloc serves callers that cannot allocate (code under HIP
// graph capture, tight serving loops): its workspace is this file-scope
// device array, of which every GPU the library runs on holds its own copy
// until the process ends.  In host code `scratch` names a host-side stand-in,
// not device memory: its device address is taken once per device with
// hipGetSymbolAddress (with that device current) and only that address is
// ever handed to a kernel.  Every call on one GPU shares that GPU's copy, so
// calls that overlap on one GPU (two streams, two threads) race.
constexpr size_t kScratchBytes = size_t(16) << 20;
constexpr int kMaxDevices = 64;

}  // namespace

static __device__ __align__(256) unsigned char scratch[kScratchBytes];

namespace {

void *g_scratch_ptr[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];
std::once_flag g_scratch_once[kMaxDevices];

// The current device's address of `scratch`, looked up on the first call on
// that device.
tw_status scratch_ptr(void **out) {
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(TW_EHIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices)
        return fail(TW_EUNSUPPORTED, "device %d: at most %d devices", dev, kMaxDevices);
    std::call_once(g_scratch_once[dev], [dev] {
        void *p = nullptr;
        g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        g_scratch_ptr[dev] = p;
    });
    if (g_scratch_err[dev] != hipSuccess)
        return fail(TW_EHIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev,
                    hipGetErrorString(g_scratch_err[dev]));
    if (!g_scratch_ptr[dev]) return fail(TW_EHIP, "no device address for scratch on device %d", dev);
    *out = g_scratch_ptr[dev];
    return TW_OK;
}

}  // namespace

extern "C" {

const char *tw_status_str(int status) {
    switch (status) {
    case TW_OK: return "TW_OK";
    case TW_EINVAL: return "TW_EINVAL";
    case TW_EUNSUPPORTED: return "TW_EUNSUPPORTED";
    case TW_EHIP: return "TW_EHIP";
    default: return "TW_UNKNOWN";
    }
}

const char *tw_last_error(void) { return g_err; }

size_t tw_workspace_bytes(int M, int K, int N, int T, int C, int R_max) {
    char saved[sizeof g_err];
    std::snprintf(saved, sizeof saved, "%s", g_err);
    const tw_status st = check_shape(M, K, N, T, C, R_max);
    std::snprintf(g_err, sizeof g_err, "%s", saved);
    if (st != TW_OK) return 0;
    size_t a = gate_ws(M, K, N), b = sparse_ws(M, K, R_max, N);
    return (a > b ? a : b) + 256;
}

// h [M][N] bf16, and when the down GEMM splits its reduction its partials
size_t tw_ffn_workspace_bytes(int M, int K, int N) {
    if (M < 0 || K <= 0 || N <= 0 || N % 128 || K % 128) return 0;
    if ((int64_t)N * K >= (int64_t(1) << 31)) return 0;
    const size_t split = tw::dense_down_split(M, K) ? tw::split_partial_bytes() : 0;
    return round_up((size_t)M * N * 2, 256) + split + 256;
}

tw_status tw_pack_gate(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N, int T,
                       int C, float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                       int32_t *ovf_rows, int32_t *ovf_count, int R_max, float *z_debug,
                       void *ws, size_t ws_bytes, void *stream, void *const *events) {
    TW_TRY(check_pack_args(x, wg_t, M, K, N, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count,
                           R_max, z_debug));
    TW_NEED(ws);
    const size_t need = tw_workspace_bytes(M, K, N, T, C, R_max);
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);
    return pack_gate_launch(x, wg_t, M, K, N, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count,
                            R_max, z_debug, ws, stream, events);
}

// The variant that allocates nothing: tw_pack_gate's kernels on the
// per-device file-scope scratch array (see the top of this file).
tw_status tw_pack_gate_noalloc(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N,
                               int T, int C, float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                               int32_t *ovf_rows, int32_t *ovf_count, int R_max, float *z_debug,
                               void *stream, void *const *events) {
    TW_TRY(check_pack_args(x, wg_t, M, K, N, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count,
                           R_max, z_debug));
    const size_t need = gate_ws(M, K, N);
    if (need > kScratchBytes)
        return fail(TW_EUNSUPPORTED,
                    "M=%d K=%d N=%d needs %zu bytes of workspace; tw_pack_gate_noalloc's "
                    "static scratch holds %zu (use tw_pack_gate with a workspace)",
                    M, K, N, need, kScratchBytes);
    void *ws = nullptr;
    TW_TRY(scratch_ptr(&ws));
    return pack_gate_launch(x, wg_t, M, K, N, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count,
                            R_max, z_debug, ws, stream, events);
}


tw_status tw_gate_dense(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N, float *z,
                        void *stream, void *const *events) {
    if (M < 0 || K <= 0 || N <= 0) return fail(TW_EINVAL, "M=%d K=%d N=%d: need M >= 0, K, N > 0", M, K, N);
    if (K % 128) return fail(TW_EUNSUPPORTED, "K=%d: must be a multiple of 128", K);
    if (N % 128) return fail(TW_EUNSUPPORTED, "N=%d: must be a multiple of 128", N);
    // tw_pack_gate's kernels, so tw_pack_gate's limits on K and on x
    if (K > 4096) return fail(TW_EUNSUPPORTED, "K=%d: at most 4096", K);
    if ((int64_t)M * K >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "M*K=%lld: x must stay under 4 GiB", (long long)M * K);
    TW_NEED_M(x);
    TW_NEED(wg_t);
    TW_NEED_M(z);
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_gate_dense(x, wg_t, M, K, N, z, s), "dense gate launch"));
    TW_TRY(record(events, 1, s));
    return TW_OK;
}

size_t tw_pack_dense_workspace_bytes(int M, int N) {
    if (M < 0 || N <= 0) return 0;
    return pack_ws(M, N) + 256;
}

tw_status tw_pack_dense(const float *z, int M, int N, int T, int C, float *tw_val,
                        int32_t *tw_idx, int32_t *tw_cnt, int32_t *ovf_rows, int32_t *ovf_count,
                        int R_max, void *ws, size_t ws_bytes, void *stream,
                        void *const *events) {
    if (M < 0 || N <= 0) return fail(TW_EINVAL, "M=%d N=%d: need M >= 0, N > 0", M, N);
    if (T != 128 && T != 256) return fail(TW_EUNSUPPORTED, "tile width T=%d: supported 128, 256", T);
    if (N % T) return fail(TW_EINVAL, "N=%d is not a multiple of T=%d", N, T);
    if (N / T > 256) return fail(TW_EUNSUPPORTED, "N/T=%d tiles per row: at most 256", N / T);
    if (C < 1 || C > T) return fail(TW_EINVAL, "capacity C=%d outside [1, T=%d]", C, T);
    if (R_max < 0 || R_max > M) return fail(TW_EINVAL, "R_max=%d outside [0, M=%d]", R_max, M);
    TW_NEED_M(z);
    TW_NEED_M(tw_val);
    TW_NEED_M(tw_idx);
    TW_NEED_M(tw_cnt);
    TW_NEED(ovf_rows);
    TW_NEED(ovf_count);
    TW_NEED(ws);
    const size_t need = tw_pack_dense_workspace_bytes(M, N);
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    uint32_t *oflag = static_cast<uint32_t *>(ws);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_pack_dense(z, M, N, T, C, tw_val, tw_idx, tw_cnt, oflag, s),
                    "dense pack launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_ovf_compact(oflag, tw::gate_col_blocks(N), tw::row_words(M), R_max,
                                           ovf_rows, ovf_count, s),
                    "ovf_compact launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

tw_status tw_sparse_ffn_fwd(const uint16_t *x, const uint16_t *wg_t, const uint16_t *wu_t,
                            const uint16_t *wd, int M, int K, int N, int T, int C,
                            const float *tw_val, const int32_t *tw_idx, const int32_t *tw_cnt,
                            const int32_t *ovf_rows, const int32_t *ovf_count, int R_max,
                            float *y, void *ws, size_t ws_bytes, void *stream,
                            void *const *events) {
    TW_TRY(check_shape(M, K, N, T, C, R_max));
    TW_NEED_M(x);
    TW_NEED(wg_t);
    TW_NEED(wu_t);
    TW_NEED(wd);
    TW_NEED_M(tw_val);
    TW_NEED_M(tw_idx);
    TW_NEED_M(tw_cnt);
    TW_NEED(ovf_rows);
    TW_NEED(ovf_count);
    TW_NEED_M(y);
    TW_NEED(ws);
    const size_t need = tw_workspace_bytes(M, K, N, T, C, R_max);
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    char *w = static_cast<char *>(ws);
    uint16_t *h = reinterpret_cast<uint16_t *>(w);
    float *partial = reinterpret_cast<float *>(w + round_up((size_t)R_max * N * 2, 256));
    float *rowpart = reinterpret_cast<float *>(w + overflow_ws(R_max, N));
    int32_t *perm = reinterpret_cast<int32_t *>(w + overflow_ws(R_max, N) +
                                                 round_up(tw::sparse_rowpart_bytes(M, K), 256));
    // heaviest-first order for the sparse kernel, written beside the
    // overflow rows' gate+up GEMM (no launch of its own)
    tw::RowOrder ord;
    if (R_max > 0 && tw::sparse_heavy_first(M)) {
        ord.tw_cnt = tw_cnt;
        ord.M = M;
        ord.NT = N / T;
        ord.C = C;
        ord.H = tw::kHeavyEntries;
        ord.perm = perm;
    }
    // All on the caller's stream: the overflow rows' dense path first (its
    // down GEMM leaves split partial tiles when the rows are few), then the
    // sparse kernel, which computes the other rows and sums those partials
    // into the overflow rows.  Running the two paths concurrently on a
    // second stream (the split partials then summed there) was measured: the
    // sparse kernel's workgroups take the CUs first, so little of the dense
    // path overlaps; warm steps gained 1-7% but the 0.5B block's cold step
    // none, and the library would have to hold streams and events.
    TW_TRY(record(events, 0, s));
    if (R_max > 0) {
        TW_TRY(launched(tw::launch_gateup(x, M, wg_t, wu_t, K, N, ovf_rows, ovf_count, R_max, h, s,
                                          ord),
                        "fallback gate+up launch"));
        TW_TRY(record(events, 1, s));
        TW_TRY(launched(tw::launch_down(h, wd, K, N, ovf_rows, ovf_count, R_max, y, partial, s),
                        "fallback down launch"));
        TW_TRY(record(events, 2, s));
    } else {
        for (int i = 1; i <= 2; ++i) TW_TRY(record(events, i, s));
    }
    TW_TRY(launched(tw::launch_sparse_updown(x, wu_t, wd, M, K, N, T, C, tw_val, tw_idx, tw_cnt,
                                             y, R_max > 0 ? partial : nullptr, ovf_rows,
                                             ovf_count, R_max, rowpart, ord.perm, s),
                    "sparse_updown launch"));
    TW_TRY(record(events, 3, s));
    TW_TRY(record(events, 4, s));
    return TW_OK;
}

tw_status tw_ffn_fwd(const uint16_t *x, const uint16_t *wg_t, const uint16_t *wu_t,
                     const uint16_t *wd, int M, int K, int N, float *y, void *ws,
                     size_t ws_bytes, void *stream, void *const *events) {
    if (M < 0 || K <= 0 || N <= 0) return fail(TW_EINVAL, "M=%d K=%d N=%d: need M >= 0, K, N > 0", M, K, N);
    if (N % 128) return fail(TW_EUNSUPPORTED, "N=%d: must be a multiple of 128", N);
    if (K % 128) return fail(TW_EUNSUPPORTED, "K=%d: must be a multiple of 128", K);
    if ((int64_t)N * K >= (int64_t(1) << 31))
        return fail(TW_EUNSUPPORTED, "N*K=%lld: weights must stay under 4 GiB", (long long)N * K);
    TW_NEED_M(x);
    TW_NEED(wg_t);
    TW_NEED(wu_t);
    TW_NEED(wd);
    TW_NEED_M(y);
    TW_NEED(ws);
    const size_t need = tw_ffn_workspace_bytes(M, K, N);
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    uint16_t *h = static_cast<uint16_t *>(ws);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_gateup(x, M, wg_t, wu_t, K, N, nullptr, nullptr, M, h, s),
                    "dense gate+up launch"));
    TW_TRY(record(events, 1, s));
    if (tw::dense_down_split(M, K)) {
        // few rows: split the reduction over N so that every CU has work
        float *partial = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                                   round_up((size_t)M * N * 2, 256));
        TW_TRY(launched(tw::launch_down(h, wd, K, N, nullptr, nullptr, M, y, partial, s),
                        "dense down launch"));
        TW_TRY(launched(tw::launch_split_reduce(partial, nullptr, nullptr, M, K, N, y, s),
                        "dense down split-reduce launch"));
    } else {
        TW_TRY(launched(tw::launch_down(h, wd, K, N, nullptr, nullptr, M, y, nullptr, s),
                        "dense down launch"));
    }
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

size_t tw_hybrid_down_workspace_bytes(int R_max) {
    if (R_max <= 0) return 0;
    return tw::split_partial_bytes() + 256;
}

tw_status tw_hybrid_pack(int M, int N, int T, int C, const float *tw_val, const int32_t *tw_idx,
                         const int32_t *tw_cnt, int P, float *hy_val, int32_t *hy_idx,
                         int32_t *hy_cnt, uint8_t *route, int32_t *bk_rows, int32_t *bk_count,
                         int R_max, void *stream, void *const *events) {
    TW_TRY(check_hybrid(M, 128, N, T, C, P, R_max));
    TW_NEED_M(tw_val);
    TW_NEED_M(tw_idx);
    TW_NEED_M(tw_cnt);
    TW_NEED_M(hy_val);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);

    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_hybrid_pack(tw_val, tw_idx, tw_cnt, M, N, T, C, P, hy_val, hy_idx,
                                           hy_cnt, route, s),
                    "hybrid pack launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_route_compact(route, M, R_max, bk_rows, bk_count, s),
                    "route compaction launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

tw_status tw_hybrid_up(const uint16_t *x, const uint16_t *wg_t, const uint16_t *wu_t, int M,
                       int K, int N, int P, const float *hy_g, const int32_t *hy_idx,
                       const int32_t *hy_cnt, const uint8_t *route, const int32_t *bk_rows,
                       const int32_t *bk_count, int R_max, float *hy_u, float *hy_h,
                       uint16_t *bk_g, uint16_t *bk_u, uint16_t *bk_h, void *stream,
                       void *const *events) {
    TW_TRY(check_hybrid(M, K, N, 128, 1, P, R_max));
    TW_NEED_M(x);
    TW_NEED(wg_t);
    TW_NEED(wu_t);
    TW_NEED_M(hy_g);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);
    TW_NEED_M(hy_h);
    if (hy_u && !aligned16(hy_u)) return fail(TW_EINVAL, "hy_u is not 16-byte aligned");
    if (R_max > 0) TW_NEED(bk_h);
    if (bk_g && !aligned16(bk_g)) return fail(TW_EINVAL, "bk_g is not 16-byte aligned");
    if (bk_u && !aligned16(bk_u)) return fail(TW_EINVAL, "bk_u is not 16-byte aligned");

    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_hybrid_up(x, wu_t, M, K, N, P, hy_g, hy_idx, hy_cnt, route, hy_u,
                                         hy_h, s),
                    "hybrid up launch"));
    TW_TRY(record(events, 1, s));
    if (R_max > 0)
        TW_TRY(launched(tw::launch_gateup_keep(x, M, wg_t, wu_t, K, N, bk_rows, bk_count, R_max,
                                               bk_h, bk_g, bk_u, s),
                        "backup gate+up launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

tw_status tw_hybrid_down(const uint16_t *wd, int M, int K, int N, int P, const float *hy_h,
                         const int32_t *hy_idx, const int32_t *hy_cnt, const uint8_t *route,
                         const int32_t *bk_rows, const int32_t *bk_count, int R_max,
                         const uint16_t *bk_h, float *y, void *ws, size_t ws_bytes, void *stream,
                         void *const *events) {
    TW_TRY(check_hybrid(M, K, N, 128, 1, P, R_max));
    TW_NEED(wd);
    TW_NEED_M(hy_h);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);
    TW_NEED_M(y);
    const size_t need = tw_hybrid_down_workspace_bytes(R_max);
    if (R_max > 0) {
        TW_NEED(bk_h);
        TW_NEED(ws);
    }
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    // the backup GEMM first (split partial tiles for few rows), then the
    // sparse-row kernel, which also sums those partials into the backup rows
    float *partial = R_max > 0 ? static_cast<float *>(ws) : nullptr;
    TW_TRY(record(events, 0, s));
    if (R_max > 0)
        TW_TRY(launched(tw::launch_down(bk_h, wd, K, N, bk_rows, bk_count, R_max, y, partial, s),
                        "backup down launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_hybrid_down(wd, M, K, N, P, hy_h, hy_idx, hy_cnt, route, y, partial,
                                           bk_rows, bk_count, R_max, s),
                    "hybrid down launch"));
    TW_TRY(record(events, 2, s));
    TW_TRY(record(events, 3, s));
    return TW_OK;
}

tw_status tw_hybrid_bwd_dh(const uint16_t *dy, const uint16_t *wd, int M, int K, int N, int P,
                           float l1, const float *hy_g, const float *hy_u, const int32_t *hy_idx,
                           const int32_t *hy_cnt, const uint8_t *route, const int32_t *bk_rows,
                           const int32_t *bk_count, int R_max, const uint16_t *bk_g,
                           const uint16_t *bk_u, float *hy_du, float *hy_dz, uint16_t *bk_du,
                           uint16_t *bk_dz, void *stream, void *const *events) {
    TW_TRY(check_hybrid(M, K, N, 128, 1, P, R_max));
    TW_NEED_M(dy);
    TW_NEED(wd);
    TW_NEED_M(hy_g);
    TW_NEED_M(hy_u);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);
    TW_NEED_M(hy_du);
    TW_NEED_M(hy_dz);
    if (R_max > 0) {
        TW_NEED(bk_g);
        TW_NEED(bk_u);
        TW_NEED(bk_du);
        TW_NEED(bk_dz);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_hybrid_dh(dy, wd, M, K, N, P, hy_g, hy_u, l1, hy_idx, hy_cnt, route,
                                         hy_du, hy_dz, s),
                    "hybrid dh launch"));
    TW_TRY(record(events, 1, s));
    if (R_max > 0)
        TW_TRY(launched(tw::launch_backup_dh(dy, M, wd, K, N, bk_rows, bk_count, R_max, bk_g, bk_u,
                                             l1, bk_du, bk_dz, s),
                        "backup dh launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

size_t tw_hybrid_bwd_dx_workspace_bytes(int R_max) { return tw_hybrid_down_workspace_bytes(R_max); }

tw_status tw_hybrid_bwd_dx(const uint16_t *wg_t, const uint16_t *wu_t, int M, int K, int N, int P,
                           const float *hy_du, const float *hy_dz, const int32_t *hy_idx,
                           const int32_t *hy_cnt, const uint8_t *route, const int32_t *bk_rows,
                           const int32_t *bk_count, int R_max, const uint16_t *bk_du,
                           const uint16_t *bk_dz, float *dx, void *ws, size_t ws_bytes,
                           void *stream, void *const *events) {
    TW_TRY(check_hybrid(M, K, N, 128, 1, P, R_max));
    TW_NEED(wg_t);
    TW_NEED(wu_t);
    TW_NEED_M(hy_du);
    TW_NEED_M(hy_dz);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);
    TW_NEED_M(dx);
    const size_t need = tw_hybrid_bwd_dx_workspace_bytes(R_max);
    if (R_max > 0) {
        TW_NEED(bk_du);
        TW_NEED(bk_dz);
        TW_NEED(ws);
    }
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    // backup rows first: dx = du W_u^T + dz W_g^T as one split GEMM whose
    // reduction runs over both products; the sparse-row kernel follows and
    // sums its partial tiles (split order) into the backup rows
    float *partial = R_max > 0 ? static_cast<float *>(ws) : nullptr;
    TW_TRY(record(events, 0, s));
    if (R_max > 0)
        TW_TRY(launched(tw::launch_down_pair(bk_du, wu_t, bk_dz, wg_t, K, N, bk_rows, bk_count,
                                             R_max, dx, partial, s),
                        "backup dx launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_hybrid_dx(wu_t, wg_t, M, K, N, P, hy_du, hy_dz, hy_idx, hy_cnt,
                                         route, dx, partial, bk_rows, bk_count, R_max, s),
                    "hybrid dx launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

size_t tw_hybrid_bwd_dw_workspace_bytes(int M, int K, int N, int P, int R_max) {
    // a shape tw_hybrid_bwd_dw rejects needs no workspace (and its sizes
    // might not be representable); the check's message is not kept
    char saved[sizeof g_err];
    std::snprintf(saved, sizeof saved, "%s", g_err);
    const tw_status st = check_hybrid(M, K, N, 128, 1, P, R_max);
    std::snprintf(g_err, sizeof g_err, "%s", saved);
    if (st != TW_OK) return 0;
    return tw::hybrid_dw_bytes(M, K, N, P, R_max) + 256;
}

tw_status tw_hybrid_bwd_dw(const uint16_t *x, const uint16_t *dy, int M, int K, int N, int P,
                           const float *hy_h, const float *hy_du, const float *hy_dz,
                           const int32_t *hy_idx, const int32_t *hy_cnt, const uint8_t *route,
                           const int32_t *bk_rows, const int32_t *bk_count, int R_max,
                           const uint16_t *bk_h, const uint16_t *bk_du, const uint16_t *bk_dz,
                           float *dwg_t, float *dwu_t, float *dwd, void *ws, size_t ws_bytes,
                           void *stream, void *const *events) {
    TW_TRY(check_hybrid(M, K, N, 128, 1, P, R_max));
    TW_NEED_M(x);
    TW_NEED_M(dy);
    TW_NEED_M(hy_h);
    TW_NEED_M(hy_du);
    TW_NEED_M(hy_dz);
    TW_NEED_M(hy_idx);
    TW_NEED_M(hy_cnt);
    TW_NEED_M(route);
    TW_NEED(bk_rows);
    TW_NEED(bk_count);
    TW_NEED(dwg_t);
    TW_NEED(dwu_t);
    TW_NEED(dwd);
    TW_NEED(ws);
    if (R_max > 0) {
        TW_NEED(bk_h);
        TW_NEED(bk_du);
        TW_NEED(bk_dz);
    }
    const size_t need = tw_hybrid_bwd_dw_workspace_bytes(M, K, N, P, R_max);
    if (ws_bytes < need) return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);

    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    hipEvent_t e1 = events ? static_cast<hipEvent_t>(events[1]) : nullptr;
    hipEvent_t e2 = events ? static_cast<hipEvent_t>(events[2]) : nullptr;
    TW_TRY(launched(tw::launch_hybrid_dw(x, dy, M, K, N, P, hy_h, hy_du, hy_dz, hy_idx, hy_cnt,
                                         route, bk_rows, bk_count, R_max, bk_h, bk_du, bk_dz,
                                         dwg_t, dwu_t, dwd, ws, s, e1, e2),
                    "weight-gradient launch"));
    TW_TRY(record(events, 3, s));
    return TW_OK;
}

}  // extern "C"

namespace {

// ---- layer norm and int8 products ------------------------------------------

bool float_type(int t) { return t == TW_BF16 || t == TW_F32; }

// Rows of x: a known type, x_stride elements apart.
tw_status check_rows(int M, int K, int max_k, int x_type, int64_t x_stride) {
    if (M < 0 || K <= 0) return fail(TW_EINVAL, "M=%d K=%d: need M >= 0, K > 0", M, K);
    if (K > max_k) return fail(TW_EUNSUPPORTED, "K=%d: at most %d", K, max_k);
    if (!float_type(x_type)) return fail(TW_EINVAL, "x_type=%d: TW_BF16 or TW_F32", x_type);
    if (x_stride < K)
        return fail(TW_EINVAL, "x_stride=%lld is below K=%d", (long long)x_stride, K);
    if (x_stride > (int64_t(1) << 40))
        return fail(TW_EUNSUPPORTED, "x_stride=%lld: at most 2^40", (long long)x_stride);
    return TW_OK;
}

// What the layer norm's forward entry points share (the norm's inputs and
// the stored sum).
tw_status check_norm(const void *x, int x_type, int64_t x_stride, const void *add, int add_type,
                     const float *gamma, const float *beta, float eps, int M, int K,
                     const void *sum) {
    TW_TRY(check_rows(M, K, tw::kNormMaxK, x_type, x_stride));
    if (!(eps >= 0.0f)) return fail(TW_EINVAL, "eps=%g: need eps >= 0", (double)eps);
    TW_NEED_M(x);
    TW_NEED(gamma);
    if (add && !float_type(add_type))
        return fail(TW_EINVAL, "add_type=%d: TW_BF16 or TW_F32", add_type);
    if (add) TW_NEED(add);
    if (beta) TW_NEED(beta);
    if (sum && !add && M > 0) return fail(TW_EINVAL, "sum is given without add");
    if (sum) TW_NEED(sum);
    return TW_OK;
}

// Shapes of an int8 product, for both products and their workspace.
tw_status check_product(int M, int K, int N, int max_k) {
    if (M < 0 || K <= 0 || N <= 0)
        return fail(TW_EINVAL, "M=%d K=%d N=%d: need M >= 0, K, N > 0", M, K, N);
    if (K % 16) return fail(TW_EUNSUPPORTED, "K=%d: must be a multiple of 16", K);
    if (K > max_k) return fail(TW_EUNSUPPORTED, "K=%d: at most %d", K, max_k);
    const int most = 1 << 24;
    if (M > most || N > most) return fail(TW_EUNSUPPORTED, "M=%d N=%d: at most 2^24 each", M, N);
    // the grid of 256 x 128 tiles
    if (((int64_t)M + 255) / 256 * (((int64_t)N + 127) / 128) > (int64_t(1) << 22))
        return fail(TW_EUNSUPPORTED, "M=%d N=%d: at most 2^37 outputs", M, N);
    return TW_OK;
}

size_t quant_ws(int M, int K) {
    return round_up((size_t)M * K, 256) + round_up((size_t)M * 4, 256);
}

// The int8 rows and scales a product reads: the caller's, or those the
// quantisation is about to write to the workspace.
struct QuantIn {
    const int8_t *q;
    const float *scale;
    int8_t *q_out;  // null: x is int8 already
    float *scale_out;
};
tw_status check_quant_in(const void *x, int x_type, int64_t x_stride, const float *x_scale, int M,
                         int K, int max_k, void *ws, size_t ws_bytes, QuantIn *in) {
    if (x_type == TW_INT8) {
        if (x_stride != K)
            return fail(TW_EINVAL, "x_stride=%lld: int8 rows are contiguous (K=%d)",
                        (long long)x_stride, K);
        TW_NEED_M(x);
        TW_NEED_M(x_scale);
        *in = QuantIn{static_cast<const int8_t *>(x), x_scale, nullptr, nullptr};
        return TW_OK;
    }
    TW_TRY(check_rows(M, K, max_k, x_type, x_stride));
    if (x_scale) return fail(TW_EINVAL, "x_scale is given, but x is not int8");
    TW_NEED_M(x);
    TW_NEED_M(ws);
    const size_t need = quant_ws(M, K);
    if (M > 0 && ws_bytes < need)
        return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);
    int8_t *q = static_cast<int8_t *>(ws);
    float *sc = M > 0 ? reinterpret_cast<float *>(q + round_up((size_t)M * K, 256)) : nullptr;
    *in = QuantIn{q, sc, q, sc};
    return TW_OK;
}

}  // namespace

extern "C" {

tw_status tw_layernorm_fwd(const void *x, int x_type, int64_t x_stride, const void *add,
                           int add_type, const float *gamma, const float *beta, float eps, int M,
                           int K, void *sum, void *y, int y_type, float *mean, float *rstd,
                           void *stream, void *const *events) {
    TW_TRY(check_norm(x, x_type, x_stride, add, add_type, gamma, beta, eps, M, K, sum));
    if (!float_type(y_type)) return fail(TW_EINVAL, "y_type=%d: TW_BF16 or TW_F32", y_type);
    TW_NEED_M(y);
    if (mean) TW_NEED(mean);
    if (rstd) TW_NEED(rstd);
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_layernorm(x, x_type, x_stride, add, add_type, gamma, beta, eps, M,
                                         K, sum, y, y_type, mean, rstd, s),
                    "layer norm launch"));
    TW_TRY(record(events, 1, s));
    return TW_OK;
}

size_t tw_layernorm_bwd_workspace_bytes(int M, int K) {
    if (M < 0 || K <= 0 || K > tw::kNormMaxK) return 0;
    return tw::layernorm_bwd_bytes(M, K);
}

tw_status tw_layernorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                           int64_t x_stride, const float *gamma, const float *mean,
                           const float *rstd, const void *dres, int M, int K, void *dx,
                           int dx_type, float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                           void *stream, void *const *events) {
    TW_TRY(check_rows(M, K, tw::kNormMaxK, x_type, x_stride));
    if (!float_type(dy_type)) return fail(TW_EINVAL, "dy_type=%d: TW_BF16 or TW_F32", dy_type);
    if (!float_type(dx_type)) return fail(TW_EINVAL, "dx_type=%d: TW_BF16 or TW_F32", dx_type);
    TW_NEED_M(dy);
    TW_NEED_M(x);
    TW_NEED(gamma);
    TW_NEED_M(mean);
    TW_NEED_M(rstd);
    TW_NEED_M(dx);
    if (dres) TW_NEED(dres);
    if (dgamma) TW_NEED(dgamma);
    if (dbeta) TW_NEED(dbeta);
    if (dgamma || dbeta) {
        TW_NEED(ws);
        const size_t need = tw_layernorm_bwd_workspace_bytes(M, K);
        if (ws_bytes < need)
            return fail(TW_EINVAL, "workspace %zu bytes < %zu needed", ws_bytes, need);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_layernorm_bwd(dy, dy_type, x, x_type, x_stride, gamma, mean, rstd,
                                             dres, M, K, dx, dx_type, dgamma, dbeta,
                                             static_cast<float *>(ws), s,
                                             events ? static_cast<hipEvent_t>(events[1]) : nullptr),
                    "layer norm gradient launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

tw_status tw_quant_rows(const void *x, int x_type, int64_t x_stride, int M, int K, int8_t *q,
                        float *scale, void *stream, void *const *events) {
    TW_TRY(check_rows(M, K, tw::kQuantMaxK, x_type, x_stride));
    TW_NEED_M(x);
    TW_NEED_M(q);
    TW_NEED_M(scale);
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_quant_rows(x, x_type, x_stride, M, K, q, scale, s),
                    "row quantisation launch"));
    TW_TRY(record(events, 1, s));
    return TW_OK;
}

tw_status tw_layernorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                             int add_type, const float *gamma, const float *beta, float eps, int M,
                             int K, void *sum, int8_t *q, float *scale, void *stream,
                             void *const *events) {
    TW_TRY(check_norm(x, x_type, x_stride, add, add_type, gamma, beta, eps, M, K, sum));
    TW_NEED_M(q);
    TW_NEED_M(scale);
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    TW_TRY(launched(tw::launch_layernorm_quant(x, x_type, x_stride, add, add_type, gamma, beta,
                                               eps, M, K, sum, q, scale, s),
                    "layer norm launch"));
    TW_TRY(record(events, 1, s));
    return TW_OK;
}

size_t tw_quant_workspace_bytes(int M, int K) {
    if (M < 0 || K <= 0 || K % 16 || K > tw::kQuantMaxK || M > (1 << 24)) return 0;
    return quant_ws(M, K) + 256;
}

tw_status tw_quant_linear(const void *x, int x_type, int64_t x_stride, const float *x_scale,
                          const int8_t *w, const float *w_scale, const float *bias, int M, int K,
                          int N, void *y, int y_type, void *ws, size_t ws_bytes, void *stream,
                          void *const *events) {
    TW_TRY(check_product(M, K, N, tw::kQuantMaxK));
    if (!float_type(y_type)) return fail(TW_EINVAL, "y_type=%d: TW_BF16 or TW_F32", y_type);
    TW_NEED(w);
    TW_NEED(w_scale);
    if (bias) TW_NEED(bias);
    TW_NEED_M(y);
    QuantIn in;
    TW_TRY(check_quant_in(x, x_type, x_stride, x_scale, M, K, tw::kQuantMaxK, ws, ws_bytes, &in));
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    const tw::QuantRows rows{x, x_type, x_stride, nullptr, nullptr, 0.0f};
    const bool fused = in.q_out && tw::quant_fused(M, K);
    if (in.q_out && !fused)
        TW_TRY(launched(tw::launch_quant_rows(x, x_type, x_stride, M, K, in.q_out, in.scale_out, s),
                        "row quantisation launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_quant_linear(in.q, in.scale, fused ? &rows : nullptr, w, w_scale,
                                            bias, M, K, N, y, y_type, s),
                    "int8 product launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

tw_status tw_quant_gateup(const void *x, int x_type, int64_t x_stride, const float *x_scale,
                          const float *gamma, const float *beta, float eps, const int8_t *wg,
                          const float *g_scale, const int8_t *wu, const float *u_scale, int M,
                          int K, int N, void *h, int h_type, void *ws, size_t ws_bytes,
                          void *stream, void *const *events) {
    const int max_k = gamma ? tw::kNormMaxK : tw::kQuantMaxK;
    TW_TRY(check_product(M, K, N, max_k));
    if (!float_type(h_type)) return fail(TW_EINVAL, "h_type=%d: TW_BF16 or TW_F32", h_type);
    if (gamma && x_type == TW_INT8) return fail(TW_EINVAL, "gamma is given, but x is int8");
    if (beta && !gamma) return fail(TW_EINVAL, "beta is given without gamma");
    if (gamma && !(eps >= 0.0f)) return fail(TW_EINVAL, "eps=%g: need eps >= 0", (double)eps);
    if (gamma) TW_NEED(gamma);
    if (beta) TW_NEED(beta);
    TW_NEED(wg);
    TW_NEED(g_scale);
    TW_NEED(wu);
    TW_NEED(u_scale);
    TW_NEED_M(h);
    QuantIn in;
    TW_TRY(check_quant_in(x, x_type, x_stride, x_scale, M, K, max_k, ws, ws_bytes, &in));
    hipStream_t s = static_cast<hipStream_t>(stream);
    TW_TRY(record(events, 0, s));
    const tw::QuantRows rows{x, x_type, x_stride, gamma, beta, eps};
    const bool fused = in.q_out && tw::quant_fused(M, K);
    if (in.q_out && !fused && gamma)
        TW_TRY(launched(tw::launch_layernorm_quant(x, x_type, x_stride, nullptr, 0, gamma, beta,
                                                   eps, M, K, nullptr, in.q_out, in.scale_out, s),
                        "layer norm launch"));
    else if (in.q_out && !fused)
        TW_TRY(launched(tw::launch_quant_rows(x, x_type, x_stride, M, K, in.q_out, in.scale_out, s),
                        "row quantisation launch"));
    TW_TRY(record(events, 1, s));
    TW_TRY(launched(tw::launch_quant_gateup(in.q, in.scale, fused ? &rows : nullptr, wg, g_scale,
                                            wu, u_scale, M, K, N, h, h_type, s),
                    "int8 product launch"));
    TW_TRY(record(events, 2, s));
    return TW_OK;
}

}  // extern "C"
