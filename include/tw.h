/*
 * tw.h -- C ABI of the TwELL sparse gated-FFN forward for AMD MI355X (gfx950).
 *
 * The block computed is the ReLU-gated feed-forward layer of "Sparser,
 * Faster, Lighter Transformer Language Models Review", section 1-1:
 *
 *     h_u = x W_u,   h_g = ReLU(x W_g),   h = h_u (elementwise) h_g,   y = h W_d
 *
 * with x [M, K] (M tokens, model dimension K) and an expanded hidden
 * dimension N.  Its two-stage inference path (section 2-2: a gate projection
 * whose epilogue builds the packed form, then the up and down projections
 * fused over the active neurons) is split over two calls:
 *
 *   tw_pack_gate       gate GEMM whose epilogue applies the ReLU and packs the
 *                      active entries of every (token row, column tile) in the
 *                      tile-wise ELLPACK layout of section 3-4, and builds the
 *                      list of rows that overflow a tile's capacity
 *                      (the dense-backup routing of sections 3-6 and 4-3);
 *   tw_sparse_ffn_fwd  per-token sparse up+down (section 3-5 equation) for the
 *                      rows that fit, and the dense path for the listed rows.
 *
 * tw_ffn_fwd is the dense gated FFN over all rows, the comparator the sparse
 * path is measured against.  tw_gate_dense + tw_pack_dense are the unfused
 * equivalent of tw_pack_gate (dense gate written to memory, then packed).
 * tw_hybrid_pack, tw_hybrid_up and tw_hybrid_down are the training forward
 * over the hybrid storage of sections 3-6 and 3-7, and tw_hybrid_bwd_dh,
 * tw_hybrid_bwd_dx and tw_hybrid_bwd_dw its backward.  tw_layernorm_fwd and
 * tw_layernorm_bwd are the layer norm in front of the block, and
 * tw_quant_gateup and tw_quant_linear its dense projections in 8-bit integers.
 * The dense training step beside it (declared at the end): the RMS norm
 * tw_rmsnorm_fwd, tw_rmsnorm_quant and tw_rmsnorm_bwd, the gated FFN with any of
 * three activations tw_gated_ffn_fwd and tw_gated_ffn_bwd, the cross entropy of an
 * output projection tw_linear_ce_fwd and tw_linear_ce_bwd, and gradient clipping,
 * tw_grad_norm and tw_grad_clip.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - bf16 values travel as raw uint16_t bit patterns.
 * - Every pointer argument except `stream` is a device pointer to memory the
 *   caller owns.  The library allocates no device memory and keeps no
 *   state between calls, so calls on different streams may run
 *   concurrently as long as their output and workspace buffers are
 *   distinct.  The one exception is tw_pack_gate_noalloc, whose workspace
 *   is a static device array inside the library, shared by every call on
 *   one GPU (see its declaration).
 * - All work is enqueued asynchronously on `stream` (a hipStream_t passed as
 *   void*; NULL is the default stream).  Nothing synchronises the host.
 * - Argument and shape errors are detected on the host before any work is
 *   enqueued and return TW_EINVAL or TW_EUNSUPPORTED; no output is touched
 *   then.  A failed kernel launch returns TW_EHIP.  tw_last_error() gives a
 *   message for the last failure of the calling thread.
 * - Device buffers must be 16-byte aligned.  When M == 0 the buffers whose
 *   size is a multiple of M may be NULL.
 * - Optional `events`: NULL, or an array of hipEvent_t (passed as void*)
 *   with one more entry than the call launches kernels, for per-kernel
 *   durations with hipEventElapsedTime.  tw_pack_gate records events[0]
 *   on `stream` before the gate, events[1] after it (one kernel; for a few
 *   token rows two: the K-sliced partial gates, then their sum and the
 *   packing) and events[2] after the overflow-list compaction.  tw_ffn_fwd
 *   (2 kernels) records events[0] before the first kernel and events[i+1]
 *   after kernel i.  tw_sparse_ffn_fwd takes 5
 *   events for 3 kernels: events[0] before any of them, events[1] and [2]
 *   after the overflow rows' gate+up and down GEMMs, events[3] after the
 *   sparse up+down kernel (which also finishes the overflow rows' split
 *   sums; for batches of 32 to 128 rows it is followed by the sum of its
 *   partial rows), events[4] together with events[3] (with R_max == 0 only
 *   the sparse kernel runs and events[0..2] are recorded together).
 *
 * Weight layout (one layout serves every path): wg_t, wu_t and wd are all
 * [N][K] row-major bf16.  wg_t and wu_t hold W_g and W_u transposed, so the
 * weights of hidden neuron j (column j of W_g / W_u) are row j, contiguous;
 * wd is W_d itself, whose row j is what neuron j adds to the output.
 *
 * Supported shapes: M >= 0, K a positive multiple of 128 and at most 4096,
 * N a positive multiple of T, T in {128, 256}, N / T <= 256, 1 <= C <= T,
 * 0 <= R_max <= M, and M * K < 2^31 (x under 4 GiB: the dense backup
 * gathers its rows with 32-bit buffer offsets).  tw_ffn_fwd has its own
 * limits, stated at its declaration.
 */
#ifndef TW_H
#define TW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tw_status {
    TW_OK = 0,
    TW_EINVAL = 1,        /* null pointer, bad size, misaligned buffer     */
    TW_EUNSUPPORTED = 2,  /* valid but outside the supported shapes above  */
    TW_EHIP = 3           /* a HIP runtime call or kernel launch failed    */
} tw_status;

/* Element type of a row buffer, where an entry point takes more than one. */
typedef enum tw_type {
    TW_BF16 = 0,
    TW_F32 = 1,
    TW_INT8 = 2,
    TW_INT32 = 3, /* targets of tw_linear_ce_fwd, tw_linear_ce_bwd */
    TW_INT64 = 4
} tw_type;

/* Activation of the gated FFN: ReLU, SiLU (g / (1 + e^-g)), GELU in its tanh
 * form (g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2). */
typedef enum tw_act { TW_RELU = 0, TW_SILU = 1, TW_GELU = 2 } tw_act;

/* Static name of a status code. */
const char *tw_status_str(int status);

/* Message describing the last non-OK status returned on the calling thread
 * (empty string if none). */
const char *tw_last_error(void);

/* Bytes of device workspace tw_pack_gate and tw_sparse_ffn_fwd need for
 * this shape (one buffer of this size serves both); 0 for arguments that
 * the entry points would reject. */
size_t tw_workspace_bytes(int M, int K, int N, int T, int C, int R_max);

/*
 * Gate GEMM + ReLU + TwELL packing + overflow routing.
 *
 * Computes z = x W_g in fp32 (bf16 products, fp32 accumulation) and, for
 * every token row m and column tile t (columns [t*T, (t+1)*T)):
 *   tw_cnt[m][t]          number of columns j in the tile with z[m][j] > 0
 *                         (strictly positive; the true count, even above C)
 *   tw_idx[m][t][s]       the s-th such j, ascending, as a global column
 *   tw_val[m][t][s]       z[m][j] (fp32) for that j
 * for s < min(tw_cnt[m][t], C); slots from min(cnt, C) to C-1 are left
 * untouched.  These are the packed values, original hidden indices and
 * per-(row, tile) counts of section 3-4 (h_v, h_I, h_nz).
 *
 * A row with any tile holding more than C active columns overflows and is
 * routed whole to the dense path (sections 3-6 and 4-3): ovf_rows receives
 * the overflowing rows in ascending order, at most R_max of them, and
 * *ovf_count their true number.  *ovf_count > R_max means that the rows past
 * the first R_max will not be recomputed: read ovf_count after the stream
 * has run and retry with a larger R_max (or C) -- the retry of section 4-3.
 *
 *   x        [M][K]          bf16, token rows
 *   wg_t     [N][K]          bf16, W_g transposed
 *   tw_val   [M][N/T][C]     fp32 out
 *   tw_idx   [M][N/T][C]     int32 out
 *   tw_cnt   [M][N/T]        int32 out
 *   ovf_rows [max(R_max,1)]  int32 out
 *   ovf_count[1]             int32 out
 *   z_debug  [M][N]          fp32 out, or NULL; receives z itself (the same
 *                            values the packing used) -- for tests
 *   ws       workspace of ws_bytes >= tw_workspace_bytes(M, K, N, T, C, R_max)
 *
 * ovf_rows and ovf_count may both be NULL (one alone is TW_EINVAL): then no
 * overflow list is built and the compaction kernel does not run (events[2]
 * is recorded right after events[1]).  tw_sparse_ffn_fwd needs the list;
 * the training path does not (tw_hybrid_pack routes rows from tw_cnt).
 */
tw_status tw_pack_gate(const uint16_t *x, const uint16_t *wg_t,
                       int M, int K, int N, int T, int C,
                       float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                       int32_t *ovf_rows, int32_t *ovf_count, int R_max,
                       float *z_debug, void *ws, size_t ws_bytes,
                       void *stream, void *const *events);

/*
 * tw_pack_gate without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same kernels, arguments, outputs and
 * error behaviour as tw_pack_gate; the workspace is instead a static device
 * array inside the library of 16 MiB per GPU (held by every GPU the library
 * runs on until the process ends; its address is looked up once per device,
 * on the first call there).  Shapes whose tw_pack_gate workspace would
 * exceed it (row-overflow bits of (N/128) * ceil(M/32) words, plus for a few
 * token rows the small-batch gate's partial gates) return TW_EUNSUPPORTED
 * with a message giving the bytes needed.  The call allocates nothing.  All
 * calls on one GPU share that GPU's array, so calls that overlap on one GPU
 * (on two streams, or from two host threads) race; calls in stream order do
 * not.  Nothing in the array needs to start at zero.
 */
tw_status tw_pack_gate_noalloc(const uint16_t *x, const uint16_t *wg_t,
                               int M, int K, int N, int T, int C,
                               float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                               int32_t *ovf_rows, int32_t *ovf_count, int R_max,
                               float *z_debug, void *stream, void *const *events);

/*
 * The unfused alternative to tw_pack_gate, in two calls: section 3-4
 * contrasts packing in the gate's epilogue with computing the dense gate,
 * writing it to memory and packing it in a separate pass (an extra write,
 * read and write of the whole gate).  These calls are that separate path,
 * kept for measuring what the fusion saves and for packing gates computed
 * elsewhere; their outputs are identical to tw_pack_gate's.
 *
 * tw_gate_dense: z = x W_g as fp32 [M][N] (the same kernel and arithmetic
 * as tw_pack_gate, so z is bitwise tw_pack_gate's z_debug).  K and N
 * multiples of 128, K <= 4096, M * K < 2^31 (tw_pack_gate's limits; other
 * shapes return TW_EUNSUPPORTED).  events: [0] before, [1] after the kernel.
 *
 * tw_pack_dense: TwELL packing and overflow routing of any fp32 gate z
 * [M][N] (active means z > 0), with exactly the outputs and conventions of
 * tw_pack_gate above (same shape limits on N, T, C, R_max).  The workspace
 * holds the row-overflow bits: ws_bytes >= tw_pack_dense_workspace_bytes
 * (tw_workspace_bytes of the same shape is always enough).  events: [0]
 * before, [1] after the packing kernel, [2] after the compaction.
 */
tw_status tw_gate_dense(const uint16_t *x, const uint16_t *wg_t, int M, int K, int N, float *z,
                        void *stream, void *const *events);
size_t tw_pack_dense_workspace_bytes(int M, int N);
tw_status tw_pack_dense(const float *z, int M, int N, int T, int C,
                        float *tw_val, int32_t *tw_idx, int32_t *tw_cnt,
                        int32_t *ovf_rows, int32_t *ovf_count, int R_max,
                        void *ws, size_t ws_bytes, void *stream, void *const *events);

/*
 * Sparse up+down for the rows that fit, dense path for the overflow list.
 *
 * For every row m with no tile over capacity (every tw_cnt[m][t] <= C), with
 * the packed (j, g) pairs of tw_pack_gate:
 *     y[m][:] = sum over packed (j, g) of (x[m] . Wu_t[j]) * g * Wd[j][:]
 * (section 3-5 equation; the up activation is a scalar per active neuron,
 * fp32 throughout).  A row with no active neuron gets y = 0.
 * For r < min(*ovf_count, R_max), the row m = ovf_rows[r] gets the dense
 * gated FFN of section 1-1 instead (h rounded to bf16 before W_d, fp32
 * accumulation).  Rows that overflow but lie past R_max are left untouched.
 *
 *   x, wg_t, wu_t, wd       as above ([M][K] and [N][K] bf16)
 *   tw_val, tw_idx, tw_cnt  the packing written by tw_pack_gate
 *   ovf_rows, ovf_count     the routing written by tw_pack_gate (device)
 *   y        [M][K]         fp32 out
 *
 * On `stream`, the overflow rows' dense path runs first: gate+up, then the
 * down GEMM, which for few rows splits its reduction over N into partial
 * tiles in the workspace.  The sparse kernel follows; it computes the rows
 * that fit and sums those partials (in split order, so the result does not
 * depend on timing) into the listed rows.  The two sets of rows are
 * disjoint.  Batches of 32 to 128 rows spread each row over several
 * workgroups, whose partial rows (in the workspace) a last small kernel
 * sums in a fixed order.  Batches of 257 to 8192 rows (with R_max > 0)
 * start their heaviest rows first, in an order that extra workgroups of the
 * gate+up launch write to the workspace from tw_cnt; each row is still
 * computed once by the same code, so y does not depend on the order.
 */
tw_status tw_sparse_ffn_fwd(const uint16_t *x, const uint16_t *wg_t,
                            const uint16_t *wu_t, const uint16_t *wd,
                            int M, int K, int N, int T, int C,
                            const float *tw_val, const int32_t *tw_idx,
                            const int32_t *tw_cnt, const int32_t *ovf_rows,
                            const int32_t *ovf_count, int R_max,
                            float *y, void *ws, size_t ws_bytes,
                            void *stream, void *const *events);

/*
 * Dense gated FFN over all M rows (section 1-1 equation): the gate and up
 * projections in one MFMA GEMM whose epilogue forms h = ReLU(g) * u rounded
 * to bf16, then the down projection into fp32 y [M][K] (when M is too small
 * for its output tiles to fill the chip, split over N and summed by a
 * second kernel; events[2] follows both).  The workspace holds h [M][N]
 * bf16 and, when the down projection splits, the partial sums:
 * ws_bytes >= tw_ffn_workspace_bytes.
 * Shapes: M >= 0, K and N positive multiples of 128, N * K < 2^31 (each
 * weight matrix under 4 GiB: 32-bit buffer offsets).  The workspace query
 * returns 0 for any other shape.
 *
 * tw_gated_ffn_fwd with TW_RELU computes the same for more shapes.  Measured
 * (us, warm; this call, that one): 1 row 2048 x 5632 25, 18; 64 rows 28, 31; 128
 * rows 32, 42; 512 rows 65, 53; 4096 x 1024 x 4096 104, 108; 4096 x 2048 x 5632
 * 274, 218; 16384 x 2048 x 8192 1435, 1195.
 */
size_t tw_ffn_workspace_bytes(int M, int K, int N);
tw_status tw_ffn_fwd(const uint16_t *x, const uint16_t *wg_t,
                     const uint16_t *wu_t, const uint16_t *wd,
                     int M, int K, int N, float *y, void *ws, size_t ws_bytes,
                     void *stream, void *const *events);

/*
 * Hybrid storage for the training forward (sections 3-6, 3-7 and 4-3).
 *
 * Training keeps the gate activation in a hybrid form built from the TwELL
 * gate (section 2-2: TwELL gate, then hybrid storage): most token rows as a
 * row-wide ELL of at most P entries (the values and original hidden indices
 * of section 3-3's ELL, in ascending column order), the few heavy rows whole
 * in a dense backup, and a binary routing vector saying which holds each
 * row.  The up and down projections then run as two separate products that
 * keep that form (section 3-7: in training they are not fused): the
 * dense-to-hybrid product (x W_u evaluated only at the stored entries, times
 * the gate) and the hybrid-to-dense product (h W_d).  The section 4-3
 * capacities are P = 128 stored entries per row and a backup of at most
 * M / 8 rows; an overflow of the backup is reported for a retry.
 *
 * Common arrays (device, caller-owned, P the sparse row capacity):
 *   hy_cnt  [M]        int32  the row's number of active neurons (the true
 *                             count, also for backup rows)
 *   hy_idx  [M][P]     int32  stored hidden index j of entry s < hy_cnt[m]
 *   hy_val / hy_u / hy_h [M][P]  fp32  gate value, up value, product of entry s
 *   route   [M]        uint8  1 if row m lives in the dense backup, else 0
 *   bk_rows [max(R_max,1)] int32  backup rows, ascending; slot r holds row bk_rows[r]
 *   bk_count[1]        int32  the true number of backup rows (may exceed R_max)
 *   bk_g / bk_u / bk_h [R_max][N] bf16  dense gate, up, product of backup slot r
 * Slots s >= hy_cnt[m] of a sparse row, and every slot of a backup row, are
 * left untouched.  A backup row past R_max (bk_count > R_max) is in neither
 * store: read bk_count after the stream has run and retry with a larger
 * R_max (or P) -- the retry of section 4-3.  Such rows get no output from
 * tw_hybrid_up or tw_hybrid_down.
 *
 * Shapes: as for tw_pack_gate (T in {128, 256}, N a multiple of T, N/T <=
 * 256, 1 <= C <= T, K a multiple of 128 and at most 4096, M*K < 2^31), and
 * N a multiple of 128, 1 <= P <= N, 0 <= R_max <= M, N*K < 2^31,
 * R_max*N < 2^31, and M*P < 2^31 (the kernels name a stored slot by the
 * 32-bit id m*P + s); other shapes return TW_EUNSUPPORTED.
 */

/*
 * TwELL -> hybrid.  Reads a TwELL packing of capacity C (tw_pack_gate's or
 * tw_pack_dense's outputs).  Row m goes to the dense backup when its total
 * count exceeds P or when one of its tiles held more than C entries (its
 * TwELL slots then lack entries); otherwise its TwELL entries are copied to
 * hy_idx / hy_val in ascending column order.  Writes hy_cnt, route and the
 * backup list.  The backup rows' dense values are produced by tw_hybrid_up.
 * events: [0] before, [1] after the packing kernel, [2] after the list.
 */
tw_status tw_hybrid_pack(int M, int N, int T, int C,
                         const float *tw_val, const int32_t *tw_idx, const int32_t *tw_cnt,
                         int P, float *hy_val, int32_t *hy_idx, int32_t *hy_cnt,
                         uint8_t *route, int32_t *bk_rows, int32_t *bk_count, int R_max,
                         void *stream, void *const *events);

/*
 * Dense-to-hybrid product of the up projection, times the gate.
 * Sparse rows: for each stored entry s (hidden index j, gate g = hy_g),
 *     hy_u[m][s] = x[m] . wu_t[j]   (fp32),   hy_h[m][s] = hy_u[m][s] * g.
 * Backup slots r < min(*bk_count, R_max), row m = bk_rows[r], all N columns
 * on the matrix cores (one GEMM over W_g and W_u, x read once):
 *     bk_g[r] = bf16(ReLU(x[m] W_g)),  bk_u[r] = bf16(x[m] W_u),
 *     bk_h[r] = bf16(ReLU(x[m] W_g) * (x[m] W_u))  (product before rounding).
 * hy_u, bk_g and bk_u may be NULL (not stored); hy_h and bk_h are required.
 * events: [0] before, [1] after the sparse-row kernel, [2] after the backup GEMM.
 */
tw_status tw_hybrid_up(const uint16_t *x, const uint16_t *wg_t, const uint16_t *wu_t,
                       int M, int K, int N, int P,
                       const float *hy_g, const int32_t *hy_idx, const int32_t *hy_cnt,
                       const uint8_t *route, const int32_t *bk_rows, const int32_t *bk_count,
                       int R_max, float *hy_u, float *hy_h,
                       uint16_t *bk_g, uint16_t *bk_u, uint16_t *bk_h,
                       void *stream, void *const *events);

/*
 * Hybrid-to-dense product of the down projection, y = h W_d (fp32 [M][K]).
 * Sparse rows: y[m] = sum over stored s of hy_h[m][s] * wd[hy_idx[m][s]]
 * (a row with no entry gets 0).  Backup slots r < min(*bk_count, R_max): the
 * row bk_rows[r] of y gets bk_h[r] W_d on the matrix cores.  The workspace
 * holds the backup GEMM's partial tiles: ws_bytes >=
 * tw_hybrid_down_workspace_bytes(R_max) (ws may be NULL when that is 0).
 * The backup GEMM runs first; the sparse-row kernel follows and also sums
 * the GEMM's partial tiles into the backup rows (in split order).
 * events: [0] before, [1] after the backup GEMM, [2] and [3] after the
 * sparse-row kernel.
 */
size_t tw_hybrid_down_workspace_bytes(int R_max);
tw_status tw_hybrid_down(const uint16_t *wd, int M, int K, int N, int P,
                         const float *hy_h, const int32_t *hy_idx, const int32_t *hy_cnt,
                         const uint8_t *route, const int32_t *bk_rows, const int32_t *bk_count,
                         int R_max, const uint16_t *bk_h, float *y,
                         void *ws, size_t ws_bytes, void *stream, void *const *events);

/*
 * Backward over the hybrid storage (section 3-7: the gradients are formed
 * from the stored sparse activations, without rebuilding a dense hidden
 * state; L1 gradient injection; the hybrid transpose for the weight
 * gradients), for the forward of tw_hybrid_pack / tw_hybrid_up /
 * tw_hybrid_down with g, u (hy_u, bk_g, bk_u) kept.  With dy = dLoss/dy
 * [M][K] (bf16) and the L1 penalty of section 3-2 on the gate activation,
 * whose gradient on a positive activation is the caller's `l1` (lambda
 * divided by the layer count and M N, in the pages' normalisation):
 *   dh = dy W_d^T,   du = dh g,   dz = (dh u + l1) where g > 0, else 0,
 *   dx = du W_u^T + dz W_g^T,
 *   dwd[j] = sum_m h[m][j] dy[m],  dwu_t[j] = sum_m du[m][j] x[m],
 *   dwg_t[j] = sum_m dz[m][j] x[m]
 * (dwu_t, dwg_t: gradients of W_u and W_g in their transposed [N][K] layout,
 * dwd of W_d [N][K]; all fp32).  Rows routed to the backup but past its room
 * (bk_count > R_max) stored nothing: they get no dx and add nothing to the
 * weight gradients.  Shapes as for the hybrid forward.
 *
 * tw_hybrid_bwd_dh (dense-to-hybrid): hy_du, hy_dz [M][P] fp32 at the stored
 * entries of sparse rows; bk_du, bk_dz [R_max][N] bf16 for backup slots (on
 * the matrix cores, from the row's stored bf16 bk_g, bk_u).  events: [0]
 * before, [1] after the sparse-row kernel, [2] after the backup GEMM.
 */
tw_status tw_hybrid_bwd_dh(const uint16_t *dy, const uint16_t *wd, int M, int K, int N, int P,
                           float l1, const float *hy_g, const float *hy_u, const int32_t *hy_idx,
                           const int32_t *hy_cnt, const uint8_t *route, const int32_t *bk_rows,
                           const int32_t *bk_count, int R_max, const uint16_t *bk_g,
                           const uint16_t *bk_u, float *hy_du, float *hy_dz, uint16_t *bk_du,
                           uint16_t *bk_dz, void *stream, void *const *events);

/*
 * tw_hybrid_bwd_dx (hybrid-to-dense): dx [M][K] fp32 for sparse rows and the
 * listed backup rows (the latter on the matrix cores: one GEMM whose
 * reduction runs over both products, du W_u^T then dz W_g^T, split into
 * partial tiles that the sparse-row kernel, which runs after it, sums in
 * split order).  ws_bytes >= tw_hybrid_bwd_dx_workspace_bytes(R_max) (ws
 * may be NULL when that is 0).  events: [0] before, [1] after the backup
 * GEMM, [2] after the sparse-row kernel.
 */
size_t tw_hybrid_bwd_dx_workspace_bytes(int R_max);
tw_status tw_hybrid_bwd_dx(const uint16_t *wg_t, const uint16_t *wu_t, int M, int K, int N, int P,
                           const float *hy_du, const float *hy_dz, const int32_t *hy_idx,
                           const int32_t *hy_cnt, const uint8_t *route, const int32_t *bk_rows,
                           const int32_t *bk_count, int R_max, const uint16_t *bk_du,
                           const uint16_t *bk_dz, float *dx, void *ws, size_t ws_bytes,
                           void *stream, void *const *events);

/*
 * tw_hybrid_bwd_dw: the three weight gradients, every row of dwg_t, dwu_t
 * and dwd written.  The sparse rows' part goes through the hybrid transpose
 * kept in the workspace: their stored entries grouped by hidden column in
 * ascending row order, so each column's gradient is a fixed-order sum; the
 * listed backup rows' part is three products on the matrix cores
 * (dwd += bk_h^T dy, dwu_t += bk_du^T x, dwg_t += bk_dz^T x over the backup
 * slots).  Results are bit-identical run to run.  ws_bytes >=
 * tw_hybrid_bwd_dw_workspace_bytes(M, K, N, P, R_max) (about 16 M P +
 * 4 R_max K bytes; 0 for a shape this call rejects).  events: [0] before,
 * [1] after the
 * transpose, [2] after the sparse rows' gradients, [3] after the backup
 * rows' products.
 */
size_t tw_hybrid_bwd_dw_workspace_bytes(int M, int K, int N, int P, int R_max);
tw_status tw_hybrid_bwd_dw(const uint16_t *x, const uint16_t *dy, int M, int K, int N, int P,
                           const float *hy_h, const float *hy_du, const float *hy_dz,
                           const int32_t *hy_idx, const int32_t *hy_cnt, const uint8_t *route,
                           const int32_t *bk_rows, const int32_t *bk_count, int R_max,
                           const uint16_t *bk_h, const uint16_t *bk_du, const uint16_t *bk_dz,
                           float *dwg_t, float *dwu_t, float *dwd, void *ws, size_t ws_bytes,
                           void *stream, void *const *events);

/*
 * Layer norm over the last dimension, forward.  For every row m, in fp32:
 *     z = x[m] (+ add[m]),  mean = sum(z) / K,
 *     rstd = 1 / sqrt(sum((z - mean)^2) / K + eps),
 *     y[m] = (z - mean) * rstd * gamma (+ beta).
 * add is the block's output joining the residual stream; its sum with x is
 * stored to `sum` (rounded to x's type; the norm uses the unrounded sum).
 *
 *   x       [M] rows of K, x_stride elements apart (x_stride >= K), bf16 or fp32
 *   add     [M][K]   bf16 or fp32, or NULL
 *   gamma   [K]      fp32
 *   beta    [K]      fp32, or NULL
 *   sum     [M][K]   x's type, or NULL; only with add
 *   y       [M][K]   bf16 or fp32
 *   mean, rstd [M]   fp32, or NULL: what tw_layernorm_bwd reads
 *
 * sum may be x itself (when x_stride == K) or, of the same type, add.
 * K from 1 to 16384, any value (odd rows included); eps >= 0.  A row holding
 * a NaN or an infinity gives NaN.  events: [0] before, [1] after the kernel.
 */
tw_status tw_layernorm_fwd(const void *x, int x_type, int64_t x_stride, const void *add,
                           int add_type, const float *gamma, const float *beta, float eps, int M,
                           int K, void *sum, void *y, int y_type, float *mean, float *rstd,
                           void *stream, void *const *events);

/*
 * Layer norm, backward: with n = (x - mean) rstd (x: the forward's z as
 * stored, in `sum` if there was an add) and t = dy gamma,
 *     dx = rstd (t - sum(t) / K - n sum(t n) / K) (+ dres),
 *     dgamma = sum over rows of dy n,   dbeta = sum over rows of dy.
 * dres is the gradient that reaches z past the norm (the residual stream's).
 *
 *   dy      [M][K]  bf16 or fp32;  x as in the forward;  mean, rstd [M]
 *   dres    [M][K]  dx's type, or NULL
 *   dx      [M][K]  bf16 or fp32
 *   dgamma, dbeta [K] fp32, each may be NULL
 * The row sums of dgamma and dbeta are taken in a fixed order (bit-identical
 * run to run).  M = 0 writes zeros to dgamma and dbeta.  ws_bytes >=
 * tw_layernorm_bwd_workspace_bytes(M, K) (ws may be NULL when dgamma and
 * dbeta both are).  events: [0] before, [1] after the row kernel, [2] after
 * the sum of dgamma and dbeta.
 */
size_t tw_layernorm_bwd_workspace_bytes(int M, int K);
tw_status tw_layernorm_bwd(const void *dy, int dy_type, const void *x, int x_type,
                           int64_t x_stride, const float *gamma, const float *mean,
                           const float *rstd, const void *dres, int M, int K, void *dx,
                           int dx_type, float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                           void *stream, void *const *events);

/*
 * 8-bit integer rows.  A row r of K values is held as int8 q and one fp32
 * scale, with top = max |r|:
 *     scale = top / 127,   q = round(r * ((1 / top) * 127))
 * (each operation rounded to fp32; halves go to the even code),
 * so |q| <= 127 and q * scale approximates r within scale / 2.  A row with
 * top < 2^-100 gets scale 0 and q = 0; a row holding a NaN or an infinity
 * gets scale NaN and q = 0 (every product with it is NaN).  Weights take the
 * same form: row n of w [N][K] holds the weights of output channel n, so
 * tw_quant_rows over a transposed weight matrix gives one scale per channel.
 *
 * tw_quant_rows quantises the rows of x (bf16 or fp32, x_stride elements
 * apart): q [M][K] int8, scale [M] fp32.  K from 1 to 65536.
 * tw_layernorm_quant quantises the layer norm of x (+ add) (arguments as in
 * tw_layernorm_fwd, K up to 16384; the normed row is not rounded in
 * between).  events: [0] before, [1] after the kernel.
 */
tw_status tw_quant_rows(const void *x, int x_type, int64_t x_stride, int M, int K, int8_t *q,
                        float *scale, void *stream, void *const *events);
tw_status tw_layernorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                             int add_type, const float *gamma, const float *beta, float eps, int M,
                             int K, void *sum, int8_t *q, float *scale, void *stream,
                             void *const *events);

/*
 * Products of 8-bit integer rows, summed exactly in 32-bit integers:
 *     p(w)[m][n] = (sum_k q[m][k] w[n][k]) * x_scale[m] * w_scale[n]
 * tw_quant_linear:  y = p(w) (+ bias)            (y [M][N])
 * tw_quant_gateup:  h = ReLU(p(wg)) * p(wu)      (h [M][N])
 * The input x is either rows of int8 (x_type TW_INT8, contiguous, with their
 * scales in x_scale) or bf16 or fp32 rows x_stride elements apart (x_scale
 * NULL), which the call quantises first as tw_quant_rows does.  With gamma,
 * tw_quant_gateup quantises their layer norm instead, as tw_layernorm_quant
 * does without add (gamma, beta NULL: no norm).
 *
 *   w, wg, wu [N][K] int8;  w_scale, g_scale, u_scale [N] fp32
 *   bias  [N] fp32, or NULL
 *   y, h  [M][N] bf16 or fp32
 *   ws    ws_bytes >= tw_quant_workspace_bytes(M, K); may be NULL for int8 x
 * K a positive multiple of 16, at most 65536 (16384 with gamma); M and N up
 * to 2^24, and at most 2^37 outputs.  Results are bit-identical run to run.
 * Calls of up to 4 float rows norm and quantise them in the product's kernel,
 * which sums a norm in another order than tw_layernorm_quant: with gamma, a
 * code whose value lies half way between two (within fp32 rounding) may
 * differ between a row in a call of few rows and the same row among many.
 * events: [0] before, [1] after the quantisation, [2] after the product
 * (events[0] and [1] are recorded together where one kernel does both).
 */
size_t tw_quant_workspace_bytes(int M, int K);
tw_status tw_quant_linear(const void *x, int x_type, int64_t x_stride, const float *x_scale,
                          const int8_t *w, const float *w_scale, const float *bias, int M, int K,
                          int N, void *y, int y_type, void *ws, size_t ws_bytes, void *stream,
                          void *const *events);
tw_status tw_quant_gateup(const void *x, int x_type, int64_t x_stride, const float *x_scale,
                          const float *gamma, const float *beta, float eps, const int8_t *wg,
                          const float *g_scale, const int8_t *wu, const float *u_scale, int M,
                          int K, int N, void *h, int h_type, void *ws, size_t ws_bytes,
                          void *stream, void *const *events);

/*
 * RMS norm over the last dimension.  For every row m, in fp32:
 *     z = x[m] (+ add[m]),  rstd = 1 / sqrt(sum(z^2) / K + eps),
 *     y[m] = z * rstd * gamma.
 * Arguments, types and limits as in tw_layernorm_fwd (there is no mean and no
 * beta); tw_rmsnorm_quant quantises the unrounded norm as tw_layernorm_quant
 * does.  A row holding a NaN gives NaN; one holding an infinity gives NaN there
 * and zeros elsewhere.  events: [0] before, [1] after the kernel.
 */
tw_status tw_rmsnorm_fwd(const void *x, int x_type, int64_t x_stride, const void *add,
                         int add_type, const float *gamma, float eps, int M, int K, void *sum,
                         void *y, int y_type, float *rstd, void *stream, void *const *events);
tw_status tw_rmsnorm_quant(const void *x, int x_type, int64_t x_stride, const void *add,
                           int add_type, const float *gamma, float eps, int M, int K, void *sum,
                           int8_t *q, float *scale, void *stream, void *const *events);

/*
 * RMS norm, backward: with n = x rstd (x: the forward's z as stored, in `sum`
 * if there was an add) and t = dy gamma,
 *     dx = rstd (t - n sum(t n) / K) (+ dres),   dgamma = sum over rows of dy n.
 * Arguments, order of the sums, workspace and events as in tw_layernorm_bwd.
 */
size_t tw_rmsnorm_bwd_workspace_bytes(int M, int K);
tw_status tw_rmsnorm_bwd(const void *dy, int dy_type, const void *x, int x_type, int64_t x_stride,
                         const float *gamma, const float *rstd, const void *dres, int M, int K,
                         void *dx, int dx_type, float *dgamma, void *ws, size_t ws_bytes,
                         void *stream, void *const *events);

/*
 * Dense gated FFN, forward: y = h W_d with h = act(g) u, g = x W_g, u = x W_u
 * (act: a tw_act).  h is rounded to bf16 between the two products; sums are
 * fp32.  (With TW_RELU also tw_ffn_fwd, which says where it is the faster one.)
 *
 *   x       [M] rows of K bf16, x_stride elements apart
 *   wg_t, wu_t, wd [N][K] bf16, as above
 *   g, u    [M][N]  bf16, each may be NULL: the projections before the
 *                   activation, which tw_gated_ffn_bwd reads
 *   y       [M][K]  bf16 or fp32
 *
 * K, N and x_stride multiples of 8, K and N at most 2^20, x_stride from K to
 * 2^20; M at most 2^24.  ws_bytes >= tw_gated_ffn_workspace_bytes(M, K, N) (0
 * for sizes the call rejects; ws may be NULL when M is 0).  Results are
 * bit-identical run to run.  events: [0] before, [1] after h, [2] after y.
 */
size_t tw_gated_ffn_workspace_bytes(int M, int K, int N);
tw_status tw_gated_ffn_fwd(const uint16_t *x, int64_t x_stride, const uint16_t *wg_t,
                           const uint16_t *wu_t, const uint16_t *wd, int act, int M, int K, int N,
                           uint16_t *g, uint16_t *u, void *y, int y_type, void *ws,
                           size_t ws_bytes, void *stream, void *const *events);

/*
 * Dense gated FFN, backward, from dy = dLoss/dy and the forward's g and u:
 *     dh = dy W_d^T,  du = dh act(g),  dz = dh u act'(g),  h = act(g) u,
 *     dx = dz W_g^T + du W_u^T,
 *     dwg_t = dz^T x,  dwu_t = du^T x,  dwd = h^T dy.
 * dz, du and h are rounded to bf16 between the products; sums are fp32.
 *
 *   dy      [M][K]  bf16;  x as in the forward;  g, u [M][N] bf16
 *   dx      [M][K]  bf16 or fp32, or NULL
 *   dwg_t, dwu_t, dwd [N][K] bf16 or fp32, all three or none (NULL)
 *
 * The weight gradients are computed after dx, which therefore must not overlap x
 * or dy where they are wanted; nor may it overlap wg_t or wu_t, a weight gradient
 * x or dy, or one output another.
 *
 * Limits as in the forward.  With M = 0 the weight gradients are zeros.
 * ws_bytes >= tw_gated_ffn_bwd_workspace_bytes(M, K, N).  events: [0] before,
 * [1] after dz, du and h, [2] after dx, [3] after the weight gradients.
 */
size_t tw_gated_ffn_bwd_workspace_bytes(int M, int K, int N);
tw_status tw_gated_ffn_bwd(const uint16_t *dy, const uint16_t *x, int64_t x_stride,
                           const uint16_t *wg_t, const uint16_t *wu_t, const uint16_t *wd, int act,
                           const uint16_t *g, const uint16_t *u, int M, int K, int N, void *dx,
                           int dx_type, void *dwg_t, void *dwu_t, void *dwd, int dw_type, void *ws,
                           size_t ws_bytes, void *stream, void *const *events);

/*
 * Softmax cross entropy of an output projection: with the logits l = x w^T
 * (never stored) and a row's target t,
 *     lse[m] = log sum_v exp(l[m][v]),   loss[m] = lse[m] - l[m][t].
 * A row whose target lies outside [0, V) is left out: its loss is 0 (lse is
 * there all the same).
 *
 *   x       [M] rows of K bf16, x_stride elements apart
 *   w       [V][K] bf16
 *   target  [M]  32- or 64-bit integers (target_type TW_INT32 or TW_INT64)
 *   loss, lse [M] fp32
 *
 * K and x_stride multiples of 8, K at most 2^20, x_stride from K to 2^20, V up
 * to 2^24, M up to 2^24.  ws_bytes >= tw_linear_ce_workspace_bytes(M, K, V).
 * Results are bit-identical run to run.  events: [0] before, [1] after the
 * kernels.
 */
size_t tw_linear_ce_workspace_bytes(int M, int K, int V);
tw_status tw_linear_ce_fwd(const uint16_t *x, int64_t x_stride, const uint16_t *w,
                           const void *target, int target_type, int M, int K, int V, float *loss,
                           float *lse, void *ws, size_t ws_bytes, void *stream,
                           void *const *events);

/*
 * Its gradient, for dloss[m] = dLoss/dloss[m] (fp32) and the forward's lse:
 *     D[m][v] = dloss[m] (exp(l[m][v] - lse[m]) - [v = t]),
 *     dx = D w,   dw = D^T x
 * (rows of D of rows that are left out, or whose dloss is 0, are 0 whatever they
 * hold; their x enters dw times 0, so for dw it has to be finite).  The logits
 * are computed again, a piece of the vocabulary at a time, and D is rounded to
 * bf16; sums are fp32.
 *
 *   dx      [M][K]  bf16 or fp32, or NULL;  dw [V][K] bf16 or fp32, or NULL
 *
 * dx must not overlap w, nor x where dw is wanted; nor dw x, dx or, unless it is
 * w itself in its type, w.
 *
 * Limits as in the forward.  With M = 0, dw is zeros.  ws_bytes >=
 * tw_linear_ce_bwd_workspace_bytes(M, K, V): a piece of D (at most 512 MB, or
 * 256 columns) and fp32 parts of dx and of a piece's dw.
 */
size_t tw_linear_ce_bwd_workspace_bytes(int M, int K, int V);
tw_status tw_linear_ce_bwd(const float *dloss, const uint16_t *x, int64_t x_stride,
                           const uint16_t *w, const void *target, int target_type,
                           const float *lse, int M, int K, int V, void *dx, int dx_type, void *dw,
                           int dw_type, void *ws, size_t ws_bytes, void *stream,
                           void *const *events);

/*
 * Gradient norm and clipping over `count` buffers of n[i] elements each:
 *     norm = sqrt(sum over all elements of g^2),
 *     out = g min(1, max_norm / (norm + eps)).
 * The arrays g, n, g_type, out and out_type are read on the host during the
 * call.  A buffer's type is TW_BF16 or TW_F32; its address is aligned to its
 * type and may be NULL where n is 0.  out[i] may be g[i] itself (of the same
 * type); otherwise no output may overlap another buffer of the call, and no
 * buffer the norm or what is needed of the workspace, nor these each other: all
 * checked.  A norm that is NaN makes every output NaN; with max_norm 0 the
 * factor is otherwise 0, whatever the norm.  n[i] at most 2^34; count at most
 * 2^20.  ws_bytes >= tw_grad_norm_workspace_bytes(count, n), which is 0 where
 * one of these is exceeded (a negative n[i], which the calls reject, counts as
 * no elements there).
 * Squares are summed in fp32, in a fixed order (bit-identical run to run).
 * norm: one fp32, aligned to 4.  events of tw_grad_norm: [0] before, [1] after;
 * of tw_grad_clip: [0] before, [1] after the squares' sums, [2] after.
 */
size_t tw_grad_norm_workspace_bytes(int count, const int64_t *n);
tw_status tw_grad_norm(int count, const void *const *g, const int64_t *n, const int *g_type,
                       float *norm, void *ws, size_t ws_bytes, void *stream, void *const *events);
tw_status tw_grad_clip(int count, const void *const *g, const int64_t *n, const int *g_type,
                       void *const *out, const int *out_type, float max_norm, float eps,
                       float *norm, void *ws, size_t ws_bytes, void *stream, void *const *events);

#ifdef __cplusplus
}
#endif

#endif /* TW_H */
