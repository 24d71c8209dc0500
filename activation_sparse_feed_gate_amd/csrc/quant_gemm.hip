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
// Three kernels.  A few rows: fragments straight into registers, K split over
// the waves of a workgroup.  Hundreds of rows: tiles over the direct-to-LDS
// ring of tw_gemm.hpp, whose 64-byte stage rows hold 64 int8 elements (the 16
// bytes a lane feeds to v_mfma_i32_32x32x32_i8 lie where
// v_mfma_f32_32x32x16_bf16 has its 8 bf16).  Thousands: 256 x 256 tiles with
// stages of whole 128-byte lines, refilled in parts.
#include <type_traits>

#include "tw_gemm.hpp"
#include "tw_norm_quant.hpp"
#include "tw_quant_rules.hpp"
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
__device__ __forceinline__ float scaled(int s0, int s1, float xs, float ws0, float ws1) {
    const float v = (float)s0 * xs * ws0;
    if constexpr (NB == 1) return v;
    // a NaN gate stays NaN
    return (v < 0.0f ? 0.0f : v) * ((float)s1 * xs * ws1);
}
template <int NB>
__device__ __forceinline__ float finish(int s0, int s1, float xs, float ws0, float ws1, float b) {
    const float v = scaled<NB>(s0, s1, xs, ws0, ws1);
    return NB == 1 ? v + b : v;
}

__device__ __forceinline__ void put(char *y, int type, size_t o, float v) {
    if (type == TW_T_F32) reinterpret_cast<float *>(y)[o] = v;
    else reinterpret_cast<uint16_t *>(y)[o] = (uint16_t)pack_bf16(v, v);
}

// ------------------------------- a few rows --------------------------------
// 16 weight rows a workgroup, MB blocks of 16 token rows; wave w of 8 takes
// the 64-element steps w, w + 8, ... of K, and the waves' sums meet in LDS.
// The time of such a product is the latency of its loads and then the weight
// stream, so a wave issues the loads of PF of its steps (weights and token
// rows) at once, after the few small ones that are waited for first: loads
// complete in order.
//
// The token rows come either as int8, read per fragment from memory (every
// workgroup reads them, mostly from L2), or, for up to 4 rows, as floats that
// each workgroup norms and quantises itself into LDS while its weights are on
// their way: that saves the quantiser's launch and the wait between the two.
constexpr int kFewWaves = 8;
constexpr int kFewPad = 16;  // bytes between quantised rows in LDS: shifts banks

struct FewRows {
    const char *x;
    int64_t x_stride;
    const float *gamma, *beta;  // gamma null: no norm
    float eps;
};

// Fused rows: WPR waves share a token row, 8 / WPR rows at once; a thread
// holds up to 2 vectors of 8 elements of its row, so 1, 2 and 4 rows may be of
// 8192, 4096 and 2048 elements (8 rows, a wave each, of 1024 only).  Measured (us,
// K x N, fused against a quantiser's launch of its own): one row, linear 5632 x
// 2048 5.3, 7.5, gateup 8.9, 10.5; two, 2048 x 5632 4.4, 6.6, gateup 7.3, 9.4, 4096 x
// 4096 6.7, 7.8, gateup 11.8, 11.5; four, 2048 x 5632 4.7, 6.8, gateup 8.3, 9.7.  The
// two sum a norm in different orders, so a code half way between two may
// differ between a call of few rows and one of many.
constexpr int kFusedRows = 4;
__host__ __device__ constexpr int fused_row_waves(int M) { return M <= 1 ? 8 : M <= 2 ? 4 : 2; }
constexpr int fused_max_k(int M) { return fused_row_waves(M) * kWave * 16; }

// The norm and quantisation of one row by WPR waves (all 8 waves take part;
// a group past the last row repeats it).  The loads are issued by the
// constructor, the rest is done by run().
template <int TX, int WPR, int VEC>
struct FusedRow {
    const FewRows &f;
    const int K, t;
    Vec8<TX> raw[VEC];
    Vec8<TW_T_F32> g[VEC], b[VEC];
    int slot = 0;

    __device__ __forceinline__ int at(int v) const { return 8 * (v * WPR * kWave + t); }
    __device__ __forceinline__ FusedRow(const FewRows &f_, int m, int K_)
        : f(f_), K(K_), t(threadIdx.x & (WPR * kWave - 1)) {
        const char *row = f.x + (int64_t)m * f.x_stride * type_bytes(TX);
#pragma unroll
        for (int v = 0; v < VEC; ++v) raw[v] = load8_whole<TX>(row, at(v), K);
        if (f.gamma) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                g[v] = load8_whole<TW_T_F32>((const char *)f.gamma, at(v), K);
        }
        if (f.beta) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                b[v] = load8_whole<TW_T_F32>((const char *)f.beta, at(v), K);
        }
    }
    // op over the row's WPR waves of their (uniform) values v; two slots of
    // red in turn, so one barrier each is enough (see RowReduce)
    template <typename Op>
    __device__ __forceinline__ float over_waves(float v, float *red, Op op) {
        float *r = red + slot * kFewWaves;
        slot ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) r[wave] = v;
        __syncthreads();
        const int first = wave & ~(WPR - 1);
        float a = r[first];
#pragma unroll
        for (int w = 1; w < WPR; ++w) a = op(a, r[first + w]);
        return a;
    }
    __device__ __forceinline__ void run(float *red, int8_t *dst, float *scale) {
        auto add = [](float a, float b) { return a + b; };
        float z[VEC][8];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            unpack8<TX>(raw[v], z[v]);
            if (at(v) >= K) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[v][i] = 0.0f;
            }
        }
        if (f.gamma) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < VEC; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += z[v][i];
            const float mean = over_waves(wave_sum(s), red, add) / K;
            s = 0.0f;
#pragma unroll
            for (int v = 0; v < VEC; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[v][i] = at(v) < K ? z[v][i] - mean : 0.0f;  // K is a multiple of 8
                    s += z[v][i] * z[v][i];
                }
            const float rstd = 1.0f / sqrtf(over_waves(wave_sum(s), red, add) / K + f.eps);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float gf[8], bf[8];
                unpack8<TW_T_F32>(g[v], gf);
                if (f.beta) unpack8<TW_T_F32>(b[v], bf);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[v][i] = at(v) < K ? z[v][i] * rstd * gf[i] + (f.beta ? bf[i] : 0.0f) : 0.0f;
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(z[v][i]) & 0x7fffffffu);
        // magnitudes compare as unsigned integers, NaN above all (row_scale)
        top = __float_as_uint(
            over_waves(__uint_as_float(wave_max(top)), red, [](float a, float b) {
                return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
            }));
        const RowScale rs = row_scale(top);
        if (t == 0) *scale = rs.scale;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (at(v) < K) *reinterpret_cast<u32x2 *>(dst + at(v)) = quant8(z[v], rs.inv);
    }
};

// MB x NC blocks of 16 token rows by 16 weight rows a workgroup.  WPR, VEC:
// of the fused rows (0: int8 rows).
// Waves a SIMD the registers leave room for: the loads in flight, the sums
// and a fused row's vectors take most of them (128 registers at 4 waves, 256
// at 2).
constexpr int few_waves(int loads, int sums, int vec) {
    return 4 * (loads + sums + 6 * vec) <= 72 ? 4 : 2;
}

template <int TX, int WPR, int VEC, int MB, int NC, int NB, int PF>
__global__ __launch_bounds__(kFewWaves *kWave,
                             few_waves(PF *(NB * NC + (TX == TW_T_INT8 ? MB : 0)), NB *NC *MB,
                                       VEC))
void quant_few_kernel(QArgs a, FewRows f, int R) {
    constexpr bool kFused = TX != TW_T_INT8;
    static_assert(!kFused || MB == 1, "fused rows: one block of 16");
    extern __shared__ __attribute__((aligned(16))) char few_smem[];
    // [NB][NC][MB][waves][64] sums; then, fused, the rows' bytes
    i32x4 *part = reinterpret_cast<i32x4 *>(few_smem);
    int8_t *rows = reinterpret_cast<int8_t *>(part + NB * NC * MB * kFewWaves * kWave);
    __shared__ float red[2 * kFewWaves], row_scales[kFusedRows];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * R, m0 = blockIdx.y * (16 * MB);
    const int l16 = lane & 15, kc = (lane >> 4) * 16;
    const int steps = (a.K + 63) / 64;

    const int8_t *wr[NB][NC], *xr[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            wr[b][c] = a.w[b].w + (size_t)min(n0 + min(16 * c + l16, R - 1), a.N - 1) * a.K;
    u32x4 wf[PF][NB][NC], xf[PF][kFused ? 1 : MB];
    // The wave's steps p0 .. p0 + PF - 1 of K (step p is p * 8 + wave): chunks
    // past a row's end read its first bytes instead, and the weights' are
    // then cleared (K is a multiple of 16: a chunk is in or out).
    auto fetch = [&](int p0) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            // no branch around loads that are in flight while the fused rows
            // are waited for: the wait could not count them
            if (!kFused && (p0 + p) * kFewWaves + wave >= steps) continue;
            const int k = ((p0 + p) * kFewWaves + wave) * 64 + kc;
            const int kk = k < a.K ? k : 0;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < NC; ++c) wf[p][b][c] = ld16(wr[b][c] + kk);
            if constexpr (!kFused) {
#pragma unroll
                for (int i = 0; i < MB; ++i) xf[p][i] = ld16(xr[i] + kk);
            }
        }
    };
    if constexpr (kFused) {
        const int m = min(wave / WPR, a.M - 1);
        const int stride = a.K + kFewPad;
        FusedRow<TX, WPR, VEC> row(f, m, a.K);
        __builtin_amdgcn_sched_barrier(0);
        fetch(0);
        __builtin_amdgcn_sched_barrier(0);
        row.run(red, rows + m * stride, row_scales + m);
        __syncthreads();
        xr[0] = rows + min(l16, a.M - 1) * stride;
    } else {
#pragma unroll
        for (int i = 0; i < MB; ++i) xr[i] = a.q + (size_t)min(m0 + i * 16 + l16, a.M - 1) * a.K;
        fetch(0);
    }
    i32x4 acc[NB][NC][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < MB; ++i) acc[b][c][i] = i32x4{};
    for (int p0 = 0; p0 * kFewWaves + wave < steps; p0 += PF) {
        if (p0) fetch(p0);
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            if ((p0 + p) * kFewWaves + wave >= steps) continue;
            const int k = ((p0 + p) * kFewWaves + wave) * 64 + kc;
            const bool in = k < a.K;
            if constexpr (kFused)
                xf[p][0] = *reinterpret_cast<const u32x4 *>(xr[0] + (in ? k : 0));
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const u32x4 w = in ? wf[p][b][c] : u32x4{};
#pragma unroll
                    for (int i = 0; i < MB; ++i)
                        acc[b][c][i] = mfma16_i8(w, xf[p][i], acc[b][c][i]);
                }
        }
    }
    // what the outputs need besides the sums: the lane's 4 columns, on their
    // way while the sums meet (a wave finishes blocks wave, wave + 8, ...)
    constexpr int kBlocks = MB * NC;
    auto place = [&](int b, int blk, int w) {
        return ((b * kBlocks + blk) * kFewWaves + w) * kWave + lane;
    };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < MB; ++i) part[place(b, c * MB + i, wave)] = acc[b][c][i];
    if (wave >= kBlocks) return __syncthreads();
    float ws[NB][4], bias[4], xs;
    auto columns = [&](int blk) {
        const int nl = n0 + 16 * (blk / MB) + 4 * (lane >> 4);
        const int m = m0 + 16 * (blk % MB) + l16;
        xs = kFused ? 0.0f : a.x_scale[min(m, a.M - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = min(nl + j, a.N - 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) ws[b][j] = a.w[b].scale[n];
            bias[j] = NB == 1 && a.bias ? a.bias[n] : 0.0f;
        }
    };
    columns(wave);
    __syncthreads();
    for (int blk = wave; blk < kBlocks; blk += kFewWaves) {
        if (blk != wave) columns(blk);
        const int nl = n0 + 16 * (blk / MB) + 4 * (lane >> 4);
        const int m = m0 + 16 * (blk % MB) + l16;
        i32x4 s[2] = {};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) s[b] += part[place(b, blk, w)];
        if (m >= a.M) continue;
        if (kFused) xs = row_scales[m];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (nl + j < min(n0 + R, a.N))
                put(a.y, a.y_type, (size_t)m * a.N + nl + j,
                    finish<NB>(s[0][j], s[1][j], xs, ws[0][j], ws[NB - 1][j], bias[j]));
    }
}

template <int TX, int WPR, int VEC, int MB, int NC, int NB, int PF>
hipError_t launch_few(const QArgs &a, const FewRows &f, hipStream_t s) {
    constexpr auto kernel = &quant_few_kernel<TX, WPR, VEC, MB, NC, NB, PF>;
    constexpr int sums = NB * NC * MB * kFewWaves * kWave * 16;
    constexpr int most = TX == TW_T_INT8 ? 0 : kFusedRows * (VEC * WPR * kWave * 8 + kFewPad);
    const hipError_t e = lds_limit_once<kernel>(sums + most);
    if (e != hipSuccess) return e;
    const int lds = sums + (TX != TW_T_INT8 ? a.M * (a.K + kFewPad) : 0);
    const int R = MB == 1 ? few_rows(a.M, a.N, NC, TX != TW_T_INT8) : 16 * NC;
    const dim3 grid((a.N + R - 1) / R, (a.M + 16 * MB - 1) / (16 * MB));
    kernel<<<grid, kFewWaves * kWave, lds, s>>>(a, f, R);
    return hipGetLastError();
}

// Loads of a wave in flight: its whole share of K where that is short, else
// as many steps as the registers hold.
template <int TX, int WPR, int VEC, int MB, int NC, int NB>
hipError_t launch_few(const QArgs &a, const FewRows &f, hipStream_t s) {
    constexpr int loads = NB * NC + (TX == TW_T_INT8 ? MB : 0);
    constexpr int most = 36 / loads < 12 ? 36 / loads : 12;
    const int share = (a.K + kFewWaves * 64 - 1) / (kFewWaves * 64);
    if constexpr (most > 2)
        if (share <= 2) return launch_few<TX, WPR, VEC, MB, NC, NB, 2>(a, f, s);
    if constexpr (most > 4)
        if (share <= 4) return launch_few<TX, WPR, VEC, MB, NC, NB, 4>(a, f, s);
    return launch_few<TX, WPR, VEC, MB, NC, NB, most>(a, f, s);
}

template <int TX, int WPR, int NB>
hipError_t launch_fused(const QArgs &a, const FewRows &f, hipStream_t s) {
    const bool one = few_fits(a.M, a.N, 1, 1);
    if (a.K <= WPR * kWave * 8)
        return one ? launch_few<TX, WPR, 1, 1, 1, NB>(a, f, s)
                   : launch_few<TX, WPR, 1, 1, 2, NB>(a, f, s);
    return one ? launch_few<TX, WPR, 2, 1, 1, NB>(a, f, s)
               : launch_few<TX, WPR, 2, 1, 2, NB>(a, f, s);
}

template <int TX, int NB>
hipError_t launch_fused(const QArgs &a, const FewRows &f, hipStream_t s) {
    if (a.M == 1) return launch_fused<TX, fused_row_waves(1), NB>(a, f, s);
    if (a.M == 2) return launch_fused<TX, fused_row_waves(2), NB>(a, f, s);
    return launch_fused<TX, fused_row_waves(kFusedRows), NB>(a, f, s);
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
            const bool past = last && kt * kPRow + chunk[j] * 16 >= a.K;
            if (row0 < BM) dma16(rx, past ? kOutside : voff[j], soff, dst);
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

// ------------------------------ large tiles --------------------------------
// 256 token rows by 256 weight rows (gateup: 128 of each matrix) a workgroup
// of 8 waves, 64 x 128 outputs each; a workgroup a CU, walking tiles, the next
// tile's first stages on their way while a tile is written.  Measured on
// 8-bit normal values, from session to session: 16384 x 8192 x 2048 207 to 238 us, 2.3
// to 2.65 POP/s (the 64-byte ring with 256 x 256 tiles 285), gateup 16384 x 2048 x
// 8192 445 to 489 us, 2.25 to 2.47 POP/s (607); on zeros, which draw less power,
// 173 and 380 us in all of them.
//
// What bounds this product is the stream of operands from L2 into LDS (loads
// alone: 150 us of the 248 that the ring above took for 16384 x 8192 x 2048
// on zeros), and a load instruction that covers whole 128-byte lines moves up
// to 1.7 times the bytes of one that covers 64-byte pieces.  So a stage is
// 128 bytes of each row, two stages fill 128 KB of LDS, and the loads of the
// stage after next enter a stage's slot in two parts, as soon as no wave reads
// what they replace:
//
//   step   matrix instructions   fragments read              loads into this slot
//   0      A x B0                B1 of this stage
//   -- X: this stage's B2, B3 have landed; its A, B0, B1 are in registers
//   1      A x B1                B2                          A, B0, B1
//   2      A x B2                B3
//   -- Y: the next stage's A, B0, B1 have landed; all of this one is in registers
//   3      A x B3                A and B0 of the next stage  B2, B3
//
// with A the wave's 64 token rows and B0 .. B3 its blocks of 32 weight rows.
// Every load has one and a half stages of arithmetic to land
// in (one barrier a stage, with the whole slot refilled at Y and waited for at
// the next Y, left the loads idle for their latency in every stage).  A step
// is 16 matrix instructions, 512 cycles with those of the SIMD's other wave, so
// its reads are there when the next step begins; the last step reads each
// fragment of the next A as soon as it has used its own.
//
// 16 x 16 x 64 instructions, because power sets the pace on real operands: out
// of registers, on 8-bit normal values, they sustain 3.7 POP/s and 32 x 32 x 32 ones
// 3.3 (4.9 and 4.8 on zeros; peak_probe.hip); in this kernel, in one session, 218 and
// 236 us.  Both halves of a block of weight rows run on a token fragment before
// the next one's: 1% over the other way.
constexpr int kWideRow = 128;           // bytes of a row in a stage
constexpr int kWideStage = 512 * kWideRow;
constexpr int kWideOut = 32 * kWideRow;  // a wave's outputs on their way to memory
constexpr int kWideLds = 2 * kWideStage + 8 * kWideOut;

// 16-byte chunk c of row r lives at chunk c ^ ((r >> 1) & 7): rows are half of
// LDS's 256 bytes of banks, so 16 consecutive rows of one logical chunk fall
// on 16 different bank groups.
__device__ __forceinline__ int wide_swz(int r) { return (r >> 1) & 7; }

template <int NB>
__global__ __launch_bounds__(512) void quant_wide_kernel(QArgs a, int row_regions) {
    constexpr int BN = 256 / NB;  // weight rows of each matrix
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int l16 = lane & 15;
    const int KT = (a.K + kWideRow - 1) / kWideRow;
    const int nbm = (a.M + 255) / 256, nbn = (a.N + BN - 1) / BN;
    const int tiles = nbm * nbn;
    settle_scalars(a.x_scale, a.w[0].scale, a.w[1].scale, a.bias, a.y, a.y_type, a.M, a.N);

    // the tile being loaded: its origin and descriptors
    int m0, n0;
    rsrc_t rx, r0, r1;
    auto at_tile = [&](int t) {
        int rb, cb;
        if (row_regions == 8) xcd_tile<8>(t, nbm, nbn, rb, cb);
        else if (row_regions == 4) xcd_tile<4>(t, nbm, nbn, rb, cb);
        else xcd_tile<2>(t, nbm, nbn, rb, cb);
        m0 = rb * 256;
        n0 = cb * BN;
        const int mr = min(256, a.M - m0), nr = min(BN, a.N - n0);  // rows in this tile
        rx = make_rsrc(a.q + (size_t)m0 * a.K, (uint64_t)mr * a.K);
        r0 = make_rsrc(a.w[0].w + (size_t)n0 * a.K, (uint64_t)nr * a.K);
        r1 = NB == 2 ? make_rsrc(a.w[1].w + (size_t)n0 * a.K, (uint64_t)nr * a.K) : r0;
    };
    // A load of a wave fetches 8 whole lines, rows 64 g + 8 wave ..+7 of group g
    // of 64: groups 0 .. 3 of x, then of the weights.  Rows past the matrix lie
    // past the descriptor's end and read zeros.
    const int lrow = 8 * wave + (lane >> 3);
    int chunk = (lane & 7) ^ wide_swz(lrow);
    uint32_t v0 = (uint32_t)lrow * a.K + chunk * 16;
    const uint32_t v64 = 64u * a.K;
    auto slot = [&](int kt, int g) {
        return smem + (kt & 1) * kWideStage + (64 * g + 8 * wave) * kWideRow;
    };
    // weight group of pair p (0: blocks 0, 1; 1: blocks 2, 3), i = 0, 1.
    // linear: groups 0, 1 are the first 128 columns' blocks, 2, 3 the others';
    // gateup: 0, 1 are the gate's rows, 2, 3 the up's
    auto load_b = [&](int kt, int p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = NB == 1 ? 2 * i + p : 2 * p + i;
            dma16(NB == 2 && p ? r1 : r0, v0 + (NB == 1 ? g : i) * v64, kt * kWideRow,
                  slot(kt, 4 + g));
        }
    };
    auto load_ab = [&](int kt) {
        // chunks past a row's end read zeros in x, so what the weights'
        // chunks hold there does not matter
        const bool past = kt * kWideRow + chunk * 16 >= a.K;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            dma16(rx, past ? kOutside : v0 + g * v64, kt * kWideRow, slot(kt, g));
        load_b(kt, 0);
    };
    constexpr int kAB = 6, kB = 2;  // loads of a wave in each part
    // Fragment of 16 rows from `row` on, one 64-byte sub-step of a stage: lane
    // l holds row l % 16, 16 bytes from 64 s + 16 (l / 16) on.
    auto read = [&](int kt, int row, int s) {
        const int c = (4 * s + (lane >> 4)) ^ wide_swz(l16);
        return lds_ld16(smem + (kt & 1) * kWideStage, (row + l16) * kWideRow + (c << 4));
    };
    // weight rows of block j; gateup: blocks 0, 1 of the gate, 2, 3 of the up
    auto b_row = [&](int j) {
        return NB == 1 ? wn * 128 + j * 32 : (j >> 1) * 128 + wn * 64 + (j & 1) * 32;
    };
    u32x4 fa[2][4], fb[2][2][2];  // [sub-step][16 rows], [register set][sub-step][16 rows]
    auto read_b = [&](int kt, int j) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) fb[j & 1][s][h] = read(kt, 256 + b_row(j) + 16 * h, s);
    };
    // [16 token rows][16 weight rows]: register r of a block is token row l16,
    // weight row 4 (lane / 16) + r
    i32x4 acc[4][8];
    auto mma = [&](int j, int s, int i, int h) {
        acc[i][2 * j + h] = mfma16_i8(fb[j & 1][s][h], fa[s][i], acc[i][2 * j + h]);
    };
    // The scheduling barriers keep each step's reads ahead of its matrix
    // instructions.
    auto step = [&](int kt, int j) {
        read_b(kt, j + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) mma(j, s, i, h);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto last_step = [&](int kt) {
        read_b(kt + 1, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mma(3, s, i, 0);
                mma(3, s, i, 1);
                __builtin_amdgcn_sched_barrier(0);
                fa[s][i] = read(kt + 1, wm * 64 + i * 16, s);
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    auto load_first = [&] {
        load_ab(0);
        load_b(0, 1);
        if (KT > 1) {
            load_ab(1);
            load_b(1, 1);
        }
    };
    // Scales of the tile at (m0, n0): of the lane's token rows (l16 of each
    // block), and of two of the wave's 128 weight rows, lane and 64 + lane (the
    // outputs of a lane are of other weight rows).
    struct Scales {
        float x[4], w[2];
    };
    // output column of the wave's weight row 64 p + c
    auto col = [&](int base, int p, int c) {
        return base + (NB == 1 ? wn * 128 + 64 * p : wn * 64) + c;
    };
    auto load_scales = [&] {
        Scales c;
#pragma unroll
        for (int i = 0; i < 4; ++i) c.x[i] = a.x_scale[min(m0 + wm * 64 + i * 16 + l16, a.M - 1)];
#pragma unroll
        for (int p = 0; p < 2; ++p)
            c.w[p] = a.w[NB == 2 ? p : 0].scale[min(col(n0, p, lane), a.N - 1)];
        return c;
    };
    at_tile(blockIdx.x);
    Scales sc = load_scales();
    load_first();
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int mt = m0, nt = n0;  // this tile; m0, n0 move on to the next below
        // (Opaque copies: what the loads below need of these is then computed
        // where it is used, not kept in registers through the k-loop.)
        asm volatile("" : "+v"(chunk), "+v"(v0));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = i32x4{};
        // What may be outstanding besides the loads below is younger: the last
        // tile's stores, 8 to 32 of them.  They are among the operations that the
        // counts below leave outstanding, so from the second tile on these waits
        // hold for more of the loads than stage 0's first six.
        if (KT > 1) wait_vmcnt<kB + kAB + kB>();
        else wait_vmcnt<kB>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[s][i] = read(0, wm * 64 + i * 16, s);
        read_b(0, 0);
        int kt = 0;
        for (; kt + 2 < KT; ++kt) {
            step(kt, 0);
            wait_vmcnt<kAB + kB>();
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();  // X
            load_ab(kt + 2);
            step(kt, 1);
            step(kt, 2);
            wait_vmcnt<kB + kAB>();
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();  // Y
            load_b(kt + 2, 1);
            last_step(kt);
        }
        if (kt + 1 < KT) {
            step(kt, 0);
            wait_vmcnt<kAB + kB>();
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();
            step(kt, 1);
            step(kt, 2);
            wait_vmcnt<kB>();
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();
            last_step(kt);
            ++kt;
        }
        step(kt, 0);
        wait_vmcnt<0>();
        __builtin_amdgcn_s_barrier();
        step(kt, 1);
        step(kt, 2);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) mma(3, s, i, h);

        // The next tile's scales and first loads (after every wave has read its
        // last fragments) are on their way while this tile is written.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        Scales next = sc;
        if (t + (int)gridDim.x < tiles) {
            at_tile(t + gridDim.x);
            next = load_scales();
            load_first();
        }
        __builtin_amdgcn_sched_barrier(0);

        // Outputs go through 4 KB of LDS a wave, 32 token rows of 128 bytes at a
        // time, so that they are stored in whole lines: a lane holds 4 consecutive
        // columns of one row.  (The lane's number is read anew: the addresses
        // below, computed ahead of the tile loop, would fill the registers that
        // the k-loop needs.)
        char *out = smem + 2 * kWideStage + wave * kWideOut;
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int lr = ln & 15, lc = 4 * (ln >> 4);
        // The columns' scales go through it first, from the lanes that hold
        // them to every lane's 4 columns of each block.
        f32x4 w[8];
#pragma unroll
        for (int p = 0; p < 2; ++p) reinterpret_cast<float *>(out)[64 * p + ln] = sc.w[p];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = *reinterpret_cast<const f32x4 *>(out + (16 * j + lc) * 4);
        auto write_out = [&](auto type) {
            constexpr bool kF32 = decltype(type)::value == TW_T_F32;
            constexpr int ES = kF32 ? 4 : 2;
            constexpr int JP = kF32 ? 2 : 4;  // blocks of 16 columns in 128 bytes
#pragma unroll
            for (int j0 = 0; j0 < 8 / NB; j0 += JP)
#pragma unroll
                for (int i0 = 0; i0 < 4; i0 += 2) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = i0; i < i0 + 2; ++i)
#pragma unroll
                        for (int j = j0; j < j0 + JP; ++j) {
                            const int ju = NB == 2 ? 4 + j : j;
                            float v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = scaled<NB>(acc[i][j][e], acc[i][ju][e], sc.x[i], w[j][e],
                                                  w[ju][e]);
                            // (read behind the next tile's first loads, which each
                            // wait here includes: 16384 x 1024 x 4096 110 us with a
                            // bias, 80 without; 16384 x 8192 x 2048 237 and 227)
                            if (NB == 1 && a.bias) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    v[e] += a.bias[min(col(nt, 0, 16 * j + lc + e), a.N - 1)];
                            }
                            const int r = 16 * (i - i0) + lr;
                            const int byte = (16 * (j - j0) + lc) * ES;
                            char *p = out + r * kWideRow + (((byte >> 4) ^ wide_swz(r)) << 4) +
                                      (byte & 15);
                            if constexpr (kF32)
                                *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
                            else
                                *reinterpret_cast<u32x2 *>(p) =
                                    u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                        }
                    const int n = col(nt, 0, 16 * j0 + (ln & 7) * (16 / ES));
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int r = it * 8 + (ln >> 3);
                        const u32x4 v =
                            lds_ld16(out, r * kWideRow + (((ln & 7) ^ wide_swz(r)) << 4));
                        const int m = mt + wm * 64 + i0 * 16 + r;
                        if (m >= a.M) continue;
                        char *p = a.y + ((size_t)m * a.N + n) * ES;
                        if (n + 16 / ES <= a.N) {
                            *reinterpret_cast<u32x4_any *>(p) = v;
                        } else {
#pragma unroll
                            for (int e = 0; e < 16 / ES; ++e) {
                                if (n + e >= a.N) continue;
                                if constexpr (kF32)
                                    reinterpret_cast<uint32_t *>(p)[e] = v[e];
                                else
                                    reinterpret_cast<uint16_t *>(p)[e] =
                                        (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                            }
                        }
                    }
                }
        };
        if (a.y_type == TW_T_F32) write_out(std::integral_constant<int, TW_T_F32>{});
        else write_out(std::integral_constant<int, TW_T_BF16>{});
        sc = next;
    }
}

template <int NB>
hipError_t launch_wide(const QArgs &a, hipStream_t s) {
    constexpr auto kernel = &quant_wide_kernel<NB>;
    const hipError_t e = lds_limit_once<kernel>(kWideLds);
    if (e != hipSuccess) return e;
    constexpr int BN = 256 / NB;
    const int64_t nbm = ((int64_t)a.M + 255) / 256, nbn = ((int64_t)a.N + BN - 1) / BN;
    const int64_t tiles = nbm * nbn;
    kernel<<<(unsigned)(tiles < 256 ? tiles : 256), 512, kWideLds, s>>>(
        a, wide_row_regions(nbm, nbn));
    return hipGetLastError();
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
    auto tiles = [&](int bm, int bn) {
        return ((int64_t)a.M + bm - 1) / bm * (((int64_t)a.N + bn - 1) / bn);
    };
    // Up to 64 rows per 128 columns or so: the smallest block whose grid fits.
    // Measured (us, K = 2048, N = 1001; K = 5632, N = 2048; K = 2048, N = 5632):
    //   32 rows   16x16 3.9, 7.7, 8.1   32x16 4.9, 10.1, 8.1   32x32 5.9, 13.1, 6.5
    //   64 rows   16x16 4.3, 12.4, 13.4   32x16 5.0, 10.2, 10.8   64x32 8.2, 18.6, 9.1
    //   128 rows  32x16 5.3, 18.9, 19.6   32x32 6.0, 13.1, 14.0   tiles 8.3, 17.2, 9.3
    // Where none fits, 64 x 64 tiles, unless they would leave most CUs idle
    // and the rows are few (N = 8192, K = 2048, 16 rows: 16x32 5.7, tiles 8.6;
    // N = 14336, K = 4096: 15.9 against 13.0).
    const FewRows none{};
    if (a.M <= 16 && few_fits(a.M, a.N, 1, 1))
        return launch_few<TW_T_INT8, 0, 0, 1, 1, NB>(a, none, s);
    if (a.M <= 16 && (few_fits(a.M, a.N, 1, 2) || a.M <= 4 || tiles(64, 64) < 192))
        return launch_few<TW_T_INT8, 0, 0, 1, 2, NB>(a, none, s);
    if (few_fits(a.M, a.N, 1, 1)) return launch_few<TW_T_INT8, 0, 0, 1, 1, NB>(a, none, s);
    if (few_fits(a.M, a.N, 2, 1)) return launch_few<TW_T_INT8, 0, 0, 2, 1, NB>(a, none, s);
    if (few_fits(a.M, a.N, 2, 2)) return launch_few<TW_T_INT8, 0, 0, 2, 2, NB>(a, none, s);
    // 64 x 32: up to 64 rows (128 rows: 18.6 against 17.2 at K = 5632)
    if (a.M <= 64 && few_fits(a.M, a.N, 4, 2))
        return launch_few<TW_T_INT8, 0, 0, 4, 2, NB>(a, none, s);
    // Larger tiles do more arithmetic per byte loaded, so the largest whose
    // grid occupies about half the chip or more.  Measured (us, linear; tiles
    // of 256 x 256, 128 x 128, 64 x 64):
    //   K = 2048, N = 5632    512 rows 25.1, 15.5, 17.6   1536 rows 27.0, 35.8, 40.4
    //   K = 5632, N = 2048   1024 rows 56.8, 29.2, 28.3   4096 rows 58.9, 66.4, 99.1
    //   K = 1024, N = 4096    512 rows 15.7, 10.9, 8.7    2048 rows 17.7, 18.2, 22.2
    if (tiles(256, 256 / NB) >= 120) return launch_wide<NB>(a, s);
    if constexpr (NB == 1) {
        if (tiles(128, 128) >= 144) return launch_tiles<128, 128, 2, 4, 4, 1>(a, s);
    } else {
        if (tiles(128, 64) >= 144) return launch_tiles<128, 64, 4, 2, 4, 2>(a, s);
    }
    return launch_tiles<64, 64, 2, 2, 4, NB>(a, s);
}

template <int NB>
hipError_t launch_fused(const QArgs &a, const QuantRows &r, hipStream_t s) {
    const FewRows f{(const char *)r.x, r.x_stride, r.gamma, r.beta, r.eps};
    if (r.x_type == TW_T_F32) return launch_fused<TW_T_F32, NB>(a, f, s);
    return launch_fused<TW_T_BF16, NB>(a, f, s);
}

}  // namespace

bool quant_fused(int M, int K) {
    return M >= 1 && M <= kFusedRows && K <= fused_max_k(M);
}

hipError_t launch_quant_linear(const int8_t *q, const float *x_scale, const QuantRows *rows,
                               const int8_t *w, const float *w_scale, const float *bias, int M,
                               int K, int N, void *y, int y_type, hipStream_t s) {
    const QArgs a{q, x_scale, {{w, w_scale}, {w, w_scale}}, bias, M, K, N, (char *)y, y_type};
    return rows ? launch_fused<1>(a, *rows, s) : launch_product<1>(a, s);
}

hipError_t launch_quant_gateup(const int8_t *q, const float *x_scale, const QuantRows *rows,
                               const int8_t *wg, const float *g_scale, const int8_t *wu,
                               const float *u_scale, int M, int K, int N, void *h, int h_type,
                               hipStream_t s) {
    const QArgs a{q, x_scale, {{wg, g_scale}, {wu, u_scale}}, nullptr, M, K, N, (char *)h, h_type};
    return rows ? launch_fused<2>(a, *rows, s) : launch_product<2>(a, s);
}

}  // namespace tw
