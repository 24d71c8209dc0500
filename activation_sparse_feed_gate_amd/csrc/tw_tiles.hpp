// tw_tiles.hpp -- bf16 products over output tiles for the dense training and
// loss kernels: C[m][n] = sum over r < R of A(m, r) B(n, r), each operand
// stored with r contiguous (kRows: one row per m or n) or with r as its row
// index (kCols), any sizes whose rows are whole 16-byte pieces, and what
// becomes of an output given by an epilogue.
//
// Edges: every lane of a direct load that would touch something outside the
// operand (a row past it, a 16-byte piece past a row's end, a reduction row
// past R) is sent past the descriptor's end instead, where it reads zeros.
// Both operands are zero there, so no NaN next to an operand enters a sum.
#pragma once

#include "tw_gemm.hpp"
#include "tw_rows.hpp"

namespace tw {

enum { kRows = 0, kCols = 1 };

// A byte offset past every descriptor made here (at most 256 rows of 2^20
// elements).
constexpr uint32_t kPastEnd = 1u << 30;
constexpr int64_t kMaxStride = 1 << 20;  // elements between operand rows

// The operands of one launch.  What a[1], b[1], ... are is the kernel's: a
// second weight matrix next to b[0] (NB = 2), further terms of the sum (SEG),
// or other products of the same shape (blockIdx.y).
struct TileArgs {
    const uint16_t *a[3], *b[3];
    int64_t lda, ldb;  // elements between rows
    int M, N, R;
    int splits;        // parts of the reduction (blockIdx.z)
};

// 32 rows x 16 reduction elements of a kCols region (32 reduction rows of 128
// columns, 256 bytes each, chunk c of row r at c ^ 4 (r % 4)): lane l receives
// column col32 + l % 32 at reduction rows 16 s + 8 (l / 32) ..+7, the layout
// of frag().
__device__ __forceinline__ u32x4 col_frag(const char *region, int col32, int s, int lane) {
    const int g4 = (lane >> 4) & 3, i16 = lane & 15;
    const int c0 = col32 + 16 * (g4 & 1) + 4 * (i16 & 3);
    i16x4 v[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int row = 16 * s + 8 * (g4 >> 1) + 4 * hh + (i16 >> 2);
        const uint32_t off = row * 256 + (((c0 >> 3) ^ (4 * (row & 3))) << 4) + (c0 & 7) * 2;
        v[hh] = lds_tr16((const lds_i16x4 *)(region + off));
    }
    const u32x2 lo = __builtin_bit_cast(u32x2, v[0]);
    const u32x2 hi = __builtin_bit_cast(u32x2, v[1]);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// ----------------------------- 128 x 128 tiles ------------------------------
// 8 waves of 64 x 32 outputs, stages of 32 reduction elements in the ring of
// kloop_pipelined.  Every operand's share of a stage is 8 KB, one direct load
// of a wave.
constexpr int kRingBM = 128, kRingBN = 128, kRingS = 4;
constexpr int kRingPart = 128 * kPRow;  // one operand of one stage

// One operand's direct loads: rows (of the kRows layout) or columns i0 ..
// i0 + 127, reduction elements 32 kt ..+31 of `R`.
template <int L>
struct RingOperand {
    const uint16_t *p;
    int64_t ld;
    int I, R, i0;
    uint32_t voff;
    int red;  // reduction element of the lane's piece within a stage
    __device__ __forceinline__ RingOperand(const uint16_t *p_, int64_t ld_, int I_, int R_, int i0_,
                                           int wave, int lane)
        : ld(ld_), I(I_), R(R_), i0(i0_) {
        if constexpr (L == kRows) {
            const int sr = 16 * wave + (lane >> 2);
            p = p_ + i0 * ld;
            red = 8 * ((lane & 3) ^ swz(sr));
            voff = i0 + sr < I ? (uint32_t)sr * (uint32_t)ld * 2 + red * 2 : kPastEnd;
        } else {
            const int row = 4 * wave + (lane >> 4);
            const int col = 8 * ((lane & 15) ^ (4 * (row & 3)));
            p = p_ + i0;
            red = row;
            voff = i0 + col < I ? (uint32_t)row * (uint32_t)ld * 2 + col * 2 : kPastEnd;
        }
    }
    __device__ __forceinline__ void issue(int kt, char *dst) const {
        const uint32_t v = kt * kPK + red < R ? voff : kPastEnd;
        if constexpr (L == kRows) {
            // (a row's last 16-byte piece lies in its padding where R is no
            // multiple of 8)
            const int rows = min(kRingBM, I - i0);
            const rsrc_t d = make_rsrc(p, ((uint64_t)(rows - 1) * ld + ((R + 7) & ~7)) * 2);
            dma16(d, v, kt * kPK * 2, dst);
        } else {
            // the descriptor moves with the stage: an operand may be larger
            // than 32-bit offsets reach
            const int rows = max(1, min(kPK, R - kt * kPK));
            const int cols = (min(kRingBN, I - i0) + 7) & ~7;
            const rsrc_t d = make_rsrc(p + (int64_t)kt * kPK * ld,
                                       ((uint64_t)(rows - 1) * ld + cols) * 2);
            dma16(d, v, 0, dst);
        }
    }
};

// An epilogue has a Row (what it keeps of one row m: row(m)) and
//   quad(z, split, row, m, n, v, u)   takes the outputs n .. n + 3 of row m (u:
//                                     those of the second weight matrix), or,
// where it reduces over the columns (kStats),
//   most(row, n, v), add(row, n, v)   two passes over a lane's outputs,
//   join<L>(row)                      lanes l and l ^ L hold one row,
//   put(row, lds, w, r)               wave column w's part of the tile's row r,
//   finish<W>(lds, r, m, cb)          joins the W wave columns.
template <int LA, int LB, int NB, int SEG, class Epi>
__global__ __launch_bounds__(512) void ring_tiles_kernel(TileArgs p, Epi epi) {
    constexpr int NI = 1 + NB, STAGE = NI * kRingPart;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int l32 = lane & 31;
    const int z = blockIdx.y, sp = blockIdx.z;
    int rb, cb;
    xcd_tile(blockIdx.x, (p.M + kRingBM - 1) / kRingBM, (p.N + kRingBN - 1) / kRingBN, rb, cb);
    const int m0 = rb * kRingBM, n0 = cb * kRingBN;
    const int KT = (p.R + kPK - 1) / kPK;

    const RingOperand<LA> a0(p.a[SEG == 2 ? 0 : z], p.lda, p.M, p.R, m0, wave, lane);
    const RingOperand<LB> b0(p.b[SEG == 2 || NB == 2 ? 0 : z], p.ldb, p.N, p.R, n0, wave, lane);
    const RingOperand<LA> a1(SEG == 2 ? p.a[1] : p.a[0], p.lda, p.M, p.R, m0, wave, lane);
    const RingOperand<LB> b1(SEG == 2 || NB == 2 ? p.b[1] : p.b[0], p.ldb, p.N, p.R, n0, wave, lane);
    auto issue = [&](int kt, char *st) {
        char *d = st + wave * 1024;
        if (SEG == 2 && kt >= KT) {
            a1.issue(kt - KT, d);
            b1.issue(kt - KT, d + kRingPart);
        } else {
            a0.issue(kt, d);
            b0.issue(kt, d + kRingPart);
            if constexpr (NB == 2) b1.issue(kt, d + 2 * kRingPart);
        }
    };
    auto fragment = [&](auto layout, const char *part, int row, int s) {
        if constexpr (decltype(layout)::value == kRows) return frag(part, row, s, lane);
        else return col_frag(part, row, s, lane);
    };
    f32x16 acc[NB][2];
#pragma unroll
    for (int o = 0; o < NB; ++o)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[o][i] = f32x16{};
    u32x4 fa[2][2], fb[2][NB];
    auto load = [&](const char *st, int s, int buf) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            fa[buf][i] = fragment(std::integral_constant<int, LA>{}, st, wm * 64 + 32 * i, s);
#pragma unroll
        for (int o = 0; o < NB; ++o)
            fb[buf][o] = fragment(std::integral_constant<int, LB>{}, st + (1 + o) * kRingPart,
                                  wn * 32, s);
    };
    // the second operand's rows are the instruction's first ones, so that a
    // lane holds 4 consecutive n of one m
    auto mma = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int o = 0; o < NB; ++o) acc[o][i] = mfma32(fb[buf][o], fa[buf][i], acc[o][i]);
    };
    const int all = SEG * KT, per = (all + p.splits - 1) / p.splits;
    kloop_pipelined<kRingS, NI>(min(sp * per, all), min(sp * per + per, all), smem, STAGE, issue,
                                load, mma);
    if constexpr (Epi::kStats) __syncthreads();  // finish() uses the ring's memory
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + wm * 64 + 32 * i + l32;
        typename Epi::Row row = epi.row(min(m, p.M - 1));
        auto each = [&](auto f) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 v, u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = acc[0][i][4 * q + e];
                    u[e] = acc[NB - 1][i][4 * q + e];
                }
                f(n0 + wn * 32 + 8 * q + 4 * (lane >> 5), v, u);
            }
        };
        if constexpr (Epi::kStats) {
            each([&](int n, f32x4 v, f32x4) { epi.most(row, n, v); });
            each([&](int n, f32x4 v, f32x4) { epi.add(row, n, v); });
            epi.template join<32>(row);
            if (lane < 32) epi.put(row, smem, wn, wm * 64 + 32 * i + l32);
        } else {
            if (m < p.M)
                each([&](int n, f32x4 v, f32x4 u) { epi.quad(z, sp, row, m, n, v, u); });
        }
    }
    if constexpr (Epi::kStats) {
        __syncthreads();
        if (tid < kRingBM && m0 + tid < p.M) epi.template finish<4>(smem, tid, m0 + tid, cb);
    }
}

template <int LA, int LB, int NB, int SEG, class Epi>
hipError_t launch_ring(const TileArgs &p, const Epi &epi, int groups, hipStream_t s) {
    constexpr auto kernel = &ring_tiles_kernel<LA, LB, NB, SEG, Epi>;
    constexpr int lds = kRingS * (1 + NB) * kRingPart;
    const hipError_t e = lds_limit_once<kernel>(lds);
    if (e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)p.M + kRingBM - 1) / kRingBM *
                          (((int64_t)p.N + kRingBN - 1) / kRingBN);
    if (tiles == 0) return hipSuccess;
    kernel<<<dim3((unsigned)tiles, groups, p.splits), 512, lds, s>>>(p, epi);
    return hipGetLastError();
}

// ------------------------------- epilogues ----------------------------------
__device__ __forceinline__ void store4(void *p, int type, int64_t at, f32x4 v) {
    if (type == TW_T_F32) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at) = v;
    } else {
        u32x2 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + at) = w;
    }
}
__device__ __forceinline__ f32x4 load4_bf16(const uint16_t *p, int64_t at) {
    const u32x2 w = *reinterpret_cast<const u32x2 *>(p + at);
    return f32x4{bf_lo(w[0]), bf_hi(w[0]), bf_lo(w[1]), bf_hi(w[1])};
}

// Outputs stored as they are: to out[z] in its type, or, where the reduction
// is taken in parts, to part[split] in fp32 (added to what is there with
// `more`: a later piece of the reduction).  ld is a multiple of 8, and N of 4.
struct EpiStore {
    static constexpr bool kStats = false;
    void *out[3];
    int type;
    float *part;  // or null
    int more;
    int M, N;
    struct Row {};
    __device__ Row row(int) const { return {}; }
    __device__ __forceinline__ void quad(int z, int split, Row &, int m, int n, f32x4 v,
                                         f32x4) const {
        if (n >= N) return;
        const int64_t at = (int64_t)m * N + n;
        if (part) {
            f32x4 *q = reinterpret_cast<f32x4 *>(part + (int64_t)split * M * N + at);
            *q = more ? *q + v : v;
        } else {
            store4(z == 0 ? out[0] : z == 1 ? out[1] : out[2], type, at, v);
        }
    }
};

// out = the sum of the parts, in their order.
template <int T>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float *__restrict__ part, int splits,
                                                        int64_t n, void *__restrict__ out) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= n) return;
    f32x4 v = *reinterpret_cast<const f32x4 *>(part + at);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(part + s * n + at);
    store4(out, T, at, v);
}
inline hipError_t launch_sum_parts(const float *part, int splits, int64_t n, void *out, int type,
                                   hipStream_t s) {
    if (n == 0) return hipSuccess;
    const unsigned grid = (unsigned)((n / 4 + 255) / 256);
    if (type == TW_T_F32) sum_parts_kernel<TW_T_F32><<<grid, 256, 0, s>>>(part, splits, n, out);
    else sum_parts_kernel<TW_T_BF16><<<grid, 256, 0, s>>>(part, splits, n, out);
    return hipGetLastError();
}

}  // namespace tw
