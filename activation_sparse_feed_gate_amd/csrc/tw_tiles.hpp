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
#include "tw_train.hpp"

namespace tw {

enum { kRows = 0, kCols = 1 };

// A byte offset past every descriptor made here: they hold at most 256 rows of
// kTileRowMost elements (2^29 bytes), or of a tile's rows those that are in the operand,
// whose buffer is no larger (the loss's D, linear_ce.hip).
constexpr uint32_t kPastEnd = 1u << 30;
static_assert(uint64_t(256) * kTileRowMost * 2 < kPastEnd, "");
// Elements between rows of a kRows operand up to which the offset of any of a tile's 256
// rows, from kPastEnd too, stays within 32 bits: one that wrapped would be read.
constexpr int64_t kTileStrideMost = 1 << 22;
static_assert(uint64_t(256) * kTileStrideMost * 2 + kPastEnd < (uint64_t(1) << 32), "");

// A tile of an output: its product, its first row and column, its size, and its place
// among the parts (-1: it takes the whole reduction).
struct Place {
    int z, m0, n0, rows, cols, part;
};

// The operands of one launch.  What a[1], b[1], ... are is the kernel's: a
// second weight matrix next to b[0] (NB = 2), a second term of the sum (SEG =
// 2: the reduction runs over both), or other products of the same shape.
struct TileArgs {
    const uint16_t *a[3], *b[3];
    int64_t lda, ldb;  // elements between rows
    int M, N, R;
    int splits = 1;  // parts of the reduction, where it is taken in parts
    int full = 0;    // the first tiles, which take the reduction whole
    int groups = 1;  // products of the same shape: a[z], b[z]
    int64_t ldb_last = 0;  // ldb of the third product
};

// Where one of an epilogue's outputs goes: rows of ld elements, the first
// `cols` columns stored (a multiple of 8); p null: nowhere.  add: to what is
// there (fp32).
struct Dest {
    void *p;
    int type;
    int64_t ld;
    int cols;
    bool add;
};

__device__ __forceinline__ void store4(void *p, int type, int64_t at, f32x4 v) {
    if (type == TW_T_F32) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at) = v;
    } else {
        u32x2 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + at) = w;
    }
}
// The 8 outputs of row m from column n on (n < cols).
__device__ __forceinline__ void put_out(const Dest &d, int m, int n, const float (&v)[8]) {
    if (!d.p) return;
    const int64_t at = m * d.ld + n;
    if (d.type == TW_T_F32) {
        f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(d.p) + at);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const f32x4 o{v[e], v[e + 1], v[e + 2], v[e + 3]};
            q[e / 4] = d.add ? q[e / 4] + o : o;
        }
    } else {
        st16(static_cast<uint16_t *>(d.p) + at,
             u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7])});
    }
}

// An epilogue has kWalk, the row blocks that walk_tile takes at a time, and, for a row m of
// the tile, a Raw (what it loads: raw(m); of(l): lane l's) and a Row made of it, and
//   Fetched, fetch(m, n)         what it loads of the 8 columns n .. n + 7 of row m,
//                                ahead of
//   values<W, ALL>(row, fetched, n, v, u, o)  which makes its kOuts outputs of columns
//                                n .. n + W - 1 from those of the product (u: of the
//                                second weights); ALL: these columns are all within N,
//   dest(o, place)               says where output o of a tile goes,
//   stores(place)                how many stores a wave makes of a tile inside the
//                                product (0, 8, 16, 24, 32 or 48), or,
// where it reduces over the columns (kStats),
//   most<W, ALL>(row, n, v), add<W, ALL>(row, n, v)   two passes over a lane's columns,
//   join<L>(row)                            lanes l and l ^ L hold one row,
//   put(row, m, cb)                         the row's block cb of 128 columns.
struct NoRaw {
    __device__ NoRaw of(int) const { return {}; }
};
struct NoFetch {};

// --------------------------------- tiles ------------------------------------
// 64 WR x 256 outputs (NB = 2: 64 WR x 128 of each weight matrix) a workgroup of 2 WR
// waves, 64 x 128 outputs each (wave row wm, wave column wn); a workgroup a CU,
// walking tiles, the next tile's first stages on their way while a tile is
// written.  WR is 4, or 2 where a product has too few tiles for the chip.  A stage is
// 64 reduction elements, 128 bytes of each of the tile's 64 WR + 256 rows; two stages
// fill 128 KB of LDS (WR = 2: 96 KB), and the loads of the stage after next enter a
// stage's slot in two parts, as soon as no wave reads what they replace:
//
//   step   matrix instructions   fragments read              loads into this slot
//   0      A x B0                B1 of this stage
//   -- X: this stage's B2, B3 have landed; its A, B0, B1 are in registers
//   1      A x B1                B2                          A, B0, B1
//   2      A x B2                B3
//   -- Y: the next stage's A, B0, B1 have landed; all of this one is in registers
//   3      A x B3                A and B0 of the next stage  B2, B3
//
// with A the wave's 64 rows and B0 .. B3 its blocks of 32 columns.  A step is 16
// matrix instructions of 16 x 16 x 32, so its reads are there when the next one
// begins.
//
// A kRows operand lies in LDS as rows of 128 bytes, chunk c of row r at c ^ ((r
// >> 1) & 7): 16 consecutive rows of one chunk fall on 16 different bank groups.
// A kCols operand is regions of 64 reduction rows of 128 columns (256
// bytes), read with the transposing ds_read_b64_tr_b16; chunk c of row r lies at c ^
// 2 f(r), f = r % 4 + 4 (r / 8 % 2): the 8 rows that 32 lanes read, two
// chunks of each, fill the 16 chunks of a row of banks once (no conflicts counted).
// Loads of either cover whole 128-byte lines.
//
// A wave's 64 x 128 outputs are 128 accumulator registers a lane, which leave room for a
// second set of B's fragments; they read 48 KB of LDS for 128 matrix instructions (24 a
// stage, for 64).  128 x 128 a wave would read a third less, but did not fit: its
// accumulators spill.
// What bounds a large product is power: on operands of zeros, where nothing toggles,
// 16384 x 8192 x 2048 and its like run at 1740 to 1830 TFLOP/s (kRows x kRows), on
// normal ones at 1330 to 1390; kRows x kCols 1650 and 1300.  16 x 16 x 32
// instructions draw less than 32 x 32 x 16 ones for the same work (alone on normal
// operands: 1957 and 1770 TFLOP/s).
constexpr int kWideCols = 256, kWideK = 64;
constexpr int kWideLine = 128;                    // bytes of a kRows row in a stage
constexpr int kWideRegion = kWideK * 256;         // 128 columns of a kCols operand
constexpr int kWideOut = 4096;                    // a wave's outputs on their way to memory
constexpr int kWideGrid = 256;                    // workgroups: one a CU
// WR wave rows of 64, two wave columns of 128.
template <int WR>
struct Wide {
    static constexpr int kWaves = 2 * WR, kThreads = 64 * kWaves, kRowsOf = 64 * WR;
    // a stage's operands
    static constexpr int kA = kRowsOf * kWideLine, kB = kWideCols * kWideLine;
    static constexpr int kSlot = kA + kB, kBytes = 2 * kSlot + kWaves * kWideOut;
    static constexpr int kPair = 8 / WR;          // loads of a wave for two column blocks
    static constexpr int kFirst = 4 + kPair;      // ... for A and two column blocks
};

__device__ __forceinline__ int line_swz(int r) { return (r >> 1) & 7; }

// wait_vmcnt<N + more> (63 at most), `more` a multiple of 8 up to 48.
template <int N>
__device__ __forceinline__ void wait_besides(int more) {
    switch (more) {
    case 8: wait_vmcnt<N + 8>(); break;
    case 16: wait_vmcnt<N + 16>(); break;
    case 24: wait_vmcnt<N + 24>(); break;
    case 32: wait_vmcnt<N + 32>(); break;
    case 48: wait_vmcnt<(N + 48 < 63 ? N + 48 : 63)>(); break;
    default: wait_vmcnt<N>(); break;
    }
}

// Which tile or part an XCD works on.  Workgroups are dealt to the 8 XCDs in turn (index
// t % 8), so item t is number shared(t) of T: each XCD gets a run of neighbours, and what
// they share comes into its L2 once.  (Measured against tiles dealt in turn, where the
// grid does not divide into rectangles: gate and up 777 x 1000 x 2728 24.1 -> 21.4 us; parts
// of dx 777 x 2048 x 5632 77 -> 52 us.)
__device__ __forceinline__ int shared(int t, int T) {
    const int x = t & 7, more = T & 7;
    return x * (T >> 3) + min(x, more) + (t >> 3);
}
// Tile number `tile` of a grid: G row blocks at a time, column block by column block, so
// that 32 neighbours share G blocks of A and 32 / G of B.  G is 8 for products stored as
// they are and for the loss, 4 where wide rows of bf16 are written (and read): dh 8192 x
// 1024 x 4096 130 -> 108 us with 4, gate and up 4096 x 2048 x 8192 with g and u 220 ->
// 212, the loss's backward pass 8192 x 2048 x 32768 2486 -> 2452; dx 8192 x 1024 x 4096
// 121 with 8, 128 with 4.
template <int G>
__device__ __forceinline__ void walk_tile(int tile, int nbm, int nbn, int &bm, int &bn) {
    const int group = tile / (G * nbn), gm = min(G, nbm - group * G);
    const int at = tile - group * G * nbn;
    bm = group * G + at % gm;
    bn = at / gm;
}

template <int WR, int LA, int LB, int NB, int SEG, class Epi>
__global__ __launch_bounds__(Wide<WR>::kThreads) void wide_tiles_kernel(TileArgs p, Epi epi) {
    using W = Wide<WR>;
    static_assert(NB == 1 || (LB == kRows && SEG == 1), "two weight matrices: rows, one term");
    constexpr int BM = W::kRowsOf, BN = kWideCols / NB;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int l16 = lane & 15;
    const int KT = (p.R + kWideK - 1) / kWideK;  // stages of one term
    const int all = SEG * KT, per = (all + p.splits - 1) / p.splits;
    const int nbm = (p.M + BM - 1) / BM, nbn = (p.N + BN - 1) / BN;
    // Items: the first p.full tiles whole, then the others in p.splits parts.
    const int tiles = nbm * nbn, rest = tiles * p.groups - p.full;
    const int items = p.full + rest * p.splits;

    // The item being loaded: its tile, product, part of the reduction.
    int m0, n0, z, part, k0, kn;
    int64_t ldb;
    rsrc_t ra[SEG], rb[SEG == 2 ? 2 : NB];  // (kRows)
    // Lane's place in a load.  kRows: rows 8 wave ..+7 of 16 WR, a chunk of 8 lanes
    // each; kCols: reduction rows 4 wave ..+3 of 8 WR, 16 chunks each.
    const int lrow = 8 * wave + (lane >> 3);
    const int chunk = (lane & 7) ^ line_swz(lrow);
    const int crow = 4 * wave + (lane >> 4);
    const int cchunk = (lane & 15) ^ (2 * ((crow & 3) | ((crow >> 3) & 1) << 2));
    uint32_t va[2], vb[2];  // offsets; kCols: of the two regions
    auto at_item = [&](int t) {
        int tile;
        part = -1;
        k0 = 0;
        kn = all;
        if (t < p.full) {
            tile = shared(t, p.full);
        } else {
            part = shared(t - p.full, rest * p.splits);
            const int sp = part / rest;
            tile = p.full + part - sp * rest;
            k0 = min(sp * per, all);
            kn = min(k0 + per, all) - k0;
        }
        z = tile / tiles;
        int bm, bn;
        walk_tile<Epi::kWalk>(tile - z * tiles, nbm, nbn, bm, bn);
        ldb = z == 2 ? p.ldb_last : p.ldb;
        m0 = bm * BM;
        n0 = bn * BN;
        const int pad = (p.R + 7) & ~7;  // a row's last piece may lie in its padding
        if constexpr (LA == kRows) {
            const int rows = min(BM, p.M - m0);
#pragma unroll
            for (int g = 0; g < SEG; ++g)
                ra[g] = make_rsrc((SEG == 2 ? p.a[g] : z == 0 ? p.a[0] : z == 1 ? p.a[1] : p.a[2]) +
                                      m0 * p.lda,
                                  ((uint64_t)(rows - 1) * p.lda + pad) * 2);
            va[0] = (uint32_t)lrow * (uint32_t)p.lda * 2 + chunk * 16;
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = 128 * q + 8 * cchunk;
                va[q] = m0 + c < p.M ? (uint32_t)crow * (uint32_t)p.lda * 2 + c * 2 : kPastEnd;
            }
        }
        if constexpr (LB == kRows) {
            const int rows = min(BN, p.N - n0);
#pragma unroll
            for (int g = 0; g < (SEG == 2 ? 2 : NB); ++g)
                rb[g] = make_rsrc((SEG == 2 || NB == 2 ? p.b[g]
                                   : z == 0            ? p.b[0]
                                   : z == 1            ? p.b[1]
                                                       : p.b[2]) +
                                      n0 * ldb,
                                  ((uint64_t)(rows - 1) * ldb + pad) * 2);
            vb[0] = (uint32_t)lrow * (uint32_t)ldb * 2 + chunk * 16;
        } else {
            // region q holds both wave columns' blocks 2 q and 2 q + 1
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = 64 * q + 8 * cchunk + (cchunk & 8 ? 64 : 0);
                vb[q] = n0 + c < p.N ? (uint32_t)crow * (uint32_t)ldb * 2 + c * 2 : kPastEnd;
            }
        }
    };
    // descriptor of a kCols operand's stage kt (it moves with the stage: an
    // operand may be larger than 32-bit offsets reach)
    auto col_rsrc = [&](const uint16_t *base, int64_t ld, int kt, int i0, int I) {
        const int rows = min(kWideK, p.R - kt * kWideK);
        const int cols = (min(kWideCols, I - i0) + 7) & ~7;
        return make_rsrc(base + (int64_t)kt * kWideK * ld + i0,
                         ((uint64_t)(rows - 1) * ld + cols) * 2);
    };
    auto group_of = [&](const uint16_t *const *q, int kt) {
        return SEG == 2 ? (kt >= KT ? q[1] : q[0]) : z == 0 ? q[0] : z == 1 ? q[1] : q[2];
    };
    // The loads of the item's stage i, begun together and issued one by one: put_a 0 ..
    // 3, put_b of pair q of the column blocks (0: B0, B1; 1: B2, B3; two matrices: the
    // gate's, the up's), 0 .. kPair - 1.
    struct Loads {
        rsrc_t d[2];  // of one operand, or two matrices
        uint32_t v[2], soff;
        char *slot;
    };
    auto begin_a = [&](int i) {
        const int kt = k0 + i, ks = SEG == 2 && kt >= KT ? kt - KT : kt;
        Loads l;
        l.slot = smem + (i & 1) * W::kSlot;
        l.soff = ks * kWideLine;
        if constexpr (LA == kRows) {
            l.d[0] = SEG == 2 && kt >= KT ? ra[SEG - 1] : ra[0];
            l.v[0] = ks * kWideK + chunk * 8 >= p.R ? kPastEnd : va[0];
        } else {
            l.d[0] = col_rsrc(group_of(p.a, kt), p.lda, ks, m0, p.M);
            l.v[0] = va[0];
            l.v[1] = va[1];
        }
        return l;
    };
    auto begin_b = [&](int i) {
        const int kt = k0 + i, ks = SEG == 2 && kt >= KT ? kt - KT : kt;
        Loads l;
        l.slot = smem + (i & 1) * W::kSlot + W::kA;
        l.soff = ks * kWideLine;
        if constexpr (LB == kRows) {
            l.d[0] = SEG == 2 && kt >= KT ? rb[SEG - 1] : rb[0];
            if constexpr (NB == 2) l.d[1] = rb[1];
            l.v[0] = ks * kWideK + chunk * 8 >= p.R ? kPastEnd : vb[0];
        } else {
            l.d[0] = col_rsrc(group_of(p.b, kt), ldb, ks, n0, p.N);
            l.v[0] = vb[0];
            l.v[1] = vb[1];
        }
        return l;
    };
    auto put_a = [&](const Loads &l, int g) {
        if constexpr (LA == kRows)
            dma16(l.d[0], l.v[0] + g * ((uint32_t)(16 * WR) * (uint32_t)p.lda * 2), l.soff,
                  l.slot + (16 * WR * g + 8 * wave) * kWideLine);
        else
            dma16(l.d[0],
                  l.v[g / W::kPair] + g % W::kPair * ((uint32_t)(8 * WR) * (uint32_t)p.lda * 2), 0,
                  l.slot + g / W::kPair * kWideRegion +
                      (8 * WR * (g % W::kPair) + 4 * wave) * 256);
    };
    auto put_b = [&](const Loads &l, int q, int g) {
        if constexpr (LB == kRows) {
            // row 16 WR g of the pair's: 64 of each wave column, or 128 of matrix q
            const int r = 16 * WR * g;
            const int row = NB == 1 ? r / 64 * 128 + q * 64 + r % 64 : r;
            dma16(l.d[NB == 2 ? q : 0], l.v[0] + row * ((uint32_t)ldb * 2), l.soff,
                  l.slot + ((NB == 2 ? q * 128 : 0) + row + 8 * wave) * kWideLine);
        } else {
            dma16(l.d[0], l.v[q] + g * ((uint32_t)(8 * WR) * (uint32_t)ldb * 2), 0,
                  l.slot + q * kWideRegion + (8 * WR * g + 4 * wave) * 256);
        }
    };
    constexpr int kAB = W::kFirst, kB = W::kPair;  // loads of a wave in each part
    auto load_first = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= kn) break;
            const Loads a = begin_a(i), b = begin_b(i);
#pragma unroll
            for (int g = 0; g < 4; ++g) put_a(a, g);
#pragma unroll
            for (int g = 0; g < 2 * kB; ++g) put_b(b, g / kB, g % kB);
        }
    };
    // Fragment of 16 rows (columns of the product's other operand) from `row` on,
    // 32 reduction elements of sub-step s: lane l holds row l % 16, elements 32 s + 8
    // (l / 16) ..+7.
    auto read_rows = [&](const char *part, int row, int s) {
        const int c = (4 * s + (lane >> 4)) ^ line_swz(l16);
        return lds_ld16(part, (row + l16) * kWideLine + (c << 4));
    };
    // the same of a kCols region, its columns 8 c ..8 c + 15
    const int fr = 8 * (lane >> 4) + (l16 >> 2);  // reduction row within a sub-step
    const int fx = 2 * ((l16 >> 2) | ((lane >> 4) & 1) << 2);
    const int fo = fr * 256 + (((l16 & 3) >> 1) << 4) + (l16 & 1) * 8;
    auto read_cols = [&](const char *region, int c, int s) {
        i16x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = lds_tr16(
                (const lds_i16x4 *)(region + fo + ((c ^ fx) << 4) + (32 * s + 4 * h) * 256));
        const u32x2 lo = __builtin_bit_cast(u32x2, v[0]);
        const u32x2 hi = __builtin_bit_cast(u32x2, v[1]);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    auto read_a = [&](int k, int i, int s) {  // 16 rows i of the wave's 64
        const char *part = smem + (k & 1) * W::kSlot;
        if constexpr (LA == kRows) return read_rows(part, wm * 64 + 16 * i, s);
        else return read_cols(part + (wm >> 1) * kWideRegion, (wm & 1) * 8 + 2 * i, s);
    };
    u32x4 fa[2][4], fb[2][2][2];  // [sub-step][16 rows], [register set][sub-step][16 columns]
    auto read_b = [&](int k, int j, int s, int h) {  // half h of block j of 32 columns
        const char *part = smem + (k & 1) * W::kSlot + W::kA;
        if constexpr (LB == kRows)
            fb[j & 1][s][h] = read_rows(
                part,
                (NB == 1 ? wn * 128 + j * 32 : (j >> 1) * 128 + wn * 64 + (j & 1) * 32) + 16 * h,
                s);
        else
            fb[j & 1][s][h] =
                read_cols(part + (j >> 1) * kWideRegion, wn * 8 + (j & 1) * 4 + 2 * h, s);
    };
    // [16 rows][16 columns]: register r of a block is row l16, column 4 (lane / 16) + r
    f32x4 acc[4][8];
    auto mma = [&](int j, int s, int i, int h) {
        acc[i][2 * j + h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, fb[j & 1][s][h]), __builtin_bit_cast(bf16x8, fa[s][i]),
            acc[i][2 * j + h], 0, 0, 0);
    };
    // A step: block j's 16 matrix instructions, two at a time, and before each pair what
    // other(0 .. 7) issues.  (The scheduling barriers keep that order: loads and
    // reads that all waves issue at once after a barrier hold up the matrix
    // instructions behind them.)
    auto step = [&](int j, auto other) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            other(q);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) mma(j, q >> 2, q & 3, h);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the fragments of stage k's block j, in the step before its own
    auto read_next = [&](int k, int j, int q) {
        if (q < 4) read_b(k, j, q >> 1, q & 1);
    };
    auto last_step = [&](int k, auto other) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            read_next(k + 1, 0, q);
            other(q);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) mma(3, q >> 2, q & 3, h);
            __builtin_amdgcn_sched_barrier(0);
            fa[q >> 2][q & 3] = read_a(k + 1, q & 3, q >> 2);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto nothing = [](int) {};
    // what the epilogue loads for the wave's rows, one a lane
    auto load_raw = [&]() { return epi.raw(min(m0 + wm * 64 + lane, p.M - 1)); };

    int after = 0;  // stores younger than a tile's first loads
    at_item(blockIdx.x);
    typename Epi::Raw raw = load_raw(), next = raw;
    load_first();
    for (int t = blockIdx.x; t < items; t += gridDim.x) {
        const int mt = m0, nt = n0, n = kn;  // m0, ... move on below
        const Place at{z, m0, n0, BM, BN, part};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{};
        // The last tile's stores are younger than the loads of stages 0 and 1, and may
        // stay on their way while these are waited for.
        if (n > 0) {
            if (n > 1) wait_besides<kB + kAB + kB>(after);
            else wait_vmcnt<kB>();
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) fa[s][i] = read_a(0, i, s);
#pragma unroll
            for (int q = 0; q < 4; ++q) read_next(0, 0, q);
            int k = 0;
            for (; k + 2 < n; ++k) {
                const Loads la = begin_a(k + 2), lb = begin_b(k + 2);
                step(0, [&](int q) { read_next(k, 1, q); });
                if (after) wait_besides<kAB + kB>(after);
                else wait_vmcnt<kAB + kB>();
                wait_lgkm0();
                __builtin_amdgcn_s_barrier();  // X
                step(1, [&](int q) {
                    read_next(k, 2, q);
                    if (q < 4) put_a(la, q);
                    else if (q < 4 + kB) put_b(lb, 0, q - 4);
                });
                step(2, [&](int q) { read_next(k, 3, q); });
                if (k) after = 0;
                if (after) wait_besides<kB + kAB>(after);
                else wait_vmcnt<kB + kAB>();
                wait_lgkm0();
                __builtin_amdgcn_s_barrier();  // Y
                last_step(k, [&](int q) {
                    if (q >= 4 && q < 4 + kB) put_b(lb, 1, q - 4);
                });
            }
            if (k + 1 < n) {
                step(0, [&](int q) { read_next(k, 1, q); });
                wait_vmcnt<kAB + kB>();
                wait_lgkm0();
                __builtin_amdgcn_s_barrier();
                step(1, [&](int q) { read_next(k, 2, q); });
                step(2, [&](int q) { read_next(k, 3, q); });
                wait_vmcnt<kB>();
                wait_lgkm0();
                __builtin_amdgcn_s_barrier();
                last_step(k, nothing);
                ++k;
            }
            step(0, [&](int q) { read_next(k, 1, q); });
            wait_vmcnt<0>();
            __builtin_amdgcn_s_barrier();
            step(1, [&](int q) { read_next(k, 2, q); });
            step(2, [&](int q) { read_next(k, 3, q); });
            step(3, nothing);
        }

        // The next tile's first loads (after every wave has read its last
        // fragments) are on their way while this tile is written.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        const bool more = t + (int)gridDim.x < items;
        if (more) {
            at_item(t + gridDim.x);
            next = load_raw();
            load_first();
        }
        __builtin_amdgcn_sched_barrier(0);

        // (The lane's number is read anew: the addresses below, computed ahead of
        // the tile loop, would fill the registers that the k-loop needs.)
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int lr = ln & 15, lc = 4 * (ln >> 4);
        const int mw = mt + wm * 64, nw = nt + wn * (BN / 2);  // the wave's outputs
        char *out = smem + 2 * W::kSlot + wave * kWideOut;
        // ALL: every row and column of the wave's outputs is one of the product's
        auto write = [&](auto whole) {
            constexpr bool ALL = decltype(whole)::value;
            if constexpr (Epi::kStats) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    typename Epi::Row row(epi, raw.of(16 * i + lr));
                    auto each = [&](auto f) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2],
                                                acc[i][j][3]};
                            f(nw + 16 * j + lc, v);
                        }
                    };
                    each([&](int n, auto &v) { epi.template most<4, ALL>(row, n, v); });
                    each([&](int n, auto &v) { epi.template add<4, ALL>(row, n, v); });
                    epi.template join<16>(row);
                    epi.template join<32>(row);
                    const int m = mw + 16 * i + lr;
                    if (ln < 16 && (ALL || (m < p.M && nw < p.N))) epi.put(row, m, nw / 128);
                }
            } else if constexpr (NB == 1) {
                // 16 rows of 64 columns at a time go through LDS, 256 bytes a row, chunk c
                // of row r at c ^ r; lanes then hold 8 consecutive columns, so that whole
                // lines are read and stored.  The next block enters LDS before this one is
                // worked on.
                const int r8 = ln >> 3, c8 = ln & 7;
                auto enter = [&](int b) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<f32x4 *>(
                            out + lr * 256 + (((4 * j + (lc >> 2)) ^ lr) << 4)) =
                            acc[b >> 1][4 * (b & 1) + j];
                    __builtin_amdgcn_wave_barrier();
                };
                const int cols = epi.dest(0, at).cols;
                // what 8 rows of a block need besides, as many of the 16 ahead as there are
                // registers for
                constexpr int kAhead = WR == 4 ? 2 : 16;
                typename Epi::Fetched got[kAhead];
                auto fetch = [&](int f) {
                    got[f % kAhead] = epi.fetch(min(mw + 8 * (f & 1) + 16 * (f >> 2) + r8, p.M - 1),
                                                min(nw + 64 * (f >> 1 & 1) + 8 * c8, cols - 8));
                };
#pragma unroll
                for (int f = 0; f < kAhead; ++f) fetch(f);
                enter(0);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const int i = b >> 1, n = nw + 64 * (b & 1) + 8 * c8;
                    float v[2][8];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = 8 * q + r8;
                            const u32x4 w = lds_ld16(out, r * 256 + (((2 * c8 + h) ^ r) << 4));
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[q][4 * h + e] = __uint_as_float(w[e]);
                        }
                    __builtin_amdgcn_wave_barrier();
                    if (b < 7) enter(b + 1);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int r = 16 * i + 8 * q + r8, m = mw + r;
                        typename Epi::Row row(epi, raw.of(r));
                        float o[Epi::kOuts][8];
                        const bool in = ALL || (m < p.M && n < cols);
                        if (in) epi.template values<8, ALL>(row, got[(2 * b + q) % kAhead], n, v[q],
                                                    v[q], o);
                        if (2 * b + q + kAhead < 16) fetch(2 * b + q + kAhead);
                        if (!in) continue;
#pragma unroll
                        for (int k = 0; k < Epi::kOuts; ++k)
                            put_out(epi.dest(k, at), m, n, o[k]);
                    }
                }
            } else {
                // The outputs (bf16) go through LDS, 32 rows of 128 bytes at a time.
#pragma unroll
                for (int i0 = 0; i0 < 4; i0 += 2) {
                    if (nw >= epi.dest(0, at).cols) continue;
                    float o[2][4][Epi::kOuts][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        typename Epi::Row row(epi, raw.of(16 * (i0 + i) + lr));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float v[4], u[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[e] = acc[i0 + i][j][e];
                                u[e] = acc[i0 + i][4 + j][e];
                            }
                            epi.template values<4, ALL>(row, {}, 0, v, u, o[i][j]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < Epi::kOuts; ++k) {
                        const Dest d = epi.dest(k, at);
                        if (!d.p) continue;
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int r = 16 * i + lr, byte = (16 * j + lc) * 2;
                                const float(&f)[4] = o[i][j][k];
                                store4(out + r * kWideLine + (((byte >> 4) ^ line_swz(r)) << 4) +
                                           (byte & 15),
                                       TW_T_BF16, 0, f32x4{f[0], f[1], f[2], f[3]});
                            }
                        __builtin_amdgcn_wave_barrier();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = 8 * q + (ln >> 3), c = ln & 7;
                            const u32x4 w =
                                lds_ld16(out, r * kWideLine + ((c ^ line_swz(r)) << 4));
                            const int m = mw + 16 * i0 + r, n = nw + 8 * c;
                            if (ALL || (m < p.M && n < d.cols))
                                st16(static_cast<uint16_t *>(d.p) + m * d.ld + n, w);
                        }
                        __builtin_amdgcn_wave_barrier();
                    }
                }
            }
        };
        const bool inside = mt + BM <= p.M && nt + BN <= p.N;
        if (inside) write(std::true_type{});
        else write(std::false_type{});
        // at least so many stores of this tile are younger than the next one's loads
        after = inside ? epi.stores(at) : 0;
        raw = next;
    }
}

template <int WR, int NB>
int64_t wide_tiles(const TileArgs &p) {  // of all products
    return ((int64_t)p.M + 64 * WR - 1) / (64 * WR) *
           (((int64_t)p.N + kWideCols / NB - 1) / (kWideCols / NB)) * p.groups;
}

template <int WR, int LA, int LB, int NB, int SEG, class Epi>
hipError_t launch_wide(const TileArgs &p, const Epi &epi, hipStream_t s) {
    using W = Wide<WR>;
    constexpr auto kernel = &wide_tiles_kernel<WR, LA, LB, NB, SEG, Epi>;
    const hipError_t e = lds_limit_once<kernel>(W::kBytes);
    if (e != hipSuccess) return e;
    const int64_t items = p.full + (wide_tiles<WR, NB>(p) - p.full) * p.splits;
    const unsigned grid = (unsigned)(items < kWideGrid ? items : kWideGrid);
    kernel<<<grid, W::kThreads, W::kBytes, s>>>(p, epi);
    return hipGetLastError();
}

// Estimated time (us) of `items` tiles of 64 WR rows over `stages` stages each.  A stage
// takes 1.0 to 1.6 us in the larger tiles and 0.55 to 0.95 in the smaller ones, the more
// the more CUs draw power and load; 8 us come before the first and after the last.  (A
// third stage of loads ahead in the smaller tiles' LDS changed nothing for the better: 1 x
// 64 stages 47 -> 55 us.)  No epilogue is counted, though dh's, which reads 4 and writes 6
// bytes an output, takes longer than its product: 4096 x 1024 x 4096 34 us estimated, 56
// to 60 measured.  It is the same work in tiles of either height, and no shape was found
// where the estimate took the slower one (dh there in the smaller tiles 72 us).
template <int WR>
double tiles_us(int64_t items, int64_t stages) {
    const double least = WR == 4 ? 1.0 : 0.55, more = WR == 4 ? 0.6 : 0.4;
    const int64_t rounds = items / kWideGrid, rest = items % kWideGrid;
    return 8.0 + stages * (rounds * (least + more) +
                           (rest ? least + more * rest / kWideGrid : 0.0));
}

// Measured (us, tiles of 128 and of 256 rows): gate and up 777 x 1000 x 2728 21, 29; 2048 x
// 2048 x 5632 82, 90; 777 x 2048 x 5632 55, 46; 4096 x 1024 x 4096 66, 57.
template <int LA, int LB, int NB, int SEG, class Epi>
hipError_t launch_tiles(TileArgs p, const Epi &epi, hipStream_t s) {
    const int64_t stages = SEG * (((int64_t)p.R + kWideK - 1) / kWideK);
    if (tiles_us<4>(wide_tiles<4, NB>(p), stages) <= tiles_us<2>(wide_tiles<2, NB>(p), stages)) {
        p.full = (int)wide_tiles<4, NB>(p);
        return launch_wide<4, LA, LB, NB, SEG>(p, epi, s);
    }
    p.full = (int)wide_tiles<2, NB>(p);
    return launch_wide<2, LA, LB, NB, SEG>(p, epi, s);
}

// ------------------------------- epilogues ----------------------------------
// Outputs stored as they are: to out[z] in its type, or, where a tile takes a part of
// the reduction, to that part in fp32 (added to what is there with `more`: a later
// piece of the reduction).  A part holds its tile alone.
struct EpiStore {
    static constexpr bool kStats = false;
    static constexpr int kWalk = 8;
    static constexpr int kOuts = 1;
    void *out[3];
    int type;
    int N;
    float *parts;
    int more;
    typedef NoRaw Raw;
    struct Row {
        __device__ Row(const EpiStore &, Raw) {}
    };
    __device__ Raw raw(int) const { return {}; }
    __device__ int stores(const Place &p) const {
        return p.part >= 0 || type == TW_T_F32 ? 32 : 16;
    }
    __device__ __forceinline__ Dest dest(int, const Place &p) const {
        if (p.part >= 0)
            return {parts + (int64_t)p.part * p.rows * p.cols - ((int64_t)p.m0 * p.cols + p.n0),
                    TW_T_F32, p.cols, N, more != 0};
        return {p.z == 0 ? out[0] : p.z == 1 ? out[1] : out[2], type, N, N, false};
    }
    typedef NoFetch Fetched;
    __device__ Fetched fetch(int, int) const { return {}; }
    template <int W, bool ALL>
    __device__ __forceinline__ void values(Row &, const Fetched &, int, const float (&v)[W],
                                           const float (&)[W], float (&o)[kOuts][W]) const {
#pragma unroll
        for (int e = 0; e < W; ++e) o[0][e] = v[e];
    }
};

// out = the sum of the parts: each of a workgroup's 4 waves takes every fourth part of
// the same 256 outputs, 4 at a time, so that the latencies of 16 parts are one (a wave
// that took them all, 8 at a time, cost a decoded row 2.5 us more).
template <int T>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float *__restrict__ part, int splits,
                                                        int64_t n, void *__restrict__ out) {
    __shared__ f32x4 sums[3][kWave];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t at = ((int64_t)blockIdx.x * kWave + lane) * 4;
    f32x4 v{};
    if (at < n)
        for (int s = wave; s < splits; s += 16) {
            f32x4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = *reinterpret_cast<const f32x4 *>(part + min(s + 4 * i, splits - 1) * n + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) v += s + 4 * i < splits ? w[i] : f32x4{};
        }
    if (wave) sums[wave - 1][lane] = v;
    __syncthreads();
    if (wave || at >= n) return;
#pragma unroll
    for (int i = 0; i < 3; ++i) v += sums[i][lane];
    store4(out, T, at, v);
}
inline hipError_t launch_sum_parts(const float *part, int splits, int64_t n, void *out, int type,
                                   hipStream_t s) {
    if (n == 0) return hipSuccess;
    const unsigned grid = (unsigned)((n / 4 + 63) / 64);
    if (type == TW_T_F32) sum_parts_kernel<TW_T_F32><<<grid, 256, 0, s>>>(part, splits, n, out);
    else sum_parts_kernel<TW_T_BF16><<<grid, 256, 0, s>>>(part, splits, n, out);
    return hipGetLastError();
}

// The same for tiles of 64 WR x 256: part s of tile full + i is number s rest + i.  A
// workgroup takes 1024 outputs of a tile, and where a grid does not hold all of them (a
// launch has at most 2^32 threads: 2^18 tiles of 256 rows) every gridDim-th.
constexpr unsigned kSumGrid = 1u << 22;
template <int WR>
__global__ __launch_bounds__(256) void sum_tiles_kernel(const float *__restrict__ parts, int splits,
                                                        int rest, int full, int nbm, int nbn,
                                                        EpiStore epi, int M) {
    constexpr int kSize = 64 * WR * kWideCols, kBlocks = kSize / 1024;  // workgroups a tile
    for (int64_t b = blockIdx.x; b < (int64_t)rest * kBlocks; b += gridDim.x) {
        const int i = (int)(b / kBlocks);
        int tile = full + i;
        const int z = tile / (nbm * nbn);
        tile -= z * (nbm * nbn);
        int bm, bn;
        walk_tile<EpiStore::kWalk>(tile, nbm, nbn, bm, bn);
        const int at = ((int)(b % kBlocks) * 256 + threadIdx.x) * 4;
        const int m = bm * 64 * WR + at / kWideCols, n = bn * kWideCols + at % kWideCols;
        if (m >= M || n >= epi.N) continue;
        const float *q = parts + (int64_t)i * kSize + at;
        f32x4 v{};
        for (int s = 0; s < splits; s += 4) {  // (4 latencies in one)
            f32x4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = *reinterpret_cast<const f32x4 *>(
                    q + (int64_t)min(s + k, splits - 1) * rest * kSize);
#pragma unroll
            for (int k = 0; k < 4; ++k) v += s + k < splits ? w[k] : f32x4{};
        }
        store4(z == 0 ? epi.out[0] : z == 1 ? epi.out[1] : epi.out[2], epi.type,
               (int64_t)m * epi.N + n, v);
    }
}

// How a product stored as it is takes its tiles: the first `full` whole and the rest in
// `splits` parts of the reduction.
struct SplitPlan {
    int rows;  // of a tile: 256 or 128
    int splits, full;
    size_t bytes;  // of the parts
};
// The plan of the least estimated time: tiles_us for the tiles taken whole, in rounds of
// the chip, and for the parts of the others; the parts' way through memory, 8 bytes an
// output and part at 4.5 TB/s, and 3 us for the kernel that adds them.  `pieces`: the
// reduction comes in pieces, every tile keeps its parts from one to the next.
// Measured (us, tiles of 128 and of 256 rows, each with its best split): down 777 x 1000
// x 2728 23, 29; 4096 x 2048 x 5632 80, 93; weight gradients 4096 x 1024 x 4096 121, 95;
// 4096 x 2048 x 5632 266, 235.
template <int SEG>
SplitPlan split_plan(const TileArgs &p, bool pieces) {
    const int64_t stages = SEG * (((int64_t)p.R + kWideK - 1) / kWideK);
    SplitPlan best{128, 1, (int)wide_tiles<2, 1>(p), 0};
    double least = 1e30;
    auto offer = [&](auto wr) {
        constexpr int WR = decltype(wr)::value;
        const int64_t tiles = wide_tiles<WR, 1>(p), size = 64 * WR * kWideCols;
        for (int s = 1; s <= 64 && s <= stages; ++s) {
            const int64_t per = (stages + s - 1) / s;
            if ((stages + per - 1) / per != s) continue;  // (every part has a stage)
            const bool parts = pieces || s > 1;
            const int64_t full = !parts ? tiles : pieces ? 0 : tiles / kWideGrid * kWideGrid;
            const int64_t rest = tiles - full;
            double us = tiles_us<WR>(full, stages) - 8.0;
            us += rest ? tiles_us<WR>(rest * s, per) : 8.0;
            if (parts) us += 3.0 + (double)rest * s * size * 8 / 4.5e6;
            if (us >= least) continue;
            least = us;
            best = {64 * WR, s, (int)full, parts ? (size_t)rest * s * size * 4 : 0};
        }
    };
    offer(std::integral_constant<int, 4>{});
    offer(std::integral_constant<int, 2>{});
    return best;
}

// A product stored as it is.  parts: split_plan's bytes; `last`: the sums are to be
// stored (with pieces: of the last one).
template <int LA, int LB, int SEG>
hipError_t launch_split(TileArgs p, const SplitPlan &plan, const EpiStore &epi, bool last,
                        hipStream_t s) {
    p.splits = plan.splits;
    p.full = plan.full;
    const hipError_t e = plan.rows == 256 ? launch_wide<4, LA, LB, 1, SEG>(p, epi, s)
                                          : launch_wide<2, LA, LB, 1, SEG>(p, epi, s);
    if (e != hipSuccess || !plan.bytes || !last) return e;
    const int nbm = (p.M + plan.rows - 1) / plan.rows, nbn = (p.N + kWideCols - 1) / kWideCols;
    const int rest = nbm * nbn * p.groups - plan.full;
    const int64_t blocks = (int64_t)(plan.rows * kWideCols / 1024) * rest;
    const unsigned grid = (unsigned)(blocks < kSumGrid ? blocks : kSumGrid);
    if (plan.rows == 256)
        sum_tiles_kernel<4><<<grid, 256, 0, s>>>(epi.parts, plan.splits, rest, plan.full, nbm, nbn,
                                                 epi, p.M);
    else
        sum_tiles_kernel<2><<<grid, 256, 0, s>>>(epi.parts, plan.splits, rest, plan.full, nbm, nbn,
                                                 epi, p.M);
    return hipGetLastError();
}

}  // namespace tw
