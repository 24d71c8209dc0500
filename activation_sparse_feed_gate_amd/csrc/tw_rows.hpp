// tw_rows.hpp -- what the row kernels (layer norm, its gradient, the int8
// quantiser) share: 8-element vectors of bf16 or fp32 rows at any alignment,
// sums and maxima over the threads of a row.
#pragma once

#include "tw_device.hpp"
#include "tw_norm_quant.hpp"

namespace tw {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 16-byte accesses at the alignment of the element type: gfx950 runs them at
// any address, so rows of odd lengths and strides take the same code.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// 8 consecutive elements as loaded (converted only when they are used, so
// that all of a row's loads are issued before the first wait).
template <int T>
struct Vec8 {
    u32x4 w[T == TW_T_F32 ? 2 : 1];
};

__host__ __device__ constexpr int type_bytes(int t) {
    return t == TW_T_F32 ? 4 : t == TW_T_BF16 ? 2 : 1;
}

// Elements e .. e+7 of a row of K; those past the end read zero.
template <int T>
__device__ __forceinline__ Vec8<T> load8(const char *row, int e, int K) {
    Vec8<T> v;
    if (e + 8 <= K) {
        const char *p = row + (size_t)e * type_bytes(T);
        v.w[0] = *reinterpret_cast<const u32x4_any *>(p);
        if constexpr (T == TW_T_F32) v.w[1] = *reinterpret_cast<const u32x4_any *>(p + 16);
    } else {
        v.w[0] = u32x4{};
        if constexpr (T == TW_T_F32) v.w[1] = u32x4{};
        if (e < K) {
#pragma unroll
            for (int i = 0; i < 7; ++i) {
                if (e + i >= K) continue;
                if constexpr (T == TW_T_F32)
                    v.w[i >> 2][i & 3] = reinterpret_cast<const uint32_t *>(row)[e + i];
                else
                    v.w[0][i >> 1] |=
                        (uint32_t) reinterpret_cast<const uint16_t *>(row)[e + i] << (16 * (i & 1));
            }
        }
    }
    return v;
}

// The same where K is a multiple of 8 (a vector is in or out): vectors past
// the end read the row's last one instead.  No branch, so nothing waits for a
// load before it is used.
template <int T>
__device__ __forceinline__ Vec8<T> load8_whole(const char *row, int e, int K) {
    const char *p = row + (size_t)min(e, K - 8) * type_bytes(T);
    Vec8<T> v;
    v.w[0] = *reinterpret_cast<const u32x4_any *>(p);
    if constexpr (T == TW_T_F32) v.w[1] = *reinterpret_cast<const u32x4_any *>(p + 16);
    return v;
}

template <bool WHOLE, int T>
__device__ __forceinline__ Vec8<T> load8_of(const char *row, int e, int K) {
    if constexpr (WHOLE) return load8_whole<T>(row, e, K);
    else return load8<T>(row, e, K);
}

template <int T>
__device__ __forceinline__ void unpack8(const Vec8<T> &v, float *f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (T == TW_T_F32) f[i] = __uint_as_float(v.w[i >> 2][i & 3]);
        else f[i] = (i & 1) ? bf_hi(v.w[0][i >> 1]) : bf_lo(v.w[0][i >> 1]);
    }
}

// Two fp32 to packed bf16, round to nearest even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

template <int T>
__device__ __forceinline__ void store8(char *row, int e, int K, const float *f) {
    if constexpr (T == TW_T_F32) {
        if (e + 8 <= K) {
            float *p = reinterpret_cast<float *>(row) + e;
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __float_as_uint(f[i]);
                b[i] = __float_as_uint(f[4 + i]);
            }
            *reinterpret_cast<u32x4_any *>(p) = a;
            *reinterpret_cast<u32x4_any *>(p + 4) = b;
        } else if (e < K) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (e + i < K) reinterpret_cast<float *>(row)[e + i] = f[i];
        }
    } else {
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        if (e + 8 <= K) {
            *reinterpret_cast<u32x4_any *>(row + (size_t)e * 2) = a;
        } else if (e < K) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (e + i < K)
                    reinterpret_cast<uint16_t *>(row)[e + i] =
                        (uint16_t)(i & 1 ? a[i >> 1] >> 16 : a[i >> 1] & 0xffffu);
        }
    }
}

__device__ __forceinline__ void store8_as(int type, char *row, int e, int K, const float *f) {
    if (type == TW_T_F32) store8<TW_T_F32>(row, e, K, f);
    else store8<TW_T_BF16>(row, e, K, f);
}

// --- sums and maxima over the threads of a row --------------------------------
template <int CTRL, int ROWMASK>
__device__ __forceinline__ uint32_t dpp0_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWMASK, 0xf, false);
}

// Largest of the 64 lanes' values (the scan of wave_sum; lanes with no
// source read 0, the identity).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp0_u32<0x111, 0xf>(v));
    v = max(v, dpp0_u32<0x112, 0xf>(v));
    v = max(v, dpp0_u32<0x114, 0xf>(v));
    v = max(v, dpp0_u32<0x118, 0xf>(v));
    v = max(v, dpp0_u32<0x142, 0xa>(v));
    v = max(v, dpp0_u32<0x143, 0xc>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Reductions over the TPR threads that hold one row: a wave, or a whole
// workgroup of TPR threads, through LDS.  Consecutive reductions alternate
// between two slots, so one barrier each is enough: a slot is written again
// only after the barrier of the reduction in between, which every thread
// enters after it has read the slot.
template <int TPR>
struct RowReduce {
    static constexpr int NW = TPR / kWave;
    float *lds;  // 2 * NW floats (unused when a row is one wave)
    int slot = 0;
    __device__ explicit RowReduce(float *p) : lds(p) {}

    __device__ __forceinline__ float sum(float v) {
        v = wave_sum(v);
        if constexpr (NW > 1) {
            float *s = lds + slot * NW;
            slot ^= 1;
            if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v += s[w];
        }
        return v;
    }
    __device__ __forceinline__ uint32_t max_u32(uint32_t v) {
        v = wave_max(v);
        if constexpr (NW > 1) {
            float *s = lds + slot * NW;
            slot ^= 1;
            if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = __uint_as_float(v);
            __syncthreads();
            v = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) v = max(v, __float_as_uint(s[w]));
        }
        return v;
    }
};

// --- int8 quantisation of a row -------------------------------------------------
// Scale of a row whose largest magnitude has the bits `top` (as an unsigned
// integer, so an infinity or NaN in the row wins): top / 127, and the factor
// (1 / top) 127 that the row is multiplied by, each operation rounded to
// fp32.  A row whose magnitudes all lie below 2^-100 (where 127 / top nears
// the end of the fp32 range) becomes
// zeros with scale 0; a row that holds an infinity or NaN gets the scale NaN
// and zeros, so that every product with it is NaN.
struct RowScale {
    float scale, inv;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    const float a = __uint_as_float(top);
    if (top >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.0f};
    if (a < 0x1p-100f) return {0.0f, 0.0f};
    return {a / 127.0f, 1.0f / a * 127.0f};
}

// round(f * inv), ties to even, as a byte.  The product is rounded to fp32
// first; |f| <= top keeps it within 127 (1 + 2^-20) (1 / top may be a
// subnormal of 21 bits), which rounds to 127.  A
// row of scale NaN has inv = 0: its bytes are forced to zero (0 * inf is NaN).
__device__ __forceinline__ uint32_t quant_byte(float f, float inv) {
#pragma clang fp contract(off)
    const float r = rintf(f * inv);
    return (uint32_t)(inv > 0.0f ? (int)r : 0) & 0xffu;
}
__device__ __forceinline__ u32x2 quant8(const float *f, float inv) {
    u32x2 q;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        q[h] = quant_byte(f[4 * h], inv) | quant_byte(f[4 * h + 1], inv) << 8 |
               quant_byte(f[4 * h + 2], inv) << 16 | quant_byte(f[4 * h + 3], inv) << 24;
    return q;
}
__device__ __forceinline__ void store_q8(int8_t *row, int e, int K, u32x2 q) {
    if (e + 8 <= K) {
        *reinterpret_cast<u32x2_any *>(row + e) = q;
    } else if (e < K) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (e + i < K) row[e + i] = (int8_t)(q[i >> 2] >> (8 * (i & 3)));
    }
}

}  // namespace tw
