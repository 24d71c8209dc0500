// grad_clip.hip -- the norm over many gradients, and clipping by it:
//   norm = sqrt(sum over all buffers of g^2),  out = g min(1, max_norm / (norm + eps)).
//
// Two passes over memory, which bounds both (the factor is known only after
// the last element).  Buffers are cut into chunks of 8192 elements, and a
// launch's workgroups walk the chunks of up to kTableMax buffers, whose
// addresses travel as kernel arguments: nothing is copied to the device, so
// a captured graph replays them.  Sums are fp32, 8 of them a thread; the
// workgroups' sums are added in fp64, in a fixed order (no atomics: the norm does
// not depend on timing).  Measured: 336 M elements in 146 buffers, bf16 clipped
// into fp32, 557 to 561 us at 4.8 TB/s; 3.9 M fp32 elements in 26 buffers 13.8 us (from cache).
#include "tw_rows.hpp"
#include "tw_train.hpp"

namespace tw {
namespace {

constexpr int kClipThreads = 256;
// Vectors of 8 a thread and chunk.  (2: 31 us for 32 over 24 M elements, but 585 for 554
// over 503 M; 8: 35 and 553.)
constexpr int kVecs = 4;
constexpr int kChunk = kClipThreads * 8 * kVecs;       // elements
constexpr int kTableMax = 96;                          // buffers a launch (3 KB of arguments)
constexpr int kClipGrid = 2048;                        // workgroups (512: 568 for 554 us)
// Parts that every workgroup of the clipping adds itself, which saves a launch (480 parts:
// 13.8 us, 14.5 with the launch); many cost more (2048: 36 and 34 us, 4096: 563 and 557).
constexpr int kPartsMax = 1024;

struct Table {
    const char *g[kTableMax];
    char *out[kTableMax];
    int64_t n[kTableMax];
    int first[kTableMax + 1];  // chunk numbers; buffer i has first[i] .. first[i + 1] - 1
    uint8_t g_type[kTableMax], out_type[kTableMax];
    int count;
};

// Runs f(type of g, address of the chunk, its elements, buffer, offset) over the
// workgroup's chunks.
template <typename F>
__device__ __forceinline__ void walk(const Table &t, F f) {
    int i = 0;
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        while (c >= t.first[i + 1]) ++i;
        const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
        const int n = (int)min((int64_t)kChunk, t.n[i] - at);
        if (t.g_type[i] == TW_T_F32)
            f(std::integral_constant<int, TW_T_F32>{}, t.g[i] + at * 4, n, i, at);
        else
            f(std::integral_constant<int, TW_T_BF16>{}, t.g[i] + at * 2, n, i, at);
    }
}

__global__ __launch_bounds__(kClipThreads) void square_sums_kernel(Table t,
                                                                   float *__restrict__ part) {
    __shared__ float red[2 * (kClipThreads / kWave)];
    RowReduce<kClipThreads> rr(red);
    float s[8] = {};
    walk(t, [&](auto type, const char *g, int n, int, int64_t) {
        constexpr int T = decltype(type)::value;
        Vec8<T> v[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) v[j] = load8<T>(g, 8 * (j * kClipThreads + threadIdx.x), n);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float f[8];
            unpack8<T>(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += f[e] * f[e];
        }
    });
    const float all = rr.sum(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
    if (threadIdx.x == 0) part[blockIdx.x] = all;
}

// The parts' sum, the same in every thread.
__device__ double sum_of_parts(const float *part, int parts, double *lds) {
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < parts; i += blockDim.x) s += part[i];
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
    const int waves = blockDim.x / kWave;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < waves; ++w) s += lds[w];
    return s;
}

__global__ __launch_bounds__(1024) void norm_kernel(const float *part, int parts, float *norm) {
    __shared__ double lds[1024 / kWave];
    const double s = sum_of_parts(part, parts, lds);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// parts > 0: the squares' sums, added here; 0: *norm is there already.
__global__ __launch_bounds__(kClipThreads) void clip_kernel(Table t, const float *part, int parts,
                                                            float max_norm, float eps,
                                                            float *norm) {
    __shared__ double lds[kClipThreads / kWave];
    float all;
    if (parts) {
        all = (float)sqrt(sum_of_parts(part, parts, lds));
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm = all;
    } else {
        all = *norm;
    }
    // (a max_norm of 0 makes zeros, also of gradients whose norm is 0: 0 / 0 there)
    const float c = max_norm > 0.0f || all != all ? max_norm / (all + eps) : 0.0f;
    const float by = c >= 1.0f ? 1.0f : c;  // a norm of NaN makes every gradient NaN
    walk(t, [&](auto type, const char *g, int n, int i, int64_t at) {
        constexpr int T = decltype(type)::value;
        char *out = t.out[i] + at * (t.out_type[i] == TW_T_F32 ? 4 : 2);
        if (out == g && by == 1.0f) return;  // as it is
        Vec8<T> v[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) v[j] = load8<T>(g, 8 * (j * kClipThreads + threadIdx.x), n);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float f[8];
            unpack8<T>(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= by;
            store8_as(t.out_type[i], out, 8 * (j * kClipThreads + threadIdx.x), n, f);
        }
    });
}

// Runs f(table) over the buffers, kTableMax of those with elements at a time (their
// chunks stay within 32 bits).
static_assert(kTableMax * (kClipMost / kChunk + 1) < (int64_t(1) << 31), "");
template <typename F>
hipError_t over_tables(int count, const void *const *g, const int64_t *n, const int *g_type,
                       void *const *out, const int *out_type, F f) {
    Table t;
    t.count = 0;
    t.first[0] = 0;
    auto flush = [&]() {
        const hipError_t e = t.count ? f(t) : hipSuccess;
        t.count = 0;
        return e;
    };
    for (int i = 0; i < count; ++i) {
        if (n[i] == 0) continue;
        const int64_t chunks = (n[i] + kChunk - 1) / kChunk;
        if (t.count == kTableMax) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        t.g[t.count] = static_cast<const char *>(g[i]);
        t.out[t.count] = out ? static_cast<char *>(out[i]) : nullptr;
        t.n[t.count] = n[i];
        t.g_type[t.count] = (uint8_t)g_type[i];
        t.out_type[t.count] = (uint8_t)(out ? out_type[i] : 0);
        t.first[t.count + 1] = t.first[t.count] + (int)chunks;
        ++t.count;
    }
    return flush();
}

unsigned grid_of(const Table &t) {
    return (unsigned)(t.first[t.count] < kClipGrid ? t.first[t.count] : kClipGrid);
}

}  // namespace

size_t grad_norm_bytes(int count, const int64_t *n) {
    // a part a workgroup of each table's launch
    int64_t parts = 0, chunks = 0;
    int in = 0;
    for (int i = 0; i < count; ++i) {
        if (n[i] <= 0) continue;
        if (in == kTableMax) {
            parts += chunks < kClipGrid ? chunks : kClipGrid;
            in = 0;
            chunks = 0;
        }
        ++in;
        chunks += (n[i] + kChunk - 1) / kChunk;
    }
    return (size_t)(parts + (chunks < kClipGrid ? chunks : kClipGrid) + 1) * 4;
}

static hipError_t square_sums(int count, const void *const *g, const int64_t *n,
                              const int *g_type, float *part, int *parts, hipStream_t s) {
    *parts = 0;
    return over_tables(count, g, n, g_type, nullptr, nullptr, [&](const Table &t) {
        square_sums_kernel<<<grid_of(t), kClipThreads, 0, s>>>(t, part + *parts);
        *parts += (int)grid_of(t);
        return hipGetLastError();
    });
}

static hipError_t norm_of_parts(const float *part, int parts, float *norm, hipStream_t s) {
    norm_kernel<<<1, 1024, 0, s>>>(part, parts, norm);
    return hipGetLastError();
}

hipError_t launch_grad_norm(int count, const void *const *g, const int64_t *n, const int *g_type,
                            float *norm, float *part, hipStream_t s) {
    int parts;
    const hipError_t e = square_sums(count, g, n, g_type, part, &parts, s);
    return e != hipSuccess ? e : norm_of_parts(part, parts, norm, s);
}

hipError_t launch_grad_clip(int count, const void *const *g, const int64_t *n, const int *g_type,
                            void *const *out, const int *out_type, float max_norm, float eps,
                            float *norm, float *part, hipStream_t s, hipEvent_t ev_norm) {
    int parts;
    hipError_t e = square_sums(count, g, n, g_type, part, &parts, s);
    if (e == hipSuccess && (parts == 0 || parts > kPartsMax)) {
        e = norm_of_parts(part, parts, norm, s);
        parts = 0;
    }
    if (e == hipSuccess && ev_norm) e = hipEventRecord(ev_norm, s);
    if (e != hipSuccess) return e;
    return over_tables(count, g, n, g_type, out, out_type, [&](const Table &t) {
        clip_kernel<<<grid_of(t), kClipThreads, 0, s>>>(t, part, parts, max_norm, eps, norm);
        return hipGetLastError();
    });
}

}  // namespace tw
