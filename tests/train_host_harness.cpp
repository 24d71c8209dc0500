// Host-only harness over the argument checks of the dense training step's entry
// points (include/tw.h), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host side and run on the CPU: every call is
// rejected before anything reaches a device (fake addresses that are never read),
// over the extremes of every size.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "tw.h"

namespace {

int g_fail = 0;

void expect(int line, bool ok) {
    if (!ok) {
        std::printf("FAIL line %d (%s)\n", line, tw_last_error());
        ++g_fail;
    }
}
#define REJECTED(call) expect(__LINE__, (call) != TW_OK && std::strlen(tw_last_error()) > 0)
#define EXPECT(call, want) expect(__LINE__, (int)(call) == (want))
#define CHECK(what) expect(__LINE__, (what))

template <typename T>
T *fake(uintptr_t a = 0x100000) {
    return reinterpret_cast<T *>(a);
}

struct Shape {
    int M = 4, K = 64, N = 72;
    int64_t stride = 64;
    size_t ws = 16;
    int act = TW_SILU, target = TW_INT64, out = TW_BF16;
    uint16_t *x = fake<uint16_t>();
};

int ffn(Shape s) {
    return tw_gated_ffn_fwd(s.x, s.stride, fake<uint16_t>(), fake<uint16_t>(), fake<uint16_t>(),
                            s.act, s.M, s.K, s.N, nullptr, nullptr, fake<void>(), s.out,
                            fake<void>(), s.ws, nullptr, nullptr);
}
int ffn_bwd(Shape s) {
    return tw_gated_ffn_bwd(fake<uint16_t>(), s.x, s.stride, fake<uint16_t>(), fake<uint16_t>(),
                            fake<uint16_t>(), s.act, fake<uint16_t>(), fake<uint16_t>(), s.M, s.K,
                            s.N, fake<void>(), s.out, fake<void>(), fake<void>(), fake<void>(),
                            TW_F32, fake<void>(), s.ws, nullptr, nullptr);
}
int ce(Shape s) {
    return tw_linear_ce_fwd(s.x, s.stride, fake<uint16_t>(), fake<void>(), s.target, s.M, s.K, s.N,
                            fake<float>(), fake<float>(), fake<void>(), s.ws, nullptr, nullptr);
}
int ce_bwd(Shape s) {
    return tw_linear_ce_bwd(fake<float>(), s.x, s.stride, fake<uint16_t>(), fake<void>(), s.target,
                            fake<float>(), s.M, s.K, s.N, fake<void>(), s.out, fake<void>(), TW_F32,
                            fake<void>(), s.ws, nullptr, nullptr);
}
int rms(Shape s) {
    return tw_rmsnorm_fwd(s.x, TW_BF16, s.stride, nullptr, 0, fake<float>(), 1e-5f, s.M, s.K,
                          nullptr, fake<void>(), s.out, nullptr, nullptr, nullptr);
}
int rms_quant(Shape s) {
    return tw_rmsnorm_quant(s.x, TW_BF16, s.stride, nullptr, 0, fake<float>(), 1e-5f, s.M, s.K,
                            nullptr, fake<int8_t>(), fake<float>(), nullptr, nullptr);
}
int rms_bwd(Shape s) {
    return tw_rmsnorm_bwd(fake<void>(), TW_BF16, s.x, TW_BF16, s.stride, fake<float>(),
                          fake<float>(), nullptr, s.M, s.K, fake<void>(), s.out, fake<float>(),
                          fake<void>(), s.ws, nullptr, nullptr);
}

}  // namespace

int main() {
    int (*const all[])(Shape) = {ffn, ffn_bwd, ce, ce_bwd, rms, rms_quant, rms_bwd};
    int (*const tiled[])(Shape) = {ffn, ffn_bwd, ce, ce_bwd};
    for (auto f : all) {
        for (int v : {INT_MIN, INT_MIN + 1, -1, 0}) {
            Shape s;
            s.K = v;
            REJECTED(f(s));
            s = {};
            if (v) {
                s.M = v;
                REJECTED(f(s));
            }
        }
        for (int64_t v : {INT64_MIN, (int64_t)-1, (int64_t)0, (int64_t)63}) {
            Shape s;
            s.stride = v;
            REJECTED(f(s));
        }
        Shape s;
        s.x = nullptr;
        REJECTED(f(s));
    }
    for (auto f : tiled) {
        for (int v : {INT_MIN, -1, 0, INT_MAX}) {
            Shape s;
            s.N = v;
            REJECTED(f(s));
        }
        for (int v : {INT_MAX, INT_MAX - 7, 65, (1 << 20) + 8}) {
            Shape s;
            s.K = v;
            s.stride = INT64_MAX;
            REJECTED(f(s));
            s.stride = (int64_t)v + 8;
            REJECTED(f(s));
        }
        Shape s;
        s.M = INT_MAX;
        REJECTED(f(s));
        s = {};
        s.stride = INT64_MAX - 7;
        EXPECT(f(s), TW_EUNSUPPORTED);
        s = {};
        s.act = 7, s.target = TW_F32;
        REJECTED(f(s));
        // sizes that are taken, workspaces that are not: each plan is computed
        for (int M : {1, 16, 17, 32, 33, 64, 65, 777, 4096, 1 << 20, 1 << 24})
            for (int K : {8, 64, 1000, 2048, 1 << 20})
                for (int N : {8, 72, 2728, 32768, 1 << 20, 1 << 24}) {
                    s = {};
                    s.M = M, s.K = K, s.N = N, s.stride = K;
                    REJECTED(f(s));
                }
    }
    // bigger sizes never need less, and the queries never overflow
    for (int K : {8, 1000, 1 << 20})
        for (int N : {8, 2728, 1 << 20})
            for (int M : {1, 65, 4096, 1 << 20}) {
                CHECK(tw_gated_ffn_workspace_bytes(M, K, N) >= (size_t)M * N * 2);
                CHECK(tw_gated_ffn_bwd_workspace_bytes(M, K, N) >= 3 * (size_t)M * N * 2);
                CHECK(tw_linear_ce_workspace_bytes(M, K, N) >= (size_t)M * ((N + 127) / 128) * 8);
                CHECK(tw_linear_ce_bwd_workspace_bytes(M, K, N) > 0);
            }
    for (int v : {INT_MIN, -1, 7, INT_MAX}) {
        CHECK(tw_gated_ffn_workspace_bytes(4, v, 64) == 0);
        CHECK(tw_gated_ffn_bwd_workspace_bytes(4, 64, v) == 0);
        CHECK(tw_linear_ce_workspace_bytes(4, v, 64) == 0);
        CHECK(tw_linear_ce_bwd_workspace_bytes(v == 7 ? -7 : v, 64, 64) == 0);
    }

    // clipping: counts, sizes, types, addresses, overlaps
    const void *g[3] = {fake<void>(0x10000), fake<void>(0x20000), fake<void>(0x30000)};
    void *out[3] = {fake<void>(0x40000), fake<void>(0x50000), fake<void>(0x60000)};
    int64_t n[3] = {100, 0, 300};
    int types[3] = {TW_BF16, TW_F32, TW_F32}, outs[3] = {TW_BF16, TW_BF16, TW_F32};
    auto clip = [&](int count, size_t ws = 4, float most = 1.0f, float eps = 0.0f) {
        return tw_grad_clip(count, g, n, types, out, outs, most, eps, fake<float>(0x1000),
                            fake<void>(0x2000), ws, nullptr, nullptr);
    };
    EXPECT(clip(3), TW_EINVAL);  // the workspace
    for (int v : {INT_MIN, -1, INT_MAX}) {
        REJECTED(clip(v));
        CHECK(tw_grad_norm_workspace_bytes(v, n) == 0);
    }
    const size_t need = tw_grad_norm_workspace_bytes(3, n);
    REJECTED(clip(3, need, -1.0f));
    REJECTED(clip(3, need, 1.0f, -1.0f));
    for (int64_t v : {INT64_MIN, (int64_t)-1, INT64_MAX, (int64_t)1 << 35}) {
        n[0] = v;
        REJECTED(clip(3, SIZE_MAX));
        n[0] = 100;
    }
    types[2] = TW_INT8;
    REJECTED(clip(3, need));
    types[2] = TW_F32;
    for (void *p : {fake<void>(0x40001), fake<void>(0), fake<void>(0x4ffff - 0x100)}) {
        out[2] = p;
        REJECTED(clip(3, need));
    }
    out[2] = fake<void>(0x40000 + 198);  // the last element of out[0]
    REJECTED(clip(3, need));
    out[2] = fake<void>(0x10000 + 196);  // within g[0]
    REJECTED(clip(3, need));
    out[2] = const_cast<void *>(g[2]);
    outs[2] = TW_BF16;  // in place of another type
    REJECTED(clip(3, need));
    outs[2] = TW_F32;
    const void *twice = g[0];
    g[0] = g[2];
    n[0] = 300, types[0] = TW_F32, outs[0] = TW_F32;
    out[0] = out[2];  // the same buffer twice
    REJECTED(clip(3, need));
    g[0] = twice;
    std::vector<int64_t> many(1 << 20, (int64_t)1 << 34);
    CHECK(tw_grad_norm_workspace_bytes(1 << 20, many.data()) > 0);
    many.assign(1 << 20, INT64_MIN);
    CHECK(tw_grad_norm_workspace_bytes(1 << 20, many.data()) > 0);
    if (g_fail == 0) std::printf("HARNESS_OK\n");
    return g_fail != 0;
}
