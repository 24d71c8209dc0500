// Host-only harness over the argument checks of the layer-norm and int8
// entry points (include/tw.h), built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host side and run on the CPU: every call
// is rejected before anything reaches a device (fake addresses that are never
// read), over the extremes of every size.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "tw.h"

namespace {

int g_fail = 0;

void expect(int line, int got, int want) {
    if (got != want || std::strlen(tw_last_error()) == 0) {
        std::printf("FAIL line %d: %d, want %d (%s)\n", line, got, want, tw_last_error());
        ++g_fail;
    }
}
#define EXPECT(call, want) expect(__LINE__, (int)(call), (want))

template <typename T>
T *fake(uintptr_t a = 0x100000) {
    return reinterpret_cast<T *>(a);
}

struct Row {
    int M = 4, K = 64, xt = TW_BF16;
    int64_t stride = 64;
    void *x = fake<void>();
};

int fwd(Row r) {
    return tw_layernorm_fwd(r.x, r.xt, r.stride, nullptr, 0, fake<float>(), nullptr, 1e-5f, r.M,
                            r.K, nullptr, fake<void>(), TW_BF16, nullptr, nullptr, nullptr, nullptr);
}
int bwd(Row r) {
    return tw_layernorm_bwd(fake<void>(), TW_BF16, r.x, r.xt, r.stride, fake<float>(),
                            fake<float>(), fake<float>(), nullptr, r.M, r.K, fake<void>(), TW_F32,
                            fake<float>(), fake<float>(), fake<void>(), 16, nullptr, nullptr);
}
int rows(Row r) {
    return tw_quant_rows(r.x, r.xt, r.stride, r.M, r.K, fake<int8_t>(), fake<float>(), nullptr,
                         nullptr);
}
int lnq(Row r) {
    return tw_layernorm_quant(r.x, r.xt, r.stride, nullptr, 0, fake<float>(), nullptr, 1e-5f, r.M,
                              r.K, nullptr, fake<int8_t>(), fake<float>(), nullptr, nullptr);
}
int linear(Row r, int N, size_t ws = 16) {
    return tw_quant_linear(r.x, r.xt, r.stride, r.xt == TW_INT8 ? fake<float>() : nullptr,
                           fake<int8_t>(), fake<float>(), nullptr, r.M, r.K, N, fake<void>(),
                           TW_BF16, fake<void>(), ws, nullptr, nullptr);
}
int gateup(Row r, int N, size_t ws = 16, const float *gamma = nullptr) {
    return tw_quant_gateup(r.x, r.xt, r.stride, nullptr, gamma, nullptr, 1e-5f, fake<int8_t>(),
                           fake<float>(), fake<int8_t>(), fake<float>(), r.M, r.K, N, fake<void>(),
                           TW_BF16, fake<void>(), ws, nullptr, nullptr);
}

}  // namespace

int main() {
    const int sizes[] = {INT_MIN, INT_MIN + 1, -1, 0};
    for (int v : sizes) {
        Row r;
        r.K = v;
        EXPECT(fwd(r), TW_EINVAL);
        EXPECT(bwd(r), TW_EINVAL);
        EXPECT(rows(r), TW_EINVAL);
        EXPECT(lnq(r), TW_EINVAL);
        EXPECT(linear(r, 64), TW_EINVAL);
        EXPECT(gateup(r, 64), TW_EINVAL);
        Row k;
        EXPECT(linear(k, v), TW_EINVAL);
        EXPECT(gateup(k, v), TW_EINVAL);
        if (v < 0) {
            k.M = v;
            EXPECT(fwd(k), TW_EINVAL);
            EXPECT(bwd(k), TW_EINVAL);
            EXPECT(rows(k), TW_EINVAL);
            EXPECT(linear(k, 64), TW_EINVAL);
        }
    }
    Row big;
    big.K = INT_MAX;
    big.stride = INT_MAX;
    EXPECT(fwd(big), TW_EUNSUPPORTED);
    EXPECT(bwd(big), TW_EUNSUPPORTED);
    EXPECT(rows(big), TW_EUNSUPPORTED);
    EXPECT(linear(big, 64), TW_EUNSUPPORTED);
    big.K = 65536;
    big.stride = 65536;
    big.M = INT_MAX;
    EXPECT(linear(big, 64), TW_EUNSUPPORTED);
    EXPECT(gateup(big, INT_MAX), TW_EUNSUPPORTED);
    big.M = 1 << 24;
    EXPECT(linear(big, 1 << 24), TW_EUNSUPPORTED);   // too many tiles
    EXPECT(linear(big, 64), TW_EINVAL);               // workspace of 2^40 bytes wanted
    EXPECT(gateup(big, 64, (size_t)1 << 40), TW_EINVAL);  // ... and the scales'
    EXPECT(gateup(big, 64, 16, fake<float>()), TW_EUNSUPPORTED);
    Row s;
    for (int64_t v : {INT64_MIN, int64_t(-64), int64_t(0), int64_t(63)}) {
        s.stride = v;
        EXPECT(fwd(s), TW_EINVAL);
        EXPECT(linear(s, 64), TW_EINVAL);
    }
    s.stride = INT64_MAX;
    EXPECT(fwd(s), TW_EUNSUPPORTED);
    EXPECT(rows(s), TW_EUNSUPPORTED);
    Row t;
    for (int v : {INT_MIN, -1, 3, INT_MAX}) {
        t.xt = v;
        EXPECT(fwd(t), TW_EINVAL);
        EXPECT(rows(t), TW_EINVAL);
        EXPECT(linear(t, 64), TW_EINVAL);
    }
    Row p;
    p.x = fake<void>(0x100008);
    EXPECT(fwd(p), TW_EINVAL);
    EXPECT(linear(p, 64, 1 << 20), TW_EINVAL);
    // workspace queries over the extremes: a size or 0, never an overflow
    size_t sum = 0;
    for (int M : {INT_MIN, -1, 0, 1, 1 << 24, INT_MAX})
        for (int K : {INT_MIN, -1, 0, 1, 16, 16384, 65536, INT_MAX}) {
            sum |= tw_quant_workspace_bytes(M, K);
            sum |= tw_layernorm_bwd_workspace_bytes(M, K);
        }
    if (sum == 0 || sum > (size_t)1 << 42) {
        std::printf("FAIL workspace queries: %zu\n", sum);
        ++g_fail;
    }
    if (g_fail) return 1;
    std::printf("HARNESS_OK\n");
    return 0;
}
