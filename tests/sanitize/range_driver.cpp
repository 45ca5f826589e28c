// Drives the validation layer of the tuning calls through alignments and
// temperatures that it accepts and refuses, over the stubs of tune_stubs.cpp.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "qt.h"

extern int qt_stub_launches;
static int failures = 0;

static void expect(const char* what, int got, int want) {
    if (got != want || qt_stub_launches != (want == QT_OK)) {
        std::printf("FAIL %s: status %d (want %d), launches %d\n", what, got, want,
                    qt_stub_launches);
        ++failures;
    }
    qt_stub_launches = 0;
}

template <typename T>
static T* at(int slot) {  // fake device addresses, 2^54 bytes apart
    return reinterpret_cast<T*>((uintptr_t)(slot + 1) << 54);
}

static int ffn(int64_t T, int64_t D, qt_dtype xt, uintptr_t xo) {
    return qt_ffn_gated(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 4, 64, D,
                        QT_ACT_SILU, at<char>(4) + xo, xt, T, at<char>(5), nullptr, at<char>(7),
                        qt_ffn_gated_workspace_bytes(T, D, 64, xt), nullptr);
}
static int bwd(int64_t T, int64_t D, qt_dtype xt, uintptr_t xo) {
    return qt_ffn_gated_bwd(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 4, 64, D,
                            QT_ACT_SILU, at<float>(4), at<char>(5), at<char>(6) + xo, xt, T,
                            at<char>(7), at<float>(8), at<float>(9), 0, at<char>(10),
                            qt_ffn_gated_bwd_workspace_bytes(T, D, 64, xt, 1, 1), nullptr);
}
static int lin(int64_t B, int64_t I, qt_dtype xt, uintptr_t xo) {
    return qt_matmul_bwd(at<uint8_t>(0), at<float>(1), 4, 64, I, at<char>(2), QT_F32,
                         at<char>(3) + xo, xt, B, at<char>(4), at<float>(5), 0, at<char>(6),
                         qt_matmul_bwd_workspace_bytes(B, I, 64, xt, 1, 1), nullptr);
}
static int loss(float tau, bool bwd) {
    if (bwd)
        return qt_distill_topk_bwd(at<char>(0), QT_BF16, 4, 64, 64, at<int32_t>(1), at<float>(2), 3,
                                   tau, at<float>(4), nullptr, at<char>(3), 64, nullptr);
    return qt_distill_topk(at<char>(0), QT_F32, 4, 64, 64, at<int32_t>(1), at<float>(2), 3, tau,
                           at<float>(4), at<float>(5), nullptr, at<char>(3), 64, nullptr, 0, nullptr);
}

int main() {
    // temperatures whose inverse (times log2 e) is no f32 number, or whose product
    // with a logarithm is none, would give NaN
    for (bool bwd : {false, true}) {
        for (float tau : {0x1p-149f, 1e-39f, 2e-39f, 0x1.fffffep-101f, 0x1.000002p100f, 0x1p127f, -1.0f,
                          0.0f, __builtin_inff(), __builtin_nanf("")})
            expect("tau", loss(tau, bwd), QT_ERR_ARG);
        for (float tau : {0x1p-100f, 1e-4f, 1.0f, 100.0f, 0x1p100f}) expect("tau", loss(tau, bwd), QT_OK);
    }
    // only forward calls that may read rows of whole groups in place want 16 bytes
    for (int T : {1, 4, 64}) {
        expect("small", ffn(T, 128, QT_BF16, 8), QT_ERR_ALIGN);
        expect("small", ffn(T, 128, QT_BF16, 16), QT_OK);
        expect("small, ragged", ffn(T, 100, QT_BF16, 2), QT_OK);
        expect("small, f32", ffn(T, 128, QT_F32, 4), QT_OK);
    }
    for (int T : {65, 4096}) expect("tile", ffn(T, 128, QT_BF16, 2), QT_OK);
    for (int T : {1, 64, 65, 4096}) {
        expect("bwd", bwd(T, 128, QT_BF16, 2), QT_OK);
        expect("bwd", bwd(T, 128, QT_F32, 4), QT_OK);
        expect("bwd", bwd(T, 128, QT_BF16, 1), QT_ERR_ALIGN);
        expect("bwd", bwd(T, 128, QT_F32, 2), QT_ERR_ALIGN);
        expect("lin", lin(T, 128, QT_BF16, 2), QT_OK);
        expect("lin", lin(T, 128, QT_F32, 4), QT_OK);
        expect("lin", lin(T, 128, QT_BF16, 1), QT_ERR_ALIGN);
        expect("lin", lin(T, 128, QT_F32, 2), QT_ERR_ALIGN);
    }
    std::printf("%d failures\n", failures);
    return failures != 0;
}
