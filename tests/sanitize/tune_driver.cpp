// Drives the validation layer of the tuning calls through valid calls at the
// ends of their ranges (sizes where products pass 32 and near 63 bits) and
// through every kind of refusal; no argument may reach undefined behaviour.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "qt.h"

extern int qt_stub_launches;
static int failures = 0;

static void expect(const char* what, int got, int want, int launches) {
    if (got != want || qt_stub_launches != launches) {
        std::printf("FAIL %s: status %d (want %d), launches %d (want %d)\n", what, got, want,
                    qt_stub_launches, launches);
        ++failures;
    }
    qt_stub_launches = 0;
}

template <typename T>
static T* at(int slot) {  // fake device addresses, 2^54 bytes apart
    return reinterpret_cast<T*>((uintptr_t)(slot + 1) << 54);
}

static int ffn(int64_t T, int64_t D, int64_t F, qt_dtype xt, int gb = 3, int ub = 4,
               int act = 0, uintptr_t xo = 0, size_t ws = SIZE_MAX) {
    return qt_ffn_gated(at<uint8_t>(0), at<float>(1), gb, at<uint8_t>(2), at<float>(3), ub, F, D,
                        (qt_act)act, at<char>(4) + xo, xt, T, at<char>(5), at<float>(6), at<char>(7),
                        ws == SIZE_MAX ? qt_ffn_gated_workspace_bytes(T, D, F, xt) : ws, nullptr);
}
static int bwd(int64_t T, int64_t D, int64_t F, qt_dtype xt, bool dx, bool ds, int acc = 0,
               size_t ws = SIZE_MAX) {
    return qt_ffn_gated_bwd(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 4, F, D,
                            QT_ACT_GELU, at<float>(4), at<char>(5), ds ? at<char>(6) : nullptr, xt, T,
                            dx ? at<char>(7) : nullptr, ds ? at<float>(8) : nullptr,
                            ds ? at<float>(9) : nullptr, acc, at<char>(10),
                            ws == SIZE_MAX ? qt_ffn_gated_bwd_workspace_bytes(T, D, F, xt, dx, ds) : ws,
                            nullptr);
}
static int lin(int64_t B, int64_t I, int64_t O, qt_dtype xt, qt_dtype yt, int bits = 3) {
    return qt_matmul_bwd(at<uint8_t>(0), at<float>(1), bits, O, I, at<char>(2), yt, at<char>(3), xt,
                         B, at<char>(4), at<float>(5), 1, at<char>(6),
                         qt_matmul_bwd_workspace_bytes(B, I, O, xt, 1, 1), nullptr);
}
static int dist(int64_t T, int64_t V, int64_t ldl, int64_t ldd, int k, float tau,
                qt_dtype lt = QT_BF16, int dst = 3) {
    return qt_distill_topk(at<char>(0), lt, T, V, ldl, at<int32_t>(1), at<float>(2), k, tau,
                           at<float>(4), at<float>(5), at<float>(6), at<char>(dst), ldd, at<char>(7),
                           qt_distill_topk_workspace_bytes(T, V, lt), nullptr);
}
static int dist_bwd(int64_t T, int64_t V, int64_t ldl, int64_t ldd, int k, float tau) {
    return qt_distill_topk_bwd(at<char>(0), QT_F32, T, V, ldl, at<int32_t>(1), at<float>(2), k, tau,
                               at<float>(4), nullptr, at<char>(3), ldd, nullptr);
}

int main() {
    const int64_t big = 1 << 20, most = 1 << 22;
    const qt_dtype types[2] = {QT_F32, QT_BF16};
    for (qt_dtype t : types) {
        for (int64_t T : {(int64_t)1, (int64_t)64, (int64_t)65, (int64_t)4097, most})
            for (int64_t D : {(int64_t)1, (int64_t)65, big})
                for (int64_t F : {(int64_t)1, (int64_t)17, big}) {
                    expect("ffn", ffn(T, D, F, t), QT_OK, 1);
                    expect("bwd", bwd(T, D, F, t, true, true), QT_OK, 1);
                    expect("bwd dx", bwd(T, D, F, t, true, false), QT_OK, 1);
                    expect("bwd ds", bwd(T, D, F, t, false, true, 1), QT_OK, 1);
                    expect("lin", lin(T, D, F, t, QT_F32), QT_OK, 1);
                    expect("lin", lin(T, D, F, t, QT_BF16, 4), QT_OK, 1);
                }
        for (int64_t T : {(int64_t)1, (int64_t)127, (int64_t)128, most})
            for (int64_t V : {(int64_t)1, (int64_t)5000, (int64_t)131073, (int64_t)INT_MAX})
                if (T < most || V < INT_MAX)  // larger spans than the fake addresses' distance
                    expect("dist", dist(T, V, V, V < INT_MAX ? V + 1 : V, 1024, 1.0f, t), QT_OK, 1);
    }
    for (int64_t bad : {(int64_t)0, (int64_t)-1, INT64_MIN, INT64_MAX, most + 1}) {
        expect("ffn T", ffn(bad, 64, 64, QT_F32), QT_ERR_SHAPE, 0);
        expect("ffn D", ffn(4, bad, 64, QT_F32), QT_ERR_SHAPE, 0);
        expect("ffn F", ffn(4, 64, bad, QT_F32), QT_ERR_SHAPE, 0);
        expect("bwd T", bwd(bad, 64, 64, QT_BF16, true, true), QT_ERR_SHAPE, 0);
        expect("bwd D", bwd(4, bad, 64, QT_BF16, true, true), QT_ERR_SHAPE, 0);
        expect("bwd F", bwd(4, 64, bad, QT_BF16, true, true), QT_ERR_SHAPE, 0);
        expect("lin", lin(4, 64, bad, QT_BF16, QT_F32), QT_ERR_SHAPE, 0);
        expect("dist T", dist(bad, 64, 64, 64, 1, 1.0f), QT_ERR_SHAPE, 0);
        if (bad != most + 1) {
            expect("dist V", dist(4, bad, bad, bad, 1, 1.0f), QT_ERR_SHAPE, 0);
            expect("dist ld", dist(4, 64, bad, 64, 1, 1.0f), QT_ERR_SHAPE, 0);
            expect("dist ldd", dist(4, 64, 64, bad, 1, 1.0f), QT_ERR_SHAPE, 0);
        }
    }
    expect("ld < V", dist(4, 64, 63, 64, 1, 1.0f), QT_ERR_SHAPE, 0);
    expect("ldd < V", dist_bwd(4, 64, 64, 63, 1, 1.0f), QT_ERR_SHAPE, 0);
    expect("bwd ok", dist_bwd(4, 64, 65, 66, 1, 1.0f), QT_OK, 1);
    for (int k : {0, -1, 1025, INT_MAX}) expect("k", dist(4, 64, 64, 64, k, 1.0f), QT_ERR_ARG, 0);
    for (float tau : {0.0f, -1.0f, __builtin_nanf(""), __builtin_inff()})
        expect("tau", dist(4, 64, 64, 64, 2, tau), QT_ERR_ARG, 0);
    expect("in place", dist(4, 64, 80, 80, 2, 1.0f, QT_BF16, 0), QT_OK, 1);
    expect("in place, other stride", dist(4, 64, 80, 81, 2, 1.0f, QT_BF16, 0), QT_ERR_ALIAS, 0);
    expect("in place, one row", dist(1, 64, 80, 81, 2, 1.0f, QT_BF16, 0), QT_OK, 1);
    expect("gradient over idx", dist(4, 64, 64, 64, 2, 1.0f, QT_BF16, 1), QT_ERR_ALIAS, 0);
    expect("gradient over loss", dist(4, 64, 64, 64, 2, 1.0f, QT_BF16, 4), QT_ERR_ALIAS, 0);
    for (int bits : {0, 2, 5, -3, 16}) {
        expect("gate bits", ffn(4, 64, 64, QT_F32, bits), QT_ERR_ARG, 0);
        expect("up bits", ffn(4, 64, 64, QT_F32, 3, bits), QT_ERR_ARG, 0);
        expect("lin bits", lin(4, 64, 64, QT_F32, QT_F32, bits), QT_ERR_ARG, 0);
    }
    expect("act", ffn(4, 64, 64, QT_F32, 3, 3, 2), QT_ERR_ARG, 0);
    expect("type", ffn(4, 64, 64, (qt_dtype)2), QT_ERR_DTYPE, 0);
    expect("type", lin(4, 64, 64, QT_F32, (qt_dtype)7), QT_ERR_DTYPE, 0);
    expect("accumulate", bwd(4, 64, 64, QT_F32, true, true, 2), QT_ERR_ARG, 0);
    expect("nothing wanted", bwd(4, 64, 64, QT_F32, false, false), QT_ERR_NULL, 0);
    // rows read in place want 16 bytes, copied ones their elements' alignment
    expect("x + 8", ffn(4, 64, 64, QT_BF16, 3, 3, 0, 8), QT_ERR_ALIGN, 0);
    expect("x + 2, ragged", ffn(4, 65, 64, QT_BF16, 3, 3, 0, 2), QT_OK, 1);
    expect("x + 1", ffn(4, 65, 64, QT_BF16, 3, 3, 0, 1), QT_ERR_ALIGN, 0);
    expect("x + 4, f32", ffn(4, 64, 64, QT_F32, 3, 3, 0, 4), QT_OK, 1);
    expect("x + 2, f32", ffn(4, 64, 64, QT_F32, 3, 3, 0, 2), QT_ERR_ALIGN, 0);
    const size_t need = qt_ffn_gated_workspace_bytes(20, 65, 64, QT_BF16);
    expect("workspace", ffn(20, 65, 64, QT_BF16, 3, 3, 0, 0, need - 1), QT_ERR_WORKSPACE, 0);
    expect("no workspace needed", ffn(4, 64, 64, QT_BF16, 3, 3, 0, 0, 0), QT_OK, 1);
    expect("bwd workspace", bwd(4, 64, 64, QT_F32, true, true, 0, 0), QT_ERR_WORKSPACE, 0);
    expect("output over input",
           qt_ffn_gated(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 3, 64, 64,
                        QT_ACT_SILU, at<char>(4), QT_BF16, 4, at<char>(4), nullptr, nullptr, 0, nullptr),
           QT_ERR_ALIAS, 0);
    expect("outputs over each other",
           qt_ffn_gated_bwd(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 3, 64, 64,
                            QT_ACT_SILU, at<float>(4), at<char>(5), at<char>(6), QT_BF16, 4, nullptr,
                            at<float>(7), at<float>(7), 0, at<char>(8), 1 << 20, nullptr),
           QT_ERR_ALIAS, 0);
    expect("one scale gradient",
           qt_ffn_gated_bwd(at<uint8_t>(0), at<float>(1), 3, at<uint8_t>(2), at<float>(3), 3, 64, 64,
                            QT_ACT_SILU, at<float>(4), at<char>(5), at<char>(6), QT_BF16, 4, nullptr,
                            at<float>(7), nullptr, 0, at<char>(8), 1 << 20, nullptr),
           QT_ERR_NULL, 0);
    expect("packed at 8",
           qt_matmul_bwd(at<uint8_t>(0) + 8, at<float>(1), 3, 64, 64, at<char>(2), QT_F32, at<char>(3),
                         QT_F32, 4, at<char>(4), nullptr, 0, at<char>(6), 1 << 20, nullptr),
           QT_ERR_ALIGN, 0);
    expect("null", qt_matmul_bwd(nullptr, at<float>(1), 3, 64, 64, at<char>(2), QT_F32, at<char>(3),
                                 QT_F32, 4, at<char>(4), nullptr, 0, at<char>(6), 1 << 20, nullptr),
           QT_ERR_NULL, 0);
    if (qt_ffn_gated_workspace_bytes(0, 1, 1, QT_F32) || qt_matmul_bwd_workspace_bytes(1, 1, big + 1, QT_F32, 1, 1) ||
        qt_distill_topk_workspace_bytes(1, INT64_MAX, QT_F32)) {
        std::printf("FAIL workspace of a refused size\n");
        ++failures;
    }
    std::printf("%d failures\n", failures);
    return failures != 0;
}
