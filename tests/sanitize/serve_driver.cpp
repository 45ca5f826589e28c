// Drives the validation layer of the serving calls through valid calls at the
// ends of their ranges and through every kind of refusal; no argument may
// reach undefined behaviour.
#include <climits>
#include <cmath>
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
static T* at(int slot) {  // fake device addresses, 2^58 bytes apart
    return reinterpret_cast<T*>((uintptr_t)(slot + 1) << 58);
}

static int write(int64_t T, int64_t ld, int64_t n, int64_t page, int64_t heads, int64_t dim,
                 qt_dtype xt = QT_BF16, int kb = 8, int vb = 4, uintptr_t off = 0) {
    return qt_kv_write(at<char>(0) + off, ld, at<char>(1), ld, xt, T, at<int32_t>(2), at<uint8_t>(3),
                       at<float>(4), kb, at<uint8_t>(5), at<float>(6), vb, n, page, heads, dim,
                       nullptr);
}
static int read(int64_t R, int64_t n, int64_t page, int64_t heads, int64_t dim,
                qt_dtype xt = QT_F32, bool k = true, bool v = true) {
    return qt_kv_read(at<int32_t>(2), R, at<uint8_t>(3), at<float>(4), 4, at<uint8_t>(5),
                      at<float>(6), 8, n, page, heads, dim, k ? at<char>(7) : nullptr,
                      v ? at<char>(8) : nullptr, xt, nullptr);
}
static int attn(int64_t B, int64_t hq, int64_t heads, int64_t dim, int64_t n, int64_t page,
                int64_t pages, int64_t window, int64_t ld, float scale = 1.0f,
                qt_dtype xt = QT_BF16, size_t ws = SIZE_MAX) {
    return qt_attn_decode(
        at<char>(0), ld, xt, B, hq, at<uint8_t>(3), at<float>(4), 8, at<uint8_t>(5), at<float>(6), 4,
        n, page, heads, dim, at<int32_t>(1), pages, at<int32_t>(2), window, scale, at<char>(7),
        at<float>(8), at<char>(9),
        ws == SIZE_MAX ? qt_attn_decode_workspace_bytes(B, hq, heads, dim, pages, page, window) : ws,
        nullptr);
}
static int moe(int64_t T, int64_t D, int64_t F, int E, int k, qt_dtype xt = QT_BF16, int bits = 3,
               int act = 0, size_t ws = SIZE_MAX) {
    return qt_moe_decode(at<char>(0), xt, T, D, F, at<float>(1), E, k, (qt_act)act, at<uint8_t>(2),
                         at<float>(3), bits, at<uint8_t>(4), at<float>(5), bits, at<uint8_t>(6),
                         at<float>(7), 7 - bits, at<char>(8), at<char>(9),
                         ws == SIZE_MAX ? qt_moe_decode_workspace_bytes(T, k, E, D, F, xt) : ws,
                         nullptr);
}

int main() {
    const int64_t most = (int64_t(1) << 31) - (1 << 16);  // slots
    for (qt_dtype t : {QT_F32, QT_BF16}) {
        for (int64_t T : {(int64_t)1, (int64_t)4097, (int64_t)1 << 22})
            for (int64_t heads : {1, 7, 1024})
                for (int64_t dim : {1, 65, 256}) {
                    expect("write", write(T, heads * dim, 9, 16, heads, dim, t), QT_OK, 1);
                    if (T < 1 << 22)  // a larger span than the fake addresses' distance
                        expect("write ld", write(T, (int64_t)1 << 38, 9, 16, heads, dim, t), QT_OK, 1);
                    expect("write n", write(T, heads * dim, most / 16, 16, heads, dim, t, 4, 4),
                           QT_OK, 1);
                    expect("read", read(T, 9, 48, heads, dim, t), QT_OK, 1);
                    expect("read K", read(T, 9, 48, heads, dim, t, true, false), QT_OK, 1);
                    expect("read V", read(T, 9, 48, heads, dim, t, false, true), QT_OK, 1);
                }
        for (int64_t B : {1, 3, 64, 65535})
            for (int64_t heads : {1, 8})
                for (int64_t per : {1, 5, 17, 256})
                    for (int64_t dim : {1, 128, 129, 256})
                        for (int64_t pages : {1, 63, 64, 65, 8192})
                            for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)1000, INT64_MAX})
                                if (B * heads * per < (1 << 20))
                                    expect("attn", attn(B, heads * per, heads, dim, 100, 16, pages,
                                                        window, heads * per * dim, 1.0f, t),
                                           QT_OK, 1);
        expect("attn longest", attn(1, 8, 8, 64, 100, 16, most / 16, 0, 512, 1.0f, t), QT_OK, 1);
        expect("attn window", attn(1, 8, 8, 64, 100, 16, most / 16, INT64_MAX, 512, 1.0f, t), QT_OK, 1);
        expect("attn blocks", attn(65535, 64, 64, 64, 100, 16, most / 16, 0, 4096, 1.0f, t),
               QT_ERR_SHAPE, 0);
        expect("attn rows", attn(65535, 512, 512, 64, 100, 16, 1, 0, 512 * 64, 1.0f, t),
               QT_ERR_SHAPE, 0);
        for (int64_t T : {1, 16})
            for (int64_t D : {(int64_t)1, (int64_t)65, (int64_t)1 << 20})
                for (int64_t F : {(int64_t)1, (int64_t)17, (int64_t)1 << 20})
                    for (int E : {1, 32, 512})
                        expect("moe", moe(T, D, F, E, E < 32 ? E : 32, t, 4, 1), QT_OK, 1);
    }
    for (int64_t bad : {(int64_t)0, (int64_t)-1, INT64_MIN, INT64_MAX, ((int64_t)1 << 62) + 16}) {
        expect("write T", write(bad, 64, 4, 16, 1, 64), QT_ERR_SHAPE, 0);
        expect("write n", write(4, 64, bad, 16, 1, 64), QT_ERR_SHAPE, 0);
        expect("write page", write(4, 64, 4, bad, 1, 64), QT_ERR_SHAPE, 0);
        expect("write heads", write(4, 64, 4, 16, bad, 64), QT_ERR_SHAPE, 0);
        expect("write dim", write(4, 64, 4, 16, 1, bad), QT_ERR_SHAPE, 0);
        expect("write ld", write(4, bad, 4, 16, 1, 64), QT_ERR_SHAPE, 0);
        expect("read R", read(bad, 4, 16, 1, 64), QT_ERR_SHAPE, 0);
        expect("read n", read(4, bad, 16, 1, 64), QT_ERR_SHAPE, 0);
        expect("attn B", attn(bad, 8, 8, 64, 9, 16, 2, 0, 512), QT_ERR_SHAPE, 0);
        expect("attn hq", attn(1, bad, 8, 64, 9, 16, 2, 0, 512), QT_ERR_SHAPE, 0);
        expect("attn heads", attn(1, 8, bad, 64, 9, 16, 2, 0, 512), QT_ERR_SHAPE, 0);
        expect("attn pages", attn(1, 8, 8, 64, 9, 16, bad, 0, 512), QT_ERR_SHAPE, 0);
        expect("attn ld", attn(1, 8, 8, 64, 9, 16, 2, 0, bad), QT_ERR_SHAPE, 0);
        expect("moe T", moe(bad, 64, 64, 8, 2), QT_ERR_SHAPE, 0);
        expect("moe D", moe(4, bad, 64, 8, 2), QT_ERR_SHAPE, 0);
        expect("moe F", moe(4, 64, bad, 8, 2), QT_ERR_SHAPE, 0);
        expect("bytes", qt_kv_bytes(bad, 16, 1, 64, 4) == 0 ? 0 : 1, 0, 0);
        expect("bytes", qt_kv_bytes(4, 16, 1, bad, 4) == 0 ? 0 : 1, 0, 0);
    }
    for (int64_t window : {(int64_t)-1, INT64_MIN})
        expect("attn window", attn(1, 8, 8, 64, 9, 16, 2, window, 512), QT_ERR_SHAPE, 0);
    for (int bad : {0, -1, INT_MIN, INT_MAX, 513}) {
        expect("moe E", moe(4, 64, 64, bad, 1), QT_ERR_SHAPE, 0);
        expect("moe k", moe(4, 64, 64, 8, bad), QT_ERR_SHAPE, 0);
        expect("write bits", write(4, 64, 4, 16, 1, 64, QT_F32, bad), QT_ERR_ARG, 0);
    }
    expect("moe bits", moe(4, 64, 64, 8, 2, QT_F32, 5), QT_ERR_ARG, 0);
    expect("moe act", moe(4, 64, 64, 8, 2, QT_F32, 3, 9), QT_ERR_ARG, 0);
    expect("moe ws", moe(4, 64, 64, 8, 2, QT_F32, 3, 0, 15), QT_ERR_WORKSPACE, 0);
    expect("attn ws", attn(1, 8, 8, 64, 9, 16, 9000, 0, 512, 1.0f, QT_F32, 1), QT_ERR_WORKSPACE, 0);
    expect("attn nan", attn(1, 8, 8, 64, 9, 16, 2, 0, 512, NAN), QT_ERR_ARG, 0);
    expect("attn inf", attn(1, 8, 8, 64, 9, 16, 2, 0, 512, -INFINITY), QT_ERR_ARG, 0);
    expect("write align", write(4, 64, 4, 16, 1, 64, QT_F32, 8, 8, 2), QT_ERR_ALIGN, 0);
    expect("type", write(4, 64, 4, 16, 1, 64, (qt_dtype)7), QT_ERR_DTYPE, 0);
    std::printf("%d failures\n", failures);
    return failures != 0;
}
