// The host rules of the tuning calls' launches (tune.h) over their documented
// sizes: every launch of a call whose buffers a card can hold has fewer than
// 2^32 threads along a dimension and covers its blocks; the sizes that no launch
// can take are known before anything is enqueued.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "tune.h"

static int failures = 0;
static int64_t checked = 0;

static void expect(bool ok, const char* what, int64_t a, int64_t b, int64_t c) {
    ++checked;
    if (!ok) {
        std::printf("FAIL %s: %lld %lld %lld\n", what, (long long)a, (long long)b, (long long)c);
        ++failures;
    }
}
static void rows(const char* what, int64_t blocks, int64_t threads, int64_t a, int64_t b) {
    const qt::GridRows g = qt::grid_rows(blocks, threads);
    const int64_t n = (int64_t)g.x * g.y;
    expect(g.x >= 1 && g.y >= 1 && g.y <= 65535 && qt::launch_fits(g.x, threads), what, a, b, g.x);
    expect(n >= blocks && n - blocks < g.y, what, a, b, n);
    expect(blocks * threads >= (1LL << 32) || g.y == 1, what, a, b, g.y);
}

int main() {
    const int64_t most = 1 << 22, big = 1 << 20;
    const double card = 288e9;
    for (int64_t T : {(int64_t)1, (int64_t)64, (int64_t)65, (int64_t)200, (int64_t)1025,
                      (int64_t)70000, most / 4 + 1, most - 1, most})
        for (int64_t D : {(int64_t)1, (int64_t)64, (int64_t)5120, (int64_t)8192, (int64_t)8256,
                          (int64_t)16384, (int64_t)40000, (int64_t)200000, big})
            for (bool bf16 : {false, true}) {
                rows("planes", qt::x_planes_blocks(T, D, true), 256, T, D);
                rows("planes in rows", qt::x_planes_blocks(T, D, false), 256, T, D);
                for (int64_t F : {(int64_t)1, (int64_t)16, (int64_t)2048, (int64_t)18432,
                                  (int64_t)50257, (int64_t)200000, big}) {
                    const double e = bf16 ? 2 : 4, G = (D + 63) / 64;
                    const qt::FfnPlan p = qt::ffn_plan(T, D, F, bf16);
                    if (T * e * (D + F) + 56.0 * F * G + p.bytes <= card)
                        expect(qt::ffn_fits(p, T, F), "ffn", T, D, F);
                    for (int nmat : {1, 2}) {
                        const qt::BwdPlan b = qt::bwd_plan(T, D, F, nmat, bf16, true, true);
                        if (T * e * (2.0 * D + F) + 28.0 * nmat * F * G + b.bytes <= card)
                            expect(qt::bwd_fits(b, T, D, F, true, true), "bwd", T, D, F);
                    }
                }
            }
    for (int64_t T : {(int64_t)1, (int64_t)127, (int64_t)128, (int64_t)1025, most - 1, most})
        for (int64_t V : {(int64_t)1, (int64_t)5000, (int64_t)16392, (int64_t)131073, qt::kDistillMaxV - 1})
            for (bool bf16 : {false, true}) {
                rows("loss", T, 1024, T, V);
                expect(qt::launch_fits(T * qt::distill_splits(T, V, bf16), 256), "split", T, V, 0);
                expect(qt::launch_fits(T * qt::distill_bwd_splits(T, V, bf16), 256), "grad", T, V, 0);
            }
    rows("loss of most rows", most, 1024, most, 0);
    expect(qt::grid_rows(most, 1024).y == 2, "2^32 threads", most, 1024, 0);
    // no card holds these; the guards see them
    expect(!qt::ffn_fits(qt::ffn_plan(most, big, big, true), most, big), "ffn", most, big, big);
    expect(!qt::bwd_fits(qt::bwd_plan(most, big, big, 2, true, true, false), most, big, big, true, false),
           "dx", most, big, big);
    expect(!qt::bwd_fits(qt::bwd_plan(most, big, big, 2, true, false, true), most, big, big, false, true),
           "ds", most, big, big);
    std::printf("%lld checks, %d failures\n", (long long)checked, failures);
    return failures != 0;
}
