// The attention's plan (host code): its chunks reach every position that a sequence
// of any length attends to, whatever the window, and none is longer than a block takes.
#include <cstdint>
#include <cstdio>

#include "serve.h"

static long failures = 0, plans = 0;

// Chunks start at multiples of a tile of 32 positions: what a sequence of n tokens needs.
static int64_t need(int64_t n, int64_t window) {
    const int64_t lo = window > 0 && window < n ? n - window : 0;
    return n - lo / 32 * 32;
}

static void check(int64_t B, int64_t heads, int64_t per, int64_t dim, int64_t pages, int64_t page,
                  int64_t window) {
    const qt::AttnPlan p = qt::attn_plan(B, heads, heads * per, dim, pages, page, window);
    const int64_t reach = pages * page;
    int64_t worst = 0;  // the longest span repeats with n every 32 positions
    for (int64_t n = reach; n > 0 && n > reach - 33; --n)
        worst = need(n, window) > worst ? need(n, window) : worst;
    if (window > 0)  // and where the window just fits
        for (int64_t n = window; n <= reach && n - window <= 33; ++n)
            worst = need(n, window) > worst ? need(n, window) : worst;
    const int64_t G = (dim + 63) / 64;
    const int64_t bytes = p.splits == 1 ? 0 : B * heads * per * p.splits * (G * 64 + 4) * 4;
    const bool ok = (int64_t)p.splits * p.chunk >= worst && p.splits >= 1 && p.chunk % 128 == 0 &&
                    p.chunk <= qt::kAttnMaxChunk && p.bytes == bytes &&
                    (p.waves == qt::kAttnWaves || (p.waves == qt::kAttnMaxWaves && p.splits == 1 && G <= 2));
    ++plans;
    if (!ok && ++failures < 10)
        std::printf("FAIL B=%lld heads=%lld per=%lld dim=%lld pages=%lld page=%lld window=%lld: "
                    "%d chunks of %d for %lld\n",
                    (long long)B, (long long)heads, (long long)per, (long long)dim, (long long)pages,
                    (long long)page, (long long)window, p.splits, p.chunk, (long long)worst);
}

int main() {
    const int64_t windows[] = {0,   1,   2,   31,  32,   33,   63,   64,   97,   127,  128, 225, 256, 257,
                               481, 500, 512, 700, 992, 993, 994, 1000, 1024, 1025, 1500, 2017, 2048, 2049,
                               4095, 4096, 30000, INT64_MAX - 40, INT64_MAX};
    for (int64_t B : {1, 3, 24, 64, 700})
        for (int64_t heads : {1, 2, 8, 64})
            for (int64_t per : {1, 8, 17, 256})
                for (int64_t dim : {1, 65, 128, 129, 256})
                    for (int64_t page : {16, 48, 64, 1008, 65536})
                        for (int64_t reach : {16, 33, 256, 272, 700, 1024, 1040, 2048, 4097, 12000, 131072})
                            for (int64_t window : windows)
                                check(B, heads, per, dim, (reach + page - 1) / page, page, window);
    // the longest tables
    for (int64_t page : {16, 48, 65536})
        for (int64_t window : windows)
            check(1, 8, 4, 128, qt::kKvMaxSlots / page, page, window);
    std::printf("%ld plans, %ld failures\n", plans, failures);
    return failures != 0;
}
