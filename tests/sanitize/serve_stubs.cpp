// Test stubs of the launchers that the validation layer of the serving calls
// (api_serve.cpp) makes, so that it can be built on the host alone with the
// sanitizers.  A stub never touches a buffer (the driver passes fake device
// addresses); it works out what its launcher would launch and reports success.
#include <hip/hip_runtime.h>

#include "serve.h"

int qt_stub_launches = 0;

namespace qt {
hipError_t launch_kv_write(const KvCache&, const KvRows&, const int32_t*, int64_t, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
hipError_t launch_kv_read(const KvCache&, const int32_t*, int64_t, void*, void*, bool, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
hipError_t launch_attn_decode(const AttnArgs& a, void*, hipStream_t) {
    const AttnPlan p = attn_plan(a.B, a.c.heads, a.q_heads, a.c.dim, a.table_pages, a.c.page,
                                 a.window);
    const int64_t tiles = (a.q_heads / a.c.heads + 15) / 16;
    const int64_t span = a.table_pages * a.c.page;
    // every position has a chunk, no chunk is larger than a block takes, the grid
    // and its rows are numbered in 31 bits
    const bool covers = a.window != 0 || (int64_t)p.splits * p.chunk >= span;
    const bool fits = p.chunk <= kAttnMaxChunk && p.chunk % 128 == 0 &&
                      (a.B * (int64_t)a.c.heads * p.splits + 7) / 8 * 8 * tiles < INT32_MAX;
    const bool short_ok = p.waves == kAttnWaves || (p.splits == 1 && a.c.groups <= 2);
    if (covers && fits && short_ok) ++qt_stub_launches;
    return hipSuccess;
}
size_t moe_layer_workspace(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F) {
    return (size_t)(T * k * (4 * (D + 3 * F) + 16) + 4 * E + 96);  // of the layer's size
}
hipError_t launch_moe_few(const FewArgs&, void*, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
}  // namespace qt

extern "C" int64_t qt_groups(int64_t I) { return I < 1 ? 0 : (I - 1) / 64 + 1; }
