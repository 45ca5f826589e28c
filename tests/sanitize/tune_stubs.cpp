// Test stubs of the launchers that the validation layer of the tuning calls
// (api_tune.cpp) makes, so that it can be built on the host alone with the
// sanitizers.  A stub never touches a buffer (the driver passes fake device
// addresses); it counts the launch and reports success.
#include <hip/hip_runtime.h>

#include "tune.h"

int qt_stub_launches = 0;

namespace qt {
hipError_t launch_ffn_gated(const FfnArgs&, void*, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
hipError_t launch_bwd(const BwdArgs&, void*, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
hipError_t launch_distill(const DistillArgs&, float*, float*, void*, int64_t, void*, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
hipError_t launch_distill_bwd(const DistillArgs&, const float*, void*, int64_t, hipStream_t) {
    ++qt_stub_launches;
    return hipSuccess;
}
}  // namespace qt

extern "C" int64_t qt_groups(int64_t I) { return I < 1 ? 0 : (I - 1) / 64 + 1; }
