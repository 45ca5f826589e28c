// Reductions over a wave in a fixed order; every lane gets the result.
#pragma once
#include <hip/hip_runtime.h>

namespace qt {

// Drops a NaN, as fmaxf does.
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

}  // namespace qt
