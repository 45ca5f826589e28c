// Host-side argument checks shared by the sources of the C-ABI layer.
#pragma once
#include "qt.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "qt_internal.h"

namespace {

using qt::kGroup;
using qt::kGroupBytes;
using qt::kGroupBytesI4;

// Overflow-checked product a*b*c of non-negative sizes; -1 on overflow.
int64_t mul3(int64_t a, int64_t b, int64_t c) {
    __int128 p = (__int128)a * b * c;
    if (p > INT64_MAX) return -1;
    return (int64_t)p;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte ranges [p, p+n) and [q, q+m) overlap.
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
    if (!p || !q || n <= 0 || m <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// gbytes: packed bytes per group (24 for int3, 32 for int4)
qt_status shape_ok(int64_t O, int64_t I, int64_t gbytes = kGroupBytes) {
    if (O < 1 || I < 1 || I > QT_MAX_I) return QT_ERR_SHAPE;
    if (mul3(O, (I + kGroup - 1) / kGroup, gbytes) < 0 || mul3(O, I, 4) < 0)
        return QT_ERR_SHAPE;
    return QT_OK;
}

[[maybe_unused]] qt_status launched(hipError_t e) { return e == hipSuccess ? QT_OK : QT_ERR_LAUNCH; }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace
