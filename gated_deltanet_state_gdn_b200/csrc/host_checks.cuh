// host_checks.cuh -- pointer checks of the C ABI's entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdn {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// [p, p + bytes) and [q, q + qbytes) intersect (both non-empty)
inline bool overlaps(const void *p, size_t bytes, const void *q, size_t qbytes)
{
    if (!p || !q || bytes == 0 || qbytes == 0) return false;
    uintptr_t a0 = (uintptr_t)p, a1 = a0 + bytes;
    uintptr_t b0 = (uintptr_t)q, b1 = b0 + qbytes;
    return a0 < b1 && b0 < a1;
}

}  // namespace gdn
