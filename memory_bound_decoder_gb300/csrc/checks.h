// Host-side checks that the entry points of the key-value cache and of what goes with it share.
#pragma once

#include <stdint.h>

#include "mbd.h"

namespace mbd {
namespace checks {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A byte range that a call reads or writes.
struct Range {
    const void* p;
    uint64_t n;
};

inline bool overlap(const Range& a, const Range& b) {
    const uint64_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

template <int N>
bool overlaps_any(const Range& a, const Range (&all)[N]) {
    for (const Range& r : all)
        if (overlap(a, r)) return true;
    return false;
}

// Bytes from the first to behind the last element of `rows` rows of `width` bf16, `stride` elements apart.
inline uint64_t rows_bytes(int64_t rows, int64_t stride, int64_t width) {
    return (uint64_t(rows - 1) * uint64_t(stride) + uint64_t(width)) * 2;
}

inline mbd_status check_stride(int64_t* stride, int64_t width) {
    if (*stride == 0) *stride = width;
    if (*stride < width) return MBD_ERR_INVALID_ARG;
    if (*stride % 8 != 0) return MBD_ERR_MISALIGNED;
    if (*stride > (int64_t{1} << 34)) return MBD_ERR_UNSUPPORTED;
    return MBD_OK;
}

}  // namespace checks
}  // namespace mbd
