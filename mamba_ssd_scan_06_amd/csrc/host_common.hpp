// Host-side helpers shared by the C entry points: the per-thread error text,
// overlap checks of buffers and overflow-safe extents of strided tensors.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {

// Records the text ssd_last_error() returns on this thread; returns `s`.
__attribute__((format(printf, 2, 3))) ssd_status fail(ssd_status s, const char *fmt, ...);

struct Range {
    const char *name;
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char *name, const void *p, size_t bytes) {
    uintptr_t lo = (uintptr_t)p;
    return Range{name, lo, p ? lo + bytes : lo};
}

inline bool overlaps(const Range &a, const Range &b) {
    return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}

// Largest extent of a tensor in elements that the kernels' 64-bit offsets are
// checked for; far beyond any memory, far below overflow.
constexpr int64_t kMaxExtent = (int64_t)1 << 46;

// Elements from the first to one past the last of a strided tensor
// [n0][n1][inner] (0 when it is empty), or -1 when a size or stride is
// negative or the extent passes kMaxExtent.
inline int64_t extent3(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner) {
    if (n0 < 0 || n1 < 0 || inner < 0) return -1;
    if (n0 == 0 || n1 == 0 || inner == 0) return 0;
    if (n0 == 1) s0 = 0;
    if (n1 == 1) s1 = 0;
    int64_t a, b, sum;
    if (s0 < 0 || s1 < 0 || __builtin_mul_overflow(n0 - 1, s0, &a) || __builtin_mul_overflow(n1 - 1, s1, &b) ||
        __builtin_add_overflow(a, b, &sum) || __builtin_add_overflow(sum, inner, &sum) || sum > kMaxExtent)
        return -1;
    return sum;
}

// Product of up to four sizes >= 0, or -1 when it passes kMaxExtent.
inline int64_t product(int64_t a, int64_t b, int64_t c = 1, int64_t d = 1) {
    int64_t r = 1;
    for (int64_t v : {a, b, c, d})
        if (v < 0 || __builtin_mul_overflow(r, v, &r) || r > kMaxExtent) return -1;
    return r;
}

}  // namespace ssd
