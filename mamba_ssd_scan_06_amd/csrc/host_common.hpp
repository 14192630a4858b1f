// Host-side helpers shared by the C entry points: the per-thread error text,
// overlap checks of buffers and overflow-safe extents of strided tensors.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kernels.hpp"
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

// Argument checks of the operators around the scan.
namespace host {

constexpr int64_t kMaxBatch = 65535;             // a grid dimension
constexpr int64_t kMaxTokens = (int64_t)1 << 31;  // token indices fit 32 bits
constexpr int64_t kMaxWide = (int64_t)1 << 20;    // channels, norm dims

inline size_t elem_size(ssd_dtype dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }
inline Elem elem(ssd_dtype dtype) { return dtype == SSD_DTYPE_BF16 ? Elem::BF16 : Elem::F32; }

inline ssd_status check_dtype(ssd_dtype dtype) {
    if (dtype != SSD_DTYPE_F32 && dtype != SSD_DTYPE_BF16) return fail(SSD_ERR_ARGS, "unknown dtype %d", (int)dtype);
    return SSD_OK;
}

struct Ptr {
    const char *name;
    const void *p;
    size_t align;
};

template <int K>
ssd_status check_align(const Ptr (&ptrs)[K]) {
    for (const Ptr &q : ptrs)
        if ((uintptr_t)q.p % q.align != 0) return fail(SSD_ERR_ALIGN, "%s is not %zu-byte aligned", q.name, q.align);
    return SSD_OK;
}

// An output that may be one of the inputs itself (an in-place update).
struct InPlace {
    int out, in;
};

// No output may overlap an input or another output, except the allowed pairs
// of identical pointers.
template <int NO, int NI, int NA>
ssd_status check_alias(const Range (&outs)[NO], const Range (&ins)[NI], const InPlace (&allowed)[NA]) {
    for (int i = 0; i < NO; ++i) {
        for (int k = 0; k < NI; ++k) {
            bool same = false;
            for (const InPlace &a : allowed)
                same = same || (a.out == i && a.in == k && outs[i].lo == ins[k].lo && outs[i].hi == ins[k].hi);
            if (!same && overlaps(outs[i], ins[k]))
                return fail(SSD_ERR_ALIAS, "%s overlaps %s", outs[i].name, ins[k].name);
        }
        for (int k = i + 1; k < NO; ++k)
            if (overlaps(outs[i], outs[k])) return fail(SSD_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[k].name);
    }
    return SSD_OK;
}

// A stride of a dimension without a second index is never used: 0 keeps it
// out of the offsets.
inline int64_t used_stride(int64_t n, int64_t stride) { return n > 1 ? stride : 0; }

inline ssd_status launched(const char *what, hipError_t r) {
    if (r != hipSuccess) return fail(SSD_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(r));
    return SSD_OK;
}

}  // namespace host
}  // namespace ssd
