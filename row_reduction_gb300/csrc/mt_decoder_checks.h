// mt_decoder_checks.h -- checks of arguments that the C entry points of the
// decoder's row operators share (decoder.cpp, step.cpp).
#pragma once

#include <stdint.h>

#include "mt_internal.h"

namespace mt {

inline bool misaligned(const void *p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}
inline bool known_dtype(int dt) { return dt >= 0 && dt < DT_COUNT; }

// Element offsets stay below this: twice the byte size of the widest type
// still fits an int64.
constexpr int64_t kMaxOffset = INT64_MAX / 16;

// |a| * b <= kMaxOffset for b >= 0 (adds to *sum, which must stay so too).
inline bool add_extent(int64_t stride, int64_t n, int64_t *sum) {
    if (n <= 1 || stride == 0) return true;
    if (stride == INT64_MIN) return false;
    const int64_t a = stride < 0 ? -stride : stride;
    if (a > (kMaxOffset - *sum) / (n - 1)) return false;
    *sum += a * (n - 1);
    return true;
}
inline bool reachable(int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
    int64_t sum = 1024;
    return add_extent(ts, tokens, &sum) && add_extent(hs, heads, &sum);
}
// Rows of an output (tokens x heads rows of dim values) do not overlap: the
// smaller stride steps over a row, the larger one over all rows of the
// other.
inline bool disjoint(int64_t ts, int64_t hs, int64_t tokens, int64_t heads,
              int64_t dim) {
    const int64_t t = ts < 0 ? -ts : ts, h = hs < 0 ? -hs : hs;
    if (tokens > 1 && t < dim) return false;
    if (heads > 1 && h < dim) return false;
    if (tokens > 1 && heads > 1)
        return t <= h ? h >= t * (tokens - 1) + dim
                      : t >= h * (heads - 1) + dim;
    return true;
}

// Largest V in {full, ..., 2, 1} whose packs of V*es bytes fit every listed
// address, stride and offset (all in `bits`, OR-ed together, in elements for
// strides and offsets and in bytes/es for addresses).
inline int widest(uint64_t bits, int full) {
    int v = full;
    while (v > 1 && (bits & (uint64_t)(v - 1))) v >>= 1;
    return v;
}

}  // namespace mt
