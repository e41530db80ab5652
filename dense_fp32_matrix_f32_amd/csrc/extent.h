// extent.h -- sizes of a call, and byte ranges of its arrays for the overlap checks of
// the entry points (host only, no HIP call).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace sgemm {

// Byte extent [lo, hi) of a rows x cols row-major array of `size`-byte elements
// with row stride ld elements (rows, cols, ld >= 1).  Sizes near the int range
// make the byte count exceed 64 bits, so it is formed in 128 bits and hi
// saturates at the top of the address space rather than wrapping below lo.
struct Extent {
    uintptr_t lo, hi;
};

inline Extent bytes_from(const void *p, unsigned __int128 bytes) {
    const uintptr_t lo = (uintptr_t)p;
    const unsigned __int128 hi = (unsigned __int128)lo + bytes;
    return {lo, hi > (unsigned __int128)UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)hi};
}

inline Extent extent(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size) {
    return bytes_from(
        p, ((unsigned __int128)(uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * size);
}

// `count` such arrays, `stride` (>= 0) elements apart.
inline Extent extent(const void *p, int64_t count, int64_t stride, int64_t rows, int64_t cols,
                     int64_t ld, size_t size) {
    return bytes_from(p, ((unsigned __int128)(uint64_t)(count - 1) * (uint64_t)stride +
                          (unsigned __int128)(uint64_t)(rows - 1) * (uint64_t)ld +
                          (uint64_t)cols) *
                             size);
}

// The operators by expert and with 4-bit weights take sizes that stay inside 31 bits
// when they are rounded up to blocks or stepped past by a grid.
constexpr int kMaxSize = INT32_MAX - 65536;

inline bool valid_size(int n) { return n >= 0 && n <= kMaxSize; }

inline bool overlaps(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace sgemm
