// Argument checks shared by the C entry points (host side): byte ranges,
// overlap, alignment.
#pragma once
#include <cstddef>
#include <cstdint>

namespace mlaq {

struct Range {
    uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
};

inline Range rng(const void* p, int64_t bytes) {
    Range r;
    if (p && bytes > 0) {
        r.lo = reinterpret_cast<uintptr_t>(p);
        r.hi = r.lo + (uintptr_t)bytes;
    }
    return r;
}

inline bool overlap(const Range& a, const Range& b) {
    return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi;
}

template <size_t NO, size_t NI>
bool any_alias(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether n rows `stride` elements apart stay below 2^58 elements, so that a
// sum of two such spans is a number of bytes in int64.
inline bool inside(int64_t n, int64_t stride) {
    return stride >= 0 && (n <= 1 || stride <= ((int64_t)1 << 58) / (n - 1));
}

constexpr int64_t kI32Max = 0x7fffffffLL;

// n / d = n * mul >> shift for 0 <= n < 2^31, d > 0: shift = 31 + the bits of d - 1, so mul is below 2^32 and the product
// below 2^63, and mul d - 2^shift < d, times n, stays below 2^shift.
struct Divisor {
    uint32_t mul, shift;
};
inline Divisor divisor(int32_t d) {
    uint32_t bits = 0;
    while (((int64_t)1 << bits) < d) ++bits;
    const uint32_t shift = 31 + bits;
    return {(uint32_t)((((uint64_t)1 << shift) + (uint64_t)d - 1) / (uint64_t)d), shift};
}

}  // namespace mlaq
