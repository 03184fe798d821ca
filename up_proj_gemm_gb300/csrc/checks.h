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

constexpr int64_t kI32Max = 0x7fffffffLL;

}  // namespace mlaq
