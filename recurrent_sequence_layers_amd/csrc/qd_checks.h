// Host-side argument checks shared by the C ABI entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace qd {

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Buf {
    const void *p;
    size_t n;
};

// Every output must be disjoint from every input and from every other output.  The one
// exception is the in-place state update: the output `same_out` may be exactly the input
// `same_in` (same address; a partial overlap is still rejected).
inline bool disjoint(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs, const void *same_in = nullptr,
                     const void *same_out = nullptr) {
    for (const Buf &o : outs) {
        for (const Buf &i : ins) {
            if (same_in && o.p == same_out && i.p == same_in && o.p == i.p) continue;
            if (overlaps(o.p, o.n, i.p, i.n)) return false;
        }
        for (const Buf &o2 : outs)
            if (&o2 != &o && overlaps(o.p, o.n, o2.p, o2.n)) return false;
    }
    return true;
}

}  // namespace qd
