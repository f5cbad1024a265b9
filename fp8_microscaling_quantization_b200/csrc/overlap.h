// overlap.h -- host-side checks of buffers that share memory.
#pragma once

#include <cstddef>

namespace bsq {

// Do [a, a + na) and [b, b + nb) share a byte?
static inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    return a && b && (const char*)a < (const char*)b + nb && (const char*)b < (const char*)a + na;
}

// A buffer of a call (NULL: not there), and whether one of the outputs shares a
// byte with an input or with another output.
struct Span {
    const void* p;
    size_t n;
};
template <int NO, int NI>
static inline bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span& s : ins)
            if (overlap(outs[i].p, outs[i].n, s.p, s.n)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
}

}  // namespace bsq
