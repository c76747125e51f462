// Argument checks shared by the newer entry points of the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gdr.h"

namespace gdr {
namespace api {

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool given16(const void *p) { return p != nullptr && aligned(p, 16); }
inline bool maybe16(const void *p) { return p == nullptr || aligned(p, 16); }
inline bool head_dim(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }
inline bool io_type(gdr_dtype_t t) { return t == GDR_F32 || t == GDR_BF16; }

struct Range {
    const void *p;
    size_t n;
};

inline bool overlap(const Range &a, const Range &b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether every output lies apart from every input and every other output.
template <size_t I, size_t O>
bool apart(const Range (&in)[I], const Range (&out)[O]) {
    for (size_t o = 0; o < O; ++o) {
        for (size_t i = 0; i < I; ++i)
            if (overlap(out[o], in[i])) return false;
        for (size_t u = o + 1; u < O; ++u)
            if (overlap(out[o], out[u])) return false;
    }
    return true;
}

}  // namespace api
}  // namespace gdr
