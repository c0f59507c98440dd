// api_check.h -- host-side checks that the C-ABI layers share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gdn2.h"

namespace gdn2 {
namespace api {

struct Span {
    const void *p;
    int64_t bytes;
};

inline bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Outputs overlap neither the inputs nor each other.
inline bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(*o, i)) return false;
        for (const Span *x = o + 1; x != outs.end(); ++x)
            if (overlap(*o, *x)) return false;
    }
    return true;
}

// a*b*.. fits in int64
inline bool product_ok(std::initializer_list<int64_t> fs) {
    int64_t x = 1;
    for (int64_t f : fs) {
        if (f < 0) return false;
        if (f != 0 && x > INT64_MAX / f) return false;
        x *= f;
    }
    return true;
}

inline gdn2_status hip_status(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP; }

inline bool workspace_ok(const void *ws, size_t have, size_t need) {
    return have >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0;
}

}  // namespace api
}  // namespace gdn2
