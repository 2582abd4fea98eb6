// Argument checks shared by the C ABI's sources: the error detail of the calling thread, buffer overlap,
// products of sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "muir.h"

namespace muir {

// Sets the thread's error detail and returns s; ok() clears it. Defined in api.cpp.
muir_status_t fail(muir_status_t s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
muir_status_t ok();

struct Range {
    const char *name;
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range(const char *name, const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + bytes : lo};
}

inline bool overlaps(const Range &x, const Range &y) {
    if (x.lo == x.hi || y.lo == y.hi) return false;
    return x.lo < y.hi && y.lo < x.hi;
}

// size = a*b*c*d with overflow detection (all factors >= 0).
inline bool mul_size(size_t &out, std::initializer_list<size_t> f) {
    size_t acc = 1;
    for (size_t x : f) {
        if (x != 0 && acc > SIZE_MAX / x) return false;
        acc *= x;
    }
    out = acc;
    return true;
}

inline muir_status_t check_hip(hipError_t err, const char *what) {
    if (err != hipSuccess) return fail(MUIR_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
    return ok();
}

}  // namespace muir
