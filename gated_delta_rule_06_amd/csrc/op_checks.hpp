// Argument checks that the C ABI's sources of the layer operators share: types, alignment, overlaps, the workspace.
#pragma once

#include <string.h>

#include "checks.hpp"

namespace muir {

inline bool known(muir_dtype_t t) { return t == MUIR_F32 || t == MUIR_BF16; }
inline size_t size_of(muir_dtype_t t) { return t == MUIR_BF16 ? 2 : 4; }
inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Buffer {
    Range r;
    size_t align;
    const char *same_as;  // an output that may be exactly this input, or NULL
};

inline Buffer buf(const char *name, const void *p, size_t bytes, size_t align = 16, const char *same_as = nullptr) {
    return Buffer{range(name, p, bytes), align, same_as};
}

// Alignment of every buffer, and no output over an input or another output.
inline muir_status_t check_buffers(const char *fn, std::initializer_list<Buffer> in, std::initializer_list<Buffer> out) {
    for (const auto *list : {&in, &out})
        for (const Buffer &x : *list)
            if (x.r.lo % x.align != 0)
                return fail(MUIR_ERR_SHAPE, "%s: %s must be %zu-byte aligned", fn, x.r.name, x.align);
    for (const Buffer &o : out) {
        for (const Buffer &x : in) {
            const bool same = o.same_as && strcmp(o.same_as, x.r.name) == 0 && o.r.lo == x.r.lo && o.r.hi == x.r.hi;
            if (!same && overlaps(o.r, x.r)) return fail(MUIR_ERR_ALIAS, "%s: %s overlaps %s", fn, o.r.name, x.r.name);
        }
        for (const Buffer &y : out)
            if (&y != &o && overlaps(o.r, y.r))
                return fail(MUIR_ERR_ALIAS, "%s: %s overlaps %s", fn, o.r.name, y.r.name);
    }
    return MUIR_OK;
}

inline muir_status_t check_workspace(const char *fn, const void *workspace, size_t have, size_t need) {
    if (need == 0) return MUIR_OK;
    if (!workspace) return fail(MUIR_ERR_WORKSPACE, "%s: workspace of %zu bytes required", fn, need);
    if (have < need) return fail(MUIR_ERR_WORKSPACE, "%s: workspace has %zu bytes, need %zu", fn, have, need);
    if (!aligned(workspace, 256)) return fail(MUIR_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", fn);
    return MUIR_OK;
}

}  // namespace muir
