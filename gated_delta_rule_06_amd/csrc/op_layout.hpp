// Sizes that the layer operators' host code and kernels share. Host-compilable.
#pragma once

#include <stddef.h>

#include <algorithm>

namespace muir {

inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

namespace hd {

constexpr int C = 64;      // tokens of a chunk
constexpr int ANCHOR = 4;  // chunks between the boundaries whose <S, A> the decay's gradient starts from

inline int chunks_of(int T) { return T / C + (T % C != 0); }
inline int groups_of(int T) { return (chunks_of(T) + ANCHOR - 1) / ANCHOR; }

}  // namespace hd

// Workgroups of the norm's backward: each keeps one row of dweight, so they are few.
inline int norm_bwd_blocks(int rows, int D) {
    const int rpb = D <= 2048 ? 4 : 1;
    return std::max(1, std::min(rows / rpb + (rows % rpb != 0), 512));
}

}  // namespace muir
