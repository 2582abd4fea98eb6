// Sizes that the layer operators' host code and kernels share. Host-compilable.
#pragma once

#include <stddef.h>

#include <algorithm>

namespace muir {

inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

namespace hd {

constexpr int C = 64;      // tokens of a chunk
// Chunks between the boundaries whose <S, A> the decay's gradient starts from. Four: 714 us for the backward of B8 T4096 H16 d128
// and a fixed decay's gradient 1.6 times as far off as the plain float32 form over 12 drawn bf16 calls; two: 748 us and 0.8
// times; one: 832 us and 1.3 times (a boundary every 64 tokens, but each token from its group's end).
constexpr int ANCHOR = 2;

inline int chunks_of(int T) { return T / C + (T % C != 0); }
inline int groups_of(int T) { return (chunks_of(T) + ANCHOR - 1) / ANCHOR; }

}  // namespace hd

// Workgroups of the norm's backward: each keeps one row of dweight, so they are few.
inline int norm_bwd_blocks(int rows, int D) {
    const int rpb = D <= 2048 ? 4 : 1;
    return std::max(1, std::min(rows / rpb + (rows % rpb != 0), 512));
}

}  // namespace muir
