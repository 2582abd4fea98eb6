// Which rows a workgroup of the attention kernels has, and where a token lies in a paged cache. Host-compilable: the same code
// runs in the kernels and, without a GPU, in their tests.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define MUIR_HD __host__ __device__ __forceinline__
#else
#define MUIR_HD inline
#endif

namespace muir {
namespace at {

constexpr float LOG2E = 1.4426950408889634f;  // the kernels take exponentials to base 2, with it in the scale

MUIR_HD int cut(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Rows of one call's sequences. Sequence s has the rows first(s) .. first(s + 1), of which the first `lens[s]` are tokens; "sequence" S is
// what lies behind the last one and has none. Offsets are cut to 0 .. N, so that whatever they hold, every access stays inside.
struct Sequences {
    const int *offsets, *lens;
    int N, S;
    bool by_place;  // the order in which blocks are taken, below
    MUIR_HD int first(int s) const {
        if (s <= 0) return 0;
        if (s > S) return N;
        return offsets ? cut(offsets[s], 0, N) : s * (N / S);
    }
    MUIR_HD int rows(int s) const {
        const int n = first(s + 1) - first(s);
        return n > 0 ? n : 0;
    }
    MUIR_HD int tokens(int s) const { return s >= S ? 0 : lens ? cut(lens[s], 0, rows(s)) : rows(s); }
};

// What a block of `R` rows has of a sequence: the sequence's first row, rows and tokens, and the block's first row in it. A block without rows, past its
// sequence's or found by offsets that do not ascend, has at >= rows; at is never below 0.
struct Block {
    int seq, lo, rows, n, at;
};
MUIR_HD Block no_block(const Sequences &q) { return Block{q.S, q.N, 0, 0, 0}; }

// A launch has N / R + S + 1 blocks, never fewer than the sequences need. By place, those with the most work go first: the place of a block in its
// sequence says how many keys its queries see, and, counted from the end, how many queries its keys have (FROM_END), so blocks are taken place by place,
// the highest first, each place over all the sequences that have it. Otherwise one sequence is taken after another, which suits a window: blocks are
// worth about the same, and neighbours share their keys.
//
// Sequences of equal length need no search.
MUIR_HD Block equal_block(const Sequences &q, int R, int i, bool from_end) {
    const int rows = q.N / q.S, per = (rows + R - 1) / R;
    if (i >= per * q.S) return no_block(q);
    const int s = q.by_place ? i % q.S : i / per, up = q.by_place ? i / q.S : i % per;
    return Block{s, s * rows, rows, q.tokens(s), (q.by_place && !from_end ? per - 1 - up : up) * R};
}
// The place of block `i`, where count(p) is how many blocks have place p or a higher one (i < count(0)), and none has `top`.
template <typename Count> MUIR_HD int search_place(int top, int i, Count count) {
    int lo = 0, hi = top;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (count(mid) > i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One sequence after another, in rising order of their blocks: also where 64 of them and more would have to be counted by place. Sequence s has the blocks from first(s) / R + s on: at most one more
// than it needs, so no sums over the lengths are needed. 64 sequences are looked at in a step: count(lo, step, hi) says how many of s = lo, lo + step, ..
// (64 of them, up to hi) have first(s) / R + s <= w.
template <typename Count> MUIR_HD int search_sequence(int S, Count count) {
    int lo = 0, hi = S;
    while (hi > lo) {
        const int step = (hi - lo) / 64 + 1, n = count(lo, step, hi);
        lo += (n > 1 ? n - 1 : 0) * step;
        hi = lo + step - 1 < hi ? lo + step - 1 : hi;
    }
    return lo;
}
// Block `w` of those, found to be in sequence `s`.
MUIR_HD Block block_in(const Sequences &q, int R, int w, int s) {
    const int lo = q.first(s), rows = q.rows(s), at = (w - lo / R - s) * R;
    return Block{s, lo, rows, q.tokens(s), at < 0 ? rows : at};
}

// Work item of a workgroup: consecutive workgroups go round the eight XCDs, so that the heads of one key head, all their blocks, run on
// one of them, whose L2 then holds that head's keys and values; what is left over eight key heads goes round by blocks. Blocks
// come in their order.
struct Item {
    int block, h;
};
MUIR_HD Item find_item(int id, int blocks, int H, int Hk) {
    const int G = H / Hk, full = Hk / 8, per = blocks * G * 8;
    int hk, rest;
    if (id < full * per) {
        hk = id / per * 8 + id % 8;
        rest = id % per / 8;
    } else {
        const int left = Hk - full * 8;
        id -= full * per;
        hk = full * 8 + id % left;
        rest = id / left;
    }
    return Item{rest / G, hk * G + rest % G};
}

// A paged cache [pages, Hk, page, d]: the page of a token, whether there is one, and the token's row among all rows.
struct Pages {
    const int *table;
    int pages, log_page, width, Hk;
    MUIR_HD int64_t room() const { return static_cast<int64_t>(width) << log_page; }
    MUIR_HD int id(int b, int pos) const { return table[static_cast<size_t>(b) * width + (pos >> log_page)]; }
    MUIR_HD bool good(int id) const { return static_cast<unsigned>(id) < static_cast<unsigned>(pages); }
    MUIR_HD size_t row(int id, int hk, int pos) const {
        return ((static_cast<size_t>(id) * Hk + hk) << log_page) + (pos & ((1 << log_page) - 1));
    }
};

// What a step's sequence has: keys in the cache, keys with the new one, the first that is seen, and the tiles of 32 from there on.
struct Span {
    int old, n, begin, t0, t1;
};
MUIR_HD Span step_span(int len, bool appends, int window, int64_t room) {
    const bool fits = len >= 0 && static_cast<int64_t>(len) + appends <= room;
    const int n = fits ? len + appends : 0, begin = window > 0 && n > window ? n - window : 0;
    return Span{fits ? len : 0, n, begin, begin / 32, (n + 31) / 32};
}

}  // namespace at
}  // namespace muir
