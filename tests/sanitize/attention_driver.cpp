// Drives the attention operators' C entry points with stand-in launchers (no GPU), and checks on the CPU what the kernels' workgroups
// take: every row once, whatever the offsets hold nothing outside the buffers, every work item once.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include <random>
#include <vector>

#include "attention_kernels.hpp"
#include "attention_layout.hpp"
#include "muir.h"

static int g_count = 0;
static hipError_t g_status = hipSuccess;

namespace muir {
static hipError_t launched() {
    ++g_count;
    return g_status;
}
hipError_t launch_attention_fwd(const AttentionCall &, void *, float *, hipStream_t) { return launched(); }
hipError_t launch_attention_bwd(const AttentionCall &, const AttentionGrads &, void *, hipStream_t) { return launched(); }
hipError_t launch_cache_append(const CacheCall &, const void *, const void *, const int *, const int *, const int *, int, int, hipStream_t) {
    return launched();
}
hipError_t launch_attention_step(const CacheCall &, const void *, const void *, const void *, const int *, void *, int, int, int, float, void *,
                                 hipStream_t) {
    return launched();
}
}  // namespace muir

static int failures = 0;
#define CHECK(x)                                      \
    do {                                              \
        if (!(x)) {                                   \
            ++failures;                               \
            printf("line %d: %s\n", __LINE__, #x);    \
        }                                             \
    } while (0)
static void expect(int got, int want, int launches, const char *what) {
    if (got != want || g_count != launches) {
        ++failures;
        printf("%s: status %d, wanted %d; %d launches, wanted %d (%s)\n", what, got, want, g_count, launches, muir_last_error());
    }
    g_count = 0;
}

template <typename T> static T *at(int i) { return reinterpret_cast<T *>((uintptr_t(1) << 40) + i * (uintptr_t(1) << 38)); }

// Block `i` of a launch as the kernels find it, the lanes one after another.
static muir::at::Block find_block(const muir::at::Sequences &q, int R, int i, int blocks, bool from_end) {
    if (!q.offsets) return muir::at::equal_block(q, R, i, from_end);
    if (q.by_place && q.S < 64) {
        std::vector<int> own(64, 0);
        int top = 0;
        for (int s = 0; s <= q.S; ++s) {
            own[s] = (q.rows(s) + R - 1) / R;
            top = own[s] > top ? own[s] : top;
        }
        auto count = [&](int p) {
            int n = 0;
            for (int x : own) n += x > p ? x - p : 0;
            return n;
        };
        if (i >= count(0)) return muir::at::no_block(q);
        const int p = muir::at::search_place(top, i, count);
        int rank = i - count(p + 1);
        CHECK(rank >= 0);
        for (int s = 0; s <= q.S; ++s)
            if (own[s] > p && rank-- == 0) return {s, q.first(s), q.rows(s), q.tokens(s), (from_end ? own[s] - 1 - p : p) * R};
        CHECK(false);
        return muir::at::no_block(q);
    }
    const int w = from_end ? i : blocks - 1 - i;
    const int s = muir::at::search_sequence(q.S, [&](int lo, int step, int hi) {
        int n = 0;
        for (int lane = 0; lane < 64; ++lane) {
            const int64_t k = int64_t(lo) + int64_t(lane) * step;
            n += k <= hi && q.first(int(k)) / R + k <= w;
        }
        return n;
    });
    CHECK(s >= 0 && s <= q.S);
    return muir::at::block_in(q, R, w, s);
}

// The blocks of a call: rows taken, each how often, and, where they are taken place by place, the most work first.
static void check_blocks(muir::at::Sequences q, int R, bool ordered) {
    const int blocks = q.N / R + q.S + 1;
    for (int turn = 0; turn < 4; ++turn) {
        const bool from_end = turn % 2;
        q.by_place = turn / 2;
        std::vector<int> taken(q.N, 0), token(q.N, 0);
        int before = INT_MAX;
        for (int i = 0; i < blocks; ++i) {
            const muir::at::Block x = find_block(q, R, i, blocks, from_end);
            CHECK(x.seq >= 0 && x.seq <= q.S && x.lo >= 0 && x.rows >= 0 && x.lo + x.rows <= q.N && x.n >= 0 && x.n <= x.rows && x.at >= 0);
            for (int r = x.at; r < x.at + R && r < x.rows; ++r) {
                ++taken[x.lo + r];
                token[x.lo + r] += r < x.n;
            }
            if (x.at >= x.rows || !q.by_place || (q.offsets && q.S >= 64)) continue;
            const int work = from_end ? (x.rows + R - 1) / R - x.at / R : x.at / R;
            CHECK(work <= before);
            before = work;
        }
        if (!ordered) continue;
        for (int s = 0; s <= q.S; ++s)
            for (int r = 0; r < q.rows(s); ++r) CHECK(token[q.first(s) + r] == (r < q.tokens(s)));
        for (int x : taken) CHECK(x == 1);
    }
}

static void check_layout() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    for (int round = 0; round < 400; ++round) {
        const int S = round % 4 == 0 ? pick(1, 5000) : pick(1, 70), most = round % 3 == 0 ? 400 : 5;
        std::vector<int> offsets(S + 1, 0), lens(S);
        for (int s = 0; s < S; ++s) {
            offsets[s + 1] = offsets[s] + (pick(0, 2) ? pick(0, most) : 0);
            lens[s] = pick(-3, most + 3);
        }
        const int N = offsets[S] + pick(0, 300), R = round % 3 == 0 ? 128 : round % 3 == 1 ? 32 : 8;
        check_blocks({offsets.data(), nullptr, N, S, false}, R, true);
        check_blocks({offsets.data(), lens.data(), N, S, false}, R, true);
        check_blocks({nullptr, lens.data(), S * most, S, false}, R, true);
        for (int &x : offsets) x = pick(0, 3) ? pick(-N - 5, 2 * N + 5) : pick(0, 1) ? INT_MAX : INT_MIN;
        check_blocks({offsets.data(), lens.data(), N, S, false}, R, false);
    }
    for (int Hk : {1, 2, 7, 8, 9, 16, 17})
        for (int G : {1, 3, 4})
            for (int blocks : {1, 5, 33}) {
                std::vector<int> seen(blocks * Hk * G, 0);
                for (int id = 0; id < blocks * Hk * G; ++id) {
                    const muir::at::Item it = muir::at::find_item(id, blocks, Hk * G, Hk);
                    CHECK(it.block >= 0 && it.block < blocks && it.h >= 0 && it.h < Hk * G);
                    ++seen[it.block * Hk * G + it.h];
                    if (it.h / G < Hk / 8 * 8) CHECK(it.h / G % 8 == id % 8);
                }
                for (int x : seen) CHECK(x == 1);
            }
    const int table[8] = {3, -1, 5, INT_MAX, 0, 1, INT_MIN, 4};
    const muir::at::Pages p{table, 5, 4, 4, 3};
    CHECK(p.room() == 64 && p.id(1, 17) == 1 && p.good(0) && p.good(4) && !p.good(5) && !p.good(-1) && !p.good(INT_MAX) && !p.good(INT_MIN));
    CHECK(p.row(4, 2, 31) == size_t((4 * 3 + 2) * 16 + 15) && p.row(1 << 30, 2, 0) == ((size_t(1) << 30) * 3 + 2) * 16);
    for (int len : {INT_MIN, -1, 0, 1, 31, 32, 63, 64, 65, INT_MAX})
        for (int append : {0, 1})
            for (int window : {0, 1, 20, 64, INT_MAX}) {
                const muir::at::Span s = muir::at::step_span(len, append, window, 64);
                const bool fits = len >= 0 && int64_t(len) + append <= 64;
                CHECK(s.n == (fits ? len + append : 0) && s.old == (fits ? len : 0) && s.begin >= 0 && s.begin <= s.n);
                CHECK(!fits || s.n - s.begin == (window && window < s.n ? window : s.n));
                CHECK(s.t0 * 32 <= s.begin && s.t1 * 32 >= s.n && s.t1 * 32 < s.n + 32 && (s.n == 0 || s.t0 < s.t1));
            }
}

int main() {
    check_layout();
    void *ws = at<void>(30);
    const size_t big = size_t(1) << 37;
    auto fwd = [&](int N, int S, int H, int Hk, int d, const int *offsets, void *o, int window, float scale, muir_dtype_t t) {
        return muir_attention_fwd(at<void>(0), at<void>(1), at<void>(2), offsets, nullptr, o, at<float>(6), N, S, H, Hk, d, window, scale, t, nullptr);
    };
    const int *off = at<int>(3);
    expect(fwd(100, 3, 4, 2, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 0, 1, "forward");
    expect(fwd(99, 3, 4, 2, 64, nullptr, at<void>(5), INT_MAX, 0.1f, MUIR_F32), 0, 1, "forward of a batch");
    expect(fwd(0, 3, 4, 2, 64, off, nullptr, 0, 0.1f, MUIR_BF16), 0, 0, "no rows");
    expect(fwd(100, 3, 4, 2, 64, nullptr, at<void>(5), 0, 0.1f, MUIR_BF16), 2, 0, "unequal batch");
    expect(fwd(100, 3, 4, 3, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 2, 0, "heads");
    expect(fwd(INT_MAX, INT_MAX, INT_MAX, 1, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 3, 0, "huge");
    expect(fwd(INT_MAX, 1, 1, 1, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 3, 0, "long");
    expect(fwd(100, INT_MAX, 1, 1, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 3, 0, "many sequences");
    expect(fwd(1 << 30, 1, 1, 1, 64, off, at<void>(5), 0, 0.1f, MUIR_BF16), 0, 1, "the longest");
    expect(fwd(100, 3, 4, 2, 64, off, at<void>(1), 0, 0.1f, MUIR_BF16), 5, 0, "alias");
    auto bwd = [&](int N, int S, int H, int d, void *dq, size_t bytes) {
        return muir_attention_bwd(at<void>(0), at<void>(1), at<void>(2), at<void>(4), at<float>(5), off, nullptr, at<void>(7), dq, at<void>(9),
                                  at<void>(10), N, S, H, H, d, 0, 0.1f, MUIR_F32, ws, bytes, nullptr);
    };
    expect(bwd(100, 3, 4, 128, at<void>(8), big), 0, 1, "backward");
    expect(bwd(0, 3, 4, 128, nullptr, 0), 0, 0, "backward of nothing");
    expect(bwd(100, 3, 4, 128, at<void>(8), 100), 4, 0, "small workspace");
    expect(bwd(100, 3, 4, 128, at<void>(7), big), 5, 0, "alias");
    expect(bwd(INT_MAX, 3, INT_MAX, 128, at<void>(8), big), 3, 0, "huge backward");
    auto append = [&](int N, int S, int Hk, int pages, int page, int width, const int *table) {
        return muir_cache_append(at<void>(0), at<void>(1), at<void>(2), at<void>(3), table, off == nullptr ? nullptr : at<int>(5), nullptr, nullptr, N,
                                 S, Hk, 64, pages, page, width, MUIR_BF16, nullptr);
    };
    expect(append(100, 3, 4, 10, 16, 4, at<int>(4)), 0, 1, "append");
    expect(append(0, 3, 4, 10, 16, 4, nullptr), 0, 0, "append nothing");
    expect(append(100, 3, 4, 10, 24, 4, at<int>(4)), 3, 0, "page");
    expect(append(100, 3, 4, 10, 16, INT_MAX, at<int>(4)), 3, 0, "wide table");
    expect(append(100, 3, 4, 0, 16, 4, at<int>(4)), 2, 0, "no pages");
    expect(append(100, 3, 4, INT_MAX, 256, 4, at<int>(4)), 5, 0, "huge cache over its inputs");
    auto step = [&](int B, int H, int Hk, int page, int width, const void *k, const void *v, void *o, size_t bytes) {
        return muir_decode_step_attention(at<void>(0), k, v, at<void>(3), at<void>(4), at<int>(5), at<int>(6), o, B, H, Hk, 128, 100, page, width, 0,
                                          0.1f, MUIR_BF16, ws, bytes, nullptr);
    };
    expect(step(3, 8, 2, 16, 100, at<void>(1), at<void>(2), at<void>(7), big), 0, 1, "step");
    expect(step(3, 8, 2, 16, 100, nullptr, nullptr, at<void>(7), big), 0, 1, "step without a token");
    expect(step(3, 8, 2, 16, 100, at<void>(1), nullptr, at<void>(7), big), 1, 0, "a key without a value");
    expect(step(3, 8, 2, 16, 100, at<void>(1), at<void>(2), at<void>(7), 100), 4, 0, "step without room");
    expect(step(INT_MAX, 8, 8, 16, 100, at<void>(1), at<void>(2), at<void>(7), big), 3, 0, "huge step");
    expect(step(3, 8, 2, 16, 100, at<void>(1), at<void>(2), at<void>(3), big), 5, 0, "alias");
    for (int B : {1, 7, 4096, INT_MAX})
        for (int width : {1, 100, 1 << 22, INT_MAX}) {
            muir_decode_step_attention_workspace_size(B, 64, 1, 128, 256, width, MUIR_F32);
            muir_attention_bwd_workspace_size(width, B, 64, 64, 128, MUIR_BF16);
        }
    g_status = hipErrorLaunchFailure;
    expect(step(3, 8, 2, 16, 100, at<void>(1), at<void>(2), at<void>(7), big), 6, 1, "launch failure");
    printf("%d failures\n", failures);
    return failures != 0;
}
