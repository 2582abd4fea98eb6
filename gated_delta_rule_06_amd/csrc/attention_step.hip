// The paged cache of keys and values: rows appended to it, and one new token of each sequence attending over it.
//
// Step: a workgroup has up to 16 query heads that share a key head and one part of a sequence's keys, its wavefronts every WAVES-th tile of
// 32 keys, each with its own running maximum, sum and output and its own tiles of keys and values in LDS (loads straight to LDS: the next keys
// while values are multiplied, the next values while keys are); they meet in LDS at the end. Where sequences and key heads do not fill the card a sequence is cut into parts, which a second kernel
// joins. Reading the cache once bounds it: B256 T4001 (mixed) H16 Hk4 d128 bf16, 1.37 GB, 207 to 218 us, 6.3 to 6.6 TB/s; B1 T32768 H16 Hk4, 67 MB, 13.9 us
// and 2.9 to 3.9 for the join. How many parts is decided by the batch and the table's room, not by lengths, which lie on the device: one sequence of 32767 among 63
// of 100 (H16 Hk4 d128 bf16, 80 MB) is walked by a workgroup to a key head and takes 285 us, among 31 146, among 7 43, alone 15; 64 of 100
// take 5.6. Scores are made transposed (16 keys by 16 heads), so that two score tiles are the operand
// of the product with the values, as in the prompt kernels. In bf16 p goes into it as two terms: rounded once, o would be 0.0020 off (2-norm, relative, B256)
// where its own rounding is 0.0017, and reading hides the second product (217 us both; B1 T32768 16.2 and 16.4 a call, 16 MB of cache 10.8 and 11.0).
// Rows behind the last token, and pages that the table does not have, are never read: their keys come as zeros and are masked.
#include "attention.hpp"
#include "attention_kernels.hpp"
#include "launch.hpp"

namespace muir {
namespace {

using namespace at;

// A few rows of a sequence, all key heads: 16 bytes a thread and turn, four turns' loads on their way at once. Eight rows to a workgroup: a prompt of 100 tokens takes
// 4.6 us, with 64 rows, in two workgroups, 15.7. B8 T4001 Hk4 d128 bf16, 94 MB read and written: 15.5 us, 6.1 TB/s.
constexpr int APPEND_ROWS = 8;
template <int ROWB>
__global__ __launch_bounds__(256) void cache_append_kernel(const unsigned char *__restrict__ k, const unsigned char *__restrict__ v,
                                                           unsigned char *__restrict__ k_cache, unsigned char *__restrict__ v_cache, Pages pg,
                                                           Sequences seqs, const int *__restrict__ start) {
    constexpr int CH = ROWB / 16, TURNS = 4;
    const Block b = find_block<APPEND_ROWS>(seqs, blockIdx.x, gridDim.x);
    if (b.at >= b.n) return;
    const int base = start ? start[b.seq] : 0, pieces = min(b.n - b.at, APPEND_ROWS) * pg.Hk * CH;
    if (base < 0) return;
    const size_t in = (static_cast<size_t>(b.lo) + b.at) * pg.Hk * ROWB;
    for (int i0 = threadIdx.x; i0 < pieces; i0 += 256 * TURNS) {
        u32x4_t ks[TURNS], vs[TURNS];
        size_t to[TURNS];
        bool keep[TURNS];
#pragma unroll
        for (int n = 0; n < TURNS; ++n) {
            const int i = min(i0 + 256 * n, pieces - 1), hk = i / CH % pg.Hk, r = i / CH / pg.Hk;
            const int64_t pos = static_cast<int64_t>(base) + b.at + r;
            ks[n] = *reinterpret_cast<const u32x4_t *>(k + in + static_cast<size_t>(i) * 16);
            vs[n] = *reinterpret_cast<const u32x4_t *>(v + in + static_cast<size_t>(i) * 16);
            keep[n] = i0 + 256 * n < pieces && pos < pg.room();
            const int id = keep[n] ? pg.id(b.seq, static_cast<int>(pos)) : -1;
            keep[n] = pg.good(id);
            to[n] = keep[n] ? pg.row(id, hk, static_cast<int>(pos)) * ROWB + i % CH * 16 : 0;
        }
#pragma unroll
        for (int n = 0; n < TURNS; ++n)
            if (keep[n]) {
                *reinterpret_cast<u32x4_t *>(k_cache + to[n]) = ks[n];
                *reinterpret_cast<u32x4_t *>(v_cache + to[n]) = vs[n];
            }
    }
}

template <typename T, int D> struct Step {
    static constexpr int KEYS = 32, TILE = KEYS * D * int(sizeof(T)), WAVES = sizeof(T) * D == 512 ? 4 : 8;
    static constexpr int ROOM = 2 * TILE, LDS = WAVES * ROOM;  // a tile of keys and one of values for each wavefront
    static_assert(ROOM >= 16 * D * 4 + 128, "outputs, maxima and sums of 16 heads pass through the tiles' room");
};

// What eight values lose when they are packed to bf16, as the second term of two.
__device__ __forceinline__ bf16x8_t rounded_off(const float (&x)[8]) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j] - static_cast<float>(static_cast<__bf16>(x[j]));
    return Op<bf16_t>::pack(r);
}

// BIG: the cache is larger than the 256 MB that the last-level cache holds, so of a program that works its way through it nothing is there when it comes to be
// read again, and its loads go past the caches: B256 T4001 (mixed) H16 Hk4 d128 bf16, 1.3 GB, 207 us (6.3 TB/s) against 233. A cache of 190 MB read again and
// again takes 33 us with ordinary loads, 38 so. Calls that read a part of 4 GB, other pages each time, with ordinary loads and so, and the same pages again
// (H16 Hk4 d128 bf16): 16 MB (B1 T8000) 11.2 and 10.8, 8.8 and 10.3; 67 MB (B1 T32767) 19.0 and 17.1, 16.7 and 15.3; 131 MB (B16 T4000) 29.0 and 25.8,
// 24.6 and 24.3; 393 MB (B64 T3000) 70.9 and 62.3, 65.9 and 62.0. So only small calls over the same pages lose, and those a program of several
// layers does not make. Where a key head has more than 16 query heads, the workgroups of its sets read the same keys, and the caches serve all but the
// first (likewise): H64 Hk2 d128 bf16 B16 T4000 26.7 and 27.2, 26.7 and 25.0; B256 T4000 289 and 321, 287 and 320; H40 Hk1 d64 B128 T4000 60 and 73, 61 and 74.
template <typename T, int D, bool BIG>
__global__ __launch_bounds__((Step<T, D>::WAVES * 64)) void attention_step_kernel(
    const T *__restrict__ q, const T *__restrict__ kn, const T *__restrict__ vn, T *k_cache, T *v_cache, Pages pg,
    const int *__restrict__ lens, T *__restrict__ o, float *__restrict__ part_o, float *__restrict__ part_s, int H, int parts, int window,
    float scale2) {
    using C = Step<T, D>;
    using Ti = Tile<T, D>;
    using frag = typename Op<T>::frag16;
    constexpr int WAVES = C::WAVES, TILE = C::TILE, QS = D / 32, NO = D / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;
    const int G = H / pg.Hk, sets = (G + 15) / 16;
    const int part = blockIdx.x % parts, set = blockIdx.x / parts % sets, bh = blockIdx.x / parts / sets, hk = bh % pg.Hk, b = bh / pg.Hk;
    const int h0 = hk * G + set * 16, heads = min(G - set * 16, 16);
    const typename Ti::template Lane<16> ln(lane);
    unsigned char *kt = smem + wv * C::ROOM, *vt = kt + TILE;

    const Span span = step_span(lens[b], kn != nullptr, window, pg.room());
    const int old = span.old, n = span.n, begin = span.begin;
    const int per = (span.t1 - span.t0 + parts - 1) / parts, from = span.t0 + part * per + wv, to = min(span.t0 + (part + 1) * per, span.t1);

    // The wavefront's tiles are from, from + WAVES, ... Each lane keeps the page of one half (16 rows, which always lie in one page) of the
    // 32 tiles that are fetched next.
    int ids = -1;
    auto look_up = [&](int tile) {
        if ((tile - from) / WAVES % 32 != 0) return;
        const int64_t pos = static_cast<int64_t>(tile + lane / 2 * WAVES) * 32 + lane % 2 * 16;
        ids = pos < n ? pg.table[static_cast<size_t>(b) * pg.width + (pos >> pg.log_page)] : -1;
    };
    auto page_of = [&](int tile, int u) { return __builtin_amdgcn_readlane(ids, 2 * ((tile - from) / WAVES % 32) + u); };
    // Which halves of a tile lie in a page that the cache has.
    auto known = [&](int tile) { return (pg.good(page_of(tile, 0)) ? 1 : 0) | (pg.good(page_of(tile, 1)) ? 2 : 0); };
    auto fetch = [&](const T *cache, int tile, unsigned char *to) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int id = page_of(tile, u), pos = tile * 32 + 16 * u, live = pg.good(id) ? min(old - pos, 16) : 0;
            Ti::template fetch<16, 1, BIG ? Ti::STREAM : 0>(to + u * 16 * Ti::ROWB, cache + (live > 0 ? pg.row(id, hk, pos) * D : 0), Ti::ROWB, live, 0, lane);
        }
    };
    int good = 0;
    if (from < to) {
        look_up(from);
        good = known(from);
        fetch(k_cache, from, kt);
        fetch(v_cache, from, vt);
    }

    frag qf[QS];
#pragma unroll
    for (int s = 0; s < QS; ++s) {
        qf[s] = frag{};
        if (col < heads) qf[s] = load8<T, 16>(q + (static_cast<size_t>(b) * H + h0 + col) * D + 32 * s + 8 * g);
    }
    f32x4_t acc[NO] = {};
    float m = LOWEST, l = 0.f;
    constexpr int LOADS = 32 / Ti::RPI;  // of one tile
    for (int tile = from; tile < to; tile += WAVES) {
        const bool more = tile + WAVES < to;
        const int p0 = tile * 32;
        own_loads_done<LOADS>();  // the values were asked for after the keys
        u32x4_t new_value;
        // The new token's row, where its page is there. A row that is not put in stays zeros: its p is 0, and what it multiplies has to be finite.
        const bool has_new = kn && p0 <= old && old < p0 + 32 && n > old && (good >> ((old - p0) >> 4) & 1);
        if (has_new && lane < Ti::CH) {
            const size_t at = (static_cast<size_t>(b) * pg.Hk + hk) * D + lane * (16 / sizeof(T));
            const u32x4_t new_key = *reinterpret_cast<const u32x4_t *>(kn + at);
            new_value = *reinterpret_cast<const u32x4_t *>(vn + at);
            *reinterpret_cast<u32x4_t *>(kt + Ti::at(old - p0, lane)) = new_key;
            if (set == 0) {
                const size_t row = pg.row(pg.id(b, old), hk, old) * D + lane * (16 / sizeof(T));
                *reinterpret_cast<u32x4_t *>(k_cache + row) = new_key;
                *reinterpret_cast<u32x4_t *>(v_cache + row) = new_value;
            }
        }
        wave_lds_sync();
        f32x4_t x[2] = {};
#pragma unroll
        for (int s = 0; s < QS; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u) x[u] = Op<T>::mma16(Ti::template row<16>(kt, 16 * u, s, ln), qf[s], x[u]);
        own_reads_done();
        int good_next = 0;
        if (more) {
            look_up(tile + WAVES);
            good_next = known(tile + WAVES);
            fetch(k_cache, tile + WAVES, kt);
        }
        if (p0 < begin || p0 + 32 > n || good != 3) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = p0 + 16 * u + 4 * g + i;
                    x[u][i] = (good >> u & 1) && pos >= begin && pos < n ? x[u][i] : -INFINITY;
                }
        }
        float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])), fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = halves_max(top) * scale2;
        if (__any(top > m + 8.f)) {
            const float now = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - now);
            l *= f;
#pragma unroll
            for (int i = 0; i < NO; ++i) acc[i] *= f;
            m = now;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[u][i] = __builtin_amdgcn_exp2f(fmaf(x[u][i], scale2, -m));
                l += x[u][i];
            }
        const float ps[8] = {x[0][0], x[0][1], x[0][2], x[0][3], x[1][0], x[1][1], x[1][2], x[1][3]};
        const frag p = Op<T>::pack16(ps);
        if (more)
            own_loads_done<LOADS>();
        else
            own_loads_done<0>();
        if (has_new && lane < Ti::CH) *reinterpret_cast<u32x4_t *>(vt + Ti::at(old - p0, lane)) = new_value;
        if (p0 < begin)  // values before the window, times p = 0, must be finite (the permutation stays inside a row)
            for (int i = lane; i < (begin - p0) * Ti::CH; i += 64) *reinterpret_cast<u32x4_t *>(vt + 16 * i) = u32x4_t{};
        wave_lds_sync();
#pragma unroll
        for (int i = 0; i < NO; ++i) {
            const frag vf = Ti::template col<16>(vt, 0, 16 * i, ln);
            if constexpr (sizeof(T) == 2) acc[i] = Op<T>::mma16(vf, rounded_off(ps), acc[i]);
            acc[i] = Op<T>::mma16(vf, p, acc[i]);
        }
        own_reads_done();
        if (more) fetch(v_cache, tile + WAVES, vt);
        good = good_next;
    }
    l += __shfl_xor(l, 16, 64);
    l = halves_sum(l);

    // The wavefronts' results: [16 heads][D] values (16-byte pieces of four, permuted by the head against bank conflicts), then maxima and sums.
    auto place = [&](int w, int h, int c) { return reinterpret_cast<float *>(smem + w * C::ROOM) + h * D + ((c ^ h) & (D / 4 - 1)) * 4; };
    auto stat = [&](int w) { return reinterpret_cast<float *>(smem + w * C::ROOM + 16 * D * 4); };
#pragma unroll
    for (int i = 0; i < NO; ++i) *reinterpret_cast<f32x4_t *>(place(wv, col, 4 * i + g)) = acc[i];
    if (g == 0) {
        stat(wv)[col] = m;
        stat(wv)[16 + col] = l;
    }
    lds_barrier();
    for (int i = threadIdx.x; i < heads * (D / 4); i += 64 * WAVES) {
        const int h = i / (D / 4), c = i % (D / 4);
        float all = LOWEST, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) all = fmaxf(all, stat(w)[h]);
        f32x4_t y = zero4();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = __builtin_amdgcn_exp2f(stat(w)[h] - all);
            sum = fmaf(stat(w)[16 + h], f, sum);
            y += *reinterpret_cast<const f32x4_t *>(place(w, h, c)) * f;
        }
        const size_t row = static_cast<size_t>(b) * H + h0 + h;
        if (parts == 1) {
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
            store4(o + row * D + 4 * c, y * inv);
        } else {
            *reinterpret_cast<f32x4_t *>(part_o + (row * parts + part) * D + 4 * c) = y;
            if (c == 0) {
                part_s[(row * parts + part) * 2] = all;
                part_s[(row * parts + part) * 2 + 1] = sum;
            }
        }
    }
}

// Joins the parts of a head, a workgroup to a head: its threads take every GROUPS-th part's four columns each, and meet in LDS, always in the same
// order.
template <typename T, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(const float *__restrict__ part_o, const float *__restrict__ part_s, T *__restrict__ o,
                                                            int parts) {
    constexpr int GROUPS = 1024 / D;
    __shared__ float sums[GROUPS];
    __shared__ f32x4_t sh[GROUPS][D / 4];
    const size_t row = blockIdx.x;
    const int group = threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
    const float *s = part_s + row * parts * 2, *y = part_o + row * parts * D + 4 * c;
    float all = LOWEST, sum = 0.f;
    for (int p = threadIdx.x & 63; p < parts; p += 64) all = fmaxf(all, s[2 * p]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) all = fmaxf(all, __shfl_xor(all, off, 64));
    f32x4_t x = zero4();
#pragma unroll 4
    for (int p = group; p < parts; p += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(s[2 * p] - all);
        sum = fmaf(s[2 * p + 1], f, sum);
        x += *reinterpret_cast<const f32x4_t *>(y + static_cast<size_t>(p) * D) * f;
    }
    sh[group][c] = x;
    if (c == 0) sums[group] = sum;
    __syncthreads();
    if (group != 0) return;
    x = zero4();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        x += sh[i][c];
        sum += sums[i];
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    store4(o + row * D + 4 * c, x * inv);
}

Pages pages_of(const CacheCall &c) {
    return Pages{c.table, c.pages, __builtin_ctz(static_cast<unsigned>(c.page)), c.width, c.Hk};
}

template <typename T, int D, bool BIG>
hipError_t launch_parts(const CacheCall &c, const void *q, const void *k, const void *v, const int *lens, void *o, int B, int H, int parts, int window,
                        float scale, float *part_o, float *part_s, hipStream_t stream) {
    using S = Step<T, D>;
    const hipError_t err = allow_lds<&attention_step_kernel<T, D, BIG>>(S::LDS);
    if (err != hipSuccess) return err;
    const int sets = (H / c.Hk + 15) / 16;
    hipLaunchKernelGGL((attention_step_kernel<T, D, BIG>), dim3(static_cast<unsigned>(B) * c.Hk * sets * parts), dim3(64 * S::WAVES), S::LDS, stream,
                       static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v), static_cast<T *>(c.k_cache),
                       static_cast<T *>(c.v_cache), pages_of(c), lens, static_cast<T *>(o), part_o, part_s, H, parts, window, scale * LOG2E);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch(const CacheCall &c, const void *q, const void *k, const void *v, const int *lens, void *o, int B, int H, int window,
                  float scale, void *workspace, hipStream_t stream) {
    // With a window there is less to divide, never more than the workspace has room for.
    const int room = c.width * c.page, parts = attention_step_parts(B, H, c.Hk, D, window ? min(room, window) : room, sizeof(T) == 2);
    float *part_o = static_cast<float *>(workspace), *part_s = part_o + static_cast<size_t>(B) * H * parts * D;
    const bool big = H / c.Hk <= 16 && 2 * static_cast<size_t>(c.pages) * c.Hk * c.page * D * sizeof(T) > size_t(256) << 20;
    const hipError_t err = big ? launch_parts<T, D, true>(c, q, k, v, lens, o, B, H, parts, window, scale, part_o, part_s, stream)
                               : launch_parts<T, D, false>(c, q, k, v, lens, o, B, H, parts, window, scale, part_o, part_s, stream);
    if (err != hipSuccess || parts == 1) return err;
    hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3(static_cast<unsigned>(B) * H), dim3(256), 0, stream, part_o, part_s,
                       static_cast<T *>(o), parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const CacheCall &c, const void *k, const void *v, const int *offsets, const int *lens, const int *start,
                               int N, int S, hipStream_t stream) {
    const int row = c.d * (c.bf16 ? 2 : 4), blocks = N / APPEND_ROWS + S + 1;
    const Sequences s{offsets, lens, N, S, false};
#define MUIR_APPEND(R)                                                                                                           \
    if (row == R) {                                                                                                              \
        hipLaunchKernelGGL((cache_append_kernel<R>), dim3(blocks), dim3(256), 0, stream, static_cast<const unsigned char *>(k), \
                           static_cast<const unsigned char *>(v), static_cast<unsigned char *>(c.k_cache),                      \
                           static_cast<unsigned char *>(c.v_cache), pages_of(c), s, start);                                     \
        return hipGetLastError();                                                                                                \
    }
    MUIR_APPEND(128) MUIR_APPEND(256) MUIR_APPEND(512)
#undef MUIR_APPEND
    return hipErrorInvalidValue;
}

hipError_t launch_attention_step(const CacheCall &c, const void *q, const void *k, const void *v, const int *lens, void *o, int B, int H,
                                 int window, float scale, void *workspace, hipStream_t stream) {
    if (c.d == 64)
        return c.bf16 ? launch<bf16_t, 64>(c, q, k, v, lens, o, B, H, window, scale, workspace, stream)
                      : launch<float, 64>(c, q, k, v, lens, o, B, H, window, scale, workspace, stream);
    if (c.d == 128)
        return c.bf16 ? launch<bf16_t, 128>(c, q, k, v, lens, o, B, H, window, scale, workspace, stream)
                      : launch<float, 128>(c, q, k, v, lens, o, B, H, window, scale, workspace, stream);
    return hipErrorInvalidValue;
}

}  // namespace muir
