// Causal softmax attention, backward. With p_ij = exp(s_ij - lse_i) made again from q, k and the forward's lse,
//   D_i = do_i . o_i     ds_ij = p_ij (do_i . v_j - D_i)
//   dq_i = scale sum_j ds_ij k_j     dk_j = scale sum_i ds_ij q_i     dv_j = sum_i p_ij do_i
// Two kernels, each with its sums in registers from the first to the last product, so no sum depends on an order and nothing is
// added atomically: dq walks a query block's keys, dk and dv walk a key block's queries, of all the heads that share it. Scores
// and do . v are made in both (7 products of which 5 are needed): one kernel would have to add dq atomically, and its bits would depend on the
// order (in float32, over blocks of 128 keys, it would go to memory and back 16 times at T4096: 8.6 GB at B8 H16 d128, more than the whole backward's time).
// bf16 B8 T4096 H16 d128: dq 0.84 ms, dkv 0.97 ms, 985 and 1140 TFLOP/s of the products made; matrix cores busy in 53 and 63 % of the cycles at 1.7 GHz,
// two workgroups to a compute unit by registers (228 and 256) and LDS. Packed with a window of 512 (13731 rows,
// H16 Hk4) 129 to 139 and 133 to 143 us, matrix cores busy in 30 and 36 %: 6.8 and 1.7 workgroups to a compute unit do not come out even.
// bf16: p and ds are rounded to bf16 for the products that sum them (half a step of each term, of either sign); everything else is
// float32. D from the rounded o is off by some e_i, and where one key has most of a row's p its ds is what that leaves: dq and dk would be 0.0029 to 0.0032 off
// (2-norm, relative) where one rounding is 0.0017. But sum_j ds_ij = 0, so dq's kernel finds e_i as the sum of its own ds, hands the
// exact D on to dk, and takes e_i sum_j p_ij k_j off dq, of that sum only the largest p of each of a wavefront's halves: the rest is
// small, and is times e_i. The same product adds what the ds of those keys lost when they were rounded, most of what a row's ds lose. dq is 0.0021 off
// then, dk 0.0024, dv 0.0023. With ds as two terms dq and dk would be 0.0018 and 0.0017, with p too dv 0.0017: forward and backward of B8 T4096 H16 d128
// 2.41 -> 2.80 and 3.11 ms, packed with a window of 512 326 -> 371 and 413 us.
#include "attention.hpp"
#include "attention_kernels.hpp"
#include "launch.hpp"
#include "op_layout.hpp"

namespace muir {
namespace {

using namespace at;

// SPLIT: a workgroup has 32 rows, and its wavefronts every WAVES-th tile of what they walk over, each in two tiles of its own, which are loaded anew as
// soon as their last product has read them; their sums meet at the end.
// dkv has eight of them where its workgroups are few and each has far to go.
template <typename T, int D, bool SPLIT, int W = 4> struct Bwd {
    static constexpr int WAVES = W, ROWS = SPLIT ? 32 : 128;
    static constexpr int STEP = SPLIT ? 32 : 64, TILE = STEP * D * int(sizeof(T));  // rows of the tiles walked over
    static constexpr int LDS = (SPLIT ? 2 * WAVES : 4) * TILE, STATS = (SPLIT ? 2 * WAVES : 4) * 64 * 4;  // lse and D, of as many tiles
    static constexpr int DQ_PER_CU = sizeof(T) * D == 512 ? 1 : 2, DKV_PER_CU = sizeof(T) * D == 512 ? 1 : 2;
    static_assert(LDS == WAVES * 64 * D * int(sizeof(T)), "a wavefront has 64 rows of the tiles' room");
    static_assert(LDS >= ROWS * D * int(sizeof(T)) && (!SPLIT || 2 * TILE >= 32 * D * 4), "the outputs pass through the tiles' room");
};

// Whether a score's sum begins at -lse / scale where rows of accumulators are queries, or at 0 and -lse is added to the exponent.
template <typename T> constexpr bool FROM_LSE = sizeof(T) == 2;

// Whether D is corrected as above: what float32 rounds off o leaves nothing to correct.
template <typename T> constexpr bool EXACT_D = sizeof(T) == 2;

// dq, and for the next kernel [H][N] of -lse (over the scale, or in base 2) and -D; a row without keys gets -infinity, so its p are zero.
template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__((64 * Bwd<T, D, SPLIT>::WAVES), (Bwd<T, D, SPLIT>::DQ_PER_CU)) void attention_dq_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ o, const T *__restrict__ dout,
    const float *__restrict__ lse, Sequences seqs, T *__restrict__ dq, float *__restrict__ tops, float *__restrict__ deltas, int blocks,
    int H, int Hk, int window, float scale) {
    using C = Bwd<T, D, SPLIT>;
    using Ti = Tile<T, D>;
    using frag = typename Op<T>::frag;
    constexpr int WAVES = C::WAVES, KEYS = C::STEP, TILE = C::TILE, QS = D / 16, NO = D / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    typename Ti::template Lane<32> ln(lane);
    const Item it = find_item(blockIdx.x, blocks, H, Hk);
    const Block b = find_block<C::ROWS>(seqs, it.block, blocks);
    if (b.at >= b.rows) return;
    const int hk = it.h / (H / Hk);
    const uint32_t kv_stride = uint32_t(Hk) * Ti::ROWB;
    const int r0 = b.at + (SPLIT ? 0 : 32 * wv), q_row = r0 + (lane & 31);
    const float scale2 = scale * LOG2E;

    const int end = min(b.at + C::ROWS, b.n);
    const int first = window ? max(b.at - window + 1, 0) / KEYS : 0;
    const int tiles = b.at < b.n ? (end + KEYS - 1) / KEYS : first;
    const T *kb = k + (static_cast<size_t>(b.lo) * Hk + hk) * D, *vb = v + (static_cast<size_t>(b.lo) * Hk + hk) * D;
    unsigned char *tile = smem + (SPLIT ? wv * 2 * TILE : 0);
    auto fetch_one = [&](const T *rows, int j, unsigned char *to) {
        Ti::template fetch<KEYS, SPLIT ? 1 : WAVES>(to, rows + static_cast<size_t>(j) * KEYS * Hk * D, kv_stride, b.n - j * KEYS, SPLIT ? 0 : wv, lane);
    };
    auto fetch = [&](int j, int buf) {
        fetch_one(kb, j, tile + buf * 2 * TILE);
        fetch_one(vb, j, tile + buf * 2 * TILE + TILE);
    };
    const int from = first + (SPLIT ? wv : 0);
    if (from < tiles) fetch(from, 0);

    const size_t own = (static_cast<size_t>(b.lo) + min(q_row, b.rows - 1)) * H + it.h;
    frag qf[QS], df[QS];
    float d = 0.f;
#pragma unroll
    for (int s = 0; s < QS; ++s) {
        qf[s] = load8<T, 32>(q + own * D + 16 * s + 8 * half);
        df[s] = load8<T, 32>(dout + own * D + 16 * s + 8 * half);
        float x[8], y[8];
        load_vec<8>(o + own * D + 16 * s + 8 * half, x);
        load_vec<8>(dout + own * D + 16 * s + 8 * half, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(x[j], y[j], d);
    }
    d = halves_sum(d);
    const float l = lse[own];
    const bool live = q_row < b.n && l != -INFINITY;
    const float top = live ? -l * LOG2E : -INFINITY;
    d = live ? d : 0.f;
    f32x16_t acc[NO] = {};
    float e[2] = {};  // sums of ds
    // About the lane's largest p so far, its last four bits the accumulator element that it was, the first key of its 32, and what its ds lost to bf16.
    // Only a p above `bar` is taken, 1/8 at first and half as much again as the last: of smaller ones there is little to correct, and each costs
    // the wavefront a look at all its scores (from 1/16 on dq took 0.91 ms at B8 T4096 H16 d128 and was 0.0020 off, from 1/8 on 0.89 and 0.0021).
    uint32_t best = 0;
    int best_at = -1;
    float rest = 0.f, bar = 0.125f;

    auto step = [&](int j, unsigned char *kt, unsigned char *vt, auto values_done) __attribute__((always_inline)) {
        if constexpr (sizeof(T) == 4) ln.again();
        const bool masked = (j + 1) * KEYS - 1 > r0 || (window && r0 + 31 - j * KEYS >= window);
#pragma unroll
        for (int t = 0; t < KEYS / 32; ++t) {
            // No query sees any of these 32 keys. d64 B8 T4096 H16 1005 -> 967 us for the whole backward, d128 as before with 30 registers fewer.
            if (!SPLIT && (j * KEYS + 32 * t > r0 + 31 || (window && r0 + 1 - (j * KEYS + 32 * (t + 1)) >= window))) continue;
            f32x16_t x = {}, y;
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = -d;
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                x = Op<T>::mma(Ti::template row<32>(kt, 32 * t, s, ln), qf[s], x);
                y = Op<T>::mma(Ti::template row<32>(vt, 32 * t, s, ln), df[s], y);
            }
            if (t == KEYS / 32 - 1) values_done();
            if (masked) {
                KEEP_BRANCH;
                const int last = q_row - j * KEYS - 32 * t - 4 * half, first_seen = window ? last - window : -1000;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = 8 * (i / 4) + i % 4;
                    x[i] = key <= last && key > first_seen ? x[i] : -INFINITY;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], scale2, top));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y[i] *= x[i];
                if constexpr (EXACT_D<T>) e[i & 1] += y[i];
            }
            if constexpr (EXACT_D<T>) {
                float most = x[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) most = fmaxf(most, x[i]);
                if (__any(most > bar)) {
                    KEEP_BRANCH;
                    uint32_t which = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) which = max(which, (__float_as_uint(x[i]) & ~15u) | static_cast<uint32_t>(i));
                    float ds = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) ds = (which & 15u) == static_cast<uint32_t>(i) ? y[i] : ds;
                    const bool more = most > bar;
                    rest = more ? ds - static_cast<float>(static_cast<__bf16>(ds)) : rest;
                    best_at = more ? j * KEYS + 32 * t : best_at;
                    best = more ? which : best;
                    bar = more ? 1.5f * most : bar;
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const frag f = acc_frag<T>(y, s);
#pragma unroll
                for (int n = 0; n < NO; ++n) acc[n] = Op<T>::mma(Ti::template col<32>(kt, 32 * t + 16 * s, 32 * n, ln), f, acc[n]);
            }
        }
    };
    if constexpr (SPLIT) {
        for (int j = from; j < tiles; j += WAVES) {
            const bool more = j + WAVES < tiles;
            own_loads_done<0>();
            step(j, tile, tile + TILE, [&]() __attribute__((always_inline)) {
                own_reads_done();
                if (more) fetch_one(vb, j + WAVES, tile + TILE);
            });
            own_reads_done();
            if (more) fetch_one(kb, j + WAVES, tile);
        }
    } else {
        auto nothing = [] {};
        auto turn = [&](int j, auto buffer) __attribute__((always_inline)) {
            constexpr int buf = decltype(buffer)::value;
            loads_done();
            if (j + 1 < tiles) fetch(j + 1, buf ^ 1);
            if (j * KEYS > r0 + 31 || (window && r0 + 1 - (j + 1) * KEYS >= window)) return;
            step(j, tile + buf * 2 * TILE, tile + buf * 2 * TILE + TILE, nothing);
        };
        for (int j = from; j < tiles; j += 2) {
            turn(j, std::integral_constant<int, 0>{});
            if (j + 1 < tiles) turn(j + 1, std::integral_constant<int, 1>{});
        }
    }
    lds_barrier();  // the tiles are free
    if constexpr (EXACT_D<T>) {
        float off = halves_sum(e[0] + e[1]);
        if constexpr (SPLIT) {
            float *sums = reinterpret_cast<float *>(smem);
            if (half == 0) sums[32 * wv + lane] = off;
            lds_barrier();
            off = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) off += sums[32 * w + (lane & 31)];
            lds_barrier();
        }
        d += off;
        // The keys come as two tiles of 32, one for each query and half, and the factors are a diagonal matrix: dq^T += k^T (rest - e p). A lane without
        // a largest p takes its own token's key, times 0, and one whose query is no token, and may hold anything, some token's.
        const int place = (best & 15u) / 4 * 8 + 4 * half + (best & 3u), mine = min(best_at >= 0 ? best_at + place : q_row, max(b.n - 1, 0));
        const auto ps = __builtin_amdgcn_permlane32_swap(best & ~15u, best & ~15u, false, false);
        const auto rests = __builtin_amdgcn_permlane32_swap(__float_as_uint(rest), __float_as_uint(rest), false, false);
        unsigned char *room = smem + wv * 64 * Ti::ROWB;
#pragma unroll
        for (int n = 0; n < 64 / Ti::RPI; ++n) {
            const int r = n * Ti::RPI + lane / Ti::CH, key = __shfl(mine, r, 64);
            const T *from = kb + static_cast<size_t>(key) * Hk * D + ((lane % Ti::CH) ^ Ti::swz(r)) * (16 / int(sizeof(T)));
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from, (lds_void *)(room + n * 1024), 16, 0, 0);
        }
        own_loads_done<0>();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float f = fmaf(-off, __uint_as_float(ps[x]), __uint_as_float(rests[x]));
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = acc_row(8 * s + i, lane) == (lane & 31) ? f : 0.f;
                const frag diagonal = Op<T>::pack(c);
#pragma unroll
                for (int n = 0; n < NO; ++n) acc[n] = Op<T>::mma(Ti::template col<32>(room, 32 * x + 16 * s, 32 * n, ln), diagonal, acc[n]);
            }
        }
        lds_barrier();  // the tiles are free again
    }
    if (half == 0 && q_row < b.rows && (!SPLIT || wv == 0)) {
        const size_t i = static_cast<size_t>(it.h) * seqs.N + b.lo + q_row;
        tops[i] = FROM_LSE<T> && live ? -l / scale : top;
        deltas[i] = -d;
    }
    T *out = dq + ((static_cast<size_t>(b.lo) + r0) * H + it.h) * D;
    if constexpr (SPLIT)
        store_sums<T, D, WAVES>(smem, acc, [&](int r) { return r0 + r < b.n ? scale : 0.f; }, out, static_cast<size_t>(H) * D, b.rows - r0, wv, lane);
    else
        store_rows<T, D>(smem + wv * 32 * Ti::ROWB, acc, scale, live, out, static_cast<size_t>(H) * D, b.rows - r0, lane);
}

// dk and dv of 128 keys of a key head, 32 to a wavefront, whose keys and values stay in registers, over the queries of all its heads. Scores have
// queries as rows, so p and ds are the operands of dv^T += do^T p and dk^T += q^T ds as they are.
template <typename T, int D, bool SPLIT, int W>
__global__ __launch_bounds__((64 * W), (Bwd<T, D, SPLIT, W>::DKV_PER_CU)) void attention_dkv_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ dout, const float *__restrict__ tops,
    const float *__restrict__ deltas, Sequences seqs, T *__restrict__ dk, T *__restrict__ dv, int blocks, int H, int Hk, int window,
    float scale) {
    using C = Bwd<T, D, SPLIT, W>;
    using Ti = Tile<T, D>;
    using frag = typename Op<T>::frag;
    constexpr int WAVES = C::WAVES, QR = C::STEP, TILE = C::TILE, QS = D / 16, NO = D / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    typename Ti::template Lane<32> ln(lane);
    const Item it = find_item(blockIdx.x, blocks, Hk, Hk);
    const Block b = find_block<C::ROWS, true>(seqs, it.block, blocks);
    if (b.at >= b.rows) return;
    const int G = H / Hk, h0 = it.h * G;
    const uint32_t q_stride = uint32_t(H) * Ti::ROWB;
    const int k0 = b.at + (SPLIT ? 0 : 32 * wv), key = k0 + (lane & 31);
    unsigned char *tile = smem + (SPLIT ? wv * 2 * TILE : 0);
    float *stats = reinterpret_cast<float *>(smem + C::LDS) + (SPLIT ? wv * 128 : 0);
    const float scale2 = scale * LOG2E;

    // Tiles of queries that see the block's keys, for each head.
    const int first = b.at / QR;
    const int end = window ? static_cast<int>(min(static_cast<int64_t>(b.n), static_cast<int64_t>(b.at) + C::ROWS + window - 1)) : b.n;
    const int per = b.at < b.n ? (end + QR - 1) / QR - first : 0, steps = per * G;
    auto fetch_one = [&](const T *rows, int i, unsigned char *to) {
        const int h = h0 + i / per, j = first + i % per;
        Ti::template fetch<QR, SPLIT ? 1 : WAVES>(to, rows + ((static_cast<size_t>(b.lo) + static_cast<size_t>(j) * QR) * H + h) * D, q_stride, b.n - j * QR,
                                                  SPLIT ? 0 : wv, lane);
    };
    auto fetch_stats = [&](int i, int buf) {
        const int h = h0 + i / per, j = first + i % per;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (!SPLIT && wv != x) continue;
            const rsrc_t r = make_rsrc((x ? deltas : tops) + static_cast<size_t>(h) * seqs.N + b.lo + static_cast<size_t>(j) * QR, min(b.n - j * QR, QR) * 4u);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(stats + (buf * 2 + x) * 64), 4, lane * 4, 0, 0, 0);
        }
    };
    auto fetch = [&](int i, int buf) {
        fetch_one(q, i, tile + buf * 2 * TILE);
        fetch_one(dout, i, tile + buf * 2 * TILE + TILE);
        fetch_stats(i, buf);
    };
    const int from = SPLIT ? wv : 0;
    if (from < steps) fetch(from, 0);

    const size_t own = (static_cast<size_t>(b.lo) + min(key, b.rows - 1)) * Hk + it.h;
    frag kf[QS], vf[QS];
#pragma unroll
    for (int s = 0; s < QS; ++s) {
        kf[s] = load8<T, 32>(k + own * D + 16 * s + 8 * half);
        vf[s] = load8<T, 32>(v + own * D + 16 * s + 8 * half);
    }
    f32x16_t dka[NO] = {}, dva[NO] = {};

    auto step = [&](int row0, unsigned char *qt, unsigned char *dt, const float *st, auto dout_done) __attribute__((always_inline)) {
        ln.again();
        // The sums begin at -lse / scale and -D of their rows, so that no subtraction is left. In float32 x begins at 0: its sum's
        // roundings would be as large as lse makes them.
        f32x16_t x = {}, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4_t l = *reinterpret_cast<const f32x4_t *>(st + 8 * i + 4 * half), d = *reinterpret_cast<const f32x4_t *>(st + 64 + 8 * i + 4 * half);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (FROM_LSE<T>) x[4 * i + r] = l[r];
                y[4 * i + r] = d[r];
            }
        }
#pragma unroll
        for (int s = 0; s < QS; ++s) {
            x = Op<T>::mma(Ti::template row<32>(qt, 0, s, ln), kf[s], x);
            y = Op<T>::mma(Ti::template row<32>(dt, 0, s, ln), vf[s], y);
        }
        // 1.14 -> 1.09 ms at B8 T4096 H16 d128; two steps ahead spill registers (1.23). The forward and dq gain nothing by it.
        if constexpr (sizeof(T) == 2 && !SPLIT) read_ahead<QS, 2, 2, 8>();
        if (row0 < k0 + 31 || row0 + 31 >= b.n || (window && row0 + 31 - k0 >= window)) {  // some query that does not see some key
            KEEP_BRANCH;
            const int from = key - row0 - 4 * half, to = min(b.n - row0 - 4 * half, window ? from + window : 1000);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 8 * (i / 4) + i % 4;
                x[i] = row >= from && row < to ? x[i] : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (FROM_LSE<T>)
                x[i] = __builtin_amdgcn_exp2f(x[i] * scale2);
            else
                x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], scale2, st[8 * (i / 4) + 4 * half + i % 4]));
            y[i] *= x[i];
        }
        if constexpr (SPLIT) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const frag p = acc_frag<T>(x, s);
#pragma unroll
                for (int n = 0; n < NO; ++n) dva[n] = Op<T>::mma(Ti::template col<32>(dt, 16 * s, 32 * n, ln), p, dva[n]);
            }
            dout_done();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const frag ds = acc_frag<T>(y, s);
#pragma unroll
                for (int n = 0; n < NO; ++n) dka[n] = Op<T>::mma(Ti::template col<32>(qt, 16 * s, 32 * n, ln), ds, dka[n]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const frag p = acc_frag<T>(x, s), ds = acc_frag<T>(y, s);
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    dva[n] = Op<T>::mma(Ti::template col<32>(dt, 16 * s, 32 * n, ln), p, dva[n]);
                    dka[n] = Op<T>::mma(Ti::template col<32>(qt, 16 * s, 32 * n, ln), ds, dka[n]);
                }
            }
            if constexpr (sizeof(T) == 2) read_ahead<2 * NO, 4, 2>();
        }
    };
    if constexpr (SPLIT) {
        for (int i = from; i < steps; i += WAVES) {
            const bool more = i + WAVES < steps;
            own_loads_done<0>();
            step((first + i % per) * QR, tile, tile + TILE, stats, [&]() __attribute__((always_inline)) {
                own_reads_done();
                if (more) fetch_one(dout, i + WAVES, tile + TILE);
            });
            own_reads_done();
            if (more) {
                fetch_one(q, i + WAVES, tile);
                fetch_stats(i + WAVES, 0);
            }
        }
    } else {
        auto turn = [&](int i, auto buffer) __attribute__((always_inline)) {
            constexpr int buf = decltype(buffer)::value;
            loads_done();
            if (i + 1 < steps) fetch(i + 1, buf ^ 1);
            const int j = first + i % per;
#pragma unroll
            for (int t = 0; t < QR / 32; ++t) {
                const int row0 = j * QR + 32 * t;
                if (row0 + 31 < k0 || row0 >= b.n || (window && row0 - (k0 + 31) >= window)) continue;  // no query sees a key
                unsigned char *qt = tile + buf * 2 * TILE + t * 32 * Ti::ROWB;
                step(row0, qt, qt + TILE, stats + buf * 128 + 32 * t, [] {});
            }
        };
        for (int i = 0; i < steps; i += 2) {
            turn(i, std::integral_constant<int, 0>{});
            if (i + 1 < steps) turn(i + 1, std::integral_constant<int, 1>{});
        }
    }
    lds_barrier();  // the tiles are free
    const size_t out = ((static_cast<size_t>(b.lo) + k0) * Hk + it.h) * D, stride = static_cast<size_t>(Hk) * D;
    if constexpr (SPLIT) {
        store_sums<T, D, WAVES>(smem, dka, [&](int r) { return k0 + r < b.n ? scale : 0.f; }, dk + out, stride, b.rows - k0, wv, lane);
        store_sums<T, D, WAVES>(smem, dva, [&](int r) { return k0 + r < b.n ? 1.f : 0.f; }, dv + out, stride, b.rows - k0, wv, lane);
    } else {
        unsigned char *room = smem + wv * 32 * Ti::ROWB;
        store_rows<T, D>(room, dka, scale, key < b.n, dk + out, stride, b.rows - k0, lane);
        store_rows<T, D>(room, dva, 1.f, key < b.n, dv + out, stride, b.rows - k0, lane);
    }
}

template <typename T, int D, bool SPLIT> hipError_t launch_dq(const AttentionCall &c, const AttentionGrads &g, float *tops, float *deltas, hipStream_t stream) {
    using B = Bwd<T, D, SPLIT>;
    const hipError_t err = allow_lds<&attention_dq_kernel<T, D, SPLIT>>(B::LDS);
    if (err != hipSuccess) return err;
    const int blocks = c.N / B::ROWS + c.S + 1;
    hipLaunchKernelGGL((attention_dq_kernel<T, D, SPLIT>), dim3(static_cast<unsigned>(blocks) * c.H), dim3(64 * B::WAVES), B::LDS, stream,
                       static_cast<const T *>(c.q), static_cast<const T *>(c.k), static_cast<const T *>(c.v), static_cast<const T *>(g.o),
                       static_cast<const T *>(g.dout), g.lse, Sequences{c.offsets, c.lens, c.N, c.S, attention_by_place(c.offsets, c.N, c.S, c.window)}, static_cast<T *>(g.dq), tops, deltas,
                       blocks, c.H, c.Hk, c.window, c.scale);
    return hipGetLastError();
}

template <typename T, int D, bool SPLIT, int W = 4> hipError_t launch_dkv(const AttentionCall &c, const AttentionGrads &g, float *tops, float *deltas, hipStream_t stream) {
    using B = Bwd<T, D, SPLIT, W>;
    const hipError_t err = allow_lds<&attention_dkv_kernel<T, D, SPLIT, W>>(B::LDS + B::STATS);
    if (err != hipSuccess) return err;
    const int blocks = c.N / B::ROWS + c.S + 1;
    hipLaunchKernelGGL((attention_dkv_kernel<T, D, SPLIT, W>), dim3(static_cast<unsigned>(blocks) * c.Hk), dim3(64 * B::WAVES), B::LDS + B::STATS,
                       stream, static_cast<const T *>(c.q), static_cast<const T *>(c.k), static_cast<const T *>(c.v),
                       static_cast<const T *>(g.dout), tops, deltas, Sequences{c.offsets, c.lens, c.N, c.S, attention_by_place(c.offsets, c.N, c.S, c.window)}, static_cast<T *>(g.dk),
                       static_cast<T *>(g.dv), blocks, c.H, c.Hk, c.window, c.scale);
    return hipGetLastError();
}

template <typename T, int D> hipError_t launch(const AttentionCall &c, const AttentionGrads &g, void *workspace, hipStream_t stream) {
    float *tops = static_cast<float *>(workspace), *deltas = tops + up256(static_cast<size_t>(c.N) * c.H * 4) / 4;
    hipError_t err;
    if constexpr (sizeof(T) == 2) {
        err = attention_split(c.N, c.S, c.H, D, c.window) ? launch_dq<T, D, true>(c, g, tops, deltas, stream) : launch_dq<T, D, false>(c, g, tops, deltas, stream);
        if (err != hipSuccess) return err;
        if (!attention_split(c.N, c.S, c.Hk, D, c.window)) return launch_dkv<T, D, false>(c, g, tops, deltas, stream);
    } else {
        err = launch_dq<T, D, true>(c, g, tops, deltas, stream);
        if (err != hipSuccess) return err;
    }
    if constexpr (sizeof(T) * D < 512)  // eight wavefronts' tiles would not fit LDS
        if (attention_far(c.N, c.S, c.H, c.Hk, c.window)) return launch_dkv<T, D, true, 8>(c, g, tops, deltas, stream);
    return launch_dkv<T, D, true>(c, g, tops, deltas, stream);
}

}  // namespace

hipError_t launch_attention_bwd(const AttentionCall &c, const AttentionGrads &g, void *workspace, hipStream_t stream) {
    if (c.d == 64) return c.bf16 ? launch<bf16_t, 64>(c, g, workspace, stream) : launch<float, 64>(c, g, workspace, stream);
    if (c.d == 128) return c.bf16 ? launch<bf16_t, 128>(c, g, workspace, stream) : launch<float, 128>(c, g, workspace, stream);
    return hipErrorInvalidValue;
}

}  // namespace muir
