// Causal softmax attention over whole prompts, forward: o_i = sum_j p_ij v_j, with the running maximum and sum of the
// softmax, one pass over the keys.
//
// A workgroup has 128 query rows of one head, 32 to a wavefront, whose queries stay in registers; keys and values come in tiles through LDS,
// the next tile's loads (straight to LDS) in flight. Scores are made transposed, S^T = K Q^T, so a lane holds scores of one query: the maximum and the
// sum are sums inside the lane and over the two halves of the wavefront, and the accumulators of P^T are the operand of O^T += V^T P^T.
// bf16: p is rounded to bf16 for that product (half a step, at most 2^-8 of each term, of either sign), its sum is taken before the rounding, and
// everything else is float32. o is 0.0022 off by it (2-norm, relative) where its own rounding is 0.0017. With p as two terms it would be that, at the price of
// a third product beside every two: B1 T32768 H16 d128 3.99 -> 5.63 ms, 24 packed sequences up to 4001 H16 Hk4 402 -> 542 us, d64 with a window of 1024
// 127 -> 174.
// The output is rescaled only where a row's maximum grew by more than 2^8 over the reference its exponentials are taken from; up to there
// they are as exact in float32 and bf16 as below 1.
//
// What bounds it. d128: the matrix cores and the card's power. B1 T32768 H16 3.95 to 4.0 ms, 1100 TFLOP/s, where a large library product makes 1361: matrix
// cores busy in 67 % of the cycles, vector instructions in 67 %, at a clock of 1.4 GHz; B8 T4096 H16 540 us, 1020 TFLOP/s, 60 and 64 % at 1.6 GHz. d64: vector instructions, of
// which there are as many to half the products: B8 T4096 H12 window 1024 127 us, vector 75 %, matrix 40 %. Few rows: the walk of the last rows' workgroup.
// Sizes tried, in us: d64 tiles of 64 keys against 32, B8 T4096 H16 331 and 351; d128 the other way, 4350 and 4160 at B1 T32768 H16, since 64 keys leave
// two workgroups to a compute unit instead of three. Two blocks of 32 queries to a wavefront, which halves the reads of LDS: 4.2 against 4.3 ms there,
// 515 against 430 for 24 packed sequences, so not kept.
#include "attention.hpp"
#include "attention_kernels.hpp"
#include "launch.hpp"

namespace muir {
namespace {

using namespace at;

// SPLIT: a workgroup has 32 rows, and its wavefronts every WAVES-th tile of their keys, each in tiles of its own; they meet at the end. There a wavefront has
// one tile of keys and one of values, and loads the next keys while it multiplies values, the next values while it multiplies keys.
template <typename T, int D, bool SPLIT> struct Fwd {
    static constexpr int WAVES = 4, ROWS = SPLIT ? 32 : 128;
    static constexpr int KEYS = D == 64 && !SPLIT ? 64 : 32, TILE = KEYS * D * int(sizeof(T));
    static constexpr int STATS = SPLIT ? (2 * WAVES + 1) * 32 * 4 : 0, LDS = (SPLIT ? 2 * WAVES : 4) * TILE + STATS;
    static constexpr int PER_CU = sizeof(T) * D == 512 ? 1 : SPLIT || KEYS == 64 ? 2 : 3;  // workgroups that registers are kept free for
    static_assert(LDS - STATS >= ROWS * D * int(sizeof(T)) && (!SPLIT || 2 * TILE >= 32 * D * 4), "the outputs pass through the tiles' room");
};

template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__((64 * Fwd<T, D, SPLIT>::WAVES), (Fwd<T, D, SPLIT>::PER_CU)) void attention_fwd_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, Sequences seqs, T *__restrict__ o, float *__restrict__ lse,
    int blocks, int H, int Hk, int window, float scale2) {
    using C = Fwd<T, D, SPLIT>;
    using Ti = Tile<T, D>;
    constexpr int WAVES = C::WAVES, KEYS = C::KEYS, TILE = C::TILE, NT = KEYS / 32, QS = D / 16, NO = D / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    typename Ti::template Lane<32> ln(lane);
    const Item it = find_item(blockIdx.x, blocks, H, Hk);
    const Block b = find_block<C::ROWS>(seqs, it.block, blocks);
    if (b.at >= b.rows) return;
    const int hk = it.h / (H / Hk);
    const uint32_t kv_stride = uint32_t(Hk) * Ti::ROWB;
    const int r0 = b.at + (SPLIT ? 0 : 32 * wv), q_row = r0 + (lane & 31);  // the wavefront's first query and the lane's, as places in the sequence

    const int end = min(b.at + C::ROWS, b.n);                        // keys that the block's rows see
    const int first = window ? max(b.at - window + 1, 0) / KEYS : 0;  // tile of the first one
    const int tiles = b.at < b.n ? (end + KEYS - 1) / KEYS : first;   // none for rows that are no tokens
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

    typename Op<T>::frag qf[QS];
    {
        const T *p = q + ((static_cast<size_t>(b.lo) + min(q_row, b.rows - 1)) * H + it.h) * D + 8 * half;
#pragma unroll
        for (int s = 0; s < QS; ++s) qf[s] = load8<T, 32>(p + 16 * s);
    }
    f32x16_t acc[NO] = {};
    float m = LOWEST, l = 0.f;  // base 2, with the scale in

    auto step = [&](int j, unsigned char *kt, unsigned char *vt, auto keys_done, auto values_needed) __attribute__((always_inline)) {
        // In bf16 the places of all operands fit beside the rest (4.00 -> 3.94 ms at B1 T32768 H16 d128); 128 rows of d64 would lose 1 % by it.
        if constexpr (sizeof(T) == 4 || (!SPLIT && D == 64)) ln.again();
        f32x16_t x[NT] = {};
#pragma unroll
        for (int s = 0; s < QS; ++s)
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t] = Op<T>::mma(Ti::template row<32>(kt, 32 * t, s, ln), qf[s], x[t]);
        keys_done();
        if ((j + 1) * KEYS - 1 > r0 || (window && r0 + 31 - j * KEYS >= window)) {  // some key that some query does not see
            KEEP_BRANCH;
            const int last = q_row - j * KEYS - 4 * half, first_seen = window ? last - window : -1000;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = 32 * t + 8 * (i / 4) + i % 4;
                    x[t][i] = key <= last && key > first_seen ? x[t][i] : -INFINITY;
                }
        }
        float top = x[0][0];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, x[t][i]), x[t][i + 1]);
        top = halves_max(top) * scale2;
        if (__any(top > m + 8.f)) {
            const float now = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - now);
            l *= f;
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[n][i] *= f;
            m = now;
        }
        float sum[2] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[t][i] = __builtin_amdgcn_exp2f(fmaf(x[t][i], scale2, -m));
                sum[i & 1] += x[t][i];
            }
            if (t == 0) values_needed();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const auto p = acc_frag<T>(x[t], s);
#pragma unroll
                for (int n = 0; n < NO; ++n) acc[n] = Op<T>::mma(Ti::template col<32>(vt, 32 * t + 16 * s, 32 * n, ln), p, acc[n]);
            }
        }
        l += sum[0] + sum[1];
    };
    if constexpr (SPLIT) {
        constexpr int LOADS = KEYS / Ti::RPI;  // of one tile
        for (int j = from; j < tiles; j += WAVES) {
            const bool more = j + WAVES < tiles;
            own_loads_done<LOADS>();  // the values were asked for after the keys
            step(
                j, tile, tile + TILE,
                [&]() __attribute__((always_inline)) {
                    own_reads_done();
                    if (more) fetch_one(kb, j + WAVES, tile);
                },
                [&]() __attribute__((always_inline)) {
                    if (more)
                        own_loads_done<LOADS>();
                    else
                        own_loads_done<0>();
                });
            own_reads_done();
            if (more) fetch_one(vb, j + WAVES, tile + TILE);
        }
    } else {
        auto nothing = [] {};
        auto turn = [&](int j, auto buffer) __attribute__((always_inline)) {
            constexpr int buf = decltype(buffer)::value;
            loads_done();  // tile j is there, and every wavefront has left the other one
            if (j + 1 < tiles) fetch(j + 1, buf ^ 1);
            if (j * KEYS > r0 + 31 || (window && r0 + 1 - (j + 1) * KEYS >= window)) return;  // the wavefront sees nothing of the tile
            step(j, tile + buf * 2 * TILE, tile + buf * 2 * TILE + TILE, nothing, nothing);
        };
        for (int j = from; j < tiles; j += 2) {
            turn(j, std::integral_constant<int, 0>{});
            if (j + 1 < tiles) turn(j + 1, std::integral_constant<int, 1>{});
        }
    }

    l = halves_sum(l);
    const bool live = q_row < b.n;
    float *stats = reinterpret_cast<float *>(smem + C::LDS - C::STATS);
    if constexpr (SPLIT) {
        if (half == 0) {
            stats[64 * wv + lane] = m;
            stats[64 * wv + 32 + lane] = l;
        }
        lds_barrier();  // and all tiles are free
        const float own = m;
        l = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = fmaxf(m, stats[64 * w + (lane & 31)]);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) l = fmaf(stats[64 * w + 32 + (lane & 31)], __builtin_amdgcn_exp2f(stats[64 * w + (lane & 31)] - m), l);
        const float f = __builtin_amdgcn_exp2f(own - m);
#pragma unroll
        for (int n = 0; n < NO; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[n][i] *= f;
    }
    const float inv = live && l != 0.f ? 1.f / l : 0.f;
    if (half == 0 && q_row < b.rows && (!SPLIT || wv == 0)) {
        if (lse) lse[(static_cast<size_t>(b.lo) + q_row) * H + it.h] = live && l != 0.f ? (m + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
        if constexpr (SPLIT) stats[64 * WAVES + lane] = inv;
    }
    T *out = o + ((static_cast<size_t>(b.lo) + r0) * H + it.h) * D;
    if constexpr (SPLIT) {
        store_sums<T, D, WAVES>(smem, acc, [&](int r) { return stats[64 * WAVES + r]; }, out, static_cast<size_t>(H) * D, b.rows - r0, wv, lane);
    } else {
        lds_barrier();  // the tiles are free
        store_rows<T, D>(smem + wv * 32 * Ti::ROWB, acc, inv, inv != 0.f, out, static_cast<size_t>(H) * D, b.rows - r0, lane);
    }
}

template <typename T, int D, bool SPLIT> hipError_t launch(const AttentionCall &c, void *o, float *lse, hipStream_t stream) {
    using F = Fwd<T, D, SPLIT>;
    const hipError_t err = allow_lds<&attention_fwd_kernel<T, D, SPLIT>>(F::LDS);
    if (err != hipSuccess) return err;
    const int blocks = c.N / F::ROWS + c.S + 1;
    hipLaunchKernelGGL((attention_fwd_kernel<T, D, SPLIT>), dim3(static_cast<unsigned>(blocks) * c.H), dim3(64 * F::WAVES), F::LDS, stream,
                       static_cast<const T *>(c.q), static_cast<const T *>(c.k), static_cast<const T *>(c.v),
                       Sequences{c.offsets, c.lens, c.N, c.S, attention_by_place(c.offsets, c.N, c.S, c.window)}, static_cast<T *>(o), lse, blocks, c.H, c.Hk, c.window, c.scale * LOG2E);
    return hipGetLastError();
}

template <typename T, int D> hipError_t launch(const AttentionCall &c, void *o, float *lse, hipStream_t stream) {
    return attention_split(c.N, c.S, c.H, D, c.window) ? launch<T, D, true>(c, o, lse, stream) : launch<T, D, false>(c, o, lse, stream);
}

}  // namespace

hipError_t launch_attention_fwd(const AttentionCall &c, void *o, float *lse, hipStream_t stream) {
    if (c.d == 64) return c.bf16 ? launch<bf16_t, 64>(c, o, lse, stream) : launch<float, 64>(c, o, lse, stream);
    if (c.d == 128) return c.bf16 ? launch<bf16_t, 128>(c, o, lse, stream) : launch<float, 128>(c, o, lse, stream);
    return hipErrorInvalidValue;
}

}  // namespace muir
