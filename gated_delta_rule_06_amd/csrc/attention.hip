// Causal softmax attention over whole prompts, forward: o_i = sum_j p_ij v_j, with the running maximum and sum of the
// softmax, one pass over the keys.
//
// A workgroup has 128 query rows of one head, 32 to a wavefront, whose queries stay in registers; keys and values come in tiles through LDS,
// the next tile's loads (straight to LDS) in flight. Scores are made transposed, S^T = K Q^T, so a lane holds scores of one query: the maximum and the
// sum are sums inside the lane and over the two halves of the wavefront, and the accumulators of P^T are the operand of O^T += V^T P^T.
// bf16: p is rounded to bf16 for that product (half a step, 2^-9 of each term, of either sign), its sum is taken before the rounding, and
// everything else is float32.
// The output is rescaled only where a row's maximum grew by more than 2^8 over the reference its exponentials are taken from; up to there
// they are as exact in float32 and bf16 as below 1.
#include "attention.hpp"
#include "attention_kernels.hpp"
#include "launch.hpp"

namespace muir {
namespace {

using namespace at;

template <typename T, int D> struct Fwd {
    static constexpr int WAVES = 4, ROWS = 32 * WAVES, KEYS = sizeof(T) == 2 ? 64 : 32;
    static constexpr int TILE = KEYS * D * int(sizeof(T)), LDS = 4 * TILE;
    static_assert(ROWS == ATTENTION_ROWS && LDS >= ROWS * D * int(sizeof(T)), "the outputs pass through the tiles' room");
};

template <typename T, int D>
__global__ __launch_bounds__(256, (sizeof(T) * D == 512 ? 1 : 2)) void attention_fwd_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                                                            Sequences seqs, T *__restrict__ o, float *__restrict__ lse, int blocks,
                                                            int H, int Hk, int window, float scale2) {
    using C = Fwd<T, D>;
    using Ti = Tile<T, D>;
    constexpr int WAVES = C::WAVES, KEYS = C::KEYS, TILE = C::TILE, NT = KEYS / 32, QS = D / 16, NO = D / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    typename Ti::template Lane<32> ln(lane);
    const Item it = find_item(blockIdx.x, blocks, H, Hk);
    const Block b = find_block<C::ROWS>(seqs, blocks - 1 - it.block);  // late blocks of a sequence first: they see the most keys
    if (b.at >= b.rows) return;
    const int hk = it.h / (H / Hk);
    const size_t row0 = static_cast<size_t>(b.lo) + b.at;  // of the block
    const uint32_t kv_stride = uint32_t(Hk) * Ti::ROWB;
    const int q_row = b.at + 32 * wv + (lane & 31);  // this lane's query, as a place in its sequence

    const int end = min(b.at + C::ROWS, b.n);                        // keys that the block's rows see
    const int first = window ? max(b.at - window + 1, 0) / KEYS : 0;  // tile of the first one
    const int tiles = b.at < b.n ? (end + KEYS - 1) / KEYS : first;   // none for rows that are no tokens
    const T *kb = k + (static_cast<size_t>(b.lo) * Hk + hk) * D, *vb = v + (static_cast<size_t>(b.lo) * Hk + hk) * D;
    auto fetch = [&](int j, int buf) {
        const size_t at = static_cast<size_t>(j) * KEYS * Hk * D;
        Ti::template fetch<KEYS, WAVES>(smem + buf * 2 * TILE, kb + at, kv_stride, b.n - j * KEYS, wv, lane);
        Ti::template fetch<KEYS, WAVES>(smem + buf * 2 * TILE + TILE, vb + at, kv_stride, b.n - j * KEYS, wv, lane);
    };
    if (first < tiles) fetch(first, 0);

    typename Op<T>::frag qf[QS];
    {
        const T *p = q + (row0 + min(32 * wv + (lane & 31), b.rows - b.at - 1)) * H * D + static_cast<size_t>(it.h) * D + 8 * half;
#pragma unroll
        for (int s = 0; s < QS; ++s) qf[s] = load8<T>(p + 16 * s);
    }
    f32x16_t acc[NO] = {};
    float m = LOWEST, l = 0.f;  // base 2, with the scale in

    const int r0 = b.at + 32 * wv;  // the wavefront's first query
    auto step = [&](int j, unsigned char *kt, unsigned char *vt) __attribute__((always_inline)) {
        ln.again();
        f32x16_t x[NT] = {};
#pragma unroll
        for (int s = 0; s < QS; ++s)
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t] = Op<T>::mma(Ti::template row<32>(kt, 32 * t, s, ln), qf[s], x[t]);
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
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const auto p = acc_frag<T>(x[t], s);
#pragma unroll
                for (int n = 0; n < NO; ++n) acc[n] = Op<T>::mma(Ti::template col<32>(vt, 32 * t + 16 * s, 32 * n, ln), p, acc[n]);
            }
        }
        l += sum[0] + sum[1];
    };
    auto turn = [&](int j, auto buffer) __attribute__((always_inline)) {
        constexpr int buf = decltype(buffer)::value;
        loads_done();  // tile j is there, and every wavefront has left the other one
        if (j + 1 < tiles) fetch(j + 1, buf ^ 1);
        if (j * KEYS > r0 + 31 || (window && r0 + 1 - (j + 1) * KEYS >= window)) return;  // the wavefront sees nothing of the tile
        step(j, smem + buf * 2 * TILE, smem + buf * 2 * TILE + TILE);
    };
    for (int j = first; j < tiles; j += 2) {
        turn(j, std::integral_constant<int, 0>{});
        if (j + 1 < tiles) turn(j + 1, std::integral_constant<int, 1>{});
    }

    l = halves_sum(l);
    const bool live = q_row < b.n;
    const float inv = live && l != 0.f ? 1.f / l : 0.f;
    if (half == 0 && q_row < b.rows && lse)
        lse[(static_cast<size_t>(b.lo) + q_row) * H + it.h] = live && l != 0.f ? (m + __builtin_amdgcn_logf(l)) * LN2 : -INFINITY;
    lds_barrier();  // the tiles are free
    unsigned char *out = smem + wv * 32 * Ti::ROWB;
#pragma unroll
    for (int n = 0; n < NO; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4_t y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = live ? acc[n][4 * i + r] * inv : 0.f;
            Ti::put4(out, lane & 31, 32 * n + 8 * i + 4 * half, y);
        }
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < 32 / Ti::RPI; ++n) {
        const int r = n * Ti::RPI + lane / Ti::CH, c = lane % Ti::CH;
        if (b.at + 32 * wv + r < b.rows)
            *reinterpret_cast<u32x4_t *>(o + ((row0 + 32 * wv + r) * H + it.h) * D + c * (16 / sizeof(T))) = *reinterpret_cast<const u32x4_t *>(out + Ti::at(r, c));
    }
}

template <typename T, int D> hipError_t launch(const AttentionCall &c, void *o, float *lse, hipStream_t stream) {
    using F = Fwd<T, D>;
    const hipError_t err = allow_lds<&attention_fwd_kernel<T, D>>(F::LDS);
    if (err != hipSuccess) return err;
    const int blocks = static_cast<int>(attention_blocks(c.N, c.S));
    hipLaunchKernelGGL((attention_fwd_kernel<T, D>), dim3(static_cast<unsigned>(blocks) * c.H), dim3(64 * F::WAVES), F::LDS, stream,
                       static_cast<const T *>(c.q), static_cast<const T *>(c.k), static_cast<const T *>(c.v),
                       Sequences{c.offsets, c.lens, c.N, c.S}, static_cast<T *>(o), lse, blocks, c.H, c.Hk, c.window, c.scale * LOG2E);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_fwd(const AttentionCall &c, void *o, float *lse, hipStream_t stream) {
    if (c.d == 64) return c.bf16 ? launch<bf16_t, 64>(c, o, lse, stream) : launch<float, 64>(c, o, lse, stream);
    if (c.d == 128) return c.bf16 ? launch<bf16_t, 128>(c, o, lse, stream) : launch<float, 128>(c, o, lse, stream);
    return hipErrorInvalidValue;
}

}  // namespace muir
