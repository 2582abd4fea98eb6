// Operands, tiles and sequences shared by the kernels of causal softmax attention (attention.hip, attention_bwd.hip,
// attention_step.hip).
//
// With s_ij = scale q_i . k_j over the keys j that query i sees (same sequence, i - window < j <= i):
//   lse_i = log sum_j exp s_ij     p_ij = exp(s_ij - lse_i)     o_i = sum_j p_ij v_j
// Exponentials are taken to base 2, with log2(e) folded into the scale.
//
// Every product over 32 rows is D[32 x 32] += A[32 x 16] B[32 x 16]^T on the matrix cores. Scores are made transposed where
// the following product sums over their rows, so that their accumulators are the next operand as they are: a lane holds one
// column, and eight consecutive accumulators are the eight contraction values of one product.
#pragma once

#include <type_traits>

#include "attention_layout.hpp"
#include "chunk_layout.hpp"
#include "common.hpp"
#include "mfma.hpp"

namespace muir {
namespace at {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

constexpr float LN2 = 0.6931471805599453f;
// A running maximum before any key: below scores of any size that a sum of products leaves exact, and finite, so that differences from it stay
// numbers.
constexpr float LOWEST = -3e38f;

// Eight contraction values of one operand row: lane l has row l % 32, and its element j is contraction index 8 (l / 32) + j
// of a product's 16 (frag), or row l % 16 and index 8 (l / 16) + j of 32 (frag16).
template <typename T> struct Op;
template <> struct Op<bf16_t> {
    using frag = bf16x8_t;
    using frag16 = bf16x8_t;
    static __device__ __forceinline__ f32x16_t mma(frag a, frag b, f32x16_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4_t mma16(frag16 a, frag16 b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Rounds to bf16, nearest even.
    static __device__ __forceinline__ frag pack(const float (&x)[8]) {
        return frag{static_cast<__bf16>(x[0]), static_cast<__bf16>(x[1]), static_cast<__bf16>(x[2]), static_cast<__bf16>(x[3]),
                    static_cast<__bf16>(x[4]), static_cast<__bf16>(x[5]), static_cast<__bf16>(x[6]), static_cast<__bf16>(x[7])};
    }
    static __device__ __forceinline__ frag16 pack16(const float (&x)[8]) { return pack(x); }
};
// float32 as three bf16 terms, each the next 8 bits of the value, so they hold all 24. A product is six of nine: the second term is below 2^-7 of the value's
// power of two and the third below 2^-15, so the three left out are together below 8 times 2^-24 of the product, always towards zero, since terms are cut off
// rather than rounded, and 0.63 times 2^-24 in the mean of values from 1 to 2. Rounding the second term to nearest would halve the bound and make it of either
// sign, and takes 96 us where cutting off takes 91 (training B3 T777 H12 d64; the first one too: 102); outputs come no nearer to 64 bits by it
// (o 4.4e-7 and 4.3e-7 off, dq 6.1e-7 both, lse 7e-8 and 6e-8). On the bf16 matrix cores that is 6 instructions of 32 cycles for
// 16 contraction values, where float32's own take 8 of 64; splitting eight values costs 44 vector instructions beside.
template <> struct Op<float> {
    struct frag {
        bf16x8_t t[3];
    };
    typedef float frag16 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x16_t mma(const frag &a, const frag &b, f32x16_t c) {
        // Smallest first: they are added to a sum that the largest then makes large.
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[2], b.t[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[1], b.t[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[1], b.t[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[1], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[0], c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4_t mma16(frag16 a, frag16 b, f32x4_t c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ frag pack(const float (&x)[8]) {
        float r[8];
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = __float_as_uint(r[2 * j]), hi = __float_as_uint(r[2 * j + 1]);
                w[j] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);  // the upper halves of both
                if (n < 2) {
                    r[2 * j] -= __uint_as_float(lo & 0xffff0000u);
                    r[2 * j + 1] -= __uint_as_float(hi & 0xffff0000u);
                }
            }
            f.t[n] = __builtin_bit_cast(bf16x8_t, w);
        }
        return f;
    }
    static __device__ __forceinline__ frag16 pack16(const float (&x)[8]) { return frag16{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}; }
};
// What a lane of an R-row product takes.
template <typename T, int R> using frag_of = std::conditional_t<R == 32, typename Op<T>::frag, typename Op<T>::frag16>;
template <typename T, int R> __device__ __forceinline__ frag_of<T, R> make_frag(const float (&x)[8]) {
    if constexpr (R == 32)
        return Op<T>::pack(x);
    else
        return Op<T>::pack16(x);
}

// Eight consecutive stored values (16-byte aligned).
template <typename T, int R> __device__ __forceinline__ frag_of<T, R> load8(const T *p) {
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const bf16x8_t *>(p);
    } else {
        float x[8];
        load_vec<8>(p, x);
        return make_frag<T, R>(x);
    }
}

// The transposing read. Through a function of a `restrict` pointer, as plain reads of LDS carry their type: without either the compiler takes it
// to read what asynchronous loads on their way are writing, and waits for all of them.
__device__ __forceinline__ s16x4_t read_transposed(lds_s16x4 *__restrict__ p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }

// A tile of token rows of D values in LDS, without padding, as the asynchronous loads write it: lane after lane 16 bytes. The
// 16-byte pieces of a row are permuted by its number so that reading one piece of 16 rows (operand rows) and 64 bytes of
// eight rows (the transposing reads) both take every bank evenly. The permutation repeats every 16 rows.
template <typename T, int D> struct Tile {
    static constexpr int ROWB = D * int(sizeof(T)), CH = ROWB / 16, RPI = 64 / CH;  // RPI: rows of one load of a wavefront
    static __device__ __forceinline__ int swz(int r) {
        return CH == 8 ? ((r & 2) << 1) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int r, int chunk) { return r * ROWB + ((chunk ^ swz(r)) << 4); }

    // A lane's place in the two kinds of operand below, for rows and columns 0 on; the others are an exclusive or with a constant and a constant
    // offset away, since whole powers of two of pieces are. `again` makes the compiler form those anew where it is called: kept in
    // registers they cost sixteen of them.
    template <int R> struct Lane {
        int row, col;
        __device__ __forceinline__ explicit Lane(int lane) {
            const int m = lane % 16, g = lane / R;
            row = at(lane % R, g * int(sizeof(T)) / 2);
            if constexpr (sizeof(T) == 2) {
                const int b = 2 * (lane % R / 16 * 16) + 8 * (m & 3);
                col = at(4 * g + (m >> 2), b >> 4) + (b & 8);
            } else {
                col = at(4 * g, lane % R >> 2) + 4 * (lane & 3);
            }
        }
        __device__ __forceinline__ void again() { asm volatile("" : "+v"(row), "+v"(col)); }
    };

    // Operand rows r0 + l % R, contraction values 16 s + 8 (l / 32) + j (32 rows) or 32 s + 8 (l / 16) + j (16 rows).
    template <int R> static __device__ __forceinline__ frag_of<T, R> row(const unsigned char *t, int r0, int s, const Lane<R> &ln) {
        const unsigned char *p = t + r0 * ROWB;
        const int x = ln.row ^ (s * (64 / R) * int(sizeof(T)) / 2 << 4);
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const bf16x8_t *>(p + x);
        } else {
            const f32x4_t a = *reinterpret_cast<const f32x4_t *>(p + x), b = *reinterpret_cast<const f32x4_t *>(p + (x ^ 16));
            return make_frag<T, R>({a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
        }
    }
    // Operand rows are the tile's columns c0 + l % R; element j is tile row r0 + 4 (l / R) + j % 4, and 256 / R rows on
    // for j >= 4: the order in which two 4-row groups of an accumulator lie in a lane. r0 is a multiple of 16.
    template <int R> static __device__ __forceinline__ frag_of<T, R> col(unsigned char *t, int r0, int c0, const Lane<R> &ln) {
        constexpr int NEXT = 256 / R, FLIP = R == 32 ? 2 << 4 : 0;  // of the permutation, eight rows on
        unsigned char *p = t + r0 * ROWB;
        const int x = ln.col ^ (c0 * int(sizeof(T)) >> 4 << 4);
        if constexpr (sizeof(T) == 2) {
            // The transposing read gives lane m of sixteen the column m of the four rows whose 32 bytes the lanes address.
            const s16x4_t lo = read_transposed((lds_s16x4 *)(p + x));
            const s16x4_t hi = read_transposed((lds_s16x4 *)(p + NEXT * ROWB + (x ^ FLIP)));
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = *reinterpret_cast<const float *>(p + (j % 4 + j / 4 * NEXT) * ROWB + (x ^ (j % 4 << 6) ^ (j / 4 * FLIP)));
            return make_frag<T, R>(f);
        }
    }
    // Four consecutive values from column c on (a multiple of 4) of row r.
    static __device__ __forceinline__ void put4(unsigned char *t, int r, int c, f32x4_t v) {
        unsigned char *p = t + at(r, c * int(sizeof(T)) >> 4);
        store4(reinterpret_cast<T *>(p) + (c & (16 / int(sizeof(T)) - 1)), v);
    }

    // ROWS rows from `base` on into the tile, by WAVES wavefronts of which this is `wv`, straight to LDS. Rows from `live`
    // on, and so what lies behind a sequence, come as zeros. `stride` is the bytes from row to row.
    // AUX: the loads' cache policy, 0 or STREAM.
    static constexpr int STREAM = 2;
    template <int ROWS, int WAVES, int AUX = 0> static __device__ __forceinline__ void fetch(unsigned char *t, const void *base, uint32_t stride, int live, int wv, int lane) {
        const rsrc_t r = make_rsrc(base, live <= 0 ? 0u : uint32_t(min(live, ROWS) - 1) * stride + ROWB);
#pragma unroll
        for (int n = 0; n < ROWS / RPI / WAVES; ++n) {
            const int r0 = (n * WAVES + wv) * RPI, i = lane / CH;
            // Only the row's place in its 16 enters the permutation, so most loads of a wavefront share their lanes' offsets.
            const uint32_t voff = i * stride + (((lane % CH) ^ swz((r0 & 15) + i)) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(t + r0 * ROWB), 16, voff, r0 * stride, 0, AUX);
        }
    }
};

// Keeps what follows it in a branch there: the compiler would rather make selects of it for everybody.
#define KEEP_BRANCH asm volatile("")

// Order of a stretch of code that multiplies operands as it reads them: one step's reads first (and FIRST others), then in turn a step's products and the reads of
// the step after it. The compiler's own order waits for each operand right after asking for it.
template <int STEPS, int READS, int PRODUCTS, int FIRST = 0> __device__ __forceinline__ void read_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, FIRST + READS, 0);
#pragma unroll
    for (int s = 1; s < STEPS; ++s) {
        __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS, 0);
}

// Waits for every load of this wavefront; the barrier behind it makes all wavefronts' tiles visible.
__device__ __forceinline__ void loads_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
}

// Waits until at most `LEFT` of this wavefront's loads are out: the ones before them, into a tile of its own, are done.
template <int LEFT> __device__ __forceinline__ void own_loads_done() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory"); }
// Before new loads into a tile of this wavefront's own: its reads of the old one are done.
__device__ __forceinline__ void own_reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Largest and sum over the two halves of a wavefront, which hold the same columns.
__device__ __forceinline__ float halves_max(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Row of accumulator element i (of 16) in a 32-row result.
__device__ __forceinline__ int acc_row(int i, int lane) { return 8 * (i / 4) + 4 * (lane / 32) + i % 4; }
// Eight accumulators as the operand of step s (of two).
template <typename T> __device__ __forceinline__ typename Op<T>::frag acc_frag(const f32x16_t &x, int s) {
    return Op<T>::pack({x[8 * s], x[8 * s + 1], x[8 * s + 2], x[8 * s + 3], x[8 * s + 4], x[8 * s + 5], x[8 * s + 6], x[8 * s + 7]});
}

// A wavefront's 32 rows, given transposed in accumulators, through its own LDS room to `rows` rows of `stride` elements, times f; zeros where not live.
template <typename T, int D>
__device__ __forceinline__ void store_rows(unsigned char *room, const f32x16_t (&acc)[D / 32], float f, bool live, T *out, size_t stride, int rows,
                                           int lane) {
    using Ti = Tile<T, D>;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4_t y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = live ? acc[n][4 * i + r] * f : 0.f;
            Ti::put4(room, lane & 31, 32 * n + 8 * i + 4 * (lane >> 5), y);
        }
    wave_lds_sync();
#pragma unroll
    for (int n = 0; n < 32 / Ti::RPI; ++n) {
        const int r = n * Ti::RPI + lane / Ti::CH, c = lane % Ti::CH;
        if (r < rows)
            *reinterpret_cast<u32x4_t *>(out + r * stride + c * (16 / sizeof(T))) = *reinterpret_cast<const u32x4_t *>(room + Ti::at(r, c));
    }
    wave_lds_sync();
}
// The same where the wavefronts of a workgroup have summands of the same 32 rows: they are added in the wavefronts' order. `factor` is of a row. The
// room, which nobody else may be using, is 32 D floats a wavefront.
template <typename T, int D, int WAVES, typename F>
__device__ __forceinline__ void store_sums(unsigned char *room, const f32x16_t (&acc)[D / 32], F factor, T *out, size_t stride, int rows, int wv,
                                           int lane) {
    using Ti = Tile<float, D>;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            Ti::put4(room + wv * 32 * Ti::ROWB, lane & 31, 32 * n + 8 * i + 4 * (lane >> 5),
                     f32x4_t{acc[n][4 * i], acc[n][4 * i + 1], acc[n][4 * i + 2], acc[n][4 * i + 3]});
    lds_barrier();
    for (int i = threadIdx.x; i < 32 * (D / 4); i += 64 * WAVES) {
        const int r = i / (D / 4), c = i % (D / 4);
        f32x4_t y = zero4();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) y += *reinterpret_cast<const f32x4_t *>(room + w * 32 * Ti::ROWB + Ti::at(r, c));
        const float f = factor(r);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = f != 0.f ? y[e] * f : 0.f;
        if (r < rows) store4(out + r * stride + 4 * c, y);
    }
    lds_barrier();
}

// Sum and largest over a wavefront of values not below 0, for everybody.
template <typename F> __device__ __forceinline__ int wave_all(int x, F f) {
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));  // from 1, 2, 4 and 8 lanes before, in rows of 16
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));  // a row's last lane to the next row
    x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));  // lane 31 to the upper half
    return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ int wave_add(int x) {
    return wave_all(x, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int wave_max(int x) {
    return wave_all(x, [](int a, int b) { return max(a, b); });
}

// Block `i` of a launch of `blocks` (FROM_END: of keys). All 64 lanes search together.
template <int R, bool FROM_END = false> __device__ __forceinline__ Block find_block(const Sequences &q, int i, int blocks) {
    if (!q.offsets) return equal_block(q, R, i, FROM_END);
    const int lane = threadIdx.x & 63;
    Block b;
    if (q.by_place && q.S < 64) {
        const int lo = q.first(lane), rows = lane <= q.S ? q.rows(lane) : 0, n = lane < q.S ? q.tokens(lane) : 0, own = (rows + R - 1) / R;
        auto count = [&](int p) { return wave_add(max(own - p, 0)); };
        if (i >= count(0)) return no_block(q);
        const int p = search_place(wave_max(own), i, count), rank = i - count(p + 1);
        const uint64_t has = __ballot(own > p);
        const bool mine = own > p && __popcll(has & ((uint64_t(1) << lane) - 1)) == rank;
        const int s = __builtin_ctzll(__ballot(mine));
        const int all = __builtin_amdgcn_readlane(own, s);
        b = Block{s, __builtin_amdgcn_readlane(lo, s), __builtin_amdgcn_readlane(rows, s), __builtin_amdgcn_readlane(n, s), (FROM_END ? all - 1 - p : p) * R};
    } else {
        const int w = FROM_END ? i : blocks - 1 - i;  // their most work is at the end, or at the start
        const int s = search_sequence(q.S, [&](int lo, int step, int hi) {
            const int k = lo + lane * step;
            return __builtin_amdgcn_readfirstlane(static_cast<int>(__popcll(__ballot(k <= hi && q.first(k) / R + k <= w))));
        });
        b = block_in(q, R, w, s);
        b.seq = __builtin_amdgcn_readfirstlane(b.seq);
        b.lo = __builtin_amdgcn_readfirstlane(b.lo);
        b.rows = __builtin_amdgcn_readfirstlane(b.rows);
        b.n = __builtin_amdgcn_readfirstlane(b.n);
        b.at = __builtin_amdgcn_readfirstlane(b.at);
    }
    return b;
}

}  // namespace at
}  // namespace muir
