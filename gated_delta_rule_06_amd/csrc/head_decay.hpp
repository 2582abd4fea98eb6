// Operands, fragments and decays shared by the kernels of linear attention with one decay per
// head (head_decay.hip, head_decay_step.hip) and the sizes of their workspaces.
//
// The recurrence, per batch element and value head (q and k shared by H / Hk value heads):
//   S_t = a_t S_{t-1} + k_t v_t^T          o_t = S_t^T q_t
// With D_ij = prod_{j<u<=i} a_u it is, over a chunk of 64 tokens with start state S_0,
//   o_i = D_i0 S_0^T q_i + sum_{j<=i} D_ij (q_i . k_j) v_j      S_64 = D_640 S_0 + sum_j D_64j k_j v_j^T
// and each gradient has the same form (x, y, z) -> sum_j D (x_i . y_j) z_j + decayed state . x_i:
//   dq: (do, v, k), state S^T, tokens in order        dk: (v, do, q), state A^T, tokens reversed
//   dv: (k, q, do), state A, tokens reversed          A_t = a_{t+1} A_{t+1} + q_t do_t^T, adjoint of S_t
// so one kernel serves the forward and the three gradients.
#pragma once

#include <type_traits>

#include "chunk_layout.hpp"
#include "common.hpp"
#include "mfma.hpp"
#include "op_layout.hpp"

namespace muir {
namespace hd {


// A fragment holds 16 rows x 32 contraction indices of an operand: lane l has row l % 16, and its
// element j is contraction index 16 (j / 4) + 4 (l / 16) + j % 4. In that order two stacked 16x16
// accumulators are a fragment as they are (their column becomes the row), so the state is multiplied
// from its registers.
template <typename T> struct Op;

template <> struct Op<bf16_t> {
    using frag = bf16x8_t;
    template <int D> static constexpr int tile_bytes() { return C * D * 2 + C; }
    // Byte offset of element (r, 4 c) of a tile [64][D]. Tiles have no padding; the 8-byte pieces of a row are permuted
    // by its number so that both reads below, 32 lanes at a time, take every bank once: `row` takes piece c of 16 rows and
    // c + 1 (or + 2, + 3), `col` takes four pieces of eight rows. Padded rows serve one of the two: with 272 bytes a row the
    // transposing reads met in pairs, 2100 of 5200 LDS cycles a chunk. The permutation keeps 16-byte pieces whole.
    // 16 bytes between blocks of 16 rows keep the compiler from reading two blocks with one instruction whose two
    // addresses lie in the same banks (1460 cycles a chunk).
    template <int D> static __device__ __forceinline__ int at(int r, int c) {
        const int f = D == 128 ? ((r & 7) << 2) | ((r >> 2) & 2) : ((r & 6) << 1) | ((r >> 2) & 2);
        return r * (D * 2) + (r >> 4) * 16 + 8 * (c ^ f);
    }
    // r0 and k0 are constants, so what is left at run time is a handful of addresses per tile width.
    template <int D> static __device__ __forceinline__ frag row(const unsigned char *t, int r0, int k0, int lane) {
        const int base = at<D>(lane & 15, lane >> 4);
        const u16x4_t a = *reinterpret_cast<const u16x4_t *>(t + ((base ^ (2 * k0)) + r0 * (D * 2 + 1)));
        const u16x4_t b = *reinterpret_cast<const u16x4_t *>(t + ((base ^ (2 * k0 + 32)) + r0 * (D * 2 + 1)));
        return __builtin_bit_cast(frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // Rows of the operand are columns c0.. of the tile. The transposing read gives lane m of a group of 16
    // the column m of the four tile rows whose 32 bytes the group's lanes address.
    template <int D> static __device__ __forceinline__ frag col(unsigned char *t, int k0, int c0, int lane) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
        const int m = lane & 15, g = lane >> 4, base = at<D>(4 * g + (m >> 2), m & 3) ^ (2 * c0);
        const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(t + (base + k0 * (D * 2 + 1))));
        const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(t + (base + (k0 + 16) * (D * 2 + 1))));
        return __builtin_bit_cast(frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // 16 bytes of row r, column piece c (of 8 elements).
    template <int D> static __device__ __forceinline__ void put16(unsigned char *t, int r, int c, u32x4_t v) {
        *reinterpret_cast<u32x4_t *>(t + at<D>(r, 2 * c)) = v;
    }
    // Four elements of row r from column 4 c on.
    template <int D> static __device__ __forceinline__ f32x4_t quad(const unsigned char *t, int r, int c) {
        const u16x4_t u = *reinterpret_cast<const u16x4_t *>(t + at<D>(r, c));
        return f32x4_t{bf16_to_f32(u[0]), bf16_to_f32(u[1]), bf16_to_f32(u[2]), bf16_to_f32(u[3])};
    }
    static __device__ __forceinline__ void floats(frag f, float (&x)[8]) {
        const u16x8_t u = __builtin_bit_cast(u16x8_t, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = bf16_to_f32(u[j]);
    }
    // Two values rounded to bf16 in one register, and, where more terms follow, what the rounding left.
    template <bool REST> static __device__ __forceinline__ uint32_t term(float &x, float &y) {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        const uint32_t p = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{x, y}, bf16x2_t));
        if constexpr (REST) {
            x -= __uint_as_float(p << 16);
            y -= __uint_as_float(p & 0xffff0000u);
        }
        return p;
    }
    // x as the sum of N bf16 fragments: each rounds what the ones before left (8 bits each, so three
    // hold a float32 to its last bit or two).
    template <int N> static __device__ __forceinline__ void split(float (&x)[8], frag (&f)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            u32x4_t u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = n + 1 < N ? term<true>(x[2 * j], x[2 * j + 1]) : term<false>(x[2 * j], x[2 * j + 1]);
            f[n] = __builtin_bit_cast(frag, u);
        }
    }
    static __device__ __forceinline__ f32x4_t mma(frag a, frag b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Four consecutive values of row r from column 4 c on, as N terms, one to each of N tiles of width D.
    template <int D, int N> static __device__ __forceinline__ void put4(unsigned char *t, int r, int c, f32x4_t v) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float w[4] = {v[0], v[1], v[2], v[3]};
            u32x2_t u;
#pragma unroll
            for (int i = 0; i < 2; ++i) u[i] = n + 1 < N ? term<true>(w[2 * i], w[2 * i + 1]) : term<false>(w[2 * i], w[2 * i + 1]);
            v = f32x4_t{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<u32x2_t *>(t + n * tile_bytes<D>() + at<D>(r, c)) = u;
        }
    }
};

template <> struct Op<float> {
    struct frag { float v[8]; };
    // Rows are padded by four elements: the eight single reads of `col` then take different banks.
    template <int D> static constexpr int tile_bytes() { return C * (D + 4) * 4; }
    template <int D> static __device__ __forceinline__ const float *elem(const unsigned char *t, int r, int c) {
        return reinterpret_cast<const float *>(t) + r * (D + 4) + c;
    }
    template <int D> static __device__ __forceinline__ frag row(const unsigned char *t, int r0, int k0, int lane) {
        const float *p = elem<D>(t, r0 + (lane & 15), k0 + 4 * (lane >> 4));
        const f32x4_t a = *reinterpret_cast<const f32x4_t *>(p);
        const f32x4_t b = *reinterpret_cast<const f32x4_t *>(p + 16);
        return frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    template <int D> static __device__ __forceinline__ frag col(unsigned char *t, int k0, int c0, int lane) {
        const float *p = elem<D>(t, k0 + 4 * (lane >> 4), c0 + (lane & 15));
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = p[(16 * (j >> 2) + (j & 3)) * (D + 4)];
        return f;
    }
    template <int D> static __device__ __forceinline__ void put16(unsigned char *t, int r, int c, u32x4_t v) {
        *reinterpret_cast<u32x4_t *>(const_cast<float *>(elem<D>(t, r, 4 * c))) = v;
    }
    template <int D> static __device__ __forceinline__ f32x4_t quad(const unsigned char *t, int r, int c) {
        return *reinterpret_cast<const f32x4_t *>(elem<D>(t, r, 4 * c));
    }
    static __device__ __forceinline__ void floats(const frag &f, float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = f.v[j];
    }
    template <int N> static __device__ __forceinline__ void split(float (&x)[8], frag (&f)[N]) {
        static_assert(N == 1, "float32 operands are one term");
#pragma unroll
        for (int j = 0; j < 8; ++j) f[0].v[j] = x[j];
    }
    static __device__ __forceinline__ f32x4_t mma(const frag &a, const frag &b, f32x4_t c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
        return c;
    }
    template <int D, int N> static __device__ __forceinline__ void put4(unsigned char *t, int r, int c, f32x4_t v) {
        static_assert(N == 1, "float32 operands are one term");
        *reinterpret_cast<f32x4_t *>(const_cast<float *>(elem<D>(t, r, 4 * c))) = v;
    }
};

// log2 of a decay. A decay of zero (or below 2^-200) becomes 2^-200, which is zero in float32 however it is
// multiplied on, and keeps the sums of logarithms finite.
__device__ __forceinline__ double log2_decay(float a) {
    const float l = log2f(a);
    return l < -200.f ? -200.0 : static_cast<double>(l);
}

// x of the lane that a DPP control names, 0 where it names none.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_or_zero(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// Inclusive sum over the lanes up to this one (shifts by 1, 2, 4 and 8 inside rows of 16 lanes, then the last lane of a row
// to the next one or two). In 64 bits: the sums reach -12800 (64 zeros) while the differences taken of them have to be
// good to 2^-24.
__device__ __forceinline__ double scan64(double x) {
    x += dpp_or_zero<0x111, 0xf>(x);
    x += dpp_or_zero<0x112, 0xf>(x);
    x += dpp_or_zero<0x114, 0xf>(x);
    x += dpp_or_zero<0x118, 0xf>(x);
    x += dpp_or_zero<0x142, 0xa>(x);
    x += dpp_or_zero<0x143, 0xc>(x);
    return x;
}

// The value of one lane for the whole wavefront.
__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

// exp2(hi + lo) to the last bit or so, for the decays of a whole chunk, which go into states. Those between two tokens of a chunk do
// without: their last bits show in no output (float32 outputs and gradients are off by the same 2e-7 to 3e-7 with and without).
__device__ __forceinline__ float exp2_pair(float hi, float lo) {
    const float n = rintf(hi);
    return __builtin_amdgcn_ldexpf(exp2_f((hi - n) + lo), static_cast<int>(n));
}
__device__ __forceinline__ float exp2_pair(double x) {
    const float hi = static_cast<float>(x);
    return exp2_pair(hi, static_cast<float>(x - hi));
}

}  // namespace hd
}  // namespace muir
