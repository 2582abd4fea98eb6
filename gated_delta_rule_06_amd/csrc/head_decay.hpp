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

#include "common.hpp"
#include "mfma.hpp"
#include "op_layout.hpp"

namespace muir {
namespace hd {

constexpr int THREADS = 256;  // four wavefronts, each with a quarter of the state's columns

// A fragment holds 16 rows x 32 contraction indices of an operand: lane l has row l % 16, and its
// element j is contraction index 16 (j / 4) + 4 (l / 16) + j % 4. In that order two stacked 16x16
// accumulators are a fragment as they are (their column becomes the row), so the state is multiplied
// from its registers.
template <typename T> struct Op;

template <> struct Op<bf16_t> {
    static constexpr int PAD = 8;  // row padding of an LDS tile: rows fall into different banks
    using frag = bf16x8_t;
    static __device__ __forceinline__ frag row(const bf16_t *t, int ld, int r0, int k0, int lane) {
        const bf16_t *p = t + (r0 + (lane & 15)) * ld + k0 + 4 * (lane >> 4);
        const u16x4_t a = *reinterpret_cast<const u16x4_t *>(p);
        const u16x4_t b = *reinterpret_cast<const u16x4_t *>(p + 16);
        return __builtin_bit_cast(frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // Rows of the operand are columns c0.. of the tile. The transposing read gives lane m of a group of 16
    // the column m of the four tile rows whose 32 bytes the group's lanes address.
    static __device__ __forceinline__ frag col(const bf16_t *t, int ld, int k0, int c0, int lane) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
        const int m = lane & 15, g = lane >> 4;
        const bf16_t *p = t + (k0 + 4 * g + (m >> 2)) * ld + c0 + 4 * (m & 3);
        const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
        const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * ld));
        return __builtin_bit_cast(frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ void floats(frag f, float (&x)[8]) {
        const u16x8_t u = __builtin_bit_cast(u16x8_t, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = bf16_to_f32(u[j]);
    }
    // x as the sum of N bf16 fragments: each rounds what the ones before left (8 bits each, so three
    // hold a float32 to its last bit or two).
    template <int N> static __device__ __forceinline__ void split(float (&x)[8], frag (&f)[N]) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            u16x8_t u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[j] = f32_to_bf16(x[j]);
                if (n + 1 < N) x[j] -= bf16_to_f32(u[j]);
            }
            f[n] = __builtin_bit_cast(frag, u);
        }
    }
    static __device__ __forceinline__ f32x4_t mma(frag a, frag b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Four consecutive values as N terms, one to each of N tiles `plane` elements apart.
    template <int N> static __device__ __forceinline__ void put4(bf16_t *p, int plane, f32x4_t v) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            u16x4_t u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = f32_to_bf16(v[i]);
                if (n + 1 < N) v[i] -= bf16_to_f32(u[i]);
            }
            *reinterpret_cast<u16x4_t *>(p + n * plane) = u;
        }
    }
};

template <> struct Op<float> {
    static constexpr int PAD = 4;
    struct frag { float v[8]; };
    static __device__ __forceinline__ frag row(const float *t, int ld, int r0, int k0, int lane) {
        const float *p = t + (r0 + (lane & 15)) * ld + k0 + 4 * (lane >> 4);
        const f32x4_t a = *reinterpret_cast<const f32x4_t *>(p);
        const f32x4_t b = *reinterpret_cast<const f32x4_t *>(p + 16);
        return frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    static __device__ __forceinline__ frag col(const float *t, int ld, int k0, int c0, int lane) {
        const float *p = t + (k0 + 4 * (lane >> 4)) * ld + c0 + (lane & 15);
        frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = p[(16 * (j >> 2) + (j & 3)) * ld];
        return f;
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
    template <int N> static __device__ __forceinline__ void put4(float *p, int, f32x4_t v) {
        static_assert(N == 1, "float32 operands are one term");
        *reinterpret_cast<f32x4_t *>(p) = v;
    }
};

// log2 of a decay. A decay of zero (or below 2^-200) becomes 2^-200, which is zero in float32 however it is
// multiplied on, and keeps the sums of logarithms finite.
__device__ __forceinline__ double log2_decay(float a) {
    const float l = log2f(a);
    return l < -200.f ? -200.0 : static_cast<double>(l);
}

// Inclusive sum over the lanes up to this one. In 64 bits: the sums reach -12800 (64 zeros) while the
// differences taken of them have to be exact to 2^-24.
__device__ __forceinline__ double scan64(double x, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    return x;
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace hd
}  // namespace muir
