// Root-mean-square norm with the residual's addition: forward, 8-bit output, backward.
//   h = x + residual (rounded to h's type, the new residual stream; the norm is taken of the rounded h)
//   rstd = (mean(h^2) + eps)^(-1/2)      y = h rstd weight
//   backward, with p = dy weight and n = h rstd: dx = rstd (p - n mean(p n)) + dh, dweight = sum over rows of dy n
// Every kernel reads and writes each element once; a row stays in registers between the sums and their use,
// TPR threads to a row with NV vectors of 8 columns each. All sums are in float32, in a fixed order.
// Memory bounds them. 32768 x 2048 bf16 (fastest of 20): forward with residual 90 us (5.9 TB/s), backward 124 (4.3 TB/s), dweight's
// sum 4.5; to e4m3 with a float32 residual 138 (5.3 TB/s).
#include <algorithm>

#include "common.hpp"
#include "mfma.hpp"
#include "op_kernels.hpp"
#include "op_layout.hpp"

namespace muir {
namespace {

constexpr int NORM_THREADS = 256;

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]) { load_vec<8>(p, x); }
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    store4(p, f32x4_t{x[0], x[1], x[2], x[3]});
    store4(p + 4, f32x4_t{x[4], x[5], x[6], x[7]});
}
__device__ __forceinline__ void store8(bf16_t *p, const float (&x)[8]) { Mma<bf16_t>::store(p, x); }

template <typename T> __device__ __forceinline__ float rounded(float x);
template <> __device__ __forceinline__ float rounded<float>(float x) { return x; }
template <> __device__ __forceinline__ float rounded<bf16_t>(float x) { return bf16_to_f32(f32_to_bf16(x)); }

// Sum over the TPR threads of a row (a wavefront, or the whole workgroup); every thread gets it.
template <int TPR> __device__ __forceinline__ float row_sum(float x, float *sh) {
    x = wave_sum(x);
    if constexpr (TPR > 64) {
        const int wv = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh[wv] = x;
        __syncthreads();
        x = (sh[0] + sh[1]) + (sh[2] + sh[3]);
    }
    return x;
}

// Largest |x| as bits: they order as the values do, and a NaN is above everything, so it is kept.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
template <int LANES> __device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), off, 64)));
    return x;
}

// h of one row into registers (and memory, with a residual), and 1 / rms.
template <typename XT, typename HT, int TPR, int NV, bool RES>
__device__ __forceinline__ float load_h(const NormCall &c, size_t row, int tr, float (&h)[NV][8], float *sh) {
    const XT *x = static_cast<const XT *>(c.x) + row * c.D;
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = 8 * (tr + TPR * n);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[n][j] = 0.f;
        if (col < c.D) load8(x + col, h[n]);
    }
    if constexpr (RES) {
        const HT *r = static_cast<const HT *>(c.residual) + row * c.D;
        HT *ho = static_cast<HT *>(c.h) + row * c.D;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = 8 * (tr + TPR * n);
            if (col >= c.D) continue;
            float r8[8];
            load8(r + col, r8);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[n][j] = rounded<HT>(h[n][j] + r8[j]);
            store8(ho + col, h[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[n][j], h[n][j], ss);
    ss = row_sum<TPR>(ss, sh);
    return 1.f / sqrtf(ss / static_cast<float>(c.D) + c.eps);
}

template <typename XT, typename HT, int TPR, int NV, bool RES>
__global__ __launch_bounds__(NORM_THREADS) void rms_norm_kernel(NormCall c, XT *y, float *rstd) {
    __shared__ float sh[4];
    const int tr = threadIdx.x % TPR;
    const size_t row = static_cast<size_t>(blockIdx.x) * (NORM_THREADS / TPR) + threadIdx.x / TPR;
    if (row >= static_cast<size_t>(c.rows)) return;  // whole rows leave: TPR threads share one
    float h[NV][8];
    const float r = load_h<XT, HT, TPR, NV, RES>(c, row, tr, h, sh);
    if (rstd && tr == 0) rstd[row] = r;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = 8 * (tr + TPR * n);
        if (col >= c.D) continue;
        float w[8];
        load8(c.weight + col, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[n][j] = h[n][j] * r * w[j];
        store8(y + row * c.D + col, h[n]);
    }
}

// 8 bits: q = round(y / scale), scale = max|y| / top over the row or over 128 columns (16 lanes). A scale below
// the smallest normal number is raised to it, and is 1 where all of y is zero.
template <typename XT, typename HT, int TPR, int NV, bool RES, bool E4M3, bool GROUP>
__global__ __launch_bounds__(NORM_THREADS) void rms_norm_8bit_kernel(NormCall c, uint8_t *y, float *scale) {
    __shared__ float sh[4];
    __shared__ uint32_t sh_max[4];
    const int tr = threadIdx.x % TPR;
    const size_t row = static_cast<size_t>(blockIdx.x) * (NORM_THREADS / TPR) + threadIdx.x / TPR;
    if (row >= static_cast<size_t>(c.rows)) return;
    float h[NV][8];
    const float r = load_h<XT, HT, TPR, NV, RES>(c, row, tr, h, sh);
    uint32_t top[NV], all = 0;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = 8 * (tr + TPR * n);
        top[n] = 0;
        if (col < c.D) {
            float w[8];
            load8(c.weight + col, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[n][j] = h[n][j] * r * w[j];
                top[n] = max(top[n], abs_bits(h[n][j]));
            }
        }
        if constexpr (GROUP) top[n] = lanes_max<16>(top[n]);
        all = max(all, top[n]);
    }
    if constexpr (!GROUP) {
        all = lanes_max<64>(all);
        if constexpr (TPR > 64) {
            if ((threadIdx.x & 63) == 0) sh_max[threadIdx.x >> 6] = all;
            __syncthreads();
            all = max(max(sh_max[0], sh_max[1]), max(sh_max[2], sh_max[3]));
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = 8 * (tr + TPR * n);
        if (col >= c.D) continue;
        const uint32_t bits = GROUP ? top[n] : all;
        float s = __uint_as_float(bits) / (E4M3 ? 448.f : 127.f);
        s = bits == 0 ? 1.f : s < 1.17549435e-38f ? 1.17549435e-38f : s;
        uint32_t q[2];
        if constexpr (E4M3) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                int v = __builtin_amdgcn_cvt_pk_fp8_f32(h[n][4 * k] / s, h[n][4 * k + 1] / s, 0, false);
                v = __builtin_amdgcn_cvt_pk_fp8_f32(h[n][4 * k + 2] / s, h[n][4 * k + 3] / s, v, true);
                q[k] = static_cast<uint32_t>(v);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                q[k] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float t = fminf(fmaxf(rintf(h[n][4 * k + j] / s), -127.f), 127.f);
                    q[k] |= (static_cast<uint32_t>(static_cast<int>(t)) & 0xffu) << (8 * j);
                }
            }
        }
        *reinterpret_cast<uint2 *>(y + row * c.D + col) = uint2{q[0], q[1]};
        if constexpr (GROUP) {
            if (col % 128 == 0) scale[row * (c.D / 128) + col / 128] = s;
        } else {
            if (col == 0) scale[row] = s;
        }
    }
}

// Backward. A workgroup takes every gridDim-th set of rows and keeps its threads' columns of dweight in
// registers; the workgroups' sums meet in `part` [gridDim, D].
template <typename YT, typename HT, int TPR, int NV>
__global__ __launch_bounds__(NORM_THREADS) void rms_norm_bwd_kernel(const YT *dy, const HT *h, const float *weight,
                                                                    const float *rstd, const HT *dh, HT *dx,
                                                                    float *part, int rows, int D) {
    constexpr int RPB = NORM_THREADS / TPR;
    __shared__ float sh[4];
    __shared__ float sh_w[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NV * 8 : 1];
    const int tr = threadIdx.x % TPR, rb = threadIdx.x / TPR;
    float dw[NV][8] = {};
    const int steps = (rows + gridDim.x * RPB - 1) / (gridDim.x * RPB);
    for (int i = 0; i < steps; ++i) {
        const size_t row = (static_cast<size_t>(i) * gridDim.x + blockIdx.x) * RPB + rb;
        const bool live = row < static_cast<size_t>(rows);  // the same for all threads of a row
        const float r = live ? rstd[row] : 0.f;
        float n8[NV][8], p8[NV][8], s = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = 8 * (tr + TPR * n);
#pragma unroll
            for (int j = 0; j < 8; ++j) n8[n][j] = p8[n][j] = 0.f;
            if (live && col < D) {
                float w[8];
                load8(dy + row * D + col, p8[n]);
                load8(h + row * D + col, n8[n]);
                load8(weight + col, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n8[n][j] *= r;
                    dw[n][j] = fmaf(p8[n][j], n8[n][j], dw[n][j]);
                    p8[n][j] *= w[j];
                    s = fmaf(p8[n][j], n8[n][j], s);
                }
            }
        }
        s = row_sum<TPR>(s, sh) / static_cast<float>(D);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = 8 * (tr + TPR * n);
            if (!live || col >= D) continue;
            float g[8] = {};
            if (dh) load8(dh + row * D + col, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = fmaf(r, p8[n][j] - n8[n][j] * s, g[j]);
            store8(dx + row * D + col, g);
        }
    }
    float *out = part + static_cast<size_t>(blockIdx.x) * D;
    if constexpr (RPB > 1) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) sh_w[rb][8 * (tr + TPR * n) + j] = dw[n][j];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += NORM_THREADS) {
            float x = 0.f;
#pragma unroll
            for (int b = 0; b < RPB; ++b) x += sh_w[b][c];
            out[c] = x;
        }
    } else {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = 8 * (tr + TPR * n);
            if (col < D) store8(out + col, dw[n]);
        }
    }
}

// dweight: 16 columns to a workgroup, four lanes to a part and 64 parts side by side. (Four parts side by side on 64
// columns were 39 us at D = 2048 with 512 parts: few loads in flight on few workgroups; this is 4.)
__global__ __launch_bounds__(256) void rms_norm_dw_kernel(const float *part, float *dweight, int parts, int D) {
    __shared__ f32x4_t sh[64][4];
    const int c = threadIdx.x & 3, p = threadIdx.x >> 2, col = blockIdx.x * 16 + 4 * c;
    f32x4_t x = zero4();
    if (col < D) {
#pragma unroll 4
        for (int i = p; i < parts; i += 64) x += *reinterpret_cast<const f32x4_t *>(part + static_cast<size_t>(i) * D + col);
    }
    sh[p][c] = x;
    for (int n = 32; n >= 1; n >>= 1) {
        __syncthreads();
        if (p < n) sh[p][c] += sh[p + n][c];
    }
    if (p == 0 && col < D)
#pragma unroll
        for (int i = 0; i < 4; ++i) dweight[col + i] = sh[0][c][i];
}

// Threads and vectors of a row by its length: a wavefront up to 2048 columns, the workgroup up to 16384.
#define MUIR_NORM_SIZES(D, F)        \
    if (D <= 512) return F(64, 1);   \
    if (D <= 1024) return F(64, 2);  \
    if (D <= 2048) return F(64, 4);  \
    if (D <= 4096) return F(256, 2); \
    if (D <= 8192) return F(256, 4); \
    return F(256, 8);

template <typename XT, typename HT, int TPR, int NV>
hipError_t norm_go(const NormCall &c, void *y, float *rstd, hipStream_t s) {
    const unsigned rpb = NORM_THREADS / TPR;
    const dim3 grid((static_cast<unsigned>(c.rows) + rpb - 1) / rpb);
    if (c.residual)
        hipLaunchKernelGGL((rms_norm_kernel<XT, HT, TPR, NV, true>), grid, dim3(NORM_THREADS), 0, s, c, static_cast<XT *>(y), rstd);
    else
        hipLaunchKernelGGL((rms_norm_kernel<XT, HT, TPR, NV, false>), grid, dim3(NORM_THREADS), 0, s, c, static_cast<XT *>(y), rstd);
    return hipGetLastError();
}

template <typename XT, typename HT> hipError_t norm_sized(const NormCall &c, void *y, float *rstd, hipStream_t s) {
#define MUIR_F(TPR, NV) norm_go<XT, HT, TPR, NV>(c, y, rstd, s)
    MUIR_NORM_SIZES(c.D, MUIR_F)
#undef MUIR_F
}

template <typename XT, typename HT, int TPR, int NV>
hipError_t norm8_go(const NormCall &c, void *y, float *scale, int fmt, int group, hipStream_t s) {
    const unsigned rpb = NORM_THREADS / TPR;
    const dim3 grid((static_cast<unsigned>(c.rows) + rpb - 1) / rpb), block(NORM_THREADS);
    uint8_t *q = static_cast<uint8_t *>(y);
#define MUIR_N8(RES, E, G)                                                                                   \
    if ((c.residual != nullptr) == RES && (fmt == 0) == E && (group != 0) == G) {                            \
        hipLaunchKernelGGL((rms_norm_8bit_kernel<XT, HT, TPR, NV, RES, E, G>), grid, block, 0, s, c, q, scale); \
        return hipGetLastError();                                                                            \
    }
    MUIR_N8(true, true, true) MUIR_N8(true, true, false) MUIR_N8(true, false, true) MUIR_N8(true, false, false)
    MUIR_N8(false, true, true) MUIR_N8(false, true, false) MUIR_N8(false, false, true) MUIR_N8(false, false, false)
#undef MUIR_N8
    return hipErrorInvalidValue;
}

template <typename XT, typename HT>
hipError_t norm8_sized(const NormCall &c, void *y, float *scale, int fmt, int group, hipStream_t s) {
#define MUIR_F(TPR, NV) norm8_go<XT, HT, TPR, NV>(c, y, scale, fmt, group, s)
    MUIR_NORM_SIZES(c.D, MUIR_F)
#undef MUIR_F
}

template <typename YT, typename HT, int TPR, int NV>
hipError_t bwd_go(const void *dy, const void *h, const float *weight, const float *rstd, const void *dh, void *dx,
                  float *part, int rows, int D, hipStream_t s) {
    hipLaunchKernelGGL((rms_norm_bwd_kernel<YT, HT, TPR, NV>), dim3(norm_bwd_blocks(rows, D)), dim3(NORM_THREADS), 0, s,
                       static_cast<const YT *>(dy), static_cast<const HT *>(h), weight, rstd,
                       static_cast<const HT *>(dh), static_cast<HT *>(dx), part, rows, D);
    return hipGetLastError();
}

template <typename YT, typename HT>
hipError_t bwd_sized(const void *dy, const void *h, const float *weight, const float *rstd, const void *dh, void *dx,
                     float *part, int rows, int D, hipStream_t s) {
#define MUIR_F(TPR, NV) bwd_go<YT, HT, TPR, NV>(dy, h, weight, rstd, dh, dx, part, rows, D, s)
    MUIR_NORM_SIZES(D, MUIR_F)
#undef MUIR_F
}

}  // namespace

hipError_t launch_rms_norm(const NormCall &c, void *y, float *rstd, hipStream_t s) {
    if (c.x_bf16) return c.h_bf16 ? norm_sized<bf16_t, bf16_t>(c, y, rstd, s) : norm_sized<bf16_t, float>(c, y, rstd, s);
    return norm_sized<float, float>(c, y, rstd, s);
}

hipError_t launch_rms_norm_8bit(const NormCall &c, void *y8, float *scale, int fmt, int group, hipStream_t s) {
    if (c.x_bf16)
        return c.h_bf16 ? norm8_sized<bf16_t, bf16_t>(c, y8, scale, fmt, group, s)
                        : norm8_sized<bf16_t, float>(c, y8, scale, fmt, group, s);
    return norm8_sized<float, float>(c, y8, scale, fmt, group, s);
}

hipError_t launch_rms_norm_bwd(const void *dy, const void *h, const float *weight, const float *rstd, const void *dh,
                               void *dx, float *dweight, int rows, int D, bool y_bf16, bool h_bf16, void *workspace,
                               hipStream_t s) {
    float *part = static_cast<float *>(workspace);
    if (rows > 0) {
        const hipError_t err =
            y_bf16 ? (h_bf16 ? bwd_sized<bf16_t, bf16_t>(dy, h, weight, rstd, dh, dx, part, rows, D, s)
                             : bwd_sized<bf16_t, float>(dy, h, weight, rstd, dh, dx, part, rows, D, s))
                   : bwd_sized<float, float>(dy, h, weight, rstd, dh, dx, part, rows, D, s);
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(rms_norm_dw_kernel, dim3((D + 15) / 16), dim3(256), 0, s, part, dweight,
                       rows > 0 ? norm_bwd_blocks(rows, D) : 0, D);
    return hipGetLastError();
}

}  // namespace muir
