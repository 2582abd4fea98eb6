// y [M, N] = x [M, K] W^T for a few rows of x and 4-bit weights: W[n, k] = (nib[n, k] - zero[n, k / G]) scale[n, k / G].
//
// What bounds it is reading the weights once (N K / 2 bytes). The products run on the matrix cores with rows m of x
// as A and 16 weight rows as B, contraction 32 at a time and so inside one group: nibbles become the bf16
// numbers 16 + nib (exact, two to three operations for two of them: the nibble moves to mantissa bits 3..6 of
// 16.0), and a group's sum is finished in float32 as scale (sum x (16 + nib) - (16 + zero) sum x). The second
// sum is a product with ones, shared by the NT weight tiles of a wavefront. float32 x goes in as three bf16
// terms (to its last bit or two).
//
// A lane loads 16 bytes, 32 weights of one row, and the four lanes of a row exchange them (4x4 transpose in
// registers) so that each product's contraction is 32 consecutive columns. The wavefronts of a workgroup split
// K; their sums meet in LDS in a fixed order.
#include "common.hpp"
#include "mfma.hpp"
#include "op_kernels.hpp"

namespace muir {
namespace {

constexpr int WAVES = 8;

// Lanes 16 g + m: on entry dword u of lane g is dword u of chunk g, on return dword g of chunk u.
__device__ __forceinline__ void exchange(uint4 &d) {
    auto a = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d = uint4{lo[0], lo[1], hi[0], hi[1]};
}

// The eight nibbles of a dword as bf16 16 + nib, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8_t nibbles(uint32_t w) {
    constexpr uint32_t M = 0x00780078u, B = 0x41804180u;
    const uint4 u{((w << 3) & M) | B, ((w >> 1) & M) | B, ((w >> 5) & M) | B, ((w >> 9) & M) | B};
    return __builtin_bit_cast(bf16x8_t, u);
}

// x of eight columns in that order, as NX bf16 terms.
template <int NX> struct XFrag { bf16x8_t f[NX]; };
__device__ __forceinline__ XFrag<1> x_frag(const bf16_t *p) {
    const u16x8_t u = *reinterpret_cast<const u16x8_t *>(p);
    return XFrag<1>{{__builtin_bit_cast(bf16x8_t, __builtin_shufflevector(u, u, 0, 4, 1, 5, 2, 6, 3, 7))}};
}
__device__ __forceinline__ XFrag<3> x_frag(const float *p) {
    float x[8];
    load_vec<8>(p, x);
    XFrag<3> r;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        u16x8_t u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = f32_to_bf16(x[j]);
            x[j] -= bf16_to_f32(u[j]);
        }
        r.f[n] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(u, u, 0, 4, 1, 5, 2, 6, 3, 7));
    }
    return r;
}

template <typename XT, typename ST, int NT, int GROUP>
__global__ __launch_bounds__(WAVES * 64) void matvec_q4_kernel(const XT *__restrict__ x, const uint8_t *__restrict__ w,
                                                               const ST *__restrict__ scale, const ST *__restrict__ zero,
                                                               XT *__restrict__ y, int M, int N, int K) {
    constexpr int NX = sizeof(XT) == 2 ? 1 : 3;
    constexpr int PER = GROUP / 32;  // products of a group
    __shared__ f32x4_t sh[WAVES][NT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int mt = blockIdx.y * 16, n0 = blockIdx.x * (16 * NT), KG = K / GROUP;
    const int steps = (K + 127) / 128;
    const int s0 = steps * wv / WAVES, s1 = steps * (wv + 1) / WAVES;
    const XT *xr = x + static_cast<size_t>(mt + m < M ? mt + m : 0) * K;
    const uint8_t *wr[NT];
    const ST *sr[NT], *zr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = min(n0 + 16 * t + m, N - 1);  // rows behind the last are computed and not stored
        wr[t] = w + static_cast<size_t>(n) * (K / 2);
        sr[t] = scale + static_cast<size_t>(n) * KG;
        zr[t] = zero ? zero + static_cast<size_t>(n) * KG : nullptr;
    }
    bf16x8_t ones;
#pragma unroll
    for (int j = 0; j < 8; ++j) ones[j] = static_cast<__bf16>(1.0f);

    f32x4_t sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = zero4();
    for (int s = s0; s < s1; ++s) {
        const int k0 = 128 * s;
        uint4 d[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            d[t] = k0 + 32 * g < K ? *reinterpret_cast<const uint4 *>(wr[t] + (k0 + 32 * g) / 2) : uint4{0, 0, 0, 0};
        XFrag<NX> fx[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + 32 * u + 8 * g;
            if (k < K && mt + m < M) {
                fx[u] = x_frag(xr + k);
            } else {
#pragma unroll
                for (int n = 0; n < NX; ++n) fx[u].f[n] = Mma<bf16_t>::zero();
            }
        }
        float sc[NT][4 / PER], zp[NT][4 / PER];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < 4 / PER; ++q) {
                const int kg = min(k0 / GROUP + q, KG - 1);
                sc[t][q] = to_f32(sr[t][kg]);
                zp[t][q] = 16.f + (zr[t] ? to_f32(zr[t][kg]) : 8.f);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) exchange(d[t]);
#pragma unroll
        for (int q = 0; q < 4 / PER; ++q) {
            f32x4_t xs = zero4(), acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = zero4();
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int u = q * PER + e;
#pragma unroll
                for (int n = NX - 1; n >= 0; --n) xs = Mma<bf16_t>::mma(fx[u].f[n], ones, xs);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t dw[4] = {d[t].x, d[t].y, d[t].z, d[t].w};
                    const bf16x8_t fw = nibbles(dw[u]);
#pragma unroll
                    for (int n = NX - 1; n >= 0; --n) acc[t] = Mma<bf16_t>::mma(fx[u].f[n], fw, acc[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[t][i] = fmaf(sc[t][q], fmaf(-zp[t][q], xs[i], acc[t][i]), sum[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) sh[wv][t][lane] = sum[t];
    __syncthreads();
    if (wv >= NT) return;
    // Wavefront t finishes weight tile t: rows m = 4 g + i of x, column n = lane % 16.
    f32x4_t r = sh[0][wv][lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) r += sh[i][wv][lane];
    const int n = n0 + 16 * wv + m;
    if (n >= N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (mt + 4 * g + i < M) elem<XT>::store(y, static_cast<size_t>(mt + 4 * g + i) * N + n, r[i]);
}

template <typename XT, typename ST, int NT>
hipError_t go(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N, int K, int group,
              hipStream_t s) {
    const dim3 grid((N + 16 * NT - 1) / (16 * NT), (M + 15) / 16), block(WAVES * 64);
#define MUIR_Q4(G)                                                                                                  \
    if (group == G) {                                                                                               \
        hipLaunchKernelGGL((matvec_q4_kernel<XT, ST, NT, G>), grid, block, 0, s, static_cast<const XT *>(x),        \
                           static_cast<const uint8_t *>(w), static_cast<const ST *>(scale),                         \
                           static_cast<const ST *>(zero), static_cast<XT *>(y), M, N, K);                           \
        return hipGetLastError();                                                                                   \
    }
    MUIR_Q4(32) MUIR_Q4(64) MUIR_Q4(128)
#undef MUIR_Q4
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_matvec_q4(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N,
                            int K, int group, bool bf16, bool scale_bf16, hipStream_t s) {
    if (bf16)
        return scale_bf16 ? go<bf16_t, bf16_t, 1>(x, w, scale, zero, y, M, N, K, group, s)
                          : go<bf16_t, float, 1>(x, w, scale, zero, y, M, N, K, group, s);
    return scale_bf16 ? go<float, bf16_t, 1>(x, w, scale, zero, y, M, N, K, group, s)
                      : go<float, float, 1>(x, w, scale, zero, y, M, N, K, group, s);
}

}  // namespace muir
