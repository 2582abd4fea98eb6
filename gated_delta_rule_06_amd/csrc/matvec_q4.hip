// y [M, N] = x [M, K] W^T for a few rows of x and 4-bit weights: W[n, k] = (nib[n, k] - zero[n, k / G]) scale[n, k / G].
//
// What bounds it is reading the weights once (N K / 2 bytes). The products run on the matrix cores with rows m of x
// as A and 16 weight rows as B, contraction 32 at a time and so inside one group: nibbles become the bf16
// numbers 16 + nib (exact, a shift and a mask-or for two of them: the nibble moves to mantissa bits 3..6 of
// 16.0), and a group's sum is finished in float32 as scale (sum x (16 + nib) - (16 + zero) sum x). The second
// sum is a product with ones, shared by the NT weight tiles of a wavefront. float32 x goes in as three bf16
// terms (to its last bit or two), and there the nibbles become nib - 8 (sign extension, a conversion and half a packing each): the
// terms of 16 + nib are up to five times as large as what is left of them, and float32 outputs showed their roundings.
//
// A workgroup walks K in tiles of 1024 columns, 128 to each of eight wavefronts (or pairs of them, half of the weight rows
// each), whose sums meet in LDS in a fixed order. A tile's weights, x and scales come as whole cache lines through LDS, the
// next tile's in flight. Reading them straight into the lanes that multiply them (16 rows, 64 bytes each, the scales one by
// one) took 2.5 times as long at M = 16, N = 16384, K = 8192, G = 64 with zeros: the vector cache looks up every row of a load on its own.
// Now 23.1 us a kernel there (3.1 TB/s) over eight sets of weights in turn, which no cache holds, and 19.1 on one set. Fetching two or three
// tiles ahead changed nothing. float32 rows take 55.6 us: their x is read in the step that uses it, by each wavefront.
// A lane takes 16 bytes, 32 weights of one row, from
// LDS, and the four lanes of a row exchange them (4x4 transpose in registers) so that each product's contraction
// is 32 consecutive columns.
#include "common.hpp"
#include "launch.hpp"
#include "mfma.hpp"
#include "op_kernels.hpp"

namespace muir {
namespace {

// Lanes 16 g + m: on entry dword u of lane g is dword u of chunk g, on return dword g of chunk u.
__device__ __forceinline__ void exchange(uint4 &d) {
    auto a = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
    auto b = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d = uint4{lo[0], lo[1], hi[0], hi[1]};
}

// The eight nibbles of a dword as bf16 16 + nib, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8_t nibbles(uint32_t w, uint32_t base) {
    constexpr uint32_t M = 0x00780078u;
    const uint4 u{((w << 3) & M) | base, ((w >> 1) & M) | base, ((w >> 5) & M) | base, ((w >> 9) & M) | base};
    return __builtin_bit_cast(bf16x8_t, u);
}

// The same as nib - 8.
__device__ __forceinline__ bf16x8_t signed_nibbles(uint32_t w) {
    constexpr int ORDER[8] = {0, 4, 1, 5, 2, 6, 3, 7};
    w ^= 0x88888888u;  // two's complement of nib - 8
    bf16x8_t f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = static_cast<__bf16>(static_cast<float>(static_cast<int>(w << (28 - 4 * ORDER[j])) >> 28));
    return f;
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

// LDS of one step: 16 NT rows of weights, 16 rows of bf16 x, the groups' scales with 16 + zero beside them.
template <typename XT, int NT, int WAVES, int GROUP> constexpr int q4_tile_bytes() {
    const int sc = 16 * NT * (WAVES * (128 / GROUP) + 1) * 8;
    return 16 * NT * (WAVES * 64 + 16) + (sizeof(XT) == 2 ? 16 * (WAVES * 256 + 16) : 0) + (sc + 15) / 16 * 16;
}

template <typename XT, typename ST, int NT, int NH, int WAVES, int GROUP, bool ZERO>
__global__ __launch_bounds__(WAVES *NH * 64) void matvec_q4_kernel(const XT *__restrict__ x, const uint8_t *__restrict__ w,
                                                               const ST *__restrict__ scale, const ST *__restrict__ zero,
                                                               XT *__restrict__ y, int M, int N, int K) {
    constexpr int NX = sizeof(XT) == 2 ? 1 : 3;
    constexpr bool XLDS = NX == 1;
    constexpr float OFFSET = NX == 1 ? 16.f : -8.f;  // what a nibble's bf16 number is more than it
    constexpr bool XSUM = NX == 1 || ZERO;           // without it nib - 8 is the weight
    constexpr int PER = GROUP / 32, NG = 4 / PER;  // products of a group, groups of a step
    constexpr int THREADS = WAVES * NH * 64, KT = WAVES * 128, NW = NT / NH;  // a wavefront has NW of the tiles of 16 rows
    constexpr int WC = KT / 32, XC = KT / 8;             // 16-byte chunks of a row of the tile
    constexpr int LW = WC * 16 + 16, LX = XC * 16 + 16;  // row strides, padded by 16 bytes: rows in different banks
    constexpr int NWL = 16 * NT * WC / THREADS, NXL = XLDS ? 16 * XC / THREADS : 1;
    static_assert(16 * NT * WC % THREADS == 0 && 16 * XC % THREADS == 0 && THREADS % WC == 0 && THREADS % XC == 0, "whole chunks");
    constexpr int SC = WAVES * NG, NSCALE = 16 * NT * SC, NSL = (NSCALE + THREADS - 1) / THREADS;  // scales of the tile
    constexpr int LS = SC + 1;                                                                    // row stride, in pairs
    constexpr int XAT = 16 * NT * LW, SAT = XAT + (XLDS ? 16 * LX : 0), TILE = q4_tile_bytes<XT, NT, WAVES, GROUP>();
    static_assert(TILE >= SAT + 16 * NT * LS * 8, "tile");
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wv = (tid >> 6) % WAVES, nh = (tid >> 6) / WAVES, m = lane & 15, g = lane >> 4;
    const int mt = blockIdx.y * 16, n0 = blockIdx.x * (16 * NT), KG = K / GROUP;
    const int tiles = (K + KT - 1) / KT, live = min(M - mt, 16), rows = N - n0;
    // One base for the workgroup; a lane's own offsets fit 32 bits (64 rows of at most 2^25 bytes).
    const uint8_t *wb = w + static_cast<size_t>(n0) * (K / 2);
    const ST *sb = scale + static_cast<size_t>(n0) * KG, *zb = ZERO ? zero + static_cast<size_t>(n0) * KG : nullptr;
    const XT *xb = x + static_cast<size_t>(mt) * K;

    uint32_t base = 0x41804180u;  // 16.0 twice, kept in a register: mask and or are then one instruction
    asm volatile("" : "+v"(base));

    // What a step needs from memory, fetched while the step before is multiplied.
    struct Step {
        uint4 w[NWL], x[NXL];
        ST sc[NSL], zp[NSL];
    };
    Step ahead;
    // A lane's offsets in the first tile; rows behind the last are the last again, computed and not stored.
    uint32_t at_w[NWL], at_s[NSL], at_x[NXL];
#pragma unroll
    for (int j = 0; j < NWL; ++j) {
        const int i = tid + THREADS * j;
        at_w[j] = static_cast<uint32_t>(min(i / WC, rows - 1)) * (K / 2) + i % WC * 16;
    }
#pragma unroll
    for (int j = 0; j < NSL; ++j) at_s[j] = static_cast<uint32_t>(min((tid + THREADS * j) / SC, rows - 1)) * KG;
#pragma unroll
    for (int j = 0; j < NXL; ++j) {
        const int i = tid + THREADS * j;
        at_x[j] = static_cast<uint32_t>(i / XC) * K + i % XC * 8;
    }
    auto fetch = [&](Step &f, int t) {
        const int kw = tid % WC * 32, kx = tid % XC * 8, left = K - t * KT;  // THREADS is a multiple of WC and XC
#pragma unroll
        for (int j = 0; j < NWL; ++j)
            f.w[j] = kw < left ? *reinterpret_cast<const uint4 *>(wb + (at_w[j] + static_cast<uint32_t>(t) * (KT / 2))) : uint4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NSL; ++j) {
            const int i = tid + THREADS * j;
            const uint32_t at = at_s[j] + min(t * SC + i % SC, KG - 1);
            if (NSCALE % THREADS == 0 || i < NSCALE) {
                f.sc[j] = sb[at];
                if constexpr (ZERO) f.zp[j] = zb[at];
            }
        }
        if constexpr (XLDS) {
#pragma unroll
            for (int j = 0; j < NXL; ++j)
                f.x[j] = kx < left && (tid + THREADS * j) / XC < live ? *reinterpret_cast<const uint4 *>(xb + (at_x[j] + static_cast<uint32_t>(t) * KT))
                                                                     : uint4{0, 0, 0, 0};
        }
    };
    bf16x8_t ones;
#pragma unroll
    for (int j = 0; j < 8; ++j) ones[j] = static_cast<__bf16>(1.0f);
    f32x4_t sum[NW];
#pragma unroll
    for (int t = 0; t < NW; ++t) sum[t] = zero4();

    auto step = [&](Step &f, int t) {
        unsigned char *lw = smem + (t & 1) * TILE, *lx = lw + XAT;
#pragma unroll
        for (int j = 0; j < NWL; ++j) {
            const int i = tid + THREADS * j;
            *reinterpret_cast<uint4 *>(lw + i / WC * LW + i % WC * 16) = f.w[j];
        }
        if constexpr (XLDS) {
#pragma unroll
            for (int j = 0; j < NXL; ++j) {
                const int i = tid + THREADS * j;
                if (i / XC < live) *reinterpret_cast<uint4 *>(lx + i / XC * LX + i % XC * 16) = f.x[j];
            }
        }
        float2 *ls = reinterpret_cast<float2 *>(lw + SAT);
#pragma unroll
        for (int j = 0; j < NSL; ++j) {
            const int i = tid + THREADS * j;
            float2 v{to_f32(f.sc[j]), OFFSET + 8.f};
            if constexpr (ZERO) v.y = OFFSET + to_f32(f.zp[j]);
            if (NSCALE % THREADS == 0 || i < NSCALE) ls[i / SC * LS + i % SC] = v;
        }
        if (t + 1 < tiles) fetch(f, t + 1);
        lds_barrier();
        // This wavefront's 128 columns of the tile.
        const int k0 = t * KT + 128 * wv;
        if (k0 >= K) return;
        XFrag<NX> fx[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = 32 * u + 8 * g;
#pragma unroll
            for (int n = 0; n < NX; ++n) fx[u].f[n] = Mma<bf16_t>::zero();
            if constexpr (XLDS) {
                if (m < live) fx[u] = x_frag(reinterpret_cast<const XT *>(lx + m * LX) + 128 * wv + k);
            } else {
                if (m < live && k0 + k < K) fx[u] = x_frag(xb + static_cast<size_t>(m) * K + k0 + k);
            }
        }
        uint4 d[NW];
#pragma unroll
        for (int n = 0; n < NW; ++n) {
            d[n] = *reinterpret_cast<const uint4 *>(lw + (16 * (nh * NW + n) + m) * LW + (4 * wv + g) * 16);
            exchange(d[n]);
        }
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            f32x4_t xs = zero4(), acc[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) acc[n] = zero4();
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int u = q * PER + e;
#pragma unroll
                for (int c = NX - 1; c >= 0; --c)
                    if constexpr (XSUM) xs = Mma<bf16_t>::mma(fx[u].f[c], ones, xs);
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    const uint32_t dw[4] = {d[n].x, d[n].y, d[n].z, d[n].w};
                    const bf16x8_t fw = NX == 1 ? nibbles(dw[u], base) : signed_nibbles(dw[u]);
#pragma unroll
                    for (int c = NX - 1; c >= 0; --c) acc[n] = Mma<bf16_t>::mma(fx[u].f[c], fw, acc[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                const float2 v = ls[(16 * (nh * NW + n) + m) * LS + wv * NG + q];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[n][i] = fmaf(v.x, XSUM ? fmaf(-v.y, xs[i], acc[n][i]) : acc[n][i], sum[n][i]);
            }
        }
    };
    fetch(ahead, 0);
    for (int t = 0; t < tiles; ++t) step(ahead, t);
    __syncthreads();
    f32x4_t *sh = reinterpret_cast<f32x4_t *>(smem);  // [WAVES][NT][64]
#pragma unroll
    for (int t = 0; t < NW; ++t) sh[(wv * NT + nh * NW + t) * 64 + lane] = sum[t];
    __syncthreads();
    const int tile = tid >> 6;
    if (tile >= NT) return;
    // Wavefront t finishes weight tile t: rows m = 4 g + i of x, column n = lane % 16.
    f32x4_t r = sh[tile * 64 + lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) r += sh[(i * NT + tile) * 64 + lane];
    const int n = n0 + 16 * tile + m;
    if (n >= N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * g + i < live) elem<XT>::store(y, static_cast<size_t>(mt + 4 * g + i) * N + n, r[i]);
}

template <typename XT, typename ST, int NT, int NH, int WAVES>
hipError_t go(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N, int K, int group,
              hipStream_t s) {
    static_assert(WAVES >= NT, "a wavefront finishes each tile");
    const dim3 grid((N + 16 * NT - 1) / (16 * NT), (M + 15) / 16), block(WAVES * NH * 64);
#define MUIR_Q4(G, Z)                                                                                               \
    if (group == G && (zero != nullptr) == Z) {                                                                     \
        auto kern = matvec_q4_kernel<XT, ST, NT, NH, WAVES, G, Z>;                                               \
        constexpr int two = 2 * q4_tile_bytes<XT, NT, WAVES, G>(), sums = WAVES * NT * 1024;                        \
        constexpr int bytes = two > sums ? two : sums;                                                              \
        const hipError_t err = allow_lds<matvec_q4_kernel<XT, ST, NT, NH, WAVES, G, Z>>(bytes);                            \
        if (err != hipSuccess) return err;                                                                          \
        hipLaunchKernelGGL(kern, grid, block, bytes, s, static_cast<const XT *>(x),                                 \
                           static_cast<const uint8_t *>(w), static_cast<const ST *>(scale),                         \
                           static_cast<const ST *>(zero), static_cast<XT *>(y), M, N, K);                           \
        return hipGetLastError();                                                                                   \
    }
    MUIR_Q4(32, false) MUIR_Q4(64, false) MUIR_Q4(128, false) MUIR_Q4(32, true) MUIR_Q4(64, true) MUIR_Q4(128, true)
#undef MUIR_Q4
    return hipErrorInvalidValue;
}

template <typename XT, typename ST>
hipError_t pick(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N, int K, int group,
                hipStream_t s) {
    // As many weight rows to a workgroup as leave one workgroup for each of the 256 compute units: x is read and unpacked
    // once for them all. us a kernel for 16, 32 and 64 rows (bf16, eight sets of weights in turn): M = 1, N = 2048, K = 2048: 3.8, 4.4, 5.6;
    // N = 8192, K = 2048: 6.8, 5.1, 5.9; N = 16384, K = 8192: 34.4, 23.7, 19.9; M = 64, N = K = 4096 (four times the workgroups): 22.0,
    // 13.7, 10.1. Sixteen wavefronts, half of the rows each, against eight with all of them: 23.1 and 23.9 at M = 16, N = 16384, K = 8192,
    // 19.8 and 21.6 at M = 1; float32 rows lose by it, 55.6 and 49.3.
    const long long work = static_cast<long long>(N) * ((M + 15) / 16);
    if (work >= 256 * 64) return go<XT, ST, 4, 2, 8>(x, w, scale, zero, y, M, N, K, group, s);
    if (work >= 256 * 32) return go<XT, ST, 2, 2, 8>(x, w, scale, zero, y, M, N, K, group, s);
    return go<XT, ST, 1, 1, 8>(x, w, scale, zero, y, M, N, K, group, s);
}

}  // namespace

hipError_t launch_matvec_q4(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N,
                            int K, int group, bool bf16, bool scale_bf16, hipStream_t s) {
    if (bf16)
        return scale_bf16 ? pick<bf16_t, bf16_t>(x, w, scale, zero, y, M, N, K, group, s)
                          : pick<bf16_t, float>(x, w, scale, zero, y, M, N, K, group, s);
    return scale_bf16 ? pick<float, bf16_t>(x, w, scale, zero, y, M, N, K, group, s)
                      : pick<float, float>(x, w, scale, zero, y, M, N, K, group, s);
}

}  // namespace muir
