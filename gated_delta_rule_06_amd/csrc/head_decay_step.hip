// One token of linear attention with one decay per head: S <- a S + k v^T, o = S^T q, in place.
//
// The state is read and written once (8 dk dv bytes a head) and that is the whole cost. Columns are
// independent, so a workgroup takes COLS of a head's dv columns: all of them where there is a head for each compute
// unit, 32 where there is not. A thread has four columns (16-byte loads) of four rows; the output sums over
// rows first inside each wavefront, then over the wavefronts through LDS, in a fixed order. State loads and
// stores are non-temporal: the state is not touched again before the next step. B256 H16 Hk4 128/128 bf16: 83 us for 541 MB, 6.5 TB/s,
// on one state (some of its 268 MB may stay in the last-level cache from call to call); B1 H16: 2.8 us.
#include "common.hpp"
#include "mfma.hpp"
#include "op_kernels.hpp"

namespace muir {
namespace {

template <typename QT, int DK, int DV, int COLS>
__global__ __launch_bounds__(DK *COLS / 16) void head_decay_step_kernel(
    const QT *__restrict__ q, const QT *__restrict__ k, const QT *__restrict__ v, const float *__restrict__ a,
    bool a_fixed, float *__restrict__ state, QT *__restrict__ o, int H, int Hk) {
    constexpr int THREADS = DK * COLS / 16, TPR = COLS / 4, GROUPS = THREADS / TPR, ROWS = DK / GROUPS;
    constexpr int NW = THREADS / 64, SLABS = DV / COLS;
    static_assert(ROWS == 4 && THREADS % 64 == 0, "shape");
    __shared__ float sh_part[NW][COLS];
    const int slab = blockIdx.x % SLABS, bh = blockIdx.x / SLABS, b = bh / H, h = bh % H;
    const int tid = threadIdx.x, c4 = tid % TPR, rg = tid / TPR, col = slab * COLS + 4 * c4;
    float *S = state + static_cast<size_t>(bh) * DK * DV + col;
    f32x4_t s[ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
        s[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t *>(S + (rg + m * GROUPS) * DV));
    const size_t ko = (static_cast<size_t>(b) * Hk + h / (H / Hk)) * DK;
    float kk[ROWS], qq[ROWS], v4[4];
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
        kk[m] = elem<QT>::load(k, ko + rg + m * GROUPS);
        qq[m] = elem<QT>::load(q, ko + rg + m * GROUPS);
    }
    load_vec<4>(v + static_cast<size_t>(bh) * DV + col, v4);
    const float decay = a[a_fixed ? h : bh];
    f32x4_t y = zero4();
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[m][c] = fmaf(decay, s[m][c], kk[m] * v4[c]);
            y[c] = fmaf(qq[m], s[m][c], y[c]);
        }
        __builtin_nontemporal_store(s[m], reinterpret_cast<f32x4_t *>(S + (rg + m * GROUPS) * DV));
    }
#pragma unroll
    for (int off = TPR; off < 64; off <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] += __shfl_xor(y[c], off, 64);
    const int wv = tid >> 6, ln = tid & 63;
    if (ln < TPR) reinterpret_cast<f32x4_t *>(sh_part[wv])[ln] = y;
    __syncthreads();
    if (tid < COLS) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) t += sh_part[i][tid];
        elem<QT>::store(o, static_cast<size_t>(bh) * DV + slab * COLS + tid, t);
    }
}

template <typename QT, int DK, int DV, int COLS>
hipError_t launch_cols(const void *q, const void *k, const void *v, const float *a, bool a_fixed, float *state,
                       void *o, int B, int H, int Hk, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(B) * H * (DV / COLS));
    hipLaunchKernelGGL((head_decay_step_kernel<QT, DK, DV, COLS>), grid, dim3(DK * COLS / 16), 0, stream,
                       static_cast<const QT *>(q), static_cast<const QT *>(k), static_cast<const QT *>(v), a,
                       a_fixed, state, static_cast<QT *>(o), H, Hk);
    return hipGetLastError();
}

template <typename QT, int DK, int DV>
hipError_t launch_sized(const void *q, const void *k, const void *v, const float *a, bool a_fixed, float *state,
                        void *o, int B, int H, int Hk, hipStream_t stream) {
    // A workgroup of a whole head is DK * DV / 16 threads, 256 to 1024; with fewer heads than compute units, split the columns.
    if (static_cast<long long>(B) * H >= 256)
        return launch_cols<QT, DK, DV, DV>(q, k, v, a, a_fixed, state, o, B, H, Hk, stream);
    return launch_cols<QT, DK, DV, 32>(q, k, v, a, a_fixed, state, o, B, H, Hk, stream);
}

}  // namespace

hipError_t launch_head_decay_step(const void *q, const void *k, const void *v, const float *a, bool a_fixed,
                                  float *state, void *o, int B, int H, int Hk, int dk, int dv, bool bf16,
                                  hipStream_t stream) {
#define MUIR_HDS(K, V)                                                                                     \
    if (dk == K && dv == V)                                                                                \
        return bf16 ? launch_sized<bf16_t, K, V>(q, k, v, a, a_fixed, state, o, B, H, Hk, stream)          \
                    : launch_sized<float, K, V>(q, k, v, a, a_fixed, state, o, B, H, Hk, stream);
    MUIR_HDS(64, 64) MUIR_HDS(64, 128) MUIR_HDS(128, 64) MUIR_HDS(128, 128)
#undef MUIR_HDS
    return hipErrorInvalidValue;
}

}  // namespace muir
