// Internal launchers of the layer operators around the chunk forward: linear attention with one decay per
// head, the root-mean-square norm, products with 4-bit weights. Arguments are validated by the C ABI layer
// (op_api.cpp) before any of these is called; each returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace muir {

// Linear attention with one decay per head. q, k [B, T, Hk, dk], v [B, T, H, dv]; a [B, T, H], or [H] with
// a_fixed; lens [B] or NULL.
struct HeadDecayCall {
    const void *q, *k, *v;
    const float *a;
    bool a_fixed;
    const int *lens;
    const float *s0;
    int B, T, H, Hk, dk, dv;
    bool bf16;
};
// Segments of the token axis that run side by side (1: one workgroup walks a whole head).
int head_decay_segments(int B, int T, int H, bool bf16);
size_t head_decay_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, bool bf16);
size_t head_decay_bwd_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv, bool bf16);
hipError_t launch_head_decay_fwd(const HeadDecayCall &c, void *o, float *s_out, void *workspace,
                                 hipStream_t stream);
struct HeadDecayGrads {
    const void *dout;
    const float *ds_out;
    void *dq, *dk, *dv;
    float *dla, *ds0;
};
hipError_t launch_head_decay_bwd(const HeadDecayCall &c, const HeadDecayGrads &g, void *workspace,
                                 hipStream_t stream);
hipError_t launch_head_decay_step(const void *q, const void *k, const void *v, const float *a,
                                  bool a_fixed, float *state, void *o, int B, int H, int Hk, int dk,
                                  int dv, bool bf16, hipStream_t stream);

// Root-mean-square norm. Types of the rows: x and y (and dy) `x_bf16`, residual and h (and dh, dx) `h_bf16`.
struct NormCall {
    const void *x, *residual;  // residual NULL: h is x and is not written
    const float *weight;
    void *h;
    int rows, D;
    bool x_bf16, h_bf16;
    float eps;
};
hipError_t launch_rms_norm(const NormCall &c, void *y, float *rstd, hipStream_t stream);
// fmt: 0 e4m3, 1 int8. group: 0 for one scale a row, else 128 columns a scale.
hipError_t launch_rms_norm_8bit(const NormCall &c, void *y8, float *scale, int fmt, int group,
                                hipStream_t stream);
size_t rms_norm_bwd_workspace_bytes(int rows, int D);
hipError_t launch_rms_norm_bwd(const void *dy, const void *h, const float *weight, const float *rstd,
                               const void *dh, void *dx, float *dweight, int rows, int D, bool y_bf16,
                               bool h_bf16, void *workspace, hipStream_t stream);

// y [M, N] = x [M, K] W^T with W [N, K] from 4-bit values, scale and zero [N, K / group].
hipError_t launch_matvec_q4(const void *x, const void *w, const void *scale, const void *zero, void *y,
                            int M, int N, int K, int group, bool bf16, bool scale_bf16,
                            hipStream_t stream);

}  // namespace muir
