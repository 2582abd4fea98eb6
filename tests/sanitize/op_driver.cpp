// Drives the layer operators' C entry points with stand-in launchers (no GPU): valid calls launch, every documented
// error returns its status without a launch, extreme sizes neither overflow nor launch.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "muir.h"
#include "op_kernels.hpp"

static int g_count = 0;
static hipError_t g_status = hipSuccess;

namespace muir {
static hipError_t launched() {
    ++g_count;
    return g_status;
}
hipError_t launch_head_decay_fwd(const HeadDecayCall &, void *, float *, void *, hipStream_t) { return launched(); }
hipError_t launch_head_decay_bwd(const HeadDecayCall &, const HeadDecayGrads &, void *, hipStream_t) { return launched(); }
hipError_t launch_head_decay_step(const void *, const void *, const void *, const float *, bool, float *, void *, int, int,
                                  int, int, int, bool, hipStream_t) {
    return launched();
}
hipError_t launch_rms_norm(const NormCall &, void *, float *, hipStream_t) { return launched(); }
hipError_t launch_rms_norm_8bit(const NormCall &, void *, float *, int, int, hipStream_t) { return launched(); }
hipError_t launch_rms_norm_bwd(const void *, const void *, const float *, const float *, const void *, void *, float *, int,
                               int, bool, bool, void *, hipStream_t) {
    return launched();
}
hipError_t launch_matvec_q4(const void *, const void *, const void *, const void *, void *, int, int, int, int, bool, bool,
                            hipStream_t) {
    return launched();
}
}  // namespace muir

static int failures = 0;
static void expect(int got, int want, int launches, const char *what) {
    if (got != want || g_count != launches) {
        ++failures;
        printf("%s: status %d, wanted %d; %d launches, wanted %d (%s)\n", what, got, want, g_count, launches, muir_last_error());
    }
    g_count = 0;
}

template <typename T> static T *at(int i) { return reinterpret_cast<T *>((uintptr_t(1) << 40) + i * (uintptr_t(1) << 36)); }

int main() {
    typedef const float cf;
    void *ws = at<void>(30);
    const size_t big = size_t(1) << 35;
    auto fwd = [&](int B, int T, int H, int Hk, int dk, int dv, const void *q, void *o, cf *s0, float *so) {
        return muir_chunk_fwd_head_decay(q, at<void>(1), at<void>(2), at<float>(3), s0, at<int>(5), o, so, B, T, H, Hk, dk, dv,
                                         1, MUIR_BF16, ws, big, nullptr);
    };
    expect(fwd(2, 100, 4, 2, 64, 128, at<void>(0), at<void>(6), nullptr, at<float>(7)), 0, 1, "forward");
    expect(fwd(2, 100, 4, 2, 64, 128, at<void>(0), at<void>(6), at<float>(7), at<float>(7)), 0, 1, "forward in place");
    expect(fwd(1, 0, 4, 2, 64, 128, nullptr, nullptr, nullptr, at<float>(7)), 0, 1, "no tokens");
    expect(fwd(1, 0, 4, 2, 64, 128, nullptr, nullptr, nullptr, nullptr), 0, 0, "nothing to do");
    expect(fwd(INT_MAX, INT_MAX, INT_MAX, 1, 64, 64, at<void>(0), at<void>(6), nullptr, nullptr), 3, 0, "huge");
    expect(fwd(1, INT_MAX, 1, 1, 64, 64, at<void>(0), at<void>(6), nullptr, nullptr), 3, 0, "long");
    expect(fwd(1, 100, 4, 3, 64, 64, at<void>(0), at<void>(6), nullptr, nullptr), 2, 0, "heads");
    expect(fwd(1, 100, 4, 2, 64, 64, nullptr, at<void>(6), nullptr, nullptr), 1, 0, "null");
    expect(fwd(1, 100, 4, 2, 64, 64, at<void>(0), at<void>(1), nullptr, nullptr), 5, 0, "alias");
    auto bwd = [&](int B, int T, int H, int per, float *dla) {
        return muir_chunk_bwd_head_decay(at<void>(0), at<void>(1), at<void>(2), at<float>(3), nullptr, nullptr, at<void>(6),
                                         nullptr, at<void>(8), at<void>(9), at<void>(10), dla, nullptr, B, T, H, H, 128, 64, per,
                                         MUIR_F32, ws, big, nullptr);
    };
    expect(bwd(2, 100, 4, 1, at<float>(11)), 0, 1, "backward");
    expect(bwd(1, 0, 4, 0, at<float>(11)), 0, 1, "backward of nothing");
    expect(bwd(1, 0, 4, 0, nullptr), 1, 0, "fixed decay without its gradient");
    expect(bwd(INT_MAX, INT_MAX, INT_MAX, 1, at<float>(11)), 3, 0, "huge backward");
    for (int T : {0, 1, 63, 64, 65, 100000, INT_MAX})
        for (int B : {1, 7, 4096, INT_MAX}) {
            muir_chunk_fwd_head_decay_workspace_size(B, T, 16, 4, 128, 128, MUIR_BF16);
            muir_chunk_bwd_head_decay_workspace_size(B, T, 16, 4, 128, 128, MUIR_F32);
            muir_rms_norm_bwd_workspace_size(T, 16384);
        }
    auto step = [&](int B, int H, float *state) {
        return muir_decode_step_head_decay(at<void>(0), at<void>(1), at<void>(2), at<float>(3), state, at<void>(5), B, H, 1, 64,
                                           64, 0, MUIR_BF16, nullptr);
    };
    expect(step(3, 4, at<float>(4)), 0, 1, "step");
    expect(step(INT_MAX, INT_MAX, at<float>(4)), 3, 0, "huge step");
    expect(step(3, 4, nullptr), 1, 0, "step without a state");
    auto norm = [&](int rows, int D, const void *res, void *h) {
        return muir_rms_norm(at<void>(0), res, at<float>(2), h, at<void>(4), nullptr, rows, D, 1e-6f, MUIR_BF16, MUIR_F32, nullptr);
    };
    expect(norm(5, 64, at<void>(1), at<void>(1)), 0, 1, "norm in place");
    expect(norm(5, 64, nullptr, nullptr), 0, 1, "norm without a residual");
    expect(norm(0, 64, nullptr, nullptr), 0, 0, "no rows");
    expect(norm(INT_MAX, 64, nullptr, nullptr), 3, 0, "too many rows");
    expect(norm(5, INT_MAX, nullptr, nullptr), 3, 0, "too long rows");
    expect(norm(5, 64, at<void>(1), nullptr), 1, 0, "residual without h");
    auto norm8 = [&](int rows, int D, int group) {
        return muir_rms_norm_8bit(at<void>(0), nullptr, at<float>(2), nullptr, at<void>(4), at<float>(5), rows, D, 0.f, MUIR_INT8,
                                  group, MUIR_F32, MUIR_F32, nullptr);
    };
    expect(norm8(5, 256, 128), 0, 1, "8 bits");
    expect(norm8(0, 256, 0), 0, 0, "8 bits of no rows");
    expect(norm8(-1, 256, 128), 2, 0, "negative rows");
    expect(norm8(5, INT_MIN, 128), 2, 0, "negative columns");
    auto normb = [&](int rows) {
        return muir_rms_norm_bwd(at<void>(0), at<void>(1), at<float>(2), at<float>(3), at<void>(4), at<void>(4), at<float>(6), rows,
                                 64, MUIR_BF16, MUIR_BF16, ws, big, nullptr);
    };
    expect(normb(9), 0, 1, "norm backward in place");
    expect(normb(0), 0, 1, "norm backward of nothing");
    auto q4 = [&](int M, int N, int K, int group) {
        return muir_matvec_q4(at<void>(0), at<void>(1), at<void>(2), at<void>(3), at<void>(4), M, N, K, group, MUIR_BF16, MUIR_F32,
                              nullptr);
    };
    expect(q4(3, 100, 256, 64), 0, 1, "q4");
    expect(q4(0, 100, 256, 64), 0, 0, "q4 of no rows");
    expect(q4(1, INT_MAX, INT_MAX, 128), 2, 0, "q4 odd K");
    expect(q4(1, INT_MAX, 1 << 30, 128), 3, 0, "huge q4");
    g_status = hipErrorLaunchFailure;
    expect(q4(3, 100, 256, 64), 6, 1, "launch failure");
    expect(step(3, 4, at<float>(4)), 6, 1, "launch failure of the step");
    printf("%d failures\n", failures);
    return failures != 0;
}
