// Internal launchers of causal softmax attention and its paged cache. Arguments are validated by the C ABI layer
// (attention_api.cpp) before any of these is called; each returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace muir {

// Rows q [N, H, d], k, v [N, Hk, d] of S sequences: offsets [S + 1] or NULL (N / S rows each), lens [S] or NULL.
struct AttentionCall {
    const void *q, *k, *v;
    const int *offsets, *lens;
    int N, S, H, Hk, d, window;  // window 0 (no limit) or below N
    float scale;
    bool bf16;
};
// Workgroups of a prompt kernel have 128 rows of one head, or 32 (split) where 128 would make too few of them, and in float32's backward.
inline long long attention_blocks(int N, int S, int rows) { return static_cast<long long>(N) / rows + S + 1; }
bool attention_split(int N, int S, int heads, int d, int window);
bool attention_far(int N, int S, int H, int Hk, int window);
// Whether a window is so short that most queries see as many keys as it has.
bool attention_even(int N, int S, int window);
bool attention_by_place(const int *offsets, int N, int S, int window);
hipError_t launch_attention_fwd(const AttentionCall &c, void *o, float *lse, hipStream_t stream);

size_t attention_bwd_workspace_bytes(int N, int H);
struct AttentionGrads {
    const void *o, *dout;
    const float *lse;
    void *dq, *dk, *dv;
};
hipError_t launch_attention_bwd(const AttentionCall &c, const AttentionGrads &g, void *workspace, hipStream_t stream);

// Paged cache: k_cache, v_cache [pages, Hk, page, d], table [B, width].
struct CacheCall {
    void *k_cache, *v_cache;
    const int *table;
    int pages, page, width, Hk, d;
    bool bf16;
};
hipError_t launch_cache_append(const CacheCall &c, const void *k, const void *v, const int *offsets, const int *lens,
                               const int *start, int N, int S, hipStream_t stream);

// Parts that a sequence's keys are split into, side by side (1: none, and no workspace).
int attention_step_parts(int B, int H, int Hk, int d, int capacity, bool bf16);
size_t attention_step_workspace_bytes(int B, int H, int Hk, int d, int capacity, bool bf16);
hipError_t launch_attention_step(const CacheCall &c, const void *q, const void *k, const void *v, const int *lens, void *o,
                                 int B, int H, int window, float scale, void *workspace, hipStream_t stream);

}  // namespace muir
