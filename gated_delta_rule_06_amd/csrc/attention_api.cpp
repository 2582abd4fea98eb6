// C ABI of causal softmax attention and its paged cache: argument validation, workspace sizes, dispatch. Every check runs on
// the host before anything is launched.
#include <math.h>

#include "attention_kernels.hpp"
#include "attention_layout.hpp"
#include "muir.h"
#include "op_checks.hpp"

namespace {

using namespace muir;

// Workgroups of a launch, which has 256 threads each (a step 512) and less than 2^32 in all.
constexpr long long kMaxBlocks = (1 << 24) - 1, kMaxStepBlocks = (1 << 23) - 1;
constexpr float kMinScale = 0x1p-64f;  // lse over the scale is still a float32
constexpr int kMaxH = 1 << 15;     // 64 rows are addressed with 32-bit offsets
constexpr int kMaxRows = 1 << 30;  // places of rows, and a few blocks behind them, are ints

muir_status_t check_heads(const char *fn, int H, int Hk, int d, muir_dtype_t type) {
    if (H < 1 || Hk < 1) return fail(MUIR_ERR_SHAPE, "%s: need H >= 1 and Hk >= 1 (got %d, %d)", fn, H, Hk);
    if (H % Hk != 0) return fail(MUIR_ERR_SHAPE, "%s: H=%d must be a multiple of Hk=%d", fn, H, Hk);
    if (!known(type)) return fail(MUIR_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, static_cast<int>(type));
    if (d != 64 && d != 128) return fail(MUIR_ERR_UNSUPPORTED, "%s: d must be 64 or 128 (got %d)", fn, d);
    if (H > kMaxH) return fail(MUIR_ERR_UNSUPPORTED, "%s: H above 2^15", fn);
    return MUIR_OK;
}

muir_status_t check_rows(const char *fn, int N, int S, const int *offsets, int per_block, int heads) {
    if (N < 0 || S < 1) return fail(MUIR_ERR_SHAPE, "%s: need N >= 0 and S >= 1 (got %d, %d)", fn, N, S);
    if (!offsets && N % S != 0) return fail(MUIR_ERR_SHAPE, "%s: without offsets N=%d must be a multiple of S=%d", fn, N, S);
    if (N > kMaxRows) return fail(MUIR_ERR_UNSUPPORTED, "%s: N above 2^30", fn);
    if (attention_blocks(N, S, per_block) * heads > kMaxBlocks)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: too many rows, sequences and heads for a call; split it", fn);
    return MUIR_OK;
}

muir_status_t check_scores(const char *fn, int window, float scale) {
    if (window < 0) return fail(MUIR_ERR_SHAPE, "%s: window must be >= 0 (got %d)", fn, window);
    if (!(scale >= kMinScale) || isinf(scale * at::LOG2E))
        return fail(MUIR_ERR_SHAPE, "%s: scale must be at least 2^-64, and times log2(e) finite", fn);
    return MUIR_OK;
}

muir_status_t check_cache(const char *fn, int pages, int page, int width) {
    if (pages < 1 || width < 1) return fail(MUIR_ERR_SHAPE, "%s: need pages >= 1 and width >= 1 (got %d, %d)", fn, pages, width);
    if (page < 16 || page > 256 || (page & (page - 1)) != 0)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: page must be 16, 32, 64, 128 or 256 (got %d)", fn, page);
    if (static_cast<long long>(width) * page > (1 << 30)) return fail(MUIR_ERR_UNSUPPORTED, "%s: more than 2^30 tokens a sequence", fn);
    return MUIR_OK;
}

size_t offset_bytes(int S) { return (static_cast<size_t>(S) + 1) * 4; }

bool step_sizes_ok(int B, int H, int Hk, int d, int page, int width, muir_dtype_t type) {
    return B >= 1 && H >= 1 && Hk >= 1 && H % Hk == 0 && H <= kMaxH && (d == 64 || d == 128) && known(type) && width >= 1 && page >= 16 &&
           page <= 256 && (page & (page - 1)) == 0 && static_cast<long long>(width) * page <= (1 << 30) &&
           static_cast<long long>(B) * Hk * ((H / Hk + 15) / 16) <= kMaxStepBlocks;
}

}  // namespace

extern "C" {

muir_status_t muir_attention_fwd(const void *q, const void *k, const void *v, const int *offsets, const int *lens, void *o, float *lse,
                                 int N, int S, int H, int Hk, int d, int window, float scale, muir_dtype_t qkv, muir_stream_t stream) {
    const char *fn = "attention_fwd";
    muir_status_t st = check_heads(fn, H, Hk, d, qkv);
    if (st == MUIR_OK) st = check_rows(fn, N, S, offsets, qkv == MUIR_BF16 ? 128 : 32, H);
    if (st == MUIR_OK) st = check_scores(fn, window, scale);
    if (st != MUIR_OK) return st;
    if (N == 0) return ok();
    if (!q || !k || !v || !o) return fail(MUIR_ERR_NULL, "%s: q, k, v and o are required", fn);
    const size_t n = static_cast<size_t>(N), nq = n * H * d * size_of(qkv), nk = n * Hk * d * size_of(qkv);
    st = check_buffers(fn,
                       {buf("q", q, nq), buf("k", k, nk), buf("v", v, nk), buf("offsets", offsets, offset_bytes(S), 4),
                        buf("lens", lens, static_cast<size_t>(S) * 4, 4)},
                       {buf("o", o, nq), buf("lse", lse, n * H * 4, 4)});
    if (st != MUIR_OK) return st;
    const AttentionCall c{q, k, v, offsets, lens, N, S, H, Hk, d, window < N ? window : 0, scale, qkv == MUIR_BF16};
    return check_hip(launch_attention_fwd(c, o, lse, static_cast<hipStream_t>(stream)), fn);
}

size_t muir_attention_bwd_workspace_size(int N, int S, int H, int Hk, int d, muir_dtype_t qkv) {
    if (N < 0 || S < 1 || H < 1 || Hk < 1 || H % Hk != 0 || H > kMaxH || (d != 64 && d != 128) || !known(qkv) ||
        N > kMaxRows || attention_blocks(N, S, qkv == MUIR_BF16 ? 128 : 32) * H > kMaxBlocks)
        return 0;
    return attention_bwd_workspace_bytes(N, H);
}

muir_status_t muir_attention_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse, const int *offsets,
                                 const int *lens, const void *dout, void *dq, void *dk, void *dv, int N, int S, int H, int Hk, int d,
                                 int window, float scale, muir_dtype_t qkv, void *workspace, size_t workspace_bytes,
                                 muir_stream_t stream) {
    const char *fn = "attention_bwd";
    muir_status_t st = check_heads(fn, H, Hk, d, qkv);
    if (st == MUIR_OK) st = check_rows(fn, N, S, offsets, qkv == MUIR_BF16 ? 128 : 32, H);
    if (st == MUIR_OK) st = check_scores(fn, window, scale);
    if (st != MUIR_OK) return st;
    if (N == 0) return ok();
    if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv)
        return fail(MUIR_ERR_NULL, "%s: every input and gradient except offsets and lens is required", fn);
    const size_t n = static_cast<size_t>(N), nq = n * H * d * size_of(qkv), nk = n * Hk * d * size_of(qkv);
    const size_t need = attention_bwd_workspace_bytes(N, H);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != MUIR_OK) return st;
    st = check_buffers(fn,
                       {buf("q", q, nq), buf("k", k, nk), buf("v", v, nk), buf("o", o, nq), buf("lse", lse, n * H * 4, 4),
                        buf("offsets", offsets, offset_bytes(S), 4), buf("lens", lens, static_cast<size_t>(S) * 4, 4), buf("dout", dout, nq)},
                       {buf("dq", dq, nq), buf("dk", dk, nk), buf("dv", dv, nk), buf("workspace", workspace, need)});
    if (st != MUIR_OK) return st;
    const AttentionCall c{q, k, v, offsets, lens, N, S, H, Hk, d, window < N ? window : 0, scale, qkv == MUIR_BF16};
    return check_hip(launch_attention_bwd(c, AttentionGrads{o, dout, lse, dq, dk, dv}, workspace, static_cast<hipStream_t>(stream)), fn);
}

muir_status_t muir_cache_append(const void *k, const void *v, void *k_cache, void *v_cache, const int *table, const int *offsets,
                                const int *lens, const int *start, int N, int S, int Hk, int d, int pages, int page, int width,
                                muir_dtype_t type, muir_stream_t stream) {
    const char *fn = "cache_append";
    muir_status_t st = check_heads(fn, Hk, Hk, d, type);
    if (st == MUIR_OK) st = check_rows(fn, N, S, offsets, 8, 1);
    if (st == MUIR_OK) st = check_cache(fn, pages, page, width);
    if (st != MUIR_OK) return st;
    if (N == 0) return ok();
    if (!k || !v || !k_cache || !v_cache || !table) return fail(MUIR_ERR_NULL, "%s: k, v, both caches and the table are required", fn);
    const size_t row = static_cast<size_t>(Hk) * d * size_of(type), n = static_cast<size_t>(N) * row;
    size_t all;
    if (!mul_size(all, {static_cast<size_t>(pages), static_cast<size_t>(page), row})) return fail(MUIR_ERR_UNSUPPORTED, "%s: sizes overflow", fn);
    st = check_buffers(fn,
                       {buf("k", k, n), buf("v", v, n), buf("table", table, static_cast<size_t>(S) * width * 4, 4),
                        buf("offsets", offsets, offset_bytes(S), 4), buf("lens", lens, static_cast<size_t>(S) * 4, 4),
                        buf("start", start, static_cast<size_t>(S) * 4, 4)},
                       {buf("k_cache", k_cache, all), buf("v_cache", v_cache, all)});
    if (st != MUIR_OK) return st;
    const CacheCall c{k_cache, v_cache, table, pages, page, width, Hk, d, type == MUIR_BF16};
    return check_hip(launch_cache_append(c, k, v, offsets, lens, start, N, S, static_cast<hipStream_t>(stream)), fn);
}

size_t muir_decode_step_attention_workspace_size(int B, int H, int Hk, int d, int page, int width, muir_dtype_t type) {
    return step_sizes_ok(B, H, Hk, d, page, width, type) ? attention_step_workspace_bytes(B, H, Hk, d, width * page, type == MUIR_BF16) : 0;
}

muir_status_t muir_decode_step_attention(const void *q, const void *k, const void *v, void *k_cache, void *v_cache, const int *table,
                                         const int *lens, void *o, int B, int H, int Hk, int d, int pages, int page, int width, int window,
                                         float scale, muir_dtype_t type, void *workspace, size_t workspace_bytes, muir_stream_t stream) {
    const char *fn = "decode_step_attention";
    if (B < 1) return fail(MUIR_ERR_SHAPE, "%s: need B >= 1 (got %d)", fn, B);
    muir_status_t st = check_heads(fn, H, Hk, d, type);
    if (st == MUIR_OK) st = check_scores(fn, window, scale);
    if (st == MUIR_OK) st = check_cache(fn, pages, page, width);
    if (st != MUIR_OK) return st;
    if (!step_sizes_ok(B, H, Hk, d, page, width, type)) return fail(MUIR_ERR_UNSUPPORTED, "%s: too many sequences and heads for a call", fn);
    if (!q || !k_cache || !v_cache || !table || !lens || !o) return fail(MUIR_ERR_NULL, "%s: a required buffer is missing", fn);
    if ((k == nullptr) != (v == nullptr)) return fail(MUIR_ERR_NULL, "%s: k and v come together", fn);
    const size_t es = size_of(type), nq = static_cast<size_t>(B) * H * d * es, nk = static_cast<size_t>(B) * Hk * d * es;
    const size_t need = muir_decode_step_attention_workspace_size(B, H, Hk, d, page, width, type);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != MUIR_OK) return st;
    size_t all;
    if (!mul_size(all, {static_cast<size_t>(pages), static_cast<size_t>(page), static_cast<size_t>(Hk) * d * es}))
        return fail(MUIR_ERR_UNSUPPORTED, "%s: sizes overflow", fn);
    st = check_buffers(fn,
                       {buf("q", q, nq), buf("k", k, nk), buf("v", v, nk), buf("table", table, static_cast<size_t>(B) * width * 4, 4),
                        buf("lens", lens, static_cast<size_t>(B) * 4, 4)},
                       {buf("k_cache", k_cache, all), buf("v_cache", v_cache, all), buf("o", o, nq), buf("workspace", workspace, need)});
    if (st != MUIR_OK) return st;
    const CacheCall c{k_cache, v_cache, table, pages, page, width, Hk, d, type == MUIR_BF16};
    return check_hip(launch_attention_step(c, q, k, v, lens, o, B, H, window, scale, workspace, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
