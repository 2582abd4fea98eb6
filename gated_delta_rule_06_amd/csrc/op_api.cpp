// C ABI of the layer operators around the chunk forward: argument validation, workspace sizes, dispatch.
// Every check runs on the host before anything is launched.
#include <math.h>

#include "muir.h"
#include "op_checks.hpp"
#include "op_kernels.hpp"

namespace {

using namespace muir;

// Largest B * H and B * (T + 64) * H: one workgroup or thread each has to fit a launch. Largest H: a chunk's 64 rows
// are addressed with 32-bit offsets.
constexpr long long kMaxHeads = 1 << 21, kMaxTokenHeads = 1LL << 31;
constexpr int kMaxH = 1 << 15;

bool head_sizes_ok(int B, int T, int H, int Hk, int dk, int dv, muir_dtype_t qkv) {
    return B >= 1 && T >= 0 && H >= 1 && Hk >= 1 && H % Hk == 0 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128) &&
           known(qkv) && H <= kMaxH && static_cast<long long>(B) * H <= kMaxHeads &&
           static_cast<long long>(B) * H <= kMaxTokenHeads / (static_cast<long long>(T) + 64);
}

muir_status_t check_head_sizes(const char *fn, int B, int T, int H, int Hk, int dk, int dv, muir_dtype_t qkv) {
    if (B < 1 || T < 0 || H < 1 || Hk < 1)
        return fail(MUIR_ERR_SHAPE, "%s: need B >= 1, T >= 0, H >= 1, Hk >= 1 (got B=%d T=%d H=%d Hk=%d)", fn, B, T, H, Hk);
    if (H % Hk != 0) return fail(MUIR_ERR_SHAPE, "%s: H=%d must be a multiple of Hk=%d", fn, H, Hk);
    if (!known(qkv)) return fail(MUIR_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, static_cast<int>(qkv));
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
        return fail(MUIR_ERR_UNSUPPORTED, "%s: dk and dv must be 64 or 128 (got %d, %d)", fn, dk, dv);
    if (!head_sizes_ok(B, T, H, Hk, dk, dv, qkv))
        return fail(MUIR_ERR_UNSUPPORTED, "%s: H above 2^15, B * H above 2^21 or B * (T + 64) * H above 2^31; split the call", fn);
    return MUIR_OK;
}

struct NormTypes {
    const char *fn;
    muir_dtype_t x, h;
};

muir_status_t check_norm(const NormTypes &t, int rows, int D) {
    if (rows < 0 || D < 1) return fail(MUIR_ERR_SHAPE, "%s: need rows >= 0 and D >= 1 (got %d, %d)", t.fn, rows, D);
    if (!known(t.x) || !known(t.h))
        return fail(MUIR_ERR_UNSUPPORTED, "%s: unknown dtype %d or %d", t.fn, static_cast<int>(t.x), static_cast<int>(t.h));
    if (t.x == MUIR_F32 && t.h == MUIR_BF16)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: a bfloat16 residual needs bfloat16 rows", t.fn);
    if (D % 8 != 0 || D > 16384)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: D must be a multiple of 8 up to 16384 (got %d)", t.fn, D);
    if (rows > (1 << 23)) return fail(MUIR_ERR_UNSUPPORTED, "%s: more than 2^23 rows; split the call", t.fn);
    return MUIR_OK;
}

// Checks of the two forward forms; `out` is y or y8.
muir_status_t check_norm_fwd(const NormTypes &t, const void *x, const void *residual, const float *weight, const void *h,
                             const void *out, const float *stat, int rows, int D, float eps, size_t out_size, size_t stats,
                             bool stat_required) {
    const muir_status_t st = check_norm(t, rows, D);
    if (st != MUIR_OK) return st;
    if (!(eps >= 0.f) || isinf(eps)) return fail(MUIR_ERR_SHAPE, "%s: eps must be finite and >= 0", t.fn);
    if ((residual == nullptr) != (h == nullptr) && rows > 0)
        return fail(MUIR_ERR_NULL, "%s: residual and h come together", t.fn);
    if (!weight || (rows > 0 && (!x || !out || (stat_required && !stat))))
        return fail(MUIR_ERR_NULL, "%s: a required buffer is missing", t.fn);
    const size_t n = static_cast<size_t>(rows) * D;
    return check_buffers(t.fn,
                         {buf("x", x, n * size_of(t.x)), buf("residual", residual, n * size_of(t.h)),
                          buf("weight", weight, static_cast<size_t>(D) * 4)},
                         {buf("h", h, n * size_of(t.h), 16, "residual"), buf("y", out, n * out_size),
                          buf(stat_required ? "scale" : "rstd", stat, stats * 4, 4)});
}

}  // namespace

extern "C" {

size_t muir_chunk_fwd_head_decay_workspace_size(int B, int T, int H, int Hk, int dk, int dv, muir_dtype_t qkv) {
    if (!head_sizes_ok(B, T, H, Hk, dk, dv, qkv)) return 0;
    return head_decay_fwd_workspace_bytes(B, T, H, dk, dv, qkv == MUIR_BF16);
}

muir_status_t muir_chunk_fwd_head_decay(const void *q, const void *k, const void *v, const float *a, const float *s0,
                                        const int *lens, void *o, float *s_out, int B, int T, int H, int Hk, int dk,
                                        int dv, int a_per_token, muir_dtype_t qkv, void *workspace,
                                        size_t workspace_bytes, muir_stream_t stream) {
    const char *fn = "chunk_fwd_head_decay";
    muir_status_t st = check_head_sizes(fn, B, T, H, Hk, dk, dv, qkv);
    if (st != MUIR_OK) return st;
    if (T > 0 && (!q || !k || !v || !a || !o)) return fail(MUIR_ERR_NULL, "%s: q, k, v, a and o are required", fn);
    const size_t need = muir_chunk_fwd_head_decay_workspace_size(B, T, H, Hk, dk, dv, qkv), es = size_of(qkv);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != MUIR_OK) return st;
    const size_t bt = static_cast<size_t>(B) * T, state = static_cast<size_t>(B) * H * dk * dv * 4;
    st = check_buffers(fn,
                       {buf("q", q, bt * Hk * dk * es), buf("k", k, bt * Hk * dk * es), buf("v", v, bt * H * dv * es),
                        buf("a", a, (a_per_token ? bt : 1) * H * 4, 4), buf("lens", lens, static_cast<size_t>(B) * 4, 4),
                        buf("s0", s0, state)},
                       {buf("o", o, bt * H * dv * es), buf("s_out", s_out, state, 16, "s0"),
                        buf("workspace", workspace, need)});
    if (st != MUIR_OK) return st;
    if (T == 0 && !s_out) return ok();
    const HeadDecayCall c{q, k, v, a, !a_per_token, lens, s0, B, T, H, Hk, dk, dv, qkv == MUIR_BF16};
    return check_hip(launch_head_decay_fwd(c, o, s_out, workspace, static_cast<hipStream_t>(stream)), fn);
}

size_t muir_chunk_bwd_head_decay_workspace_size(int B, int T, int H, int Hk, int dk, int dv, muir_dtype_t qkv) {
    if (!head_sizes_ok(B, T, H, Hk, dk, dv, qkv)) return 0;
    return head_decay_bwd_workspace_bytes(B, T, H, Hk, dk, dv, qkv == MUIR_BF16);
}

muir_status_t muir_chunk_bwd_head_decay(const void *q, const void *k, const void *v, const float *a, const float *s0,
                                        const int *lens, const void *dout, const float *ds_out, void *dq, void *dk,
                                        void *dv, float *dla, float *ds0, int B, int T, int H, int Hk, int dk_, int dv_,
                                        int a_per_token, muir_dtype_t qkv, void *workspace, size_t workspace_bytes,
                                        muir_stream_t stream) {
    const char *fn = "chunk_bwd_head_decay";
    muir_status_t st = check_head_sizes(fn, B, T, H, Hk, dk_, dv_, qkv);
    if (st != MUIR_OK) return st;
    if (T > 0 && (!q || !k || !v || !a || !dout || !dq || !dk || !dv || !dla))
        return fail(MUIR_ERR_NULL, "%s: every input and gradient except s0, lens, ds_out and ds0 is required", fn);
    if (!a_per_token && !dla) return fail(MUIR_ERR_NULL, "%s: dla is required", fn);
    const size_t need = muir_chunk_bwd_head_decay_workspace_size(B, T, H, Hk, dk_, dv_, qkv), es = size_of(qkv);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != MUIR_OK) return st;
    const size_t bt = static_cast<size_t>(B) * T, state = static_cast<size_t>(B) * H * dk_ * dv_ * 4;
    const size_t nk = bt * Hk * dk_ * es, nv = bt * H * dv_ * es, na = (a_per_token ? bt : 1) * H * 4;
    st = check_buffers(fn,
                       {buf("q", q, nk), buf("k", k, nk), buf("v", v, nv), buf("a", a, na, 4),
                        buf("lens", lens, static_cast<size_t>(B) * 4, 4), buf("s0", s0, state), buf("dout", dout, nv),
                        buf("ds_out", ds_out, state)},
                       {buf("dq", dq, nk), buf("dk", dk, nk), buf("dv", dv, nv), buf("dla", dla, na, 4),
                        buf("ds0", ds0, state), buf("workspace", workspace, need)});
    if (st != MUIR_OK) return st;
    const HeadDecayCall c{q, k, v, a, !a_per_token, lens, s0, B, T, H, Hk, dk_, dv_, qkv == MUIR_BF16};
    const HeadDecayGrads g{dout, ds_out, dq, dk, dv, dla, ds0};
    return check_hip(launch_head_decay_bwd(c, g, workspace, static_cast<hipStream_t>(stream)), fn);
}

muir_status_t muir_decode_step_head_decay(const void *q, const void *k, const void *v, const float *a, float *state,
                                          void *o, int B, int H, int Hk, int dk, int dv, int a_per_token,
                                          muir_dtype_t qkv, muir_stream_t stream) {
    const char *fn = "decode_step_head_decay";
    muir_status_t st = check_head_sizes(fn, B, 1, H, Hk, dk, dv, qkv);
    if (st != MUIR_OK) return st;
    if (!q || !k || !v || !a || !state || !o) return fail(MUIR_ERR_NULL, "%s: a required buffer is missing", fn);
    const size_t es = size_of(qkv), nk = static_cast<size_t>(B) * Hk * dk * es, nv = static_cast<size_t>(B) * H * dv * es;
    st = check_buffers(fn,
                       {buf("q", q, nk), buf("k", k, nk), buf("v", v, nv),
                        buf("a", a, static_cast<size_t>(a_per_token ? B : 1) * H * 4, 4)},
                       {buf("state", state, static_cast<size_t>(B) * H * dk * dv * 4), buf("o", o, nv)});
    if (st != MUIR_OK) return st;
    return check_hip(launch_head_decay_step(q, k, v, a, !a_per_token, state, o, B, H, Hk, dk, dv, qkv == MUIR_BF16,
                                            static_cast<hipStream_t>(stream)),
                     fn);
}

muir_status_t muir_rms_norm(const void *x, const void *residual, const float *weight, void *h, void *y, float *rstd,
                            int rows, int D, float eps, muir_dtype_t x_type, muir_dtype_t h_type, muir_stream_t stream) {
    const NormTypes t{"rms_norm", x_type, residual ? h_type : x_type};
    const muir_status_t st = check_norm_fwd(t, x, residual, weight, h, y, rstd, rows, D, eps, size_of(x_type),
                                            static_cast<size_t>(rows), false);
    if (st != MUIR_OK) return st;
    if (rows == 0) return ok();
    const NormCall c{x, residual, weight, h, rows, D, t.x == MUIR_BF16, t.h == MUIR_BF16, eps};
    return check_hip(launch_rms_norm(c, y, rstd, static_cast<hipStream_t>(stream)), t.fn);
}

muir_status_t muir_rms_norm_8bit(const void *x, const void *residual, const float *weight, void *h, void *y8,
                                 float *scale, int rows, int D, float eps, muir_format_t format, int group,
                                 muir_dtype_t x_type, muir_dtype_t h_type, muir_stream_t stream) {
    const NormTypes t{"rms_norm_8bit", x_type, residual ? h_type : x_type};
    if (format != MUIR_E4M3 && format != MUIR_INT8)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: unknown format %d", t.fn, static_cast<int>(format));
    if (group != 0 && group != 128) return fail(MUIR_ERR_UNSUPPORTED, "%s: group must be 0 or 128 (got %d)", t.fn, group);
    if (group != 0 && D > 0 && D % group != 0)
        return fail(MUIR_ERR_SHAPE, "%s: D=%d must be a multiple of the group, %d", t.fn, D, group);
    const size_t scales = static_cast<size_t>(rows < 0 ? 0 : rows) * (group ? D / group : 1);
    const muir_status_t st = check_norm_fwd(t, x, residual, weight, h, y8, scale, rows, D, eps, 1, scales, true);
    if (st != MUIR_OK) return st;
    if (rows == 0) return ok();
    const NormCall c{x, residual, weight, h, rows, D, t.x == MUIR_BF16, t.h == MUIR_BF16, eps};
    return check_hip(launch_rms_norm_8bit(c, y8, scale, format == MUIR_E4M3 ? 0 : 1, group,
                                          static_cast<hipStream_t>(stream)),
                     t.fn);
}

size_t muir_rms_norm_bwd_workspace_size(int rows, int D) {
    if (rows < 0 || rows > (1 << 23) || D < 1 || D % 8 != 0 || D > 16384) return 0;
    return rms_norm_bwd_workspace_bytes(rows, D);
}

muir_status_t muir_rms_norm_bwd(const void *dy, const void *h, const float *weight, const float *rstd, const void *dh,
                                void *dx, float *dweight, int rows, int D, muir_dtype_t y_type, muir_dtype_t h_type,
                                void *workspace, size_t workspace_bytes, muir_stream_t stream) {
    const NormTypes t{"rms_norm_bwd", y_type, h_type};
    muir_status_t st = check_norm(t, rows, D);
    if (st != MUIR_OK) return st;
    if (!weight || !dweight || (rows > 0 && (!dy || !h || !rstd || !dx)))
        return fail(MUIR_ERR_NULL, "%s: a required buffer is missing", t.fn);
    const size_t need = muir_rms_norm_bwd_workspace_size(rows, D), n = static_cast<size_t>(rows) * D;
    st = check_workspace(t.fn, workspace, workspace_bytes, need);
    if (st != MUIR_OK) return st;
    st = check_buffers(t.fn,
                       {buf("dy", dy, n * size_of(y_type)), buf("h", h, n * size_of(h_type)),
                        buf("weight", weight, static_cast<size_t>(D) * 4), buf("rstd", rstd, static_cast<size_t>(rows) * 4, 4),
                        buf("dh", dh, n * size_of(h_type))},
                       {buf("dx", dx, n * size_of(h_type), 16, "dh"), buf("dweight", dweight, static_cast<size_t>(D) * 4, 4),
                        buf("workspace", workspace, need)});
    if (st != MUIR_OK) return st;
    return check_hip(launch_rms_norm_bwd(dy, h, weight, rstd, dh, dx, dweight, rows, D, y_type == MUIR_BF16,
                                         h_type == MUIR_BF16, workspace, static_cast<hipStream_t>(stream)),
                     t.fn);
}

muir_status_t muir_matvec_q4(const void *x, const void *w, const void *scale, const void *zero, void *y, int M, int N,
                             int K, int group, muir_dtype_t x_type, muir_dtype_t scale_type, muir_stream_t stream) {
    const char *fn = "matvec_q4";
    if (M < 0 || N < 1 || K < 1) return fail(MUIR_ERR_SHAPE, "%s: need M >= 0, N >= 1, K >= 1 (got %d, %d, %d)", fn, M, N, K);
    if (!known(x_type) || !known(scale_type))
        return fail(MUIR_ERR_UNSUPPORTED, "%s: unknown dtype %d or %d", fn, static_cast<int>(x_type), static_cast<int>(scale_type));
    if (group != 32 && group != 64 && group != 128)
        return fail(MUIR_ERR_UNSUPPORTED, "%s: group must be 32, 64 or 128 (got %d)", fn, group);
    if (K % group != 0) return fail(MUIR_ERR_SHAPE, "%s: K=%d must be a multiple of the group, %d", fn, K, group);
    if (M > 64) return fail(MUIR_ERR_UNSUPPORTED, "%s: at most 64 rows (got %d): more are a matrix product", fn, M);
    if (N > (1 << 26) || K > (1 << 26)) return fail(MUIR_ERR_UNSUPPORTED, "%s: N and K up to 2^26", fn);
    if (!w || !scale || (M > 0 && (!x || !y))) return fail(MUIR_ERR_NULL, "%s: x, w, scale and y are required", fn);
    const size_t nk = static_cast<size_t>(N) * K, ns = nk / group * size_of(scale_type), ss = size_of(scale_type);
    const muir_status_t st = check_buffers(
        fn,
        {buf("x", x, static_cast<size_t>(M) * K * size_of(x_type)), buf("w", w, nk / 2), buf("scale", scale, ns, ss),
         buf("zero", zero, ns, ss)},
        {buf("y", y, static_cast<size_t>(M) * N * size_of(x_type), size_of(x_type))});
    if (st != MUIR_OK) return st;
    if (M == 0) return ok();
    return check_hip(launch_matvec_q4(x, w, scale, zero, y, M, N, K, group, x_type == MUIR_BF16, scale_type == MUIR_BF16,
                                      static_cast<hipStream_t>(stream)),
                     fn);
}

}  // extern "C"
