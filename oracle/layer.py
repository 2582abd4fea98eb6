"""Plain 64-bit forms of the layer operators (torch on the CPU, token by token): linear attention with one decay
per head, the root-mean-square norm, products with 4-bit weights. Independent of the HIP kernels."""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else x.detach().double().cpu()


def _prepared(q, k, v, a, s0, lens, *more):
    """Inputs in 64 bits, key heads repeated, tokens behind a sequence's end made neutral (k = v = 0, a = 1)."""
    B, T, H = v.shape[:3]
    rep = H // q.shape[2]
    a = _f64(a).expand(B, T, H)
    end = torch.full((B,), T) if lens is None else lens.cpu().long().clamp(0, T)
    live = torch.arange(T)[None] < end[:, None]
    m = live[:, :, None, None]
    q, k = (torch.where(m, _f64(x).repeat_interleave(rep, 2), 0.0) for x in (q, k))
    v = torch.where(m, _f64(v), 0.0)
    s0 = torch.zeros(B, H, q.shape[-1], v.shape[-1], dtype=torch.float64) if s0 is None else _f64(s0)
    more = [torch.where(m, _f64(x), 0.0) for x in more]
    return (q, k, v, torch.where(live[..., None], a, 1.0), s0, live, rep, *more)


def head_decay_forward(q, k, v, a, s0=None, lens=None):
    """o [B,T,H,dv] and the final state, of S <- a S + k v^T, o = S^T q."""
    q, k, v, a, S, live, _ = _prepared(q, k, v, a, s0, lens)
    o = torch.zeros_like(v)
    for t in range(v.shape[1]):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = (q[:, t, :, :, None] * S).sum(2)
    return o, S


def head_decay_backward(q, k, v, a, do, s0=None, ds=None, lens=None):
    """Gradients {"q", "k", "v", "la", "s0"} by the adjoint A of each token's state, and "edge": <S, A> before the
    adjoint takes in the token itself. The decay's is a_t <S_{t-1}, A_t>."""
    fixed = a.dim() == 1
    q, k, v, a, S, live, rep, do = _prepared(q, k, v, a, s0, lens, do)
    B, T, H = v.shape[:3]
    states = [S]
    for t in range(T):
        states.append(a[:, t, :, None, None] * states[-1] + k[:, t, :, :, None] * v[:, t, :, None, :])
    A = torch.zeros_like(S) if ds is None else _f64(ds).clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    la, edge = torch.zeros(B, T, H, dtype=torch.float64), torch.zeros(B, T, H, dtype=torch.float64)
    for t in reversed(range(T)):
        edge[:, t] = (states[t + 1] * A).sum((-1, -2))
        A = A + q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = (states[t + 1] * do[:, t, :, None, :]).sum(-1)
        dk[:, t] = (A * v[:, t, :, None, :]).sum(-1)
        dv[:, t] = (A * k[:, t, :, :, None]).sum(-2)
        A = a[:, t, :, None, None] * A
        la[:, t] = (states[t] * A).sum((-1, -2))
    m = live[:, :, None, None]
    shared = lambda x: torch.where(m, x, 0.0).unflatten(2, (H // rep, rep)).sum(3)  # noqa: E731
    la = torch.where(live[..., None], la, 0.0)
    return {"q": shared(dq), "k": shared(dk), "v": torch.where(m, dv, 0.0), "la": la.sum((0, 1)) if fixed else la,
            "s0": A, "edge": edge, "qh": dq, "kh": dk}


def rms_norm(x, weight, residual=None, eps=1e-6):
    """(y, h, rstd); h is rounded to the residual's type, as the operator's definition says."""
    h = _f64(x) if residual is None else (_f64(x) + _f64(residual)).to(residual.dtype).double()
    rstd = (h.square().mean(-1) + eps) ** -0.5
    return h * rstd[..., None] * _f64(weight), h, rstd


def rms_norm_backward(dy, h, weight, eps=1e-6, dh=None):
    """(dx, dweight) by differentiating the definition."""
    h64, w64 = _f64(h).clone().requires_grad_(), _f64(weight).clone().requires_grad_()
    y = h64 * (h64.square().mean(-1, keepdim=True) + eps) ** -0.5 * w64
    dx, dw = torch.autograd.grad(y, (h64, w64), _f64(dy))
    return (dx if dh is None else dx + _f64(dh)), dw


def q4_weights(w, scale, zero, group):
    """[N, K] in 64 bits."""
    w = w.cpu()
    n = torch.stack([w & 15, w >> 4], -1).flatten(1).double()
    z = 8.0 if zero is None else _f64(zero).repeat_interleave(group, 1)
    return (n - z) * _f64(scale).repeat_interleave(group, 1)
