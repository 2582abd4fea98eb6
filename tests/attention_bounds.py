"""How far the attention kernels' outputs may be off, element by element, from the sizes of what they sum.

u is half a step of the type, finfo.eps / 2: 2^-8 for bfloat16 and 2^-24 for float32; w = 2^-24. Per row i:
- a score is a float32 sum of d products, so off by at most d w scale sum|q k|; its exponent is a product, a difference and an
  exponential, a few w of the exponent's size, which is at most the scores' size: e_i = (d + 8) w scale max_j sum|q_i k_j|.
- p_ij (numerator and denominator) is off by (2 e_i + n w) p_ij, n the number of its row's keys, and by u p_ij where it is rounded for a product.
- o_i sums p_ij v_j in float32 and is rounded once: r_i sum p|v| + u |o|, with r_i = u + 2 e_i + 2 n w (u itself only in bfloat16; in float32 a w more).
- ds_ij = p_ij (do_i . v_j - do_i . o_i): p's error times the difference, and p times the errors of both products: (d + 1) w |do|.|v|,
  and |do| . (error of o) + (d + 1) w |do|.|o|.
- dq, dk, dv sum those with k, q, do in float32 (n w more) and are rounded once.
- An exponential below 2^-126, the smallest normal float32, comes as zero, and so may a product of it: every p and ds is off by up to TINY = 2^-120
  beside the above (the differences that p is multiplied with are below 2^6 here), every sum of n of them by n TINY times its largest factor.
  Without this a key that every query all but ignores (p = e^-720 where scores differ by 720) would have to have a gradient of 1e-313."""
import torch

W = 2.0 ** -24
TINY = 2.0 ** -120


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _parts(q, k, v, lo, n, h, window, scale):
    from oracle import attention as oa
    f = lambda x: x.detach().double().cpu()  # noqa: E731
    rep = q.shape[1] // k.shape[1]
    Q, K, V = f(q[lo:lo + n, h]), f(k[lo:lo + n, h // rep]), f(v[lo:lo + n, h // rep])
    seen = oa.visible(n, window)
    p = torch.softmax(torch.where(seen, scale * (Q @ K.T), -torch.inf), 1)
    e = (q.shape[2] + 8) * W * scale * torch.where(seen, Q.abs() @ K.abs().T, 0.0).amax(1)
    return Q, K, V, p, e, f


def forward_bounds(q, k, v, where, window=0, scale=None):
    """(bound of o, bound of lse)."""
    N, H, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    u = half_step(q.dtype)
    bo, bl = torch.zeros(N, H, d, dtype=torch.float64), torch.zeros(N, H, dtype=torch.float64)
    for lo, n in where:
        for h in range(H if n else 0):
            Q, K, V, p, e, _ = _parts(q, k, v, lo, n, h, window, scale)
            r = (u + 2 * e + 2 * (n + 8) * W)[:, None]
            bo[lo:lo + n, h] = r * (p @ V.abs()) + u * (p @ V).abs() + n * TINY * V.abs().max()
            # A logarithm of a sum that is off by e_i + n w, and roundings of values up to the scores' size.
            bl[lo:lo + n, h] = 2 * e + 2 * (n + 8) * W
    return bo, bl


def backward_bounds(q, k, v, do, where, window=0, scale=None):
    N, H, d = q.shape
    rep, scale = H // k.shape[1], d ** -0.5 if scale is None else scale
    u = half_step(q.dtype)
    out = {n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("q", q), ("k", k), ("v", v))}
    sums = {n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("q", q), ("k", k), ("v", v))}
    bo, _ = forward_bounds(q, k, v, where, window, scale)
    for lo, n in where:
        r = slice(lo, lo + n)
        for h in range(H if n else 0):
            Q, K, V, p, e, f = _parts(q, k, v, lo, n, h, window, scale)
            G = f(do[r, h])
            g = h // rep
            o, dp = p @ V, G @ V.T
            D = (G * o).sum(1, keepdim=True)
            rel = (u + 2 * e + 2 * (n + 8) * W)[:, None]
            ds = p * (dp - D)
            # The p of the backward comes from the rounded lse, off as the forward's sum is.
            eds = p * (2 * rel * (dp - D).abs() + (d + 1) * W * (G.abs() @ V.abs().T)
                       + ((G.abs() * (bo[r, h] + (d + 1) * W * o.abs())).sum(1, keepdim=True)))
            m = rep * n
            out["q"][r, h] = scale * (eds @ K.abs() + n * W * (ds.abs() @ K.abs()) + n * TINY * K.abs().max())
            out["k"][r, g] += scale * (eds.T @ Q.abs() + m * W * (ds.abs().T @ Q.abs()) + n * TINY * Q.abs().max())
            out["v"][r, g] += (p * (2 * rel)).T @ G.abs() + m * W * (p.T @ G.abs()) + n * TINY * G.abs().max()
            sums["q"][r, h] = scale * ds @ K
            sums["k"][r, g] += scale * ds.T @ Q
            sums["v"][r, g] += p.T @ G
    return {n: out[n] + u * (sums[n].abs() + out[n]) for n in out}
