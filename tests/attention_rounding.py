"""The bf16 attention passes in 64 bits with the roundings that the kernels make, and nothing else: how far off those put the outputs, in the 2-norm."""
import torch

from oracle import attention as oa


def rounded(x):
    return x.to(torch.bfloat16).double()


def backward(q, k, v, do, where, window=0, scale=None, taken=1.0, handed=1.0, rest=1.0):
    """{"q", "k", "v"} from bf16 rows. The forward rounds p and o, so D = do . o is off by e_i, which is the sum of the row's ds. Of e_i sum_j p_ij k_j and of what
    rounding ds lost, one p of a row's even and of its odd groups of four keys (a wavefront's two halves) is put right in dq: 32 keys after 32 are looked through,
    and the largest of them is taken if it is above 1/8 and above 1.5 times the last one taken. dk is made with the exact D. `taken` and `handed` are how often
    e_i is taken off in dq and handed on to dk, `rest` how often the lost part is added: 1 in the kernels, anything else is a mistake to be noticed."""
    N, H, d = q.shape
    rep, scale = H // k.shape[1], d ** -0.5 if scale is None else scale
    out = {n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("q", q), ("k", k), ("v", v))}
    for lo, n in where:
        if n == 0:
            continue
        seen, r = oa.visible(n, window), slice(lo, lo + n)
        half = torch.arange(n) // 4 % 2
        for h in range(H):
            Q, K, V, G = (x.double() for x in (q[r, h], k[r, h // rep], v[r, h // rep], do[r, h]))
            s = torch.where(seen, scale * (Q @ K.T), -torch.inf)
            x = torch.exp(s - s.amax(1, keepdim=True))
            total = x.sum(1, keepdim=True)
            o, p = rounded(rounded(x) @ V / total), x / total
            dp, D = G @ V.T, (G * o).sum(1, keepdim=True)
            ds = p * (dp - D)
            e = ds.sum(1, keepdim=True)
            dq = rounded(ds) @ K
            for which in (0, 1):
                bar, top, at = torch.full((n, 1), 0.125).double(), torch.zeros(n, 1).double(), torch.zeros(n, 1).long()
                for j in range(0, n, 32):
                    most, place = torch.where(half[j:j + 32] == which, p[:, j:j + 32], 0.0).max(1, keepdim=True)
                    more = most > bar
                    top, at, bar = torch.where(more, most, top), torch.where(more, place + j, at), torch.where(more, 1.5 * most, bar)
                lost = (ds - rounded(ds)).gather(1, at)
                dq += torch.where(top > 0, rounded(rest * lost - taken * e * top), 0.0) * K[at[:, 0]]
            out["q"][r, h] = rounded(scale * dq)
            out["k"][r, h // rep] += scale * rounded(p * (dp - D - handed * e)).T @ Q
            out["v"][r, h // rep] += rounded(p).T @ G
    return {"q": out["q"], "k": rounded(out["k"]), "v": rounded(out["v"])}


def off(got, want):
    """2-norm of the difference, relative."""
    return ((got.double().cpu() - want).norm() / want.norm()).item()
