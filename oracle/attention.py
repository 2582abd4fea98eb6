"""Plain 64-bit forms of causal softmax attention and its paged cache (torch on the CPU, sequence by sequence and head by
head). Independent of the HIP kernels."""
from __future__ import annotations

import torch


def _f64(x):
    return x.detach().double().cpu()


def spans(n, offsets=None, lens=None, count=None):
    """(first row, tokens) of each sequence of n rows: by offsets, else `count` equal parts; lengths cut to the rows."""
    if offsets is None:
        at = [i * (n // count) for i in range(count + 1)]
    else:
        at = [0] + [min(max(int(x), 0), n) for x in offsets[1:]]
    out = []
    for i in range(len(at) - 1):
        rows = max(at[i + 1] - at[i], 0)
        out.append((at[i], rows if lens is None else min(max(int(lens[i]), 0), rows)))
    return out


def visible(n, window=0):
    """[n, n]: does token i see token j."""
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    return (j <= i) & ((i - j < window) if window else torch.ones(n, n, dtype=torch.bool))


def forward(q, k, v, where, window=0, scale=None):
    """(o, lse) of flat rows q [N,H,d], k, v [N,Hk,d] with the sequences `where`."""
    N, H, d = q.shape
    rep, scale = H // k.shape[1], d ** -0.5 if scale is None else scale
    o, lse = torch.zeros(N, H, d, dtype=torch.float64), torch.full((N, H), -torch.inf, dtype=torch.float64)
    for lo, n in where:
        if n == 0:
            continue
        seen = visible(n, window)
        for h in range(H):
            Q, K, V = _f64(q[lo:lo + n, h]), _f64(k[lo:lo + n, h // rep]), _f64(v[lo:lo + n, h // rep])
            s = torch.where(seen, scale * (Q @ K.T), -torch.inf)
            lse[lo:lo + n, h] = torch.logsumexp(s, 1)
            o[lo:lo + n, h] = torch.exp(s - lse[lo:lo + n, h, None]) @ V
    return o, lse


def backward(q, k, v, do, where, window=0, scale=None):
    """{"q", "k", "v"}: the formulas, summed over the heads that share a key head."""
    N, H, d = q.shape
    rep, scale = H // k.shape[1], d ** -0.5 if scale is None else scale
    out = {n: torch.zeros(x.shape, dtype=torch.float64) for n, x in (("q", q), ("k", k), ("v", v))}
    for lo, n in where:
        if n == 0:
            continue
        seen, r = visible(n, window), slice(lo, lo + n)
        for h in range(H):
            Q, K, V, G = _f64(q[r, h]), _f64(k[r, h // rep]), _f64(v[r, h // rep]), _f64(do[r, h])
            p = torch.softmax(torch.where(seen, scale * (Q @ K.T), -torch.inf), 1)
            dp = G @ V.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            out["q"][r, h] = scale * ds @ K
            out["k"][r, h // rep] += scale * ds.T @ Q
            out["v"][r, h // rep] += p.T @ G
    return out


def cached(cache, table, b, n):
    """(rows [n, Hk, d], there [n]) of sequence b's first n tokens; a token in no page is not there."""
    pages, _, page, _ = cache.shape
    rows, there = [], []
    for p in range(n):
        i = int(table[b, p // page])
        there.append(0 <= i < pages)
        rows.append(cache[i if there[-1] else 0, :, p % page])
    return (torch.stack(rows) if rows else cache[0, :, 0][None][:0]), torch.tensor(there, dtype=torch.bool)


def append(k, v, k_cache, v_cache, table, where, start=None):
    """The caches (copies) with the rows of the sequences `where` put in."""
    out = k_cache.clone().cpu(), v_cache.clone().cpu()
    pages, page, width = k_cache.shape[0], k_cache.shape[2], table.shape[1]
    for s, (lo, n) in enumerate(where):
        first = 0 if start is None else int(start[s])
        for t in range(n if first >= 0 else 0):
            p = first + t
            if p < width * page and 0 <= int(table[s, p // page]) < pages:
                for new, cache in zip((k, v), out):
                    cache[int(table[s, p // page]), :, p % page] = new[lo + t].cpu()
    return out


def step(q, k, v, k_cache, v_cache, table, lens, window=0, scale=None):
    """(o, k_cache, v_cache, size) after one token of each sequence; size is the sum of p |v|, what roundings of p are relative to."""
    B, H, d = q.shape
    Hk, page, width = k_cache.shape[1], k_cache.shape[2], table.shape[1]
    rep, scale = H // Hk, d ** -0.5 if scale is None else scale
    table, kc, vc = table.cpu(), k_cache.clone().cpu(), v_cache.clone().cpu()
    o, size = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n + (k is not None) > width * page:
            continue
        if k is not None:
            i = int(table[b, n // page])
            if 0 <= i < kc.shape[0]:
                kc[i, :, n % page], vc[i, :, n % page] = k[b].cpu(), v[b].cpu()
            n += 1
        (K, there), (V, _) = cached(kc, table, b, n), cached(vc, table, b, n)
        if window and n > window:
            K, V, there = K[-window:], V[-window:], there[-window:]
        if not there.any():
            continue
        for h in range(H):
            K64, V64 = _f64(K[there, h // rep]), _f64(V[there, h // rep])
            p = torch.softmax(scale * (K64 @ _f64(q[b, h])), 0)
            o[b, h], size[b, h] = p @ V64, p @ V64.abs()
    return o, kc, vc, size
