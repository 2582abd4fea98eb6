"""The root-mean-square norm against its definition in 64 bits. A row's sum of D squares is off by at most D F relative
(F one float32 rounding), halved by the root; the few operations after it add 8 F."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from oracle import layer

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, FL = torch.bfloat16, torch.float32


def rows(device, n, D, xt, rt, seed=0):
    g = torch.Generator().manual_seed(seed + D)
    x = torch.randn(n, D, generator=g).to(xt)
    res = None if rt is None else (2 * torch.randn(n, D, generator=g)).to(rt)
    w = 1 + 0.3 * torch.randn(D, generator=g)
    return [t if t is None else t.to(device) for t in (x, res, w)]


def close(got, want, bound, name):
    assert torch.isfinite(got.float()).all(), name
    over = ((got.double().cpu() - want).abs() - bound).max().item() if want.numel() else -1
    print(f"  {name}: over its bound by {over:.3e}", flush=True)
    assert over <= 0, name


SIZES = [(1, 8), (3, 64), (5, 520), (2, 1016), (7, 2048), (4, 2056), (3, 4096), (2, 8192), (2, 8200), (1, 16384), (1030, 128)]
TYPES = [(BF, None), (BF, BF), (BF, FL), (FL, None), (FL, FL)]


@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("n,D", SIZES)
def test_forward_and_backward(device, n, D, xt, rt):
    x, res, w = rows(device, n, D, xt, rt)
    y, h, rstd = muir.rms_norm(x, w, res)
    y64, h64, r64 = layer.rms_norm(x, w, res)
    e = (D / 2 + 8) * F
    assert torch.equal(h.double().cpu(), h64)
    close(rstd, r64, e * r64, "rstd")
    close(y, y64, (U[xt] + e * (1 + U[xt])) * y64.abs(), "y")
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(n, D, generator=g).to(xt).to(device)
    dh = torch.randn(n, D, generator=g).to(h.dtype).to(device)
    for more in (None, dh):
        dx, dw = muir.rms_norm_bwd(dy, h, w, rstd, dh=more)
        dx64, dw64 = layer.rms_norm_backward(dy, h, w, dh=more)
        # p and n are off by 4 F and e; the mean of p n by D F of its terms' sum.
        p, nn = (dy.double() * w.double()).cpu(), h64 * r64[..., None]
        terms = r64[..., None] * (p.abs() + nn.abs() * (p * nn).abs().mean(-1, keepdim=True))
        mag = dx64.abs() + terms + (0 if more is None else more.double().cpu().abs())
        close(dx, dx64, U[h.dtype] * dx64.abs() + (D * F + 3 * e) * mag, "dx")
        close(dw, dw64, (n * F + 2 * e) * (dy.double().cpu() * nn).abs().sum(0) + 1e-30, "dweight")


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("int8", 127.0)])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("n,D", [(1, 128), (5, 640), (3, 2048), (2, 2176), (2, 5120), (1, 16384)])
def test_8bit(device, n, D, xt, rt, group, fmt, top):
    x, res, w = rows(device, n, D, xt, rt)
    y, scale, h = muir.rms_norm_8bit(x, w, res, format=fmt, group=group)
    y64, h64, _ = layer.rms_norm(x, w, res)
    assert torch.equal(h.double().cpu(), h64)
    e = (D / 2 + 10) * F
    v = y64.view(n, -1, group or D)
    s64 = v.abs().amax(-1) / top
    got = scale.double().cpu().view(n, -1)
    assert scale.shape == ((n, D // 128) if group else (n,))
    assert ((got - s64).abs() <= e * s64).all()
    # Half a step of the 8-bit value (e4m3: 2^-4 of it, at least 2^-10; int8: 1/2), and the quotient's own error.
    q = y.float().double().cpu().view(n, -1, group or D)
    r = v / got[..., None]
    half = torch.maximum(2.0 ** -4 * r.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) if fmt == "e4m3" else 0.5
    close(q, r, half + 2 * e * r.abs(), "8-bit values")
    assert q.abs().max() <= top


def test_rows_of_zeros_small_and_special_values(device):
    x = torch.zeros(4, 256, device=device)
    x[1] = 1e-30
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    w = torch.ones(256, device=device)
    y, h, rstd = muir.rms_norm(x, w, eps=1e-6)
    assert y[0].abs().max() == 0 and torch.isfinite(y[1]).all()
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 7])
    for fmt in ("e4m3", "int8"):
        for group in (0, 128):
            q, s, _ = muir.rms_norm_8bit(x, w, format=fmt, group=group)
            assert (s[0] == 1).all() and q[0].float().abs().max() == 0
            assert torch.isnan(s[2]).all()
            assert not torch.isfinite(s[3]).all()
    # A weight of almost nothing: the scale stays a normal number and the values finite.
    q, s, _ = muir.rms_norm_8bit(torch.ones(1, 128, device=device), torch.full((128,), 1e-42, device=device))
    assert s.item() >= 1.17549435e-38 and torch.isfinite(q.float()).all()
    # A NaN weight is kept in its own group only.
    w[200] = float("nan")
    q, s, _ = muir.rms_norm_8bit(torch.ones(1, 256, device=device), w, group=128)
    assert torch.isfinite(s[0, 0]) and torch.isnan(s[0, 1])


def test_no_rows_leading_dimensions_and_in_place(device):
    w = torch.ones(64, device=device)
    y, h, rstd = muir.rms_norm(torch.empty(0, 3, 64, device=device), w)
    assert y.shape == (0, 3, 64) and rstd.shape == (0, 3)
    dx, dw = muir.rms_norm_bwd(y, h, w, rstd)
    assert dx.shape == (0, 3, 64) and dw.abs().max().item() == 0
    x, res, _ = rows(device, 6, 64, BF, FL)
    a = muir.rms_norm(x.view(2, 3, 64), w, res.view(2, 3, 64))
    keep = res.clone()
    b = muir.rms_norm(x, w, keep, h=keep)
    assert a[0].shape == (2, 3, 64) and a[2].shape == (2, 3) and b[1] is keep
    assert torch.equal(a[0].view(6, 64), b[0]) and torch.equal(a[1].view(6, 64), keep)
    dy, dh = torch.randn(6, 64, device=device).to(BF), torch.randn(6, 64, device=device)
    want = muir.rms_norm_bwd(dy, keep, w, b[2], dh=dh)
    got = muir.rms_norm_bwd(dy, keep, w, b[2], dh=dh, dx=dh)
    assert got[0] is dh and torch.equal(want[0], dh) and torch.equal(want[1], got[1])


def test_gradient_against_differences(device):
    x, _, w = rows(device, 3, 64, FL, None)
    y, h, rstd = muir.rms_norm(x, w)
    dy = torch.randn(3, 64, generator=torch.Generator().manual_seed(3)).to(device)
    dx, dw = muir.rms_norm_bwd(dy, h, w, rstd)
    loss = lambda a, b: (layer.rms_norm(a, b)[0] * dy.double().cpu()).sum()  # noqa: E731
    x64, w64 = x.double().cpu(), w.double().cpu()
    r = torch.randn(3, 64, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    rw = r[0].clone()
    for got, want, scale in (((dx.double().cpu() * r).sum(), (loss(x64 + 1e-5 * r, w64) - loss(x64 - 1e-5 * r, w64)) / 2e-5, r.abs().sum()),
                             ((dw.double().cpu() * rw).sum(), (loss(x64, w64 + 1e-5 * rw) - loss(x64, w64 - 1e-5 * rw)) / 2e-5, rw.abs().sum())):
        # 80 F of terms of size up to 10, and the difference's second-order error, 1e-10 of third derivatives.
        assert abs(got - want) <= (80 * F * 10 + 1e-8) * scale


def test_graph_replays_and_other_stream(device):
    x, res, w = rows(device, 40, 2048, BF, BF)
    dy = torch.randn(40, 2048, device=device).to(BF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, rstd = muir.rms_norm(x, w, res)
        dx, dw = muir.rms_norm_bwd(dy, h, w, rstd)
        q, s, _ = muir.rms_norm_8bit(x, w, res)
    for i in range(3):
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream(device)
        with torch.cuda.stream(side):
            ey, eh, er = muir.rms_norm(x, w, res)
            edx, edw = muir.rms_norm_bwd(dy, eh, w, er)
            eq, es, _ = muir.rms_norm_8bit(x, w, res)
        side.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, edx) and torch.equal(dw, edw)
        assert torch.equal(q.view(torch.uint8), eq.view(torch.uint8)) and torch.equal(s, es)
