"""Products with 4-bit weights against 64 bits. A sum of K products and K / group finishing steps in float32, the
group's own sums at most 31 / 1 times the weights they stand for (16 + nib against nib - zero): bounded by
(K + 4) F sum |x| (16 + 15 + |zero| + 16) scale over the groups, an absolute bound that needs no luck."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from oracle import layer

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, FL = torch.bfloat16, torch.float32


def make(device, M, N, K, group, xt, st, zeros, seed=0):
    g = torch.Generator().manual_seed(seed + M * 7 + N)
    x = torch.randn(M, K, generator=g).to(xt)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scale = (0.01 + 0.02 * torch.rand(N, K // group, generator=g)).to(st)
    zero = (torch.rand(N, K // group, generator=g) * 15).to(st) if zeros else None
    return [t if t is None else t.to(device) for t in (x, w, scale, zero)]


def check(y, x, w, scale, zero, group):
    K = x.shape[-1]
    x64 = x.double().cpu()
    want = x64 @ layer.q4_weights(w, scale, zero, group).T.contiguous()
    size = (47 + (0 if zero is None else zero.double().cpu().abs())) * scale.double().cpu()
    if zero is None:
        size = size + 8 * scale.double().cpu()
    # Products are summed inside a group (group F), then over the groups (K / group F, twice for the finishing steps).
    steps = (group + 2 * K // group + 8) * F
    bound = steps * (x64.abs() @ size.repeat_interleave(group, 1).T.contiguous())
    d = (y.double().cpu() - want).abs()
    bound = U[x.dtype] * want.abs() + bound * (1 + U[x.dtype])
    print(f"  worst {d.max().item():.3e}, over its bound by {(d - bound).max().item():.3e}", flush=True)
    assert torch.isfinite(y).all() and (d <= bound).all()


@pytest.mark.parametrize("xt,st", [(BF, BF), (BF, FL), (FL, BF), (FL, FL)])
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 1, 32, 32, False), (1, 16, 128, 128, True), (2, 17, 64, 64, True), (3, 100, 96, 32, False), (1, 2048, 2048, 128, False),
    (16, 257, 1088, 64, True), (17, 40, 160, 32, True), (64, 33, 256, 128, False), (33, 300, 4224, 128, True), (5, 1000, 8192, 64, False),
])
def test_product(device, M, N, K, group, zeros, xt, st):
    x, w, scale, zero = make(device, M, N, K, group, xt, st, zeros)
    y = muir.matvec_q4(x, w, scale, zero, group=group)
    torch.cuda.synchronize()
    check(y, x, w, scale, zero, group)


def test_every_nibble_and_position(device):
    """One-hot rows read single weights: exact in float32, every value at every place of a 128-column block."""
    K, N = 256, 32
    nib = (torch.arange(N)[:, None] * 5 + torch.arange(K)[None] * 3) % 16
    w = (nib[:, 0::2] + 16 * nib[:, 1::2]).to(torch.uint8).to(device)
    scale = torch.ones(N, K // 32, device=device)
    for k0 in range(0, K, 64):
        x = torch.zeros(64, K, device=device)
        x[torch.arange(64), k0 + torch.arange(64)] = 1
        y = muir.matvec_q4(x, w, scale, group=32)
        assert torch.equal(y.cpu(), (nib[:, k0:k0 + 64].T - 8).float())


def test_no_rows_dimensions_repeats_and_graph(device):
    x, w, scale, zero = make(device, 6, 96, 256, 64, BF, BF, True)
    assert muir.matvec_q4(x[:0], w, scale, zero, group=64).shape == (0, 96)
    y = muir.matvec_q4(x, w, scale, zero, group=64)
    assert torch.equal(muir.matvec_q4(x.view(2, 3, 256), w, scale, zero, group=64).view(6, 96), y)
    assert torch.equal(muir.matvec_q4(x[3], w, scale, zero, group=64), y[3])
    guard = torch.full((8, 96), 7.0, device=device, dtype=BF)
    muir.matvec_q4(x, w, scale, zero, group=64, y=guard[:6])
    assert torch.equal(guard[:6], y) and (guard[6:] == 7).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = muir.matvec_q4(x, w, scale, zero, group=64)
    for _ in range(3):
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, muir.matvec_q4(x, w, scale, zero, group=64))
