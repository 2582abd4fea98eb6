"""The layer operators together, as a program uses them: a training pass through norm and attention, and a decode loop
of norm, 4-bit projections, attention step and 8-bit norm."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from oracle import layer

pytestmark = pytest.mark.gpu


def test_training_pass_gradients_against_differences(device):
    """L = <o, c> with o the attention over normed rows: the gradient of the rows and the norm's weight through both
    backward passes, against differences of the same chain in 64 bits."""
    B, T, H, d = 1, 100, 2, 64
    g = torch.Generator().manual_seed(0)
    x, res = torch.randn(B, T, H * d, generator=g), torch.randn(B, T, H * d, generator=g)
    w = 1 + 0.2 * torch.randn(H * d, generator=g)
    a = torch.exp(-0.2 * torch.rand(B, T, H, generator=g))
    c = torch.randn(B, T, H, d, generator=g)
    dev = [t.to(device) for t in (x, res, w, a, c)]
    y, h, rstd = muir.rms_norm(dev[0], dev[2], dev[1])
    heads = (y / 8).view(B, T, H, d)
    o, _ = muir.chunk_fwd_head_decay(heads, heads, heads, dev[3])
    grads = muir.chunk_bwd_head_decay(heads, heads, heads, dev[3], do=dev[4])
    dy = ((grads["q"] + grads["k"] + grads["v"]) / 8).view(B, T, H * d)
    dx, dw = muir.rms_norm_bwd(dy, h, dev[2], rstd)

    def loss(e, rx, rw):
        hh = (x.double() + res.double()) + e * rx
        yy = hh * (hh.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * (w.double() + e * rw) / 8
        yy = yy.view(B, T, H, d)
        return (layer.head_decay_forward(yy, yy, yy, a)[0] * c.double()).sum()

    rx, rw = torch.randn(B, T, H * d, generator=g).double(), torch.randn(H * d, generator=g).double()
    want = (loss(1e-5, rx, rw) - loss(-1e-5, rx, rw)) / 2e-5
    got = (dx.double().cpu() * rx).sum() + (dw.double().cpu() * rw).sum()
    size = (dx.double().cpu() * rx).abs().sum() + (dw.double().cpu() * rw).abs().sum()
    # Each factor of the chain is good to its own test's bound, about 600 roundings of 2^-24 of its magnitudes, which
    # cancellation makes larger than the result by less than 16 here (positive and negative terms of like size).
    assert abs(got - want) <= 600 * 16 * 2.0 ** -24 * size


def test_decode_loop(device):
    """Four tokens through residual, norm, projections, step, output projection and the 8-bit norm; eager and as one
    captured graph, which agree bit for bit, and against 64 bits."""
    B, H, Hk, d, D = 3, 4, 2, 64, 256
    g = torch.Generator().manual_seed(2)
    qkv = (2 * Hk + H) * d

    def weights(n, k):
        return (torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).to(device),
                (0.01 * torch.rand(n, k // 64, generator=g)).to(torch.bfloat16).to(device))

    w_in, w_out = weights(qkv, D), weights(D, H * d)
    norm = (1 + 0.1 * torch.randn(D, generator=g)).to(device)
    a = torch.rand(H, generator=g).to(device)
    stream = torch.randn(B, D, generator=g).to(device)
    x = torch.zeros(B, D, dtype=torch.bfloat16, device=device)
    state = torch.zeros(B, H, d, d, device=device)

    def token():
        y, h, _ = muir.rms_norm(x, norm, stream, h=stream)
        p = muir.matvec_q4(y, *w_in, group=64).view(B, 2 * Hk + H, d)
        q, k, v = (t.contiguous() for t in p.split([Hk, Hk, H], 1))
        o = muir.decode_step_head_decay(q, k, v, a, state)
        x.copy_(muir.matvec_q4(o.view(B, H * d), *w_out, group=64))
        return p, o, *muir.rms_norm_8bit(x, norm, stream)

    start = [t.clone() for t in (stream, x, state)]
    s64, x64, st64 = (t.double().cpu() for t in start)
    W1, W2 = layer.q4_weights(*w_in, None, 64), layer.q4_weights(*w_out, None, 64)
    eager = []
    for _ in range(4):
        p, o, q8, scale, h = token()
        eager.append([t.clone() for t in (p, o, q8.view(torch.uint8), scale, h, x, stream, state)])
        # 64 bits from the values that the kernels rounded to, operator by operator.
        y64, s64, _ = layer.rms_norm(x64, norm, s64.float())
        p64 = y64 @ W1.T.contiguous()
        close = lambda got, want, tol: (got.double().cpu() - want).abs().max() <= tol * want.abs().max()  # noqa: E731
        assert close(p.view(B, -1), p64, 2 * 2.0 ** -8 * 4)  # y and p rounded to bf16; a sum of 256 terms can grow it fourfold
        q, k, v = (t.double().cpu() for t in p.split([Hk, Hk, H], 1))
        rep = lambda t: t.repeat_interleave(H // Hk, 1)  # noqa: E731
        st64 = a.double().cpu()[None, :, None, None] * st64 + rep(k)[..., None] * v[..., None, :]
        assert close(state, st64, 2.0 ** -20)
        assert close(o, (rep(q)[..., None] * st64).sum(2), 2.0 ** -8 + 2.0 ** -16)
        x64 = x.double().cpu()
        assert close(x, o.double().cpu().view(B, -1) @ W2.T.contiguous(), 2.0 ** -8 + 2.0 ** -14)
    for t, s in zip((stream, x, state), start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, o, q8, scale, h = token()
    for t, s in zip((stream, x, state), start):
        t.copy_(s)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((p, o, q8.view(torch.uint8), scale, h, x, stream, state), eager[i]):
            assert torch.equal(got, want)
