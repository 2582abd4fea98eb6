"""Attention's operators as a program uses them: a prompt, its cache and the steps after it; a layer's training step; captured graphs, other streams and
calls at once. Every attention output is checked against 64 bits from the inputs that the run gave it."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from attention_bounds import W, backward_bounds, forward_bounds
from oracle import attention as oa

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32


def close(got, want, bound):
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), (off - bound).max()


@pytest.mark.parametrize("dt,d", [(BF, 128), (BF, 64), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("window", [0, 40])
def test_prompt_cache_steps(device, dt, d, window):
    """Prompts of different lengths (one empty) into a cache that is full of NaN, a second part of each prompt behind the first, then steps: each step's
    output is the row that the whole sequence's prompt pass has there."""
    B, H, Hk, page, first, steps = 4, 4, 2, 16, [50, 0, 1, 33], 20
    second = [7, 0, 16, 40]
    total = [a + b + steps for a, b in zip(first, second)]
    T = max(total)
    g = torch.Generator().manual_seed(d + window)
    q, k, v = ((s * torch.randn(B, T, h, d, generator=g)).to(dt) for h, s in ((H, 2), (Hk, 1), (Hk, 1)))
    width = -(-T // page)
    table = torch.randperm(B * width, generator=g).int().view(B, width).to(device)
    kc, vc = (torch.full((B * width, Hk, page, d), float("nan"), dtype=dt, device=device) for _ in range(2))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    where = [(b * T, n) for b, n in enumerate(total)]
    rows = [x.view(B * T, -1, d) for x in (q, k, v)]
    want, _ = oa.forward(*rows, where, window)
    bound, _ = forward_bounds(*rows, where, window)
    want, bound = want.view(B, T, H, d), bound.view(B, T, H, d)
    D = [x.to(device) for x in (q, k, v)]
    o, _ = muir.attention_fwd(*D, lens=ints(first), window=window)
    muir.cache_append(D[1], D[2], kc, vc, table, lens=ints(first))
    for b in range(B):
        close(o[b, :first[b]], want[b, :first[b]], bound[b, :first[b]])
    # The rest of each prompt, packed.
    offsets = [0]
    for n in second:
        offsets.append(offsets[-1] + n)
    rest = [torch.cat([x[b, first[b]:first[b] + second[b]] for b in range(B)]).contiguous() for x in D[1:]]
    muir.cache_append(*rest, kc, vc, table, ints(offsets), start=ints(first))
    lens = ints([a + b for a, b in zip(first, second)])
    for t in range(steps):
        at = lens.tolist()
        x = [torch.stack([y[b, at[b]] for b in range(B)]) for y in D]
        o = muir.decode_step_attention(*x, kc, vc, table, lens, window=window)
        lens += 1
        for b in range(B):
            close(o[b], want[b, at[b]], bound[b, at[b]])
    for b in range(B):
        for p in range(total[b]):
            for cache, x in ((kc, D[1]), (vc, D[2])):
                assert torch.equal(cache[table[b, p // page], :, p % page], x[b, p])


def test_hybrid_stack(device):
    """A layer of linear attention with a decay per head, then one of softmax attention over a window, each behind a norm and with a residual: prompts of two
    lengths, then steps, in bfloat16. The recurrent state and the cache go from one to the other."""
    B, T, D, H, Hk, d, page, window = 2, 90, 256, 4, 2, 64, 16, 32
    g = torch.Generator().manual_seed(5)
    w = [[(torch.randn(D, h * d, generator=g) / 16).to(BF).to(device) for h in (H, Hk, Hk)] + [(torch.randn(H * d, D, generator=g) / 16).to(BF).to(device)]
         for _ in range(2)]
    w[0][2] = (torch.randn(D, H * d, generator=g) / 16).to(BF).to(device)  # a value head for each query head there, q and k shared
    w[0][0] = w[0][1].flip(1).contiguous()
    norm = [torch.rand(D, generator=g).to(device) + .5 for _ in range(2)]
    decay = torch.linspace(.9, .99, H, device=device)
    lens = torch.tensor([90, 61], dtype=torch.int32, device=device)
    width = 10
    table = torch.randperm(B * width, generator=g).int().view(B, width).to(device)
    kc, vc = (torch.full((B * width, Hk, page, d), float("nan"), dtype=BF, device=device) for _ in range(2))
    heads = lambda y, m: (y @ m).view(*y.shape[:-1], -1, d)  # noqa: E731
    x = torch.randn(B, T, D, generator=g).to(BF).to(device)
    y, h, _ = muir.rms_norm(x, norm[0])
    o, state = muir.chunk_fwd_head_decay(heads(y, w[0][0]), heads(y, w[0][1]), heads(y, w[0][2]), decay, lens=lens)
    y, h, _ = muir.rms_norm(o.flatten(-2) @ w[0][3], norm[1], h)
    q, k, v = (heads(y, m) for m in w[1][:3])
    o, _ = muir.attention_fwd(q, k, v, lens=lens, window=window)
    muir.cache_append(k, v, kc, vc, table, lens=lens)
    where = [(b * T, int(n)) for b, n in enumerate(lens)]
    rows = [z.reshape(B * T, -1, d).cpu() for z in (q, k, v)]
    close(o.view(B * T, H, d), oa.forward(*rows, where, window)[0], forward_bounds(*rows, where, window)[0])
    seen = [[z[b, :int(lens[b])].cpu() for z in (q, k, v)] for b in range(B)]
    for _ in range(8):
        x = torch.randn(B, D, generator=g).to(BF).to(device)
        y, h, _ = muir.rms_norm(x, norm[0])
        o = muir.decode_step_head_decay(heads(y, w[0][0]), heads(y, w[0][1]), heads(y, w[0][2]), decay, state)
        y, h, _ = muir.rms_norm(o.flatten(-2) @ w[0][3], norm[1], h)
        new = [heads(y, m) for m in w[1][:3]]
        o = muir.decode_step_attention(*new, kc, vc, table, lens, window=window)
        lens += 1
        for b in range(B):
            seen[b] = [torch.cat([s, z[b:b + 1].cpu()]) for s, z in zip(seen[b], new)]
            n = int(lens[b])
            close(o[b], oa.forward(*seen[b], [(0, n)], window)[0][-1], forward_bounds(*seen[b], [(0, n)], window)[0][-1])
        h = h + (o.flatten(-2) @ w[1][3])
        assert torch.isfinite(h).all()


def test_layer_gradient_against_differences(device):
    """The gradient of <attention(norm(x) Wq, norm(x) Wk, norm(x) Wv), G> with respect to x, by rms_norm, attention and their backward passes in float32,
    against a central difference of the same in 64 bits. The projections are 64-bit products rounded to float32.

    The bound: the norm's y is off by (D / 2 + 8) w of itself at most (a sum of D squares, a root, two products), so a score by (D + 16) w S with S its
    absolute sum, 2 of the d + 8 = 72 that backward_bounds counts: p and ds, twice that and what is counted there already: 5 bounds. They go through the
    projections' and the norm's own gradients as they are, with (D + 8) w of the terms on top."""
    T, D, H, Hk, d, window, e = 70, 128, 2, 1, 64, 30, 1e-5
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, D, generator=g)
    weight = torch.rand(D, generator=g) + .5
    G = torch.randn(T, H, d, generator=g)
    M = [torch.randn(D, h * d, generator=g).double() / D ** .5 for h in (H, Hk, Hk)]
    y, h, rstd = muir.rms_norm(x.to(device), weight.to(device))
    f32 = [(y.double().cpu() @ m).float().view(T, -1, d) for m in M]
    q, k, v = (z.to(device).view(1, T, -1, d) for z in f32)
    o, lse = muir.attention_fwd(q, k, v, window=window)
    grads = muir.attention_bwd(q, k, v, o, lse, do=G.to(device).view(1, T, H, d), window=window)
    dy = sum(grads[n].double().cpu().view(T, -1) @ m.T for n, m in zip("qkv", M))
    dx, _ = muir.rms_norm_bwd(dy.float().to(device), h, weight.to(device), rstd)

    def loss(z):
        n = z * torch.rsqrt((z * z).mean(1, keepdim=True) + 1e-6) * weight.double()
        return (oa.forward(*((n @ m).view(T, -1, d) for m in M), [(0, T)], window)[0] * G.double()).sum()

    bounds = backward_bounds(*f32, G, [(0, T)], window)
    by = sum(5 * bounds[n].view(T, -1) @ m.abs().T for n, m in zip("qkv", M))
    r, hat, w64 = rstd.double().cpu()[:, None], h.double().cpu() * rstd.double().cpu()[:, None], weight.double()
    through = lambda z: r * (w64 * z + hat.abs() * (w64 * z * hat.abs()).mean(1, keepdim=True))  # noqa: E731
    bx = through(by) + (D + 8) * W * through(dy.abs())
    for seed in range(4):
        u = torch.randn(T, D, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        want = (loss(x.double() + e * u) - loss(x.double() - e * u)) / (2 * e)
        got = (dx.double().cpu() * u).sum()
        # The difference's own error: e^2 times a third derivative, whose size is that of G times the cube of a score's change per unit (about 10).
        assert abs(got - want) <= (bx * u.abs()).sum() + e * e * 1e3 * G.abs().sum()


def prompt(device, dt, B, T, H, Hk, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, T, h, d, generator=g).to(dt).to(device) for h in (H, Hk, Hk, H)]


def both(x, **more):
    q, k, v, do = x
    o, lse = muir.attention_fwd(q, k, v, **more)
    return [o, lse, *muir.attention_bwd(q, k, v, o, lse, do=do, **more).values()]


@pytest.mark.parametrize("dt,T,H", [(BF, 300, 3), (BF, 400, 64), (FL, 300, 3)])
def test_other_stream_and_graph_replays_of_a_prompt(device, dt, T, H):
    x = prompt(device, dt, 2, T, H, H, 64, 1)
    lens = torch.tensor([T, T - 30], dtype=torch.int32, device=device)
    want = both(x, lens=lens, window=200)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device)
    with torch.cuda.stream(side):
        got = both(x, lens=lens, window=200)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both(x, lens=lens, window=200)
    for i in range(4):
        for n, t in enumerate(x):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(10 * i + n)).to(dt))
        lens.copy_(torch.tensor([T - 50 * i, i], dtype=torch.int32))
        eager = both(x, lens=lens, window=200)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))


@pytest.mark.parametrize("dt", [BF, FL])
def test_graph_replays_of_steps(device, dt):
    """A captured step is replayed for many tokens: the lengths that it reads go up inside the graph. One sequence is split over workgroups."""
    for B, room in ((1, 4096), (3, 128)):
        H, Hk, d, page, T, steps = 4, 2, 64, 32, 100, 12
        g = torch.Generator().manual_seed(B)
        width = room // page
        table = torch.randperm(B * width, generator=g).int().view(B, width).to(device)
        new = [torch.randn(steps, B, h, d, generator=g).to(dt).to(device) for h in (H, Hk, Hk)]
        k, v = (torch.randn(B, T, Hk, d, generator=g).to(dt).to(device) for _ in range(2))

        def start():
            kc, vc = (torch.full((B * width, Hk, page, d), float("nan"), dtype=dt, device=device) for _ in range(2))
            muir.cache_append(k, v, kc, vc, table)
            return kc, vc, torch.full((B,), T, dtype=torch.int32, device=device)

        kc, vc, lens = start()
        want = []
        for t in range(steps):
            want.append(muir.decode_step_attention(*(x[t] for x in new), kc, vc, table, lens))
            lens += 1
        kept = kc, vc
        kc, vc, lens = start()
        x = [y[0].clone() for y in new]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = muir.decode_step_attention(*x, kc, vc, table, lens)
            lens += 1
        for t in range(steps):
            for a, b in zip(x, new):
                a.copy_(b[t])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want[t]), t
        for a, b in zip((kc, vc), kept):
            assert torch.equal(a.nan_to_num(9.), b.nan_to_num(9.))


def test_two_calls_at_once(device):
    """Prompts on two streams, and steps of a split sequence, share nothing."""
    xs = [prompt(device, BF, 1, 900, 8, 8, 128, i) for i in range(2)]
    caches = [prompt(device, BF, 80, 64, 2, 2, 64, 5 + i)[:2] for i in range(2)]  # [pages, page, heads, d]
    caches = [[c.transpose(1, 2).contiguous() for c in cs] for cs in caches]
    table = torch.arange(80, dtype=torch.int32, device=device).view(1, 80)
    lens = torch.tensor([5000], dtype=torch.int32, device=device)
    qs = [torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(i)).to(BF).to(device) for i in range(2)]
    step = lambda i: muir.decode_step_attention(qs[i], None, None, *caches[i], table, lens)  # noqa: E731
    want = [[*both(x), step(i)] for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device) for _ in xs]
    got = [[], []]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append([*both(xs[i]), step(i)])
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_two_graphs_with_one_workspace(device):
    """Two captured backward passes of different sizes may share a workspace and outputs' memory where they run one after the other."""
    xs = [prompt(device, BF, 1, n, 2, 2, 64, n) for n in (300, 130)]
    size = max(muir.attention_bwd_workspace_size(n, 1, 2, 2, 64, muir.MUIR_BF16) for n in (300, 130))
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    fwd = [muir.attention_fwd(*x[:3]) for x in xs]
    want = [muir.attention_bwd(*x[:3], *f, do=x[3]) for x, f in zip(xs, fwd)]
    torch.cuda.synchronize()
    graphs, kept = [], []
    for x, f in zip(xs, fwd):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kept.append(muir.attention_bwd(*x[:3], *f, do=x[3], workspace=ws))
    for _ in range(3):
        for graph, k, w in zip(graphs, kept, want):
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(k[n], w[n]) for n in w)


def test_one_tensor_for_several_arguments(device):
    """q, k, v and do may be the same tensor; inputs are only read."""
    x = torch.randn(1, 200, 4, 64, generator=torch.Generator().manual_seed(0)).to(BF).to(device)
    keep = x.clone()
    a, b = both([x] * 4), both([x.clone() for _ in range(4)])
    assert torch.equal(x, keep) and all(torch.equal(s, t) for s, t in zip(a, b))
