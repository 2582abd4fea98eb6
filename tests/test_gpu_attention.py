"""Causal softmax attention over whole prompts, forward and backward, against its formulas in 64 bits. Bounds: attention_bounds."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from attention_bounds import backward_bounds, forward_bounds
from oracle import attention as oa

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32


def make(device, dt, lead, H, Hk, d, seed, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    q = sharp * torch.randn(*lead, H, d, generator=g)
    k, v, do = torch.randn(*lead, Hk, d, generator=g), torch.randn(*lead, Hk, d, generator=g), torch.randn(*lead, H, d, generator=g)
    return [x.to(dt).to(device) for x in (q, k, v, do)]


def flat(x):
    return x.reshape(-1, *x.shape[-2:])


def check(q, k, v, do, where, offsets=None, lens=None, window=0, scale=None):
    """Both passes against 64 bits; rows that are no token have zeros and -inf."""
    o, lse = muir.attention_fwd(q, k, v, offsets, lens=lens, window=window, scale=scale)
    grads = muir.attention_bwd(q, k, v, o, lse, offsets, do=do, lens=lens, window=window, scale=scale)
    torch.cuda.synchronize()
    Q, K, V, G = (flat(x).cpu() for x in (q, k, v, do))
    token = torch.zeros(len(Q), dtype=torch.bool)
    for lo, n in where:
        token[lo:lo + n] = True
    want, wl = oa.forward(Q, K, V, where, window, scale)
    bo, bl = forward_bounds(Q, K, V, where, window, scale)
    got, gl = flat(o).double().cpu(), lse.reshape(-1, lse.shape[-1]).double().cpu()
    assert (got[~token] == 0).all() and (gl[~token] == -torch.inf).all()
    assert ((got - want).abs() <= bo)[token].all(), ((got - want).abs() - bo)[token].max()
    assert ((gl - wl).abs() <= bl)[token].all(), ((gl - wl).abs() - bl)[token].max()
    want, bounds = oa.backward(Q, K, V, G, where, window, scale), backward_bounds(Q, K, V, G, where, window, scale)
    for n in muir.ATTENTION_GRADS:
        got = flat(grads[n]).double().cpu()
        assert grads[n].shape == {"q": q, "k": k, "v": v}[n].shape
        assert (got[~token] == 0).all(), n
        off = (got - want[n]).abs()
        assert (off <= bounds[n])[token].all(), (n, (off / bounds[n])[token].max())
    return o, lse, grads


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 300])
def test_lengths(device, dt, d, T):
    q, k, v, do = make(device, dt, (1, T), 2, 2, d, T)
    check(q, k, v, do, [(0, T)])


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("H,Hk", [(3, 1), (8, 2), (12, 12), (9, 9), (17, 17)])
def test_shared_heads(device, dt, H, Hk):
    q, k, v, do = make(device, dt, (2, 150), H, Hk, 64, H)
    check(q, k, v, do, [(0, 150), (150, 150)])


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 100, 128, 129, 399, 400, 2 ** 31 - 1])
def test_windows(device, dt, d, window):
    q, k, v, do = make(device, dt, (1, 400), 2, 1, d, window % 1000)
    check(q, k, v, do, [(0, 400)], window=window)


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("window", [0, 70])
def test_padded_batch_does_not_read_behind_lengths(device, dt, window):
    """Lengths from none to all, one cut from beyond; NaN and infinity in the rows behind them."""
    B, T = 6, 260
    q, k, v, do = make(device, dt, (B, T), 4, 2, 64, 5)
    lens = [0, 1, 129, 259, 260, 1000]
    for b, n in enumerate(lens):
        q[b, n:], do[b, n:] = float("nan"), float("inf")
        k[b, n:], v[b, n:] = float("inf"), float("nan")
    where = [(b * T, min(n, T)) for b, n in enumerate(lens)]
    ln = torch.tensor(lens, dtype=torch.int32, device=device)
    check(q, k, v, do, where, lens=ln, window=window)
    ln[0] = -7
    o, _ = muir.attention_fwd(q, k, v, lens=ln, window=window)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("dt,d", [(BF, 128), (FL, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_packed_sequences(device, dt, d, window):
    """Empty sequences in front, between and last, rows behind the last one with NaN in them; sequences do not see each other."""
    lens = [0, 5, 130, 0, 1, 0, 256, 77, 3, 0]
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    N = offsets[-1] + 141
    q, k, v, do = make(device, dt, (N,), 4, 2, d, 11)
    for x in (q, k, v, do):
        x[offsets[-1]:] = float("nan")
    off = torch.tensor(offsets, dtype=torch.int32, device=device)
    check(q, k, v, do, oa.spans(N, offsets), off, window=window)
    tokens = torch.tensor([max(n - 2, 0) for n in lens], dtype=torch.int32, device=device)
    check(q, k, v, do, oa.spans(N, offsets, tokens), off, lens=tokens, window=window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(32, 32), (64, 32)])
@pytest.mark.parametrize("window", [0, 70])
def test_plenty_of_blocks(device, d, H, Hk, window):
    """So many heads and sequences that bfloat16 takes 128 rows to a workgroup for queries and keys: packed, and padded with lengths."""
    lens = [0, 1, 129, 128, 33, 0, 140, 127, 64, 0, 31, 65]
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    N = offsets[-1] + 5
    q, k, v, do = make(device, BF, (N,), H, Hk, d, d + H)
    for x in (q, k, v, do):
        x[offsets[-1]:] = float("nan")
    check(q, k, v, do, oa.spans(N, offsets), torch.tensor(offsets, dtype=torch.int32, device=device), window=window)
    B, T = 8, 135
    q, k, v, do = make(device, BF, (B, T), H, Hk, d, d + H + 1)
    lens = [135, 0, 1, 128, 129, 97, 32, 134]
    for b, n in enumerate(lens):
        for x in (q, k, v, do):
            x[b, n:] = float("nan")
    check(q, k, v, do, [(b * T, n) for b, n in enumerate(lens)], lens=torch.tensor(lens, dtype=torch.int32, device=device), window=window)


@pytest.mark.parametrize("dt,H,Hk", [(BF, 4, 1), (BF, 32, 32), (FL, 4, 2)])
@pytest.mark.parametrize("S", [1, 62, 63, 64, 65, 130])
@pytest.mark.parametrize("window", [0, 3])
def test_sequence_counts(device, dt, H, Hk, S, window):
    """As many packed sequences as lanes count at once, one fewer, more; some empty, rows behind the last, tokens left out by lengths."""
    g = torch.Generator().manual_seed(S)
    n = torch.randint(0, 12, (S,), generator=g)
    n[S // 2] = 140
    n[::5] = 0
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).int()
    lens = (n - torch.randint(0, 3, (S,), generator=g)).clamp_min(0).int()
    N = int(offsets[-1]) + 40
    q, k, v, do = make(device, dt, (N,), H, Hk, 64, S)
    check(q, k, v, do, oa.spans(N, offsets.tolist(), lens.tolist()), offsets.to(device), lens=lens.to(device), window=window)


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
def test_long_rows_with_many_heads(device, dt, d):
    """Rows with more tiles of keys than are in flight at once, in many workgroups; the last rows of several sequences."""
    q, k, v, do = make(device, dt, (2, 517), 45, 45, d, 77)
    heads = [0, 22, 44]
    o, lse = muir.attention_fwd(q, k, v)
    g = muir.attention_bwd(q, k, v, o, lse, do=do)
    Q, K, V, G = (flat(x)[:, heads].cpu() for x in (q, k, v, do))
    where = [(0, 517), (517, 517)]
    want, wl = oa.forward(Q, K, V, where)
    bo, bl = forward_bounds(Q, K, V, where)
    assert ((flat(o)[:, heads].double().cpu() - want).abs() <= bo).all() and ((lse.flatten(0, 1)[:, heads].double().cpu() - wl).abs() <= bl).all()
    want, bounds = oa.backward(Q, K, V, G, where), backward_bounds(Q, K, V, G, where)
    for n in muir.ATTENTION_GRADS:
        assert ((flat(g[n])[:, heads].double().cpu() - want[n]).abs() <= bounds[n]).all(), n


def test_many_short_sequences(device):
    """More sequences than lanes that look for them, many empty."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (5000,), generator=g)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).int()
    N = int(offsets[-1])
    q, k, v, do = make(device, FL, (N,), 1, 1, 64, 4)
    check(q, k, v, do, oa.spans(N, offsets.tolist()), offsets.to(device))


@pytest.mark.parametrize("dt", [BF, FL])
def test_scores_far_apart(device, dt):
    """Scores of hundreds, rising along the keys, falling, and equal; a scale of its own."""
    T, d = 200, 64
    q, k, v, do = make(device, dt, (3, T), 1, 1, d, 9)
    ramp = torch.linspace(-30, 30, T).to(dt).to(device)
    for b, r in enumerate((ramp, -ramp, 0 * ramp)):
        q[b], k[b] = 0, 0
        q[b, :, 0, 0], k[b, :, 0, 0] = 8, r
    check(q, k, v, do, [(b * T, T) for b in range(3)], scale=1.5)


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("T,H", [(1, 1), (5, 1), (70, 1), (100, 300)])
def test_scores_near_the_lowest(device, dt, T, H):
    """Every score the same and about -2e32: exponentials are 1, so o is the mean of the values seen, their sum off by at most n w."""
    q, k, v, _ = make(device, dt, (1, T), H, H, 64, T)
    q.zero_()
    k.zero_()
    q[..., 0], k[..., 0] = 2.0 ** 57, -2.0 ** 53
    o, lse = muir.attention_fwd(q, k, v)
    n = torch.arange(1, T + 1)[:, None, None]
    V = v[0].double().cpu()
    off = (o[0].double().cpu() - V.cumsum(0) / n).abs()
    u = torch.finfo(dt).eps / 2
    assert (off <= (u + 2 * (n + 8) * 2.0 ** -24) * V.abs().cumsum(0) / n).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("T,H", [(60, 1), (100, 300)])
@pytest.mark.parametrize("up", [True, False])
def test_large_scores(device, dt, T, H, up):
    """Scores of up to 2^29, some 2^22 apart, rising or falling along the keys: each query has one key, the last it sees or the first. The score's own rounding
    is in both of numerator and denominator. bf16: the exponential is rounded once and so is the output, two half steps, and a few of float32. float32: the
    product of three terms leaves out three parts of up to 2^-24 each and adds six, then come a reciprocal, its product with the sum and the storing:
    12 times 2^-24."""
    q, k, v, _ = make(device, dt, (1, T), H, H, 64, T)
    q.zero_()
    k.zero_()
    q[..., 0] = 2.0 ** 16
    k[0, :, :, 0] = ((1 if up else -1) * torch.arange(T, device=device)[:, None] * 2.0 ** 9).to(dt)
    o, lse = muir.attention_fwd(q, k, v)
    want = v[0].double().cpu() if up else v[0, :1].double().cpu().expand(T, H, 64)
    bound = 2.1 * 2.0 ** -8 if dt is BF else 12 * 2.0 ** -24
    assert ((o[0].double().cpu() - want).abs() <= bound * want.abs()).all() and torch.isfinite(lse).all()


def test_no_rows(device):
    x = torch.zeros(2, 0, 2, 64, device=device)
    o, lse = muir.attention_fwd(x, x, x)
    assert o.shape == x.shape and lse.shape == (2, 0, 2)
    g = muir.attention_bwd(x, x, x, o, lse, do=x)
    assert all(g[n].shape == x.shape for n in g)


def test_offsets_that_are_none(device):
    """Offsets beyond the rows are cut to them, and descending ones make empty sequences: nothing is read or written outside."""
    q, k, v, do = make(device, BF, (100,), 2, 1, 64, 6)
    for offsets in ([0, 60, 1000], [0, 2 ** 31 - 1, 50], [0, -5, 100], [7, 60, 40, 100]):
        off = torch.tensor(offsets, dtype=torch.int32, device=device)
        room = torch.full((300, 2, 64), 7.0, dtype=BF, device=device)
        o, lse = muir.attention_fwd(q, k, v, off, o=room[100:200])
        g = muir.attention_bwd(q, k, v, o, lse, off, do=do)
        torch.cuda.synchronize()
        assert (room[:100] == 7).all() and (room[200:] == 7).all() and g["q"].shape == q.shape
    off = torch.tensor([0, 60, 1000], dtype=torch.int32, device=device)
    check(q, k, v, do, [(0, 60), (60, 40)], off)


def test_gradients_against_differences(device):
    """<dq, a> + <dk, b> + <dv, c> against a central difference of <o, do> in 64 bits."""
    T, H, Hk, d, e = 150, 4, 2, 64, 1e-5
    q, k, v, do = make(device, FL, (1, T), H, Hk, d, 21)
    o, lse = muir.attention_fwd(q, k, v, window=90)
    g = muir.attention_bwd(q, k, v, o, lse, do=do, window=90)
    gen = torch.Generator().manual_seed(1)
    x = [flat(t).double().cpu() for t in (q, k, v)]
    r = [torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in x]
    D = flat(do).double().cpu()
    loss = lambda s: (oa.forward(*[t + s * u for t, u in zip(x, r)], [(0, T)], 90)[0] * D).sum()  # noqa: E731
    want = (loss(e) - loss(-e)) / (2 * e)
    bounds = backward_bounds(*(flat(t).cpu() for t in (q, k, v, do)), [(0, T)], 90)
    got = sum((flat(g[n]).double().cpu() * u).sum() for n, u in zip("qkv", r))
    slack = sum((bounds[n] * u.abs()).sum() for n, u in zip("qkv", r))
    # The difference itself: e^2 times a third derivative, of the order of the cube of the scores' change (here about 10 per unit).
    assert abs(got - want) <= slack + 1e-6 * abs(want) + e * e * 1e3 * D.abs().sum()


def test_without_lse(device):
    """The C entry takes NULL for lse."""
    q, k, v, _ = make(device, BF, (2, 90), 4, 2, 64, 3)
    o = torch.full_like(q, float("nan"))
    st = muir.lib().muir_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, o.data_ptr(), None, 180, 2, 4, 2, 64, 0, 0.125, muir.MUIR_BF16,
                                       torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(o, muir.attention_fwd(q, k, v)[0])


def test_the_same_bits_again(device):
    q, k, v, do = make(device, BF, (2, 700), 8, 2, 128, 8)
    a = muir.attention_fwd(q, k, v)
    ga = muir.attention_bwd(q, k, v, *a, do=do)
    for _ in range(3):
        b = muir.attention_fwd(q, k, v)
        gb = muir.attention_bwd(q, k, v, *b, do=do)
        assert all(torch.equal(x, y) for x, y in zip((*a, *ga.values()), (*b, *gb.values())))


def test_rows_past_32_bits(device):
    """q and o of more than 2^32 elements: the last sequence of a long packed call, with a window, against 64 bits."""
    H, Hk, d, n = 64, 1, 128, 200
    tail = make(device, BF, (n,), H, Hk, d, 2)
    lead = (1 << 32) // (H * d) + 1000 - n
    q, k, v, do = (torch.zeros(lead + n, h, d, dtype=BF, device=device) for h in (H, Hk, Hk, H))
    for x, t in zip((q, k, v, do), tail):
        x[lead:] = t
    off = torch.tensor([0, lead // 2, lead, lead + n], dtype=torch.int32, device=device)
    o, lse = muir.attention_fwd(q, k, v, off, window=64)
    assert (o[:lead] == 0).all()
    g = muir.attention_bwd(q, k, v, o, lse, off, do=do, window=64)
    t = [x.cpu() for x in tail]
    want, wl = oa.forward(*t[:3], [(0, n)], 64)
    bo, bl = forward_bounds(*t[:3], [(0, n)], 64)
    assert ((o[lead:].double().cpu() - want).abs() <= bo).all() and ((lse[lead:].double().cpu() - wl).abs() <= bl).all()
    want, bounds = oa.backward(*t, [(0, n)], 64), backward_bounds(*t, [(0, n)], 64)
    for m in muir.ATTENTION_GRADS:
        assert (g[m][:lead] == 0).all() and ((g[m][lead:].double().cpu() - want[m]).abs() <= bounds[m]).all(), m
