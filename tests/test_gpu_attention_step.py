"""Keys and values appended to a paged cache, and one new token attending over it, against 64 bits."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from attention_bounds import W, half_step
from oracle import attention as oa

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32


def setup(device, dt, lens, H, Hk, d, page, seed, extra=1, spare=2):
    """Caches with NaN wherever no token is, pages in no order; table rows end with -1."""
    g = torch.Generator().manual_seed(seed)
    B, width = len(lens), max(-(-(max(n, 0) + extra) // page) for n in lens)
    need = [-(-(max(n, 0) + extra) // page) for n in lens]
    ids = torch.randperm(sum(need) + spare, generator=g).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    kc = torch.full((sum(need) + spare, Hk, page, d), float("nan"), dtype=dt)
    vc = kc.clone()
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        for p in range(max(n, 0)):
            kc[table[b, p // page], :, p % page] = torch.randn(Hk, d, generator=g).to(dt)
            vc[table[b, p // page], :, p % page] = torch.randn(Hk, d, generator=g).to(dt)
    q = (2 * torch.randn(B, H, d, generator=g)).to(dt)
    k, v = torch.randn(B, Hk, d, generator=g).to(dt), torch.randn(B, Hk, d, generator=g).to(dt)
    return [x.to(device) for x in (q, k, v, kc, vc, table, torch.tensor(lens, dtype=torch.int32))]


def same(x, y):
    x, y = x.cpu(), y.cpu()
    return torch.equal(torch.isnan(x), torch.isnan(y)) and torch.equal(x.nan_to_num(), y.nan_to_num())


def check(q, k, v, kc, vc, table, lens, window=0, scale=None):
    want, k1, v1, size = oa.step(q, k, v, kc, vc, table, lens, window, scale)
    o = muir.decode_step_attention(q, k, v, kc, vc, table, lens, window=window, scale=scale)
    torch.cuda.synchronize()
    assert same(kc, k1) and same(vc, v1)
    u, d, n = half_step(q.dtype), q.shape[-1], int(lens.max()) + 1
    # As attention_bounds says for o; scores here: |q . k| <= sum|q k| <= 6 d of these inputs (2 x normal times normal, mean 1.3).
    e = (d + 8) * W * (d ** -0.5 if scale is None else scale) * 6 * d
    bound = (u + 2 * e + 2 * (n + 8) * W) * size + u * want.abs()
    off = (o.double().cpu() - want).abs()
    assert (off <= bound).all(), (off - bound).max()
    return o


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (8, 2), (16, 1), (20, 1), (34, 2)])
def test_step(device, dt, d, H, Hk):
    check(*setup(device, dt, [0, 1, 31, 32, 33, 100, 257], H, Hk, d, 16, H + d))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 2, 33, 200, 2 ** 31 - 1])
def test_pages_and_windows(device, page, window):
    for dt in (BF, FL):
        check(*setup(device, dt, [0, 15, 16, 255, 256, 300], 4, 2, 64, page, page), window=window)


@pytest.mark.parametrize("dt,d", [(BF, 128), (FL, 64), (FL, 128), (BF, 64)])
def test_split_over_a_long_cache(device, dt, d):
    """One sequence, so its keys are split; long enough that a wavefront has more tiles than it keeps the pages of, with a table much wider than needed."""
    q, k, v, kc, vc, table, lens = setup(device, dt, [5000], 4, 2, d, 16, 1)
    assert muir.decode_step_attention_workspace_size(1, 4, 2, d, 16, table.shape[1], muir.MUIR_BF16 if dt is BF else muir.MUIR_F32) > 0
    check(q, k, v, kc, vc, table, lens)
    wide = torch.full((1, 4000), -1, dtype=torch.int32, device=device)
    wide[:, :table.shape[1]] = table
    check(q, k, v, kc, vc, wide, lens, window=1000)
    check(q, k, v, kc, vc, wide, lens)


def test_long_without_a_split(device):
    """So many sequences that none is split, and a wavefront walks many tiles."""
    lens = [9000] + [3] * 300
    q, k, v, kc, vc, table, lens = setup(device, BF, lens, 4, 2, 64, 64, 2)
    check(q, k, v, kc, vc, table, lens)


def test_read_only(device):
    """Without a new token nothing is written, and an empty sequence has nothing to see."""
    q, _, _, kc, vc, table, lens = setup(device, BF, [0, 1, 40, 64], 4, 2, 64, 32, 7, extra=0)
    o = check(q, None, None, kc, vc, table, lens)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("B,n", [(200, 40), (1, 3000)])
def test_scores_near_the_lowest(device, dt, B, n):
    """Every score the same and about -2e32 (as of a prompt): o is the mean of the cached values."""
    q, _, _, kc, vc, table, lens = setup(device, dt, [n] * B, 2, 1, 64, 64, 4, extra=0)
    q.zero_()
    kc.zero_()
    q[..., 0], kc[..., 0] = 2.0 ** 57, -2.0 ** 53
    o = muir.decode_step_attention(q, None, None, kc, vc, table, lens)
    u = torch.finfo(dt).eps / 2
    for b in range(B):
        V = oa.cached(vc.cpu(), table.cpu(), b, n)[0][:, 0].double()
        assert ((o[b].double().cpu() - V.mean(0)).abs() <= (u + 2 * (n + 8) * W) * V.abs().mean(0)).all()


def test_left_out_and_missing(device):
    """Negative lengths and full tables take no part; tokens in no page are not seen, and a new token in none is not kept."""
    q, k, v, kc, vc, table, lens = setup(device, BF, [50, -1, 64, 63, 20, 40, -2 ** 31, 2 ** 31 - 1][:6], 4, 2, 64, 16, 8)
    table = table[:, :4].contiguous()  # 64 tokens of room: the third sequence has no place for its new one
    table[0, 1] = kc.shape[0]
    table[3, 3] = -1
    table[4] = -5
    table[5, 0], table[5, 2] = 2 ** 31 - 1, -2 ** 31
    o = check(q, k, v, kc, vc, table, lens)
    assert (o[1] == 0).all() and (o[2] == 0).all() and (o[4] == 0).all()
    for n in (-2 ** 31, 2 ** 31 - 1):
        lens[5] = n
        assert (check(q, k, v, kc, vc, table, lens)[5] == 0).all()


def test_shared_prefix_pages(device):
    """Two sequences read the same first pages; each has its own last one."""
    q, k, v, kc, vc, table, lens = setup(device, BF, [70, 75], 4, 2, 64, 16, 9)
    table[1, :4] = table[0, :4]
    check(q, k, v, kc, vc, table, lens)


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("packed", [False, True])
def test_append(device, dt, d, packed):
    g = torch.Generator().manual_seed(d)
    lens, Hk, page, T = [0, 1, 100, 64, 37], 3, 16, 100
    start = [0, 15, 3, -1, 60]
    if packed:
        offsets = [0]
        for n in lens:
            offsets.append(offsets[-1] + n)
        lead, where = (offsets[-1] + 9,), oa.spans(offsets[-1] + 9, offsets)
        off, ln = torch.tensor(offsets, dtype=torch.int32, device=device), None
    else:
        lead, where, off = (len(lens), T), oa.spans(T * len(lens), None, lens, len(lens)), None
        ln = torch.tensor(lens, dtype=torch.int32, device=device)
    k, v = (torch.randn(*lead, Hk, d, generator=g).to(dt).to(device) for _ in range(2))
    kc, vc = (torch.randn(40, Hk, page, d, generator=g).to(dt).to(device) for _ in range(2))
    table = torch.randperm(40, generator=g)[:5 * 6].view(5, 6).int()
    table[2, 2], table[4, 4] = -1, 40
    st = torch.tensor(start, dtype=torch.int32, device=device)
    for s in (None, st):
        want = oa.append(k.view(-1, Hk, d), v.view(-1, Hk, d), kc, vc, table, where, s)
        muir.cache_append(k, v, kc, vc, table.to(device), off, lens=ln, start=s)
        assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_cache_past_32_bits(device):
    """Pages whose bytes and elements lie past 2^32."""
    Hk, page, d = 4, 256, 128
    pages = (1 << 32) // (Hk * page * d) + 40
    kc, vc = (torch.empty(pages, Hk, page, d, dtype=BF, device=device) for _ in range(2))
    q, k, v, ks, vs, table, lens = setup(device, BF, [700, 300], 8, Hk, d, page, 3)
    far = pages - ks.shape[0]
    kc[far:], vc[far:] = ks, vs
    table = torch.where(table >= 0, table + far, table)
    g = torch.Generator().manual_seed(0)
    new = [torch.randn(1, 300, Hk, d, generator=g).to(BF).to(device) for _ in range(2)]
    muir.cache_append(*new, kc, vc, table[1:].contiguous())
    muir.cache_append(*new, ks, vs, (table[1:] - far).contiguous())
    o = muir.decode_step_attention(q, k, v, kc, vc, table, lens)
    near = muir.decode_step_attention(q, k, v, ks, vs, torch.where(table >= 0, table - far, table), lens)
    assert torch.equal(o, near) and same(kc[far:], ks) and same(vc[far:], vs)


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
def test_large_cache(device, dt, d):
    """Caches of more than 256 MB, read past the last-level cache: the bits that a small cache gives, which other tests check."""
    Hk, page = 2, 64
    pages = (1 << 28) // (2 * Hk * page * d * dt.itemsize) + 20
    q, k, v, ks, vs, table, lens = setup(device, dt, [0, 1, 70, 900, 64], 6, Hk, d, page, d)
    kc, vc = (torch.full((pages, Hk, page, d), float("nan"), dtype=dt, device=device) for _ in range(2))
    far = pages - ks.shape[0]
    kc[far:], vc[far:] = ks, vs
    for window in (0, 100):
        o = muir.decode_step_attention(q, k, v, kc, vc, torch.where(table >= 0, table + far, table), lens, window=window)
        near = muir.decode_step_attention(q, k, v, ks, vs, table, lens, window=window)
        assert torch.isfinite(o).all() and torch.equal(o, near) and same(kc[far:], ks) and same(vc[far:], vs)
    assert torch.isnan(kc[:far]).all() and torch.isnan(vc[:far]).all()


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("window", [1, 255, 600, 1500, 2047])
def test_windows_over_a_long_cache(device, dt, d, window):
    """A window leaves fewer parts than the workspace, whose size knows of no window, has room for."""
    check(*setup(device, dt, [2500, 1, 900], 4, 2, d, 32, window), window=window)
