"""Arguments of softmax attention at their limits, on the device."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from test_gpu_attention import BF, FL, make
from test_gpu_attention_step import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40 + 7, 2 ** 63, 2 ** 64 + 2])
def test_windows_beyond_an_int(device, window):
    """A window longer than any sequence is no limit, however many bits it takes; one below 0 is refused."""
    q, k, v, do = make(device, BF, (1, 90), 2, 1, 64, 1)
    o, lse = muir.attention_fwd(q, k, v, window=window)
    want = muir.attention_fwd(q, k, v)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g, want = muir.attention_bwd(q, k, v, o, lse, do=do, window=window), muir.attention_bwd(q, k, v, o, lse, do=do)
    assert all(torch.equal(g[n], want[n]) for n in want)
    x = setup(device, BF, [70], 2, 1, 64, 16, 2)
    o = muir.decode_step_attention(*x, window=window)
    assert torch.equal(o, muir.decode_step_attention(*x))
    for call in (lambda w: muir.attention_fwd(q, k, v, window=w), lambda w: muir.attention_bwd(q, k, v, q, lse, do=do, window=w),
                 lambda w: muir.decode_step_attention(*x, window=w)):
        with pytest.raises(muir.MuirError):
            call(-window)


def between(rows, like, device, align=1):
    """(room, the tensor of `rows` rows in its middle): guard rows of 7 on both sides."""
    n = -(-rows // align) * align
    room = torch.full((3 * n, *like.shape[1:]), 7, dtype=like.dtype, device=device)
    return room, room[n:n + rows]


@pytest.mark.parametrize("dt,H,Hk", [(BF, 2, 1), (BF, 64, 4), (BF, 256, 128), (FL, 2, 1), (FL, 24, 2)])
@pytest.mark.parametrize("window", [0, 20])
def test_nothing_is_written_outside(device, dt, H, Hk, window):
    """Offsets that are none (beyond the rows, negative, descending), and some that are: o, lse, the gradients and the workspace lie between rows that stay as
    they were, for blocks of 32 and of 128 rows and eight wavefronts."""
    N, d = 100, 64
    q, k, v, do = make(device, dt, (N,), H, Hk, d, 6)
    size = muir.attention_bwd_workspace_size(N, 3, H, Hk, d, muir.MUIR_BF16 if dt is BF else muir.MUIR_F32)
    for offsets in ([0, 30, 60, 100], [0, 60, 1000, 1000], [0, 2 ** 31 - 1, 50, 60], [0, -5, 100, -2 ** 31], [7, 60, 40, 100], [50, 40, 30, 20], [0, 0, 0, 0],
                    [0, 100, 0, 100], [0, 99, 1, 100]):
        off = torch.tensor(offsets, dtype=torch.int32, device=device)
        rooms = {n: between(N, x, device) for n, x in (("o", q), ("lse", torch.empty(N, H)), ("q", q), ("k", k), ("v", v))}
        rooms["workspace"] = between(size, torch.empty(size, dtype=torch.uint8), device, 256)
        o, lse = muir.attention_fwd(q, k, v, off, window=window, o=rooms["o"][1], lse=rooms["lse"][1])
        muir.attention_bwd(q, k, v, o, lse, off, do=do, window=window, out={n: rooms[n][1] for n in "qkv"}, workspace=rooms["workspace"][1])
        torch.cuda.synchronize()
        for n, (room, x) in rooms.items():
            at = len(room) // 3
            assert (room[:at] == 7).all() and (room[at + len(x):] == 7).all(), (n, offsets)


@pytest.mark.parametrize("dt,Hk", [(BF, 2), (FL, 3)])
def test_an_append_writes_nothing_outside(device, dt, Hk):
    """The same for the caches, with starts and pages that are none."""
    N, d, page, pages = 100, 64, 16, 12
    _, k, v, _ = make(device, dt, (N,), Hk, Hk, d, 7)
    table = torch.tensor([[0, 11, 5], [-1, 3, 12], [2 ** 31 - 1, 7, -2 ** 31]], dtype=torch.int32, device=device)
    for offsets in ([0, 30, 60, 100], [0, 2 ** 31 - 1, 50, 60], [0, -5, 100, -2 ** 31], [50, 40, 30, 20], [0, 99, 1, 100]):
        for start in ([0, 0, 0], [-1, 47, 2 ** 31 - 1], [40, 10, -2 ** 31]):
            rooms = [between(pages, torch.empty(pages, Hk, page, d, dtype=dt), device) for _ in range(2)]
            ints = [torch.tensor(x, dtype=torch.int32, device=device) for x in (offsets, start)]
            muir.cache_append(k, v, rooms[0][1], rooms[1][1], table, ints[0], start=ints[1])
            torch.cuda.synchronize()
            assert all((room[:pages] == 7).all() and (room[2 * pages:] == 7).all() for room, _ in rooms), (offsets, start)
