"""What a step of softmax attention does not see: NaN and infinity there reach nothing."""
import pytest
import torch

from test_gpu_attention_step import BF, FL, check, setup

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dt,d,H,Hk", [(BF, 64, 4, 2), (BF, 128, 20, 1), (FL, 64, 4, 2), (FL, 128, 34, 2)])
def test_new_tokens_in_no_page(device, dt, d, H, Hk, bad):
    """A new token whose page does not exist may hold anything: first of its sequence, first of a page, inside one, alone in the table."""
    lens = [0, 16, 20, 37, 70, 33]
    q, k, v, kc, vc, table, n = setup(device, dt, lens, H, Hk, d, 16, d + H)
    for b in range(5):
        table[b, lens[b] // 16] = (-1, kc.shape[0], -7, 2 ** 31 - 1, -2 ** 31)[b]
        k[b], v[b] = bad, bad
    table[3] = -1
    o = check(q, k, v, kc, vc, table, n)
    assert (o[0] == 0).all() and (o[3] == 0).all()


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dt,d,H,Hk", [(BF, 64, 4, 2), (BF, 128, 20, 1), (FL, 64, 4, 2), (FL, 128, 34, 2)])
@pytest.mark.parametrize("window", [1, 16, 17, 31, 32, 33, 100])
def test_tokens_before_the_window(device, dt, d, H, Hk, window, bad):
    """Cached tokens that the window has left behind may hold anything, also in the window's own page and the same 32 tokens."""
    lens = [0, 1, 31, 32, 33, 47, 64, 100, 257]
    q, k, v, kc, vc, table, n = setup(device, dt, lens, H, Hk, d, 16, window)
    for b, old in enumerate(lens):
        for p in range(max(old + 1 - window, 0)):
            kc[table[b, p // 16], :, p % 16], vc[table[b, p // 16], :, p % 16] = bad, bad
    check(q, k, v, kc, vc, table, n, window=window)


@pytest.mark.parametrize("window", [300, 1500])
def test_tokens_before_the_window_of_a_split_sequence(device, window):
    q, k, v, kc, vc, table, n = setup(device, BF, [5000], 4, 2, 128, 64, window)
    p = 5001 - window
    kc[table[0, :p // 64].long()] = vc[table[0, :p // 64].long()] = float("nan")
    kc[table[0, p // 64], :, :p % 64] = vc[table[0, p // 64], :, :p % 64] = float("nan")
    check(q, k, v, kc, vc, table, n, window=window)
