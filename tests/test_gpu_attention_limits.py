"""Arguments of softmax attention at their limits, on the device."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from test_gpu_attention import BF, make
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
