"""The attention operators give the same bits again, with other work before and between."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from test_gpu_attention import BF, FL, make
from test_gpu_attention_step import same, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("B,T,H,Hk,d,window", [(1, 512, 8, 2, 64, 0), (2, 300, 64, 64, 64, 0), (2, 300, 64, 32, 128, 50), (1, 900, 4, 4, 128, 0)])
def test_prompts(device, dt, B, T, H, Hk, d, window):
    q, k, v, do = make(device, dt, (B, T), H, Hk, d, T)
    lens = torch.tensor([T, T - 37][:B], dtype=torch.int32, device=device)
    other = make(device, dt, (3, 211), 6, 3, d, 1)

    def run():
        o, lse = muir.attention_fwd(q, k, v, lens=lens, window=window)
        return [o, lse, *muir.attention_bwd(q, k, v, o, lse, do=do, lens=lens, window=window).values()]

    first = run()
    for _ in range(5):
        muir.attention_bwd(*other[:3], *muir.attention_fwd(*other[:3]), do=other[3])
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("lens", [[5000], [0, 33, 700, 64]])
def test_steps(device, dt, d, lens):
    q, k, v, kc, vc, table, n = setup(device, dt, lens, 4, 2, d, 32, d)
    other = setup(device, dt, [3000], 4, 2, d, 64, 1)
    first = muir.decode_step_attention(q, k, v, kc, vc, table, n)
    kept = kc.clone(), vc.clone()
    for _ in range(5):
        muir.decode_step_attention(*other)
        assert torch.equal(first, muir.decode_step_attention(q, k, v, kc, vc, table, n)) and same(kc, kept[0]) and same(vc, kept[1])
