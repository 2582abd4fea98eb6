"""How near a step of softmax attention comes to 64 bits in bfloat16: its output's own rounding is all it loses."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from attention_bounds import W, half_step
from oracle import attention as oa
from test_gpu_attention_step import BF, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(4, 2), (20, 1)])
@pytest.mark.parametrize("lens,window", [([3, 31, 32, 100, 257, 300], 0), ([3, 31, 32, 100, 257, 300], 70), ([5000], 0)])
def test_one_rounding(device, d, H, Hk, lens, window):
    """p goes into its product as two bfloat16 terms, which leave out 2^-16 of it (a half step of a half step). So o is off by that and by what float32 leaves,
    both of sum p|v| (attention_bounds: scores off by e, n terms added), and then by its one rounding; the sizes are those of the inputs. Over all elements,
    in the 2-norm, that is the error that rounding the 64-bit output makes, and the first part on top."""
    q, k, v, kc, vc, table, n = setup(device, BF, lens, H, Hk, d, 64, d + H)
    want, _, _, size = oa.step(q, k, v, kc, vc, table, n, window)
    got = muir.decode_step_attention(q, k, v, kc, vc, table, n, window=window).double().cpu()
    # |q . k| is at most |q| |k|, and so is sum|q k|; the largest of the call.
    K = torch.cat([kc.double().nan_to_num().flatten(0, 2), k.double().flatten(0, 1)]).norm(dim=1).max()
    e = (d + 8) * W * d ** -0.5 * q.double().norm(dim=2).max().cpu() * K.cpu()
    u = half_step(BF)
    inner = (u * u + 2 * e + 2 * (max(lens) + 9) * W) * size
    off = (got - want).abs()
    assert (off <= (1 + u) * inner + u * want.abs()).all(), (off - inner - u * want.abs()).max()
    rounding = (want.to(BF).double() - want).norm()
    assert off.norm() <= rounding + (1 + u) * inner.norm(), (off.norm() / want.norm(), rounding / want.norm())
