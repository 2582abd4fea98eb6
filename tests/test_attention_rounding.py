"""The corrections that the bf16 backward of softmax attention makes: how far off its gradients are with them, over all elements, and that a correction left out, turned
round or made too often would be seen."""
import pytest
import torch

import attention_rounding as ar
import gated_delta_rule_06_amd as muir
from oracle import attention as oa

BF = torch.bfloat16
# Queries so sharp, or windows so short, that one key has most of a row: there the corrections are largest. (sequences, tokens, H, Hk, d, window, sharpness)
FEW = [(1, 300, 2, 2, 64, 0, 6), (1, 300, 2, 2, 128, 0, 6), (2, 300, 4, 2, 64, 2, 4), (2, 300, 4, 2, 128, 3, 4)]   # blocks of 32 rows
FAR = [(1, 512, 8, 2, 64, 0, 6), (1, 512, 8, 2, 128, 0, 6)]                                                          # eight wavefronts for dk and dv
MANY = [(2, 300, 64, 64, 64, 0, 6), (2, 300, 64, 64, 128, 0, 6), (2, 300, 64, 64, 64, 3, 4), (2, 300, 128, 64, 128, 2, 4)]  # blocks of 128 rows


def make(S, T, H, Hk, d, window, sharp):
    g = torch.Generator().manual_seed(T + H + d + window)
    x = [(s * torch.randn(S, T, h, d, generator=g)).to(BF) for h, s in ((H, sharp), (Hk, 1), (Hk, 1), (H, 1))]
    return x, [y.flatten(0, 1) for y in x], [(i * T, T) for i in range(S)]


# The kernels' sums are float32 and their exponentials off by a few 2^-24, so their roundings fall otherwise than the ones in 64 bits here, and of 40000 and more
# elements the 2-norm of the roundings is the same to a percent; where wavefronts share a row's keys each puts a p of its own right, and less is left.
ROOM = 1.05


@pytest.mark.parametrize("case", FEW + FAR)
def test_a_mistake_would_be_seen(case):
    """Corrections planted wrongly in the 64-bit form come out above what is allowed, by as much again."""
    _, x, where = make(*case)
    want = oa.backward(*x, where, case[5])
    off = lambda **how: {n: ar.off(g, want[n]) for n, g in ar.backward(*x, where, case[5], **how).items()}  # noqa: E731
    right = off()
    for how, where_seen in ((dict(taken=0), "q"), (dict(taken=-1), "q"), (dict(taken=3), "q"), (dict(rest=0), "q"), (dict(rest=-1), "q"),
                            (dict(handed=0), "k"), (dict(handed=-1), "k"), (dict(handed=3), "k")):
        assert off(**how)[where_seen] > ROOM * ROOM * right[where_seen], how


@pytest.mark.gpu
@pytest.mark.parametrize("case", FEW + FAR + MANY)
def test_gradients_over_all_elements(device, case):
    x, rows, where = make(*case)
    want, right = oa.backward(*rows, where, case[5]), ar.backward(*rows, where, case[5])
    q, k, v, do = (y.to(device) for y in x)
    o, lse = muir.attention_fwd(q, k, v, window=case[5])
    got = muir.attention_bwd(q, k, v, o, lse, do=do, window=case[5])
    for n in muir.ATTENTION_GRADS:
        off, most = ar.off(got[n].flatten(0, 1), want[n]), ROOM * ar.off(right[n], want[n])
        print(f"{n} {off:.5f} of {most:.5f}")
        assert off <= most, (n, off, most)
