"""Linear attention with one decay per head: bf16 outputs as exact as their one rounding.

Beside that rounding (U of the output) the operands of the last products are two bf16 terms each, the decayed products and
the state alike: the first term leaves at most U of a value and the second U of that, so U * U of each part's magnitudes, on top
of the float32 sums (kf, test_gpu_head_decay)."""
import pytest
import torch

from test_gpu_head_decay import (CASES, U, absolute, backward, backward64, forward, forward64, ids, inputs, kf, within)

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
BF_CASES = [c for c in CASES if c[6] == "bf16"]


def case_inputs(device, case):
    B, T, H, Hk, dk, dv, _, fixed, lens, s0, kind = case
    return inputs(device, B, T, H, Hk, dk, dv, BF, fixed, lens, s0, kind, T + 1)


def bound(want, mag, T):
    u = U[BF]
    return u * want.abs() + (u * u + kf(T)) * (1 + u) * mag + 1e-30


@pytest.mark.parametrize("case", BF_CASES, ids=ids)
def test_outputs_keep_all_but_their_own_rounding(device, case):
    x = case_inputs(device, case)
    o, _ = forward(x)
    torch.cuda.synchronize()
    within(o, forward64(x)[0], bound(forward64(x)[0], forward64(absolute(x))[0], case[1]), "o")


@pytest.mark.parametrize("case", BF_CASES, ids=ids)
def test_value_gradients_keep_all_but_their_own_rounding(device, case):
    x = case_inputs(device, case)
    g = backward(x)
    torch.cuda.synchronize()
    want, mag = backward64(x), backward64(absolute(x))
    within(g["v"], want["v"], bound(want["v"], mag["v"], case[1]), "dv")
