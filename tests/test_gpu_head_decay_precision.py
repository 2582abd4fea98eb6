"""Linear attention with one decay per head: bf16 outputs as exact as their one rounding, decay gradients that keep their relative
accuracy, float32 states that are rounded once a chunk.

The outputs: beside that rounding (U of the output) the operands of the last products are two bf16 terms each, the decayed products and
the state alike: the first term leaves at most U of a value and the second U of that, so U * U of each part's magnitudes, on top
of the float32 sums (kf, test_gpu_head_decay)."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from test_gpu_head_decay import (CASES, F, U, absolute, backward, backward64, forward, forward64, ids, inputs, kf, within)

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


# A decay's gradient is a difference: <S, A> at the nearer end of its group of 128 tokens, plus q.dq - k.dk summed over the
# tokens in between. A token's own product (q.k)(do.v) is in both and left out of both, so what the difference was rounded by
# is bounded by the other terms alone. Where the decay is strong they are small, and the gradient keeps its relative accuracy.


def dla_bound(x):
    T, H = x["v"].shape[1:3]
    rep = H // x["q"].shape[2]
    mag = backward64(absolute(x))
    up = lambda n: x[n].double().abs().cpu().repeat_interleave(rep, 2)  # noqa: E731
    q, k, v, do = up("q"), up("k"), x["v"].double().abs().cpu(), x["do"].double().abs().cpu()
    live = torch.ones(x["v"].shape[0], T, 1, dtype=torch.float64)
    if x["lens"] is not None:
        live = (torch.arange(T)[None] < x["lens"].cpu().clamp(0, T)[:, None]).double()[..., None]
    own = (q * k).sum(-1) * (do * v).sum(-1)
    terms = live * ((q * mag["qh"]).sum(-1) + (k * mag["kh"]).sum(-1) - 2 * own).clamp_min(0)
    total = torch.zeros_like(terms)
    for t0 in range(0, T, 128):
        part = terms[:, t0:t0 + 128]
        before = part.cumsum(1) - part
        from_end = part.flip(1).cumsum(1).flip(1) + mag["edge"][:, min(t0 + 127, T - 1)][:, None]
        from_start = before + (mag["edge"][:, t0 - 1][:, None] if t0 else 0.0)
        first = (torch.arange(part.shape[1]) < 64)[None, :, None] & (t0 > 0 or x["s0"] is None)
        total[:, t0:t0 + 128] = torch.where(first, from_start, from_end)
    # The row sums' own chains (kf), 128 tokens in 64 bits, <S, A>'s 64-lane sums of 64 terms and its parts.
    bound = (kf(T) * (2 if rep > 1 else 1) + 256 * F) * total * live
    return (bound.sum((0, 1)) if x["a"].dim() == 1 else bound) + 1e-30


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("s0", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,lens", [
    (1, 1, 2, 2, 64, 64, None), (1, 2, 2, 1, 128, 128, None), (2, 64, 2, 2, 64, 128, None), (2, 65, 2, 1, 128, 64, [65, 33]),
    (1, 129, 2, 2, 128, 128, None), (3, 300, 4, 2, 64, 64, [300, 190, 0]), (1, 900, 2, 2, 64, 128, None)])
@pytest.mark.parametrize("a", [1e-5, 1e-3, 0.05, 0.9])
def test_decay_gradients_keep_their_relative_accuracy(device, a, B, T, H, Hk, dk, dv, lens, s0, typ):
    for fixed in (False, True):
        x = inputs(device, B, T, H, Hk, dk, dv, {"bf16": BF, "f32": torch.float32}[typ], fixed, lens, s0, "slow", T)
        x["a"].mul_(a)
        g = backward(x)
        torch.cuda.synchronize()
        want = backward64(x)["la"]
        within(g["la"], want, dla_bound(x) + U[torch.float32] * want.abs(), f"dla, {'fixed' if fixed else 'per token'}")


def test_a_long_float32_state_is_rounded_once_a_chunk(device):
    """512 chunks of a state that hardly decays, one walk to a head. Each chunk rounds the state twice at most (its decay, and its
    sum with the chunk's own), by F / sqrt(3) of it in the mean square, and it grows as the root of the chunks: together
    F sqrt(512 / 3) in the 2-norm; a chunk's own sum of 64 products adds F sqrt(64 / 3)."""
    B, T, H, d = 4, 32768, 64, 64
    g = torch.Generator(device=device).manual_seed(3)
    q, k, v = (torch.randn(B, T, H, d, device=device, generator=g) for _ in range(3))
    a = torch.exp2(-1e-5 * (1 + torch.arange(H, device=device) / H))
    assert muir.chunk_fwd_head_decay_workspace_size(B, T, H, H, d, d, muir.MUIR_F32) == 0
    _, s = muir.chunk_fwd_head_decay(q, k, v, a)
    want = torch.zeros(B, H, d, d, dtype=torch.float64, device=device)
    log = torch.log2(a.double())[None, :, None]
    to_end = torch.exp2(log * (63 - torch.arange(64, device=device)))
    for c in range(0, T, 64):
        kc = k[:, c:c + 64].double().permute(0, 2, 3, 1).contiguous() * to_end[:, :, None]
        want = want * torch.exp2(64 * log)[..., None] + torch.matmul(kc, v[:, c:c + 64].double().transpose(1, 2).contiguous())
    off = ((s.double() - want).norm() / want.norm()).item()
    print(f"  state off by {off:.3e}", flush=True)
    assert off <= F * ((512 / 3) ** 0.5 + (64 / 3) ** 0.5)
