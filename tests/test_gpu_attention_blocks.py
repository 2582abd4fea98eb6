"""float32 prompts with so many heads and sequences that the forward takes 128 rows to a workgroup."""
import pytest
import torch

from oracle import attention as oa
from test_gpu_attention import FL, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(32, 32), (64, 32)])
@pytest.mark.parametrize("window", [0, 1, 70])
def test_float32(device, d, H, Hk, window):
    """Packed, with empty sequences and rows behind the last, and padded with lengths; NaN in all rows that are no token."""
    lens = [0, 1, 129, 128, 33, 0, 140, 127, 64, 0, 31, 65]
    offsets = [0]
    for n in lens:
        offsets.append(offsets[-1] + n)
    N = offsets[-1] + 5
    x = make(device, FL, (N,), H, Hk, d, d + H)
    for y in x:
        y[offsets[-1]:] = float("nan")
    check(*x, oa.spans(N, offsets), torch.tensor(offsets, dtype=torch.int32, device=device), window=window)
    B, T = 9, 135
    x = make(device, FL, (B, T), H, Hk, d, d + H + 1)
    lens = [135, 0, 1, 128, 129, 97, 32, 134, 135]
    for b, n in enumerate(lens):
        for y in x:
            y[b, n:] = float("nan")
    check(*x, [(b * T, n) for b, n in enumerate(lens)], lens=torch.tensor(lens, dtype=torch.int32, device=device), window=window)
