"""Products of float32 rows with 4-bit weights where every sum is an integer below 2^24: the results are exact, so no
operand may be larger than the weight it stands for."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(1, 16, 128, 128), (4, 33, 96, 32), (16, 260, 1088, 64), (2, 17000, 256, 32)])
def test_float32_rows_are_exact_below_24_bits(device, M, N, K, group, zeros):
    g = torch.Generator().manual_seed(M + N)
    # One large odd number a row, a few small ones: |nib - zero| <= 8 keeps the sums below 8 (2^20 + 1) + 8 * 15 * 8 < 2^24.
    x = torch.zeros(M, K)
    x[torch.arange(M), torch.randint(0, K, (M,), generator=g)] = 2.0 ** 20 + 1 + 2 * torch.randint(0, 1000, (M,), generator=g)
    for _ in range(8):
        x[torch.arange(M), torch.randint(0, K, (M,), generator=g)] += torch.randint(-15, 16, (M,), generator=g)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scale = torch.ones(N, K // group)
    zero = torch.randint(7, 9, (N, K // group), generator=g).float() if zeros else None
    y = muir.matvec_q4(x.to(device), w.to(device), scale.to(device), None if zero is None else zero.to(device), group=group)
    assert torch.equal(y.double().cpu(), x.double() @ layer.q4_weights(w, scale, zero, group).T.contiguous())
