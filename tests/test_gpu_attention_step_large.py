"""A step over a cache larger than the last-level cache whose key heads have more query heads than a workgroup takes."""
import pytest
import torch

import gated_delta_rule_06_amd as muir
from test_gpu_attention_step import BF, FL, same, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 128), (FL, 64), (FL, 128)])
@pytest.mark.parametrize("H,Hk", [(32, 2), (34, 2), (40, 1)])
def test_sets_of_query_heads(device, dt, d, H, Hk):
    """16, 17 and 40 query heads to a key head, with a small and a large cache: the same bits, which other tests check for the small one."""
    page = 64
    pages = (1 << 28) // (2 * Hk * page * d * dt.itemsize) + 20
    q, k, v, ks, vs, table, lens = setup(device, dt, [0, 1, 70, 900, 64], H, Hk, d, page, d)
    kc, vc = (torch.full((pages, Hk, page, d), float("nan"), dtype=dt, device=device) for _ in range(2))
    far = pages - ks.shape[0]
    kc[far:], vc[far:] = ks, vs
    for window in (0, 100):
        o = muir.decode_step_attention(q, k, v, kc, vc, torch.where(table >= 0, table + far, table), lens, window=window)
        near = muir.decode_step_attention(q, k, v, ks, vs, table, lens, window=window)
        assert torch.isfinite(o).all() and torch.equal(o, near) and same(kc[far:], ks) and same(vc[far:], vs)
    assert torch.isnan(kc[:far]).all() and torch.isnan(vc[:far]).all()
