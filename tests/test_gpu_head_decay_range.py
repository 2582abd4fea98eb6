"""Linear attention with one decay per head where a chunk's whole decay lies below the normal float32 range: the state from
before such a chunk is gone, and what the chunk itself added has to decay as the recurrence says in the weaker chunk
that follows. Bounds as for the ordinary decays (test_gpu_head_decay)."""
import pytest
import torch

from test_gpu_head_decay import backward, check_backward, check_forward, forward, inputs

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("T,lens", [(65, None), (129, None), (193, [193, 130]), (700, [650, 67])])
@pytest.mark.parametrize("a", [0.197, 0.2, 0.206, 0.22])
def test_fixed_decay_then_a_part_of_a_chunk(device, a, T, lens, typ):
    """64 log2 a is -150 to -140: full chunks below the normal range, the last one with few tokens."""
    x = inputs(device, 1 if lens is None else 2, T, 2, 1, 64, 128, TYPES[typ], True, lens, True, "slow", T)
    x["a"].fill_(a)
    o, s = forward(x)
    g = backward(x)
    torch.cuda.synchronize()
    check_forward(x, o, s)
    check_backward(x, g)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("total", [-126.5, -135.3, -146.0, -148.0, -149.4])
@pytest.mark.parametrize("T,lens", [(192, None), (330, [330, 200, 64]), (1000, [1000, 450, 0])])
def test_one_chunk_below_the_normal_range_between_slow_ones(device, T, lens, total, typ):
    """One token of each second chunk takes the chunk's decay to 2^total; all the others are near 1."""
    x = inputs(device, 1 if lens is None else 3, T, 2, 2, 128, 64, TYPES[typ], False, lens, True, "slow", T)
    x["a"].fill_(0.999)
    x["a"][:, 10::128] = 2.0 ** total
    o, s = forward(x)
    g = backward(x)
    torch.cuda.synchronize()
    check_forward(x, o, s)
    check_backward(x, g)
