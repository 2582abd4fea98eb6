"""Limits of the attention operators' arguments, without a GPU."""
import pytest

import gated_delta_rule_06_amd as muir
from test_attention_abi import APPEND, APPEND_ARGS, BWD, BWD_ARGS, FWD, FWD_ARGS, STEP, STEP_ARGS, call

# The kernels take exponentials to base 2: the scale times log2(e) = 1.4427 has to be a finite float32, below 2^128 - 2^103.
TOO_LARGE, LARGEST = 2.3587e38, 2.3586e38


@pytest.mark.parametrize("name,names,args", [("muir_attention_fwd", FWD, FWD_ARGS), ("muir_attention_bwd", BWD, BWD_ARGS),
                                             ("muir_decode_step_attention", STEP, STEP_ARGS)])
def test_scales_that_overflow_in_base_2(name, names, args):
    for scale in (TOO_LARGE, 2.5e38, 3.4e38):
        st, msg = call(name, names, args, dict(scale=scale))
        assert st == 2 and "scale" in msg, msg
    # One that does not is taken, and the next check speaks.
    st, msg = call(name, names, args, dict(scale=LARGEST, q=None))
    assert st == 1 and muir.status_string(st) == "MUIR_ERR_NULL", msg


def test_how_many_rows_an_append_takes():
    """N / 8 + S + 1 workgroups, up to 2^24 - 1 of them; the next check speaks where they are taken."""
    for N, S, status in (((1 << 27) - 56, 5, 1), ((1 << 27) - 48, 5, 3), (1 << 27, 5, 3), (0, (1 << 24) - 2, 0), (0, (1 << 24) - 1, 3), ((1 << 30) + 1, 1, 3)):
        st, msg = call("muir_cache_append", APPEND, APPEND_ARGS, dict(N=N, S=S, k=None))
        assert st == status, (N, S, st, msg)
