"""float32 products of the attention operators: three truncated bf16 terms a value, six of their nine products. What that leaves out, in numpy, and that the kernels
leave out just that."""
import numpy as np
import pytest
import torch

import gated_delta_rule_06_amd as muir

U = 2.0 ** -24


def terms(x):
    """The kernels' three terms of float32 values: the upper 16 bits of what is left, in 64 bits."""
    r, out = np.asarray(x, np.float32).copy(), []
    for _ in range(3):
        t = (r.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(t.astype(np.float64))
        r = r - t
    return out


def left_out(a, b):
    """Of the product, relative."""
    A, B = terms(a), terms(b)
    return (A[1] * B[2] + A[2] * B[1] + A[2] * B[2]) / (a.astype(np.float64) * b)


def values(n, seed):
    """Pairs: any, of either sign and over a few powers of two; then those with the longest lower terms."""
    r = np.random.default_rng(seed)
    a, b = ((1 + r.random(n)) * 2.0 ** r.integers(-2, 3, n) * r.choice([-1, 1], n) for _ in range(2))
    a, b = a.astype(np.float32), b.astype(np.float32)
    a[::4], b[::4] = 1 + 2.0 ** -7 - 2.0 ** -23 * r.integers(1, 60, len(a[::4])), 1 + 2.0 ** -7 - 2.0 ** -23
    return a, b


def test_what_six_products_leave_out():
    """The second term is below 2^-7 of the value's power of two and the third below 2^-15, of the value's sign: two products below 2^-22 and one far smaller
    are left out, 8 w of the product and never of the other sign; three terms hold the value."""
    a, b = values(400000, 0)
    A, off = terms(a), left_out(a, b)
    assert (sum(A) == a).all()
    e = 2.0 ** np.floor(np.log2(np.abs(a)))
    assert (np.abs(A[1]) < 2.0 ** -7 * e).all() and (np.abs(A[2]) < 2.0 ** -15 * e).all()
    assert off.min() >= 0 and 7.5 * U < off.max() < 8.01 * U
    r = np.random.default_rng(1)
    mean = left_out(*((1 + r.random(400000)).astype(np.float32) for _ in range(2))).mean()
    assert 0.6 * U < mean < 0.67 * U


@pytest.mark.gpu
@pytest.mark.parametrize("N,d", [(100, 64), (4096, 64), (100, 128), (4096, 128)])
def test_the_kernels_leave_out_just_that(device, N, d):
    """Sequences of one token, whose lse is their score a b, blocks of 32 and of 128 rows. Beside what is left out: the sum of the six products is rounded where the
    largest is added (2 w, should the matrix core truncate; the others are 2^-6 of it), times log2(e) (w), the maximum and the logarithm of the sum are added (w),
    times ln 2 (w), both constants together 2^-26; the exponential and the logarithm, of a number that is 1 but for the score's rounding, are off by one unit
    in the last place of 1: 2 w each, of 1, before the product with ln 2. Products of at least a quarter, so that this is seen beside them."""
    a, b = values(N, N + d)
    big = np.abs(a.astype(np.float64) * b) >= 0.25
    a, b = a[big], b[big]
    q, k, v = (torch.zeros(len(a), 1, 1, d, device=device) for _ in range(3))
    at = d // 2 + 3
    q[:, 0, 0, at], k[:, 0, 0, at] = torch.from_numpy(a).to(device), torch.from_numpy(b).to(device)
    _, lse = muir.attention_fwd(q, k, v, scale=1.0)
    exact = a.astype(np.float64) * b
    want = exact * (1 - left_out(a, b))
    off = np.abs(lse.view(-1).double().cpu().numpy() - want)
    # (2 + 1 + 1 + 1 + 1/4) w of the size, and 4 w of 1 times ln 2.
    assert (off <= (5.25 * np.abs(exact) + 4 * np.log(2)) * U).all(), (off / np.abs(exact) / U).max()
