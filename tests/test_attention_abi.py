"""The attention operators' argument checks without a GPU, what their workgroups take, and the oracle's forms against each other."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_06_amd as muir
from oracle import attention as oa

BASE, STRIDE = 1 << 40, 1 << 34


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * STRIDE + off)


BF, FL = muir.MUIR_BF16, muir.MUIR_F32


def call(name, names, args, over):
    args = {**args, **over}
    st = getattr(muir.lib(), name)(*[args[n] for n in names], None)
    return st, muir.last_error()


SIZES = ["N", "S", "H", "Hk", "d", "window", "scale", "dt"]
SIZE_ARGS = dict(N=1000, S=5, H=6, Hk=3, d=64, window=0, scale=0.125, dt=BF)
BAD_SIZES = [
    (dict(N=-1), 2), (dict(S=0), 2), (dict(H=0), 2), (dict(Hk=0), 2), (dict(Hk=4), 2), (dict(d=32), 3), (dict(d=96), 3), (dict(d=256), 3),
    (dict(dt=2), 3), (dict(window=-1), 2), (dict(scale=0.0), 2), (dict(scale=-1.0), 2), (dict(scale=float("nan")), 2),
    (dict(scale=float("inf")), 2), (dict(scale=2.0 ** -65), 2), (dict(N=(1 << 30) + 1, H=1, Hk=1), 3), (dict(N=1 << 30), 3), (dict(S=1 << 24), 3), (dict(H=1 << 16, Hk=1), 3),
    (dict(N=1001, offsets=None), 2),
]
FWD = ["q", "k", "v", "offsets", "lens", "o", "lse", *SIZES]
FWD_ARGS = dict({n: fake(i) for i, n in enumerate(FWD[:7])}, **SIZE_ARGS)


@pytest.mark.parametrize("over,status", BAD_SIZES + [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(q=fake(0, 8)), 2), (dict(o=fake(5, 2)), 2),
    (dict(offsets=fake(3, 2)), 2), (dict(lse=fake(6, 2)), 2), (dict(o=fake(0)), 5), (dict(o=fake(1, 256)), 5), (dict(lse=fake(5)), 5), (dict(lse=fake(3)), 5),
    (dict(lse=fake(4)), 5),
])
def test_forward_refusals(over, status):
    st, msg = call("muir_attention_fwd", FWD, FWD_ARGS, over)
    assert st == status and msg, msg


BWD = ["q", "k", "v", "o", "lse", "offsets", "lens", "dout", "dq", "dk", "dv", *SIZES, "ws", "wsb"]
BWD_ARGS = dict({n: fake(i) for i, n in enumerate(BWD[:11])}, **SIZE_ARGS, ws=fake(20), wsb=1 << 33)


@pytest.mark.parametrize("over,status", BAD_SIZES + [
    (dict(lse=None), 1), (dict(o=None), 1), (dict(dout=None), 1), (dict(dk=None), 1), (dict(ws=None), 4), (dict(wsb=64), 4),
    (dict(ws=fake(20, 16)), 4), (dict(dq=fake(0)), 5), (dict(dq=fake(7)), 5), (dict(dk=fake(10)), 5), (dict(ws=fake(4)), 5), (dict(dv=fake(10, 8)), 2),
])
def test_backward_refusals(over, status):
    st, msg = call("muir_attention_bwd", BWD, BWD_ARGS, over)
    assert st == status and msg, msg


CACHE = [(dict(pages=0), 2), (dict(width=0), 2), (dict(page=8), 3), (dict(page=48), 3), (dict(page=512), 3), (dict(page=0), 3),
         (dict(page=256, width=1 << 23), 3), (dict(table=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(d=80), 3), (dict(dt=5), 3)]
APPEND = ["k", "v", "k_cache", "v_cache", "table", "offsets", "lens", "start", "N", "S", "Hk", "d", "pages", "page", "width", "dt"]
APPEND_ARGS = dict({n: fake(i) for i, n in enumerate(APPEND[:8])}, N=1000, S=5, Hk=3, d=64, pages=100, page=16, width=20, dt=BF)


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(N=-1), 2), (dict(S=0), 2), (dict(Hk=0), 2), (dict(N=999, offsets=None), 2), (dict(k=None), 1), (dict(k_cache=fake(1)), 5), (dict(v_cache=fake(2, 64)), 5),
    (dict(k_cache=fake(4)), 5), (dict(v_cache=fake(7)), 5), (dict(k=fake(0, 4)), 2), (dict(start=fake(7, 1)), 2),
])
def test_append_refusals(over, status):
    st, msg = call("muir_cache_append", APPEND, APPEND_ARGS, over)
    assert st == status and msg, msg


STEP = ["q", "k", "v", "k_cache", "v_cache", "table", "lens", "o", "B", "H", "Hk", "d", "pages", "page", "width", "window", "scale", "dt", "ws", "wsb"]
STEP_ARGS = dict({n: fake(i) for i, n in enumerate(STEP[:8])}, B=5, H=6, Hk=3, d=64, pages=100, page=16, width=200, window=0, scale=0.125,
                 dt=BF, ws=fake(20), wsb=1 << 33)


@pytest.mark.parametrize("over,status", CACHE + [
    (dict(B=0), 2), (dict(H=7), 2), (dict(window=-3), 2), (dict(scale=0.0), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(lens=None), 1),
    (dict(o=None), 1), (dict(B=1 << 24, Hk=1, H=1), 3), (dict(B=1 << 23, Hk=1, H=1), 3), (dict(scale=2.0 ** -65), 2), (dict(ws=None), 4), (dict(wsb=16), 4), (dict(o=fake(0)), 5), (dict(o=fake(3)), 5),
    (dict(k_cache=fake(2)), 5), (dict(ws=fake(4)), 5), (dict(q=fake(0, 8)), 2), (dict(table=fake(5, 1)), 2),
])
def test_step_refusals(over, status):
    st, msg = call("muir_decode_step_attention", STEP, STEP_ARGS, over)
    assert st == status and msg, msg


def test_workspace_sizes():
    bwd, step = muir.attention_bwd_workspace_size, muir.decode_step_attention_workspace_size
    assert bwd(1000, 5, 6, 3, 64, BF) >= 2 * 4 * 1000 * 6 and bwd(0, 1, 6, 3, 64, BF) == 0
    for bad in [(-1, 1, 2, 1, 64, BF), (10, 0, 2, 1, 64, BF), (10, 1, 3, 2, 64, BF), (10, 1, 2, 1, 32, BF), (10, 1, 2, 1, 64, 9), ((1 << 30) + 1, 1, 1, 1, 64, BF)]:
        assert bwd(*bad) == 0
    assert step(1, 16, 4, 128, 64, 512, BF) > 0 and step(1, 16, 4, 128, 16, 1, BF) == 0 and step(4096, 16, 16, 128, 64, 512, BF) == 0
    for bad in [(0, 2, 1, 64, 16, 100, BF), (1, 3, 2, 64, 16, 100, BF), (1, 2, 1, 64, 17, 100, BF), (1, 2, 1, 64, 16, 0, BF), (1, 2, 1, 64, 16, 1 << 30, BF)]:
        assert step(*bad) == 0


def test_binding_refuses_host_tensors_and_bad_shapes():
    x, off, lens = torch.zeros(2, 4, 2, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c, t = torch.zeros(9, 2, 16, 64), torch.zeros(2, 4, dtype=torch.int32)
    for bad in (lambda: muir.attention_fwd(x, x, x), lambda: muir.attention_fwd(x[0], x[0], x[0]), lambda: muir.attention_fwd(x, x, x, off),
                lambda: muir.attention_fwd(x[0, 0], x, x), lambda: muir.attention_fwd("q", x, x), lambda: muir.attention_bwd(x, x, x, x, x, do=x),
                lambda: muir.cache_append(x, x, c, c, t), lambda: muir.cache_append(x[0], x[0], c, c, t),
                lambda: muir.decode_step_attention(x[0], x[0], x[0], c, c, t, lens), lambda: muir.decode_step_attention(x, x, x, c, c, t, lens),
                lambda: muir.decode_step_attention(x[0], x[0], None, c, c, t, lens)):
        with pytest.raises((ValueError, TypeError)):
            bad()


HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_host_logic_is_clean_under_sanitizers(tmp_path):
    """The argument checks, and which rows, work items and cache rows the kernels take, under the address and undefined-behaviour sanitizers."""
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("needs g++ and the HIP runtime headers")
    csrc = os.path.join(ROOT, "gated_delta_rule_06_amd", "csrc")
    exe = tmp_path / "attention_driver"
    cmd = [cxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}", f"-I{csrc}",
           *[os.path.join(csrc, f) for f in ("api.cpp", "sizes.cpp", "attention_api.cpp", "attention_sizes.cpp")],
           os.path.join(HERE, "sanitize", "stub_kernels.cpp"), os.path.join(HERE, "sanitize", "attention_driver.cpp"), "-o", str(exe)]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-4000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=1"})
    assert out.returncode == 0 and out.stdout.startswith("0 failures"), out.stdout + out.stderr[-2000:]


@pytest.mark.parametrize("window", [0, 1, 5])
def test_oracle_gradients_are_the_forwards_derivative(window):
    g = torch.Generator().manual_seed(window)
    N, H, Hk, d = 14, 4, 2, 64
    q, k, v, do = (torch.randn(N, h, d, generator=g, dtype=torch.float64) for h in (H, Hk, Hk, H))
    where = oa.spans(N, [0, 3, 3, 11], [3, 0, 7])
    assert where == [(0, 3), (3, 0), (3, 7)]
    grads = oa.backward(q, k, v, do, where, window)
    r = [torch.randn(x.shape, generator=g, dtype=torch.float64) for x in (q, k, v)]
    loss = lambda e: (oa.forward(q + e * r[0], k + e * r[1], v + e * r[2], where, window)[0] * do).sum()  # noqa: E731
    want = (loss(1e-6) - loss(-1e-6)) / 2e-6
    assert abs(sum((grads[n] * x).sum() for n, x in zip("qkv", r)) - want) < 1e-6 * (1 + abs(want))


def test_oracle_step_continues_the_prompt():
    g = torch.Generator().manual_seed(4)
    T, H, Hk, d = 40, 4, 2, 64
    q, k, v = (torch.randn(T, h, d, generator=g) for h in (H, Hk, Hk))
    table = torch.tensor([[2, 0, 3]])
    kc, vc = oa.append(k[:-1], v[:-1], torch.zeros(4, Hk, 16, d), torch.zeros(4, Hk, 16, d), table, [(0, T - 1)])
    o, kc, vc, _ = oa.step(q[-1:], k[-1:], v[-1:], kc, vc, table, [T - 1], 20)
    assert torch.allclose(o[0], oa.forward(q, k, v, [(0, T)], 20)[0][-1], atol=1e-12)
    assert torch.equal(kc[0, :, 5], k[21]) and torch.equal(vc[3, :, 7], v[39])
