"""The layer operators' argument checks without a GPU: the C entry points refuse bad arguments on the host before
anything is launched, and the binding refuses host tensors."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_06_amd as muir

BASE, STRIDE = 1 << 40, 1 << 34


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * STRIDE + off)


BF, FL = muir.MUIR_BF16, muir.MUIR_F32


def call(name, names, args, over):
    args = dict(args)
    args.update(over)
    st = getattr(muir.lib(), name)(*[args[n] for n in names], None)
    return st, muir.last_error()


FWD = ["q", "k", "v", "a", "s0", "lens", "o", "s_out", "B", "T", "H", "Hk", "dk", "dv", "per", "dt", "ws", "wsb"]
FWD_ARGS = dict({n: fake(i) for i, n in enumerate(FWD[:8])}, B=2, T=1000, H=6, Hk=3, dk=64, dv=128, per=1, dt=BF,
                ws=fake(20), wsb=1 << 33)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), 2), (dict(T=-1), 2), (dict(H=0), 2), (dict(Hk=0), 2), (dict(Hk=4), 2), (dict(Hk=12), 2), (dict(dk=32), 3),
    (dict(dv=96), 3), (dict(dt=3), 3), (dict(B=1 << 21), 3), (dict(T=(1 << 31) - 1), 3), (dict(q=None), 1), (dict(a=None), 1),
    (dict(o=None), 1), (dict(ws=None), 4), (dict(wsb=100), 4), (dict(ws=fake(20, 16)), 4), (dict(q=fake(0, 8)), 2),
    (dict(a=fake(3, 2)), 2), (dict(lens=fake(5, 2)), 2), (dict(o=fake(2)), 5), (dict(o=fake(2, 4096)), 5),
    (dict(s_out=fake(4, 256)), 5), (dict(s_out=fake(0)), 5), (dict(ws=fake(7)), 5), (dict(o=fake(5)), 5), (dict(o=fake(7)), 5),
])
def test_forward_refusals(over, status):
    st, msg = call("muir_chunk_fwd_head_decay", FWD, FWD_ARGS, over)
    assert st == status and msg, msg


BWD = ["q", "k", "v", "a", "s0", "lens", "dout", "ds_out", "dq", "dk", "dv", "dla", "ds0", "B", "T", "H", "Hk", "DK", "DV",
       "per", "dt", "ws", "wsb"]
BWD_ARGS = dict({n: fake(i) for i, n in enumerate(BWD[:13])}, B=2, T=1000, H=6, Hk=3, DK=64, DV=128, per=1, dt=BF,
                ws=fake(20), wsb=1 << 33)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), 2), (dict(Hk=4), 2), (dict(DK=0), 3), (dict(dt=2), 3), (dict(dout=None), 1), (dict(dla=None), 1), (dict(dq=None), 1),
    (dict(ws=None), 4), (dict(wsb=64), 4), (dict(dv=fake(11)), 5), (dict(ds0=fake(7)), 5), (dict(dq=fake(0)), 5), (dict(dk=fake(8)), 5),
    (dict(dout=fake(6, 4)), 2), (dict(ws=fake(3)), 5), (dict(T=0, per=0, dla=None), 1),
])
def test_backward_refusals(over, status):
    st, msg = call("muir_chunk_bwd_head_decay", BWD, BWD_ARGS, over)
    assert st == status and msg, msg


def test_workspace_sizes():
    fwd, bwd = muir.chunk_fwd_head_decay_workspace_size, muir.chunk_bwd_head_decay_workspace_size
    assert fwd(1, 64, 2, 1, 64, 64, BF) == 0 and fwd(1, 32768, 16, 16, 128, 128, BF) > 0
    assert bwd(1, 64, 2, 1, 64, 64, BF) > bwd(1, 64, 2, 2, 64, 64, BF) > 0
    assert bwd(1, 0, 2, 2, 64, 64, BF) == 0
    for bad in [(0, 64, 2, 1, 64, 64, BF), (1, -1, 2, 1, 64, 64, BF), (1, 64, 3, 2, 64, 64, BF), (1, 64, 2, 1, 32, 64, BF),
                (1, 64, 2, 1, 64, 64, 9), (1 << 22, 64, 2, 1, 64, 64, BF)]:
        assert fwd(*bad) == 0 and bwd(*bad) == 0
    assert muir.rms_norm_bwd_workspace_size(0, 64) == 0 and muir.rms_norm_bwd_workspace_size(1, 12) == 0
    assert muir.rms_norm_bwd_workspace_size(5, 64) > 0


STEP = ["q", "k", "v", "a", "state", "o", "B", "H", "Hk", "dk", "dv", "per", "dt"]
STEP_ARGS = dict({n: fake(i) for i, n in enumerate(STEP[:6])}, B=2, H=6, Hk=3, dk=64, dv=128, per=1, dt=BF)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), 2), (dict(Hk=5), 2), (dict(dk=65), 3), (dict(dt=-1), 3), (dict(B=1 << 20), 3), (dict(state=None), 1), (dict(o=None), 1),
    (dict(o=fake(4, 64)), 5), (dict(state=fake(2)), 5), (dict(o=fake(0)), 5), (dict(state=fake(4, 8)), 2),
])
def test_step_refusals(over, status):
    st, msg = call("muir_decode_step_head_decay", STEP, STEP_ARGS, over)
    assert st == status and msg, msg


NORM = ["x", "residual", "weight", "h", "y", "rstd", "rows", "D", "eps", "xt", "ht"]
NORM_ARGS = dict({n: fake(i) for i, n in enumerate(NORM[:6])}, rows=10, D=64, eps=1e-6, xt=BF, ht=FL)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 2), (dict(D=0), 2), (dict(D=12), 3), (dict(D=16392), 3), (dict(rows=(1 << 23) + 1), 3), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(xt=FL, ht=BF), 3), (dict(xt=4), 3), (dict(h=None), 1),
    (dict(residual=None), 1), (dict(x=None), 1), (dict(weight=None), 1), (dict(y=None), 1), (dict(y=fake(0)), 5), (dict(h=fake(1, 64)), 5),
    (dict(h=fake(0)), 5), (dict(y=fake(3)), 5), (dict(x=fake(0, 2)), 2), (dict(rstd=fake(5, 2)), 2), (dict(rstd=fake(4)), 5),
])
def test_norm_refusals(over, status):
    st, msg = call("muir_rms_norm", NORM, NORM_ARGS, over)
    assert st == status and msg, msg


NORM8 = ["x", "residual", "weight", "h", "y", "scale", "rows", "D", "eps", "fmt", "group", "xt", "ht"]
NORM8_ARGS = dict({n: fake(i) for i, n in enumerate(NORM8[:6])}, rows=10, D=256, eps=1e-6, fmt=0, group=128, xt=BF, ht=BF)


@pytest.mark.parametrize("over,status", [
    (dict(fmt=2), 3), (dict(group=64), 3), (dict(group=-1), 3), (dict(D=192), 2), (dict(scale=None), 1), (dict(scale=fake(4)), 5),
    (dict(y=fake(1)), 5), (dict(rows=-5), 2), (dict(xt=FL), 3),
])
def test_norm_8bit_refusals(over, status):
    st, msg = call("muir_rms_norm_8bit", NORM8, NORM8_ARGS, over)
    assert st == status and msg, msg


NORMB = ["dy", "h", "weight", "rstd", "dh", "dx", "dweight", "rows", "D", "yt", "ht", "ws", "wsb"]
NORMB_ARGS = dict({n: fake(i) for i, n in enumerate(NORMB[:7])}, rows=10, D=64, yt=BF, ht=FL, ws=fake(20), wsb=1 << 30)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 2), (dict(D=4), 3), (dict(yt=FL, ht=BF), 3), (dict(dy=None), 1), (dict(dweight=None), 1), (dict(ws=None), 4),
    (dict(wsb=8), 4), (dict(dx=fake(0)), 5), (dict(dx=fake(4, 64)), 5), (dict(dweight=fake(2)), 5), (dict(ws=fake(1)), 5),
])
def test_norm_backward_refusals(over, status):
    st, msg = call("muir_rms_norm_bwd", NORMB, NORMB_ARGS, over)
    assert st == status and msg, msg


Q4 = ["x", "w", "scale", "zero", "y", "M", "N", "K", "group", "xt", "st"]
Q4_ARGS = dict({n: fake(i) for i, n in enumerate(Q4[:5])}, M=4, N=100, K=256, group=64, xt=BF, st=BF)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), 2), (dict(N=0), 2), (dict(K=0), 2), (dict(K=96), 2), (dict(group=16), 3), (dict(group=256), 3), (dict(M=65), 3),
    (dict(N=(1 << 26) + 1), 3), (dict(xt=7), 3), (dict(st=7), 3), (dict(x=None), 1), (dict(w=None), 1), (dict(scale=None), 1),
    (dict(y=None), 1), (dict(y=fake(0)), 5), (dict(y=fake(1, 128)), 5), (dict(w=fake(1, 4)), 2), (dict(scale=fake(2, 1)), 2),
])
def test_q4_refusals(over, status):
    st, msg = call("muir_matvec_q4", Q4, Q4_ARGS, over)
    assert st == status and msg, msg


def test_binding_refuses_host_tensors_and_bad_ranks():
    x = torch.zeros(1, 4, 2, 64)
    a = torch.ones(1, 4, 2)
    for bad in (lambda: muir.chunk_fwd_head_decay(x, x, x, a), lambda: muir.decode_step_head_decay(x[0], x[0], x[0], a[0], x),
                lambda: muir.chunk_bwd_head_decay(x, x, x, a, do=x), lambda: muir.chunk_fwd_head_decay(x[0], x, x, a),
                lambda: muir.rms_norm(x, torch.ones(64)), lambda: muir.rms_norm_bwd(x, x, torch.ones(64), a),
                lambda: muir.rms_norm_8bit(x, torch.ones(64), format="e5m2"), lambda: muir.matvec_q4(x, x, x),
                lambda: muir.matvec_q4(torch.zeros(1, 100), torch.zeros(4, 50, dtype=torch.uint8), x, group=64)):
        with pytest.raises((ValueError, TypeError)):
            bad()


HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_host_logic_is_clean_under_sanitizers(tmp_path):
    """The argument checks and sizes under the address and undefined-behaviour sanitizers, with launchers that count."""
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("needs g++ and the HIP runtime headers")
    csrc = os.path.join(ROOT, "gated_delta_rule_06_amd", "csrc")
    exe = tmp_path / "op_driver"
    cmd = [cxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{os.path.join(ROOT, 'include')}", f"-I{csrc}",
           *[os.path.join(csrc, f) for f in ("api.cpp", "sizes.cpp", "op_api.cpp", "op_sizes.cpp")],
           os.path.join(HERE, "sanitize", "stub_kernels.cpp"), os.path.join(HERE, "sanitize", "op_driver.cpp"), "-o", str(exe)]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-4000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env={**os.environ, "ASAN_OPTIONS": "detect_leaks=1"})
    assert out.returncode == 0 and out.stdout.startswith("0 failures"), out.stdout + out.stderr[-2000:]
