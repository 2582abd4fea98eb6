"""Python binding of libmuir: channel-wise gated delta-rule linear attention with
matched-filter readout (Muir), hand-written HIP kernels for AMD CDNA4 (gfx950).

The binding only marshals arguments: it checks tensor dtypes, shapes and devices,
allocates outputs and the workspace with PyTorch, passes raw device pointers and the
current HIP stream to the C ABI declared in ``include/muir.h``, and raises
``MuirError`` with the library's message on a non-zero status. Every step of the
computation runs in the library's kernels; there is no fallback. Importing works
without a GPU (argument validation can be exercised on the CPU), but the library
itself must be built (``python -m gated_delta_rule_06_amd._build``).
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "MuirError", "lib", "chunk_fwd", "chunk_fwd_workspace_size", "chunk_fwd_prepare",
    "chunk_fwd_scan", "chunk_fwd_scalar_erase", "chunk_fwd_scalar_erase_workspace_size",
    "chunk_fwd_scalar_erase_solve",
    "chunk_fwd_scalar_erase_scan", "lowrank_gates", "chunk_fwd_lowrank", "decode_step",
    "chunk_bwd", "chunk_bwd_workspace_size", "BWD_GRADS",
    "chunk_fwd_head_decay", "chunk_fwd_head_decay_workspace_size", "chunk_bwd_head_decay",
    "chunk_bwd_head_decay_workspace_size", "HEAD_DECAY_GRADS", "decode_step_head_decay",
    "rms_norm", "rms_norm_bwd", "rms_norm_bwd_workspace_size", "rms_norm_8bit", "matvec_q4",
    "status_string", "last_error", "version", "MUIR_F32", "MUIR_BF16", "STATUS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuir.so")

MUIR_F32, MUIR_BF16 = 0, 1
STATUS = {0: "MUIR_OK", 1: "MUIR_ERR_NULL", 2: "MUIR_ERR_SHAPE", 3: "MUIR_ERR_UNSUPPORTED",
          4: "MUIR_ERR_WORKSPACE", 5: "MUIR_ERR_ALIAS", 6: "MUIR_ERR_HIP"}


class MuirError(RuntimeError):
    """A libmuir call returned a non-zero status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib():
    """The loaded ``libmuir.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m gated_delta_rule_06_amd._build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.muir_chunk_fwd_workspace_size.argtypes = [i] * 6 + [i]
        L.muir_chunk_fwd_workspace_size.restype = sz
        L.muir_chunk_fwd.argtypes = [vp] * 11 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd.restype = i
        L.muir_chunk_fwd_noalloc.argtypes = [vp] * 11 + [i] * 7 + [vp]
        L.muir_chunk_fwd_noalloc.restype = i
        L.muir_chunk_fwd_noalloc_max_workspace.argtypes = []
        L.muir_chunk_fwd_noalloc_max_workspace.restype = sz
        L.muir_chunk_fwd_prepare.argtypes = [vp] * 5 + [i] * 6 + [vp, sz, vp]
        L.muir_chunk_fwd_prepare.restype = i
        L.muir_chunk_fwd_scan.argtypes = [vp] * 6 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_scan.restype = i
        L.muir_chunk_fwd_gated.argtypes = [vp] * 12 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_gated.restype = i
        L.muir_chunk_fwd_scan_gated.argtypes = [vp] * 7 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_scan_gated.restype = i
        L.muir_chunk_fwd_scalar_erase.argtypes = [vp] * 11 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_scalar_erase.restype = i
        L.muir_chunk_fwd_scalar_erase_workspace_size.argtypes = [i] * 6
        L.muir_chunk_fwd_scalar_erase_workspace_size.restype = sz
        L.muir_chunk_fwd_scalar_erase_solve.argtypes = [vp] * 3 + [i] * 6 + [vp, sz, vp]
        L.muir_chunk_fwd_scalar_erase_solve.restype = i
        L.muir_chunk_fwd_scalar_erase_scan.argtypes = [vp] * 3 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_scalar_erase_scan.restype = i
        L.muir_chunk_fwd_lowrank_workspace_size.argtypes = [i] * 6
        L.muir_chunk_fwd_lowrank_workspace_size.restype = sz
        L.muir_chunk_fwd_lowrank.argtypes = [vp] * 16 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_lowrank.restype = i
        L.muir_lowrank_gates.argtypes = [vp] * 13 + [i] * 4 + [vp]
        L.muir_lowrank_gates.restype = i
        L.muir_lowrank_output_gate.argtypes = [vp] * 4 + [i] * 4 + [vp]
        L.muir_lowrank_output_gate.restype = i
        L.muir_chunk_fwd_lowrank_gated_workspace_size.argtypes = [i] * 6
        L.muir_chunk_fwd_lowrank_gated_workspace_size.restype = sz
        L.muir_chunk_fwd_lowrank_gated.argtypes = [vp] * 18 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_fwd_lowrank_gated.restype = i
        L.muir_chunk_bwd_workspace_size.argtypes = [i] * 7
        L.muir_chunk_bwd_workspace_size.restype = sz
        L.muir_chunk_bwd.argtypes = [vp] * 20 + [i] * 7 + [vp, sz, vp]
        L.muir_chunk_bwd.restype = i
        L.muir_decode_step.argtypes = [vp] * 10 + [i] * 5 + [vp]
        L.muir_decode_step.restype = i
        f = ctypes.c_float
        L.muir_chunk_fwd_head_decay_workspace_size.argtypes = [i] * 7
        L.muir_chunk_fwd_head_decay_workspace_size.restype = sz
        L.muir_chunk_fwd_head_decay.argtypes = [vp] * 8 + [i] * 8 + [vp, sz, vp]
        L.muir_chunk_fwd_head_decay.restype = i
        L.muir_chunk_bwd_head_decay_workspace_size.argtypes = [i] * 7
        L.muir_chunk_bwd_head_decay_workspace_size.restype = sz
        L.muir_chunk_bwd_head_decay.argtypes = [vp] * 13 + [i] * 8 + [vp, sz, vp]
        L.muir_chunk_bwd_head_decay.restype = i
        L.muir_decode_step_head_decay.argtypes = [vp] * 6 + [i] * 7 + [vp]
        L.muir_decode_step_head_decay.restype = i
        L.muir_rms_norm.argtypes = [vp] * 6 + [i, i, f, i, i, vp]
        L.muir_rms_norm.restype = i
        L.muir_rms_norm_bwd_workspace_size.argtypes = [i, i]
        L.muir_rms_norm_bwd_workspace_size.restype = sz
        L.muir_rms_norm_bwd.argtypes = [vp] * 7 + [i] * 4 + [vp, sz, vp]
        L.muir_rms_norm_bwd.restype = i
        L.muir_rms_norm_8bit.argtypes = [vp] * 6 + [i, i, f, i, i, i, i, vp]
        L.muir_rms_norm_8bit.restype = i
        L.muir_matvec_q4.argtypes = [vp] * 5 + [i] * 6 + [vp]
        L.muir_matvec_q4.restype = i
        L.muir_status_string.argtypes = [i]
        L.muir_status_string.restype = ctypes.c_char_p
        L.muir_last_error.argtypes = []
        L.muir_last_error.restype = ctypes.c_char_p
        L.muir_version.argtypes = []
        L.muir_version.restype = i
        L.muir_state_bytes.argtypes = [i] * 4
        L.muir_state_bytes.restype = sz
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().muir_status_string(int(status)).decode()


def last_error() -> str:
    return lib().muir_last_error().decode()


def version() -> int:
    return int(lib().muir_version())


def state_bytes(B: int, H: int, dk: int, dv: int) -> int:
    """Bytes of the fp32 recurrent state of B sequences x H heads (``muir_state_bytes``)."""
    return int(lib().muir_state_bytes(B, H, dk, dv))


def _check(status: int):
    if status != 0:
        raise MuirError(status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    import torch
    if device.type != "cuda":
        return None
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return MUIR_F32
    if t.dtype == torch.bfloat16:
        return MUIR_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _require(t, name, dtype=None, shape=None, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (the library has no host path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def chunk_fwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int, chunk: int,
                             dtype_code: int) -> int:
    return int(lib().muir_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, dtype_code))


def chunk_fwd(q, k, v, a, g, e, w, r, s0=None, *, chunk: int = 64, o=None, s_out=None,
              return_state: bool = True, workspace=None, og=None):
    """Chunkwise forward over whole sequences (``muir_chunk_fwd``).

    q, k [B,T,H,dk] and v [B,T,H,dv] in float32 or bfloat16 (same dtype); a, g
    [B,T,H,dk], e, w [B,T,H,dv] and r [H,dk] float32; s0 [B,H,dk,dv] float32 or None.
    Returns (o, s_out): o [B,T,H,dv] in the q/k/v dtype and the final state (or None
    with ``return_state=False``). ``s_out`` may be passed (it may be ``s0`` itself for
    an in-place update); ``workspace`` may be a pre-allocated uint8 device tensor.
    With ``og`` ([B,T,H,dv] float32) the output-gate epilogue runs
    (``muir_chunk_fwd_gated``): o is multiplied by og elementwise as it is stored.
    """
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, q.dtype, (B, T, H, dk if name != "v" else dv), dev)
    for name, t, d in (("a", a, dk), ("g", g, dk), ("e", e, dv), ("w", w, dv)):
        _require(t, name, torch.float32, (B, T, H, d), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    if s0 is not None:
        _require(s0, "s0", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    else:
        _require(o, "o", q.dtype, (B, T, H, dv), dev)
    if s_out is None and return_state:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    elif s_out is not None:
        _require(s_out, "s_out", torch.float32, (B, H, dk, dv), dev)
    need = chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _require(workspace, "workspace", torch.uint8, None, dev)
    if og is None:
        status = lib().muir_chunk_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(g), _ptr(e), _ptr(w), _ptr(r), _ptr(s0),
            _ptr(o), _ptr(s_out), B, T, H, dk, dv, chunk, code, _ptr(workspace),
            workspace.numel(), _stream(dev))
    else:
        _require(og, "og", torch.float32, (B, T, H, dv), dev)
        status = lib().muir_chunk_fwd_gated(
            _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(g), _ptr(e), _ptr(w), _ptr(og), _ptr(r),
            _ptr(s0), _ptr(o), _ptr(s_out), B, T, H, dk, dv, chunk, code, _ptr(workspace),
            workspace.numel(), _stream(dev))
    _check(status)
    return o, s_out


def chunk_bwd_workspace_size(B: int, T: int, H: int, dk: int, dv: int, chunk: int,
                            dtype_code: int) -> int:
    return int(lib().muir_chunk_bwd_workspace_size(B, T, H, dk, dv, chunk, dtype_code))


BWD_GRADS = ("q", "k", "v", "la", "g", "e", "w", "r", "s0")


def chunk_bwd(q, k, v, a, g, e, w, r, s0=None, *, do, ds_out=None, chunk: int = 64,
              workspace=None, out=None):
    """Backward pass of ``chunk_fwd`` (``muir_chunk_bwd``).

    Inputs as for ``chunk_fwd``, plus ``do`` (dL/do, [B,T,H,dv], the q/k/v dtype) and
    ``ds_out`` (dL/ds_out, [B,H,dk,dv] float32 or None). Returns a dict of float32
    gradients keyed by ``BWD_GRADS``: "la" is a * dL/da, "r" is [H,dk], "s0" is
    [B,H,dk,dv]. ``out`` may hold pre-allocated tensors under those keys.
    """
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        _require(t, name, q.dtype, (B, T, H, dk if name in ("q", "k") else dv), dev)
    for name, t, d in (("a", a, dk), ("g", g, dk), ("e", e, dv), ("w", w, dv)):
        _require(t, name, torch.float32, (B, T, H, d), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    for name, t in (("s0", s0), ("ds_out", ds_out)):
        if t is not None:
            _require(t, name, torch.float32, (B, H, dk, dv), dev)
    shapes = {n: (B, T, H, dk if n in ("q", "k", "la", "g") else dv) for n in BWD_GRADS}
    shapes["r"] = (H, dk)
    shapes["s0"] = (B, H, dk, dv)
    out = dict(out or {})
    for n, shp in shapes.items():
        if n in out:
            _require(out[n], "d" + n, torch.float32, shp, dev)
        else:
            out[n] = torch.empty(shp, dtype=torch.float32, device=dev)
    need = chunk_bwd_workspace_size(B, T, H, dk, dv, chunk, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _require(workspace, "workspace", torch.uint8, None, dev)
    status = lib().muir_chunk_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(g), _ptr(e), _ptr(w), _ptr(r), _ptr(s0),
        _ptr(do), _ptr(ds_out), *[_ptr(out[n]) for n in BWD_GRADS],
        B, T, H, dk, dv, chunk, code, _ptr(workspace), workspace.numel(), _stream(dev))
    _check(status)
    return out


def chunk_fwd_prepare(q, k, a, g, r, *, chunk: int, workspace):
    """Parallel phase of the chunk forward (``muir_chunk_fwd_prepare``) into ``workspace``."""
    import torch
    B, T, H, dk = q.shape
    dev = q.device
    code = _dtype_code(q)
    _require(q, "q", q.dtype, (B, T, H, dk), dev)
    _require(k, "k", q.dtype, (B, T, H, dk), dev)
    for name, t in (("a", a), ("g", g)):
        _require(t, name, torch.float32, (B, T, H, dk), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    _require(workspace, "workspace", torch.uint8, None, dev)
    _check(lib().muir_chunk_fwd_prepare(
        _ptr(q), _ptr(k), _ptr(a), _ptr(g), _ptr(r), B, T, H, dk, chunk, code,
        _ptr(workspace), workspace.numel(), _stream(dev)))


def chunk_fwd_scan(v, e, w, s0=None, *, chunk: int, workspace, o, s_out=None, og=None):
    """Sequential phase of the chunk forward (``muir_chunk_fwd_scan``) from ``workspace``;
    with ``og`` the output-gate epilogue (``muir_chunk_fwd_scan_gated``)."""
    import torch
    B, T, H, dv = v.shape
    dev = v.device
    code = _dtype_code(v)
    for name, t in (("e", e), ("w", w)):
        _require(t, name, torch.float32, (B, T, H, dv), dev)
    _require(o, "o", v.dtype, (B, T, H, dv), dev)
    if s0 is not None:
        _require(s0, "s0", torch.float32, (B, H, dv, dv), dev)
    if s_out is not None:
        _require(s_out, "s_out", torch.float32, (B, H, dv, dv), dev)
    _require(workspace, "workspace", torch.uint8, None, dev)
    if og is None:
        _check(lib().muir_chunk_fwd_scan(
            _ptr(v), _ptr(e), _ptr(w), _ptr(s0), _ptr(o), _ptr(s_out), B, T, H, dv, dv, chunk,
            code, _ptr(workspace), workspace.numel(), _stream(dev)))
    else:
        _require(og, "og", torch.float32, (B, T, H, dv), dev)
        _check(lib().muir_chunk_fwd_scan_gated(
            _ptr(v), _ptr(e), _ptr(w), _ptr(og), _ptr(s0), _ptr(o), _ptr(s_out), B, T, H, dv,
            dv, chunk, code, _ptr(workspace), workspace.numel(), _stream(dev)))


def chunk_fwd_scalar_erase_workspace_size(B: int, T: int, H: int, dk: int, dv: int,
                                          chunk: int) -> int:
    return int(lib().muir_chunk_fwd_scalar_erase_workspace_size(B, T, H, dk, dv, chunk))


def chunk_fwd_scalar_erase(q, k, v, a, g, e, w, r, s0=None, *, chunk: int = 256, o=None,
                           s_out=None, return_state: bool = True, workspace=None):
    """Chunk forward with one erase strength per token (``muir_chunk_fwd_scalar_erase``).

    As :func:`chunk_fwd` (bfloat16 q/k/v only) except ``e`` is [B,T,H] float32: the
    result equals the channel-wise forward with e broadcast over the value channels.
    Returns (o, s_out). ``workspace`` (uint8, at least
    :func:`chunk_fwd_scalar_erase_workspace_size` bytes) may be passed.
    """
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    code = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, q.dtype, (B, T, H, dk if name != "v" else dv), dev)
    for name, t, d in (("a", a, dk), ("g", g, dk), ("w", w, dv)):
        _require(t, name, torch.float32, (B, T, H, d), dev)
    _require(e, "e", torch.float32, (B, T, H), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    if s0 is not None:
        _require(s0, "s0", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    else:
        _require(o, "o", q.dtype, (B, T, H, dv), dev)
    if s_out is None and return_state:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    elif s_out is not None:
        _require(s_out, "s_out", torch.float32, (B, H, dk, dv), dev)
    need = chunk_fwd_scalar_erase_workspace_size(B, T, H, dk, dv, chunk)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    else:
        _require(workspace, "workspace", torch.uint8, None, dev)
    _check(lib().muir_chunk_fwd_scalar_erase(
        _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(g), _ptr(e), _ptr(w), _ptr(r), _ptr(s0),
        _ptr(o), _ptr(s_out), B, T, H, dk, dv, chunk, code, _ptr(workspace),
        workspace.numel(), _stream(dev)))
    return o, s_out


def chunk_fwd_scalar_erase_solve(v, e, w, *, chunk: int, workspace):
    """The chunk-parallel phase (``muir_chunk_fwd_scalar_erase_solve``) on a workspace that
    :func:`chunk_fwd_prepare` (bf16 q/k/v) filled: the inverse, then the per-chunk products.
    Run it once per prepare."""
    import torch
    B, T, H, dv = v.shape
    dev = v.device
    _require(v, "v", torch.bfloat16, (B, T, H, dv), dev)
    _require(e, "e", torch.float32, (B, T, H), dev)
    _require(w, "w", torch.float32, (B, T, H, dv), dev)
    _require(workspace, "workspace", torch.uint8, None, dev)
    _check(lib().muir_chunk_fwd_scalar_erase_solve(
        _ptr(v), _ptr(e), _ptr(w), B, T, H, dv, chunk, MUIR_BF16, _ptr(workspace),
        workspace.numel(), _stream(dev)))


def chunk_fwd_scalar_erase_scan(s0=None, *, B: int, T: int, H: int, d: int, chunk: int,
                                workspace, o, s_out=None):
    """The sequential phase and the readout (``muir_chunk_fwd_scalar_erase_scan``) from a
    solved workspace; o [B,T,H,d] bfloat16 is written."""
    import torch
    dev = o.device
    _require(o, "o", torch.bfloat16, (B, T, H, d), dev)
    if s0 is not None:
        _require(s0, "s0", torch.float32, (B, H, d, d), dev)
    if s_out is not None:
        _require(s_out, "s_out", torch.float32, (B, H, d, d), dev)
    _require(workspace, "workspace", torch.uint8, None, dev)
    _check(lib().muir_chunk_fwd_scalar_erase_scan(
        _ptr(s0), _ptr(o), _ptr(s_out), B, T, H, d, d, chunk, MUIR_BF16, _ptr(workspace),
        workspace.numel(), _stream(dev)))


def lowrank_gates(z, U, c, *, H: int, d: int, which=("a", "e", "w", "g"), out=None):
    """Gates from the fused low-rank projection (``muir_lowrank_gates``).

    z [B,T,512] bfloat16; U a dict of up-projections {"decay": [H,d,64], "erase": [H,d,64],
    "write": [H,d,128], "read": [H,d,128]} bfloat16 and c the matching offsets [H,d]
    float32. Returns a dict of the requested gates among a (decay), e, w, g, each
    [B,T,H,d] float32 (``out`` may supply them)."""
    import torch
    B, T, R = z.shape
    dev = z.device
    _require(z, "z", torch.bfloat16, (B, T, 512), dev)
    names = {"a": ("decay", 64), "e": ("erase", 64), "w": ("write", 128), "g": ("read", 128)}
    out = dict(out or {})
    args = []
    for gname in ("a", "e", "w", "g"):
        n, r = names[gname]
        if gname in which:
            _require(U[n], "U_" + n, torch.bfloat16, (H, d, r), dev)
            _require(c[n], "c_" + n, torch.float32, (H, d), dev)
            if gname not in out:
                out[gname] = torch.empty((B, T, H, d), dtype=torch.float32, device=dev)
            _require(out[gname], gname, torch.float32, (B, T, H, d), dev)
            args.append((U[n], c[n], out[gname]))
        else:
            args.append((None, None, None))
    _check(lib().muir_lowrank_gates(
        _ptr(z), *[_ptr(x[0]) for x in args], *[_ptr(x[1]) for x in args],
        *[_ptr(x[2]) for x in args], B, T, H, d, _stream(dev)))
    return {k: v for k, v in out.items() if k in which}


def _chunk_fwd_lowrank(q, k, v, z, U, c, r, s0, chunk, o, s_out, return_state, workspace,
                       gated: bool):
    import torch
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, torch.bfloat16, (B, T, H, dk if name != "v" else dv), dev)
    _require(z, "z", torch.bfloat16, (B, T, 512), dev)
    names = ("decay", "erase", "write", "read") + (("output",) if gated else ())
    for n in names:
        _require(U[n], "U_" + n, torch.bfloat16, (H, dk, 64 if n in ("decay", "erase") else 128), dev)
        _require(c[n], "c_" + n, torch.float32, (H, dk), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    if s0 is not None:
        _require(s0, "s0", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    if s_out is None and return_state:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    size = (lib().muir_chunk_fwd_lowrank_gated_workspace_size if gated
            else lib().muir_chunk_fwd_lowrank_workspace_size)
    need = int(size(B, T, H, dk, dv, chunk))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    ups = [_ptr(U[n]) for n in ("decay", "erase", "write", "read")]
    offs = [_ptr(c[n]) for n in ("decay", "erase", "write", "read")]
    tail = (_ptr(r), _ptr(s0), _ptr(o), _ptr(s_out), B, T, H, dk, dv, chunk, MUIR_BF16,
            _ptr(workspace), workspace.numel(), _stream(dev))
    if gated:
        _check(lib().muir_chunk_fwd_lowrank_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(z), *ups,
                                                  _ptr(U["output"]), *offs, _ptr(c["output"]), *tail))
    else:
        _check(lib().muir_chunk_fwd_lowrank(_ptr(q), _ptr(k), _ptr(v), _ptr(z), *ups, *offs, *tail))
    return o, s_out


def chunk_fwd_lowrank(q, k, v, z, U, c, r, s0=None, *, chunk: int = 256, o=None, s_out=None,
                      return_state: bool = True, workspace=None):
    """Chunk forward with the gates made from the low-rank gate projection inside the call
    (``muir_chunk_fwd_lowrank``). q, k, v bfloat16 as for :func:`chunk_fwd`; z, U, c as for
    :func:`lowrank_gates` (all four gates). Returns (o, s_out)."""
    return _chunk_fwd_lowrank(q, k, v, z, U, c, r, s0, chunk, o, s_out, return_state, workspace,
                              False)


def chunk_fwd_lowrank_gated(q, k, v, z, U, c, r, s0=None, *, chunk: int = 256, o=None,
                            s_out=None, return_state: bool = True, workspace=None):
    """As :func:`chunk_fwd_lowrank` with the output gate too (``muir_chunk_fwd_lowrank_gated``):
    U and c also hold "output" ([H, d, 128] bf16, [H, d] fp32); the readout is o * og."""
    return _chunk_fwd_lowrank(q, k, v, z, U, c, r, s0, chunk, o, s_out, return_state, workspace,
                              True)


def lowrank_output_gate(z, Uo, co, *, out=None):
    """The output gate og [B, T, H, d] fp32 from z's output slice (``muir_lowrank_output_gate``):
    z [B, T, 512] bf16, Uo [H, d, 128] bf16, co [H, d] fp32."""
    import torch
    B, T, _ = z.shape
    H, d, _ = Uo.shape
    dev = z.device
    _require(z, "z", torch.bfloat16, (B, T, 512), dev)
    _require(Uo, "Uo", torch.bfloat16, (H, d, 128), dev)
    _require(co, "co", torch.float32, (H, d), dev)
    if out is None:
        out = torch.empty((B, T, H, d), dtype=torch.float32, device=dev)
    _require(out, "og", torch.float32, (B, T, H, d), dev)
    _check(lib().muir_lowrank_output_gate(_ptr(z), _ptr(Uo), _ptr(co), _ptr(out), B, T, H, d,
                                          _stream(dev)))
    return out


def decode_step(q, k, v, a, g, e, w, r, state, *, o=None):
    """One recurrent step per (batch, head), updating ``state`` in place.

    q, k [B,H,dk], v [B,H,dv] (float32 or bfloat16); a, g [B,H,dk], e, w [B,H,dv],
    r [H,dk] float32; state [B,H,dk,dv] float32. Returns o [B,H,dv] (q/k/v dtype).
    """
    import torch
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    code = _dtype_code(q)
    for name, t, d in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        _require(t, name, q.dtype, (B, H, d), dev)
    for name, t, d in (("a", a, dk), ("g", g, dk), ("e", e, dv), ("w", w, dv)):
        _require(t, name, torch.float32, (B, H, d), dev)
    _require(r, "r", torch.float32, (H, dk), dev)
    _require(state, "state", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=dev)
    else:
        _require(o, "o", q.dtype, (B, H, dv), dev)
    status = lib().muir_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(g), _ptr(e), _ptr(w), _ptr(r),
        _ptr(state), _ptr(o), B, H, dk, dv, code, _stream(dev))
    _check(status)
    return o


# The layer operators below are called once per token and layer: their checks are one expression per tensor, and the
# message is made only when it is false.

def _is(t, name, dtype, shape, index):
    """``t`` is a contiguous GPU tensor of this type and shape on device ``index`` (or the error says what is not)."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == index and index >= 0
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    import torch
    _require(t, name, dtype, shape, torch.device("cuda", max(index, 0)))


def _call(fn, index, *args):
    """One library call on device ``index``'s current stream, with that device current."""
    import torch
    if index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        raise MuirError(status, last_error())


def _at(t):
    return None if t is None else t.data_ptr()


def _out(t, name, dtype, shape, like):
    """``t`` checked as an output beside ``like``, or a new tensor."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _is(t, name, dtype, shape, like.get_device())
    return t


def _workspace(t, need, like):
    """(pointer's tensor, bytes): ``t`` checked, a new one, or none where none is needed."""
    import torch
    if t is None:
        return (torch.empty(need, dtype=torch.uint8, device=like.device), need) if need else (None, 0)
    _is(t, "workspace", torch.uint8, t.shape, like.get_device())
    return t, t.numel()


def _rank(t, name, n):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")


def _head_decay_inputs(q, k, v, a, s0, lens):
    import torch
    _rank(q, "q", 4)
    _rank(v, "v", 4)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    i, dt = q.get_device(), q.dtype
    _is(q, "q", dt, (B, T, Hk, dk), i)
    _is(k, "k", dt, (B, T, Hk, dk), i)
    _is(v, "v", dt, (B, T, H, dv), i)
    code = _dtype_code(q)
    _rank(a, "a", 1 if getattr(a, "ndim", 3) == 1 else 3)
    per_token = a.ndim == 3
    _is(a, "a", torch.float32, (B, T, H) if per_token else (H,), i)
    if s0 is not None:
        _is(s0, "s0", torch.float32, (B, H, dk, dv), i)
    if lens is not None:
        _is(lens, "lens", torch.int32, (B,), i)
    return (B, T, H, Hk, dk, dv), int(per_token), code, i


@functools.lru_cache(maxsize=256)
def chunk_fwd_head_decay_workspace_size(B: int, T: int, H: int, Hk: int, dk: int, dv: int,
                                        dtype_code: int) -> int:
    return int(lib().muir_chunk_fwd_head_decay_workspace_size(B, T, H, Hk, dk, dv, dtype_code))


def chunk_fwd_head_decay(q, k, v, a, s0=None, *, lens=None, o=None, s_out=None,
                         return_state: bool = True, workspace=None):
    """Linear attention with one decay per head over whole sequences
    (``muir_chunk_fwd_head_decay``): S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

    q, k [B,T,Hk,dk] and v [B,T,H,dv] in float32 or bfloat16 (same dtype), each key head
    shared by H / Hk value heads; a [B,T,H] or [H] float32 in [0, 1]; s0 [B,H,dk,dv]
    float32 or None; lens [B] int32 or None: the tokens of each sequence, those behind
    are not read and their rows of o are zeros. Returns (o, s_out): o [B,T,H,dv] and the
    state after each sequence's last token (None with ``return_state=False``). ``s_out``
    may be ``s0`` itself. A NaN or infinity in a token can reach every output of its chunk of
    64 tokens, earlier ones too.
    """
    import torch
    sizes, per_token, code, i = _head_decay_inputs(q, k, v, a, s0, lens)
    B, T, H, Hk, dk, dv = sizes
    o = _out(o, "o", q.dtype, (B, T, H, dv), q)
    if s_out is not None or return_state:
        s_out = _out(s_out, "s_out", torch.float32, (B, H, dk, dv), q)
    workspace, size = _workspace(workspace, chunk_fwd_head_decay_workspace_size(*sizes, code), q)
    _call(lib().muir_chunk_fwd_head_decay, i, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          a.data_ptr(), _at(s0), _at(lens), o.data_ptr(), _at(s_out), B, T, H, Hk, dk, dv,
          per_token, code, _at(workspace), size)
    return o, s_out


@functools.lru_cache(maxsize=256)
def chunk_bwd_head_decay_workspace_size(B: int, T: int, H: int, Hk: int, dk: int, dv: int,
                                        dtype_code: int) -> int:
    return int(lib().muir_chunk_bwd_head_decay_workspace_size(B, T, H, Hk, dk, dv, dtype_code))


HEAD_DECAY_GRADS = ("q", "k", "v", "la", "s0")


def chunk_bwd_head_decay(q, k, v, a, s0=None, *, do, ds_out=None, lens=None, workspace=None,
                         out=None):
    """Backward pass of :func:`chunk_fwd_head_decay` (``muir_chunk_bwd_head_decay``).

    Inputs as for the forward, plus ``do`` (dL/do, [B,T,H,dv], the q/k/v dtype) and
    ``ds_out`` (dL/ds_out, [B,H,dk,dv] float32 or None). Returns a dict keyed by
    ``HEAD_DECAY_GRADS``: "q", "k" and "v" shaped and typed as the inputs (shared heads
    summed), "la" = a * dL/da float32 shaped as a, "s0" [B,H,dk,dv] float32. Gradients of
    tokens behind ``lens`` are zeros. ``out`` may hold pre-allocated tensors under those keys.
    """
    import torch
    sizes, per_token, code, i = _head_decay_inputs(q, k, v, a, s0, lens)
    B, T, H, Hk, dk, dv = sizes
    f32 = torch.float32
    _is(do, "do", q.dtype, (B, T, H, dv), i)
    if ds_out is not None:
        _is(ds_out, "ds_out", f32, (B, H, dk, dv), i)
    out = dict(out) if out else {}
    for n, dtype, shape in (("q", q.dtype, q.shape), ("k", q.dtype, k.shape),
                            ("v", q.dtype, v.shape), ("la", f32, a.shape),
                            ("s0", f32, (B, H, dk, dv))):
        out[n] = _out(out.get(n), "d" + n, dtype, shape, q)
    workspace, size = _workspace(workspace, chunk_bwd_head_decay_workspace_size(*sizes, code), q)
    _call(lib().muir_chunk_bwd_head_decay, i, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          a.data_ptr(), _at(s0), _at(lens), do.data_ptr(), _at(ds_out),
          *[out[n].data_ptr() for n in HEAD_DECAY_GRADS], B, T, H, Hk, dk, dv, per_token, code,
          _at(workspace), size)
    return out


def decode_step_head_decay(q, k, v, a, state, *, o=None):
    """One token of :func:`chunk_fwd_head_decay`'s recurrence, updating ``state`` in place
    (``muir_decode_step_head_decay``).

    q, k [B,Hk,dk], v [B,H,dv] (float32 or bfloat16); a [B,H] or [H] float32; state
    [B,H,dk,dv] float32. Returns o [B,H,dv] (q/k/v dtype).
    """
    import torch
    _rank(q, "q", 3)
    _rank(v, "v", 3)
    B, Hk, dk = q.shape
    _, H, dv = v.shape
    i, dt = q.get_device(), q.dtype
    _is(q, "q", dt, (B, Hk, dk), i)
    _is(k, "k", dt, (B, Hk, dk), i)
    _is(v, "v", dt, (B, H, dv), i)
    code = _dtype_code(q)
    _rank(a, "a", 1 if getattr(a, "ndim", 2) == 1 else 2)
    per_token = a.ndim == 2
    _is(a, "a", torch.float32, (B, H) if per_token else (H,), i)
    _is(state, "state", torch.float32, (B, H, dk, dv), i)
    if o is None:
        o = torch.empty_like(v)
    else:
        _is(o, "o", dt, (B, H, dv), i)
    _call(lib().muir_decode_step_head_decay, i, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          a.data_ptr(), state.data_ptr(), o.data_ptr(), B, H, Hk, dk, dv, per_token, code)
    return o


def _norm_inputs(x, weight, residual, h):
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a torch.Tensor with at least one dimension")
    shape, i = x.shape, x.get_device()
    D = shape[-1]
    code = hcode = _dtype_code(x)
    _is(x, "x", x.dtype, shape, i)
    _is(weight, "weight", torch.float32, (D,), i)
    if residual is not None:
        _is(residual, "residual", getattr(residual, "dtype", None), shape, i)
        hcode = _dtype_code(residual)
        if h is None:
            h = torch.empty_like(residual)
        else:
            _is(h, "h", residual.dtype, shape, i)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    return x.numel() // D if D else 0, D, i, code, hcode, h


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6, y=None, h=None):
    """Root-mean-square norm over the last dimension with the residual's addition
    (``muir_rms_norm``): h = x + residual, y = h / rms(h) * weight.

    x [..., D] float32 or bfloat16; weight [D] float32; residual like x, or float32 beside
    bfloat16 x, or None. Returns (y, h, rstd): y like x, h like residual (x itself without
    one), rstd [...] float32, which :func:`rms_norm_bwd` takes. ``h`` may be ``residual``
    itself (in place).
    """
    import torch
    rows, D, i, code, hcode, h = _norm_inputs(x, weight, residual, h)
    if y is None:
        y = torch.empty_like(x)
    else:
        _is(y, "y", x.dtype, x.shape, i)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _call(lib().muir_rms_norm, i, x.data_ptr(), _at(residual), weight.data_ptr(), _at(h),
          y.data_ptr(), rstd.data_ptr(), rows, D, eps, code, hcode)
    return y, x if residual is None else h, rstd


@functools.lru_cache(maxsize=256)
def rms_norm_bwd_workspace_size(rows: int, D: int) -> int:
    return int(lib().muir_rms_norm_bwd_workspace_size(rows, D))


def rms_norm_bwd(dy, h, weight, rstd, *, dh=None, dx=None, dweight=None, workspace=None):
    """Backward pass of :func:`rms_norm` (``muir_rms_norm_bwd``).

    dy [..., D] in y's dtype; h and rstd from the forward; ``dh`` the gradient that reaches h
    from the residual stream, in h's dtype, or None. Returns (dx, dweight): dx in h's dtype,
    the gradient of x and of the residual alike, and dweight [D] float32. ``dx`` may be
    ``dh`` itself.
    """
    import torch
    if not isinstance(h, torch.Tensor) or h.dim() < 1:
        raise TypeError("h must be a torch.Tensor with at least one dimension")
    shape, i = h.shape, h.get_device()
    D = shape[-1]
    rows = h.numel() // D if D else 0
    hcode = _dtype_code(h)
    _is(h, "h", h.dtype, shape, i)
    _is(dy, "dy", getattr(dy, "dtype", None), shape, i)
    code = _dtype_code(dy)
    _is(weight, "weight", torch.float32, (D,), i)
    _is(rstd, "rstd", torch.float32, shape[:-1], i)
    if dh is not None:
        _is(dh, "dh", h.dtype, shape, i)
    dx = _out(dx, "dx", h.dtype, shape, h)
    dweight = _out(dweight, "dweight", torch.float32, (D,), h)
    workspace, size = _workspace(workspace, rms_norm_bwd_workspace_size(rows, D), h)
    _call(lib().muir_rms_norm_bwd, i, dy.data_ptr(), h.data_ptr(), weight.data_ptr(),
          rstd.data_ptr(), _at(dh), dx.data_ptr(), dweight.data_ptr(), rows, D, code, hcode,
          _at(workspace), size)
    return dx, dweight


def rms_norm_8bit(x, weight, residual=None, *, eps: float = 1e-6, format: str = "e4m3",
                  group: int = 0, y=None, scale=None, h=None):
    """:func:`rms_norm` with its output in 8 bits (``muir_rms_norm_8bit``).

    ``format`` "e4m3" (torch.float8_e4m3fn) or "int8"; one float32 scale for each row
    (``group=0``) or each 128 columns (``group=128``). Returns (y, scale, h): the 8-bit
    values [..., D], scale [...] or [..., D / 128] with y * scale the normed rows, and h as
    :func:`rms_norm`.
    """
    import torch
    if format == "e4m3":
        fmt, dtype = 0, torch.float8_e4m3fn
    elif format == "int8":
        fmt, dtype = 1, torch.int8
    else:
        raise ValueError(f'format must be "e4m3" or "int8", got {format!r}')
    rows, D, i, code, hcode, h = _norm_inputs(x, weight, residual, h)
    y = _out(y, "y", dtype, x.shape, x)
    shape = x.shape[:-1] + ((D // group,) if group > 0 else ())
    scale = _out(scale, "scale", torch.float32, shape, x)
    _call(lib().muir_rms_norm_8bit, i, x.data_ptr(), _at(residual), weight.data_ptr(), _at(h),
          y.data_ptr(), scale.data_ptr(), rows, D, eps, fmt, group, code, hcode)
    return y, scale, x if residual is None else h


def matvec_q4(x, w, scale, zero=None, *, group: int = 128, y=None):
    """Product of up to 64 rows with 4-bit weights (``muir_matvec_q4``):
    y[m, n] = sum_k x[m, k] (nib[n, k] - zero[n, k / group]) scale[n, k / group].

    x [..., K] float32 or bfloat16; w [N, K / 2] uint8, columns 2j (low half) and 2j + 1
    (high half) in byte j of a row; scale [N, K / group] float32 or bfloat16; zero the same
    or None for 8; group 32, 64 or 128. Returns y [..., N] in x's dtype.
    """
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a torch.Tensor with at least one dimension")
    _rank(w, "w", 2)
    K, N, i = x.shape[-1], w.shape[0], x.get_device()
    code = _dtype_code(x)
    if group <= 0 or K % 2 or K % group:
        raise ValueError(f"K={K} must be a multiple of the group, {group}")
    _is(x, "x", x.dtype, x.shape, i)
    _is(w, "w", torch.uint8, (N, K // 2), i)
    _is(scale, "scale", getattr(scale, "dtype", None), (N, K // group), i)
    scode = _dtype_code(scale)
    if zero is not None:
        _is(zero, "zero", scale.dtype, (N, K // group), i)
    y = _out(y, "y", x.dtype, x.shape[:-1] + (N,), x)
    _call(lib().muir_matvec_q4, i, x.data_ptr(), w.data_ptr(), scale.data_ptr(), _at(zero),
          y.data_ptr(), x.numel() // K if K else 0, N, K, group, code, scode)
    return y
