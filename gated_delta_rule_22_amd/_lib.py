"""ctypes binding of ``libckda.so`` (declared in ``include/ckda.h``).

Argument marshalling only: shapes and dtypes are read from torch tensors,
outputs and the workspace are allocated with torch (device memory), and the
current HIP stream is passed through.  Every step of the computation runs in
the library's kernels.  There is no fallback: if the library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# CKDA_LIB names another build of the same library (e.g. a host-sanitized one).
LIB_PATH = os.environ.get("CKDA_LIB") or os.path.join(_PKG, "libckda.so")

CKDA_BF16 = 0
CKDA_F32 = 1

_lib = None


class CkdaError(RuntimeError):
    pass


def library() -> ctypes.CDLL:
    """Load ``libckda.so`` once and declare its signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise CkdaError(f"{LIB_PATH} is not built; run `python -m gated_delta_rule_22_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.ckda_abi_version.argtypes = []
        lib.ckda_abi_version.restype = ci
        lib.ckda_status_string.argtypes = [ci]
        lib.ckda_status_string.restype = ctypes.c_char_p
        lib.ckda_forward_workspace_bytes.argtypes = [ci] * 7
        lib.ckda_forward_workspace_bytes.restype = sz
        lib.ckda_forward_ex_workspace_bytes.argtypes = [ci] * 8
        lib.ckda_forward_ex_workspace_bytes.restype = sz
        lib.ckda_forward.argtypes = [vp] * 7 + [ci] * 7 + [vp, vp, vp, sz, vp]
        lib.ckda_forward.restype = ci
        lib.kda_forward.argtypes = [vp] * 7 + [ci] * 7 + [vp, vp, vp, sz, vp]
        lib.kda_forward.restype = ci
        lib.ckda_forward_ex.argtypes = [vp] * 7 + [ci] * 8 + [vp, vp, vp, sz, vp]
        lib.ckda_forward_ex.restype = ci
        lib.ckda_forward_noalloc.argtypes = [vp] * 7 + [ci] * 8 + [vp, vp, vp]
        lib.ckda_forward_noalloc.restype = ci
        lib.ckda_forward_noalloc_max_bytes.argtypes = []
        lib.ckda_forward_noalloc_max_bytes.restype = sz
        lib.ckda_backward_workspace_bytes.argtypes = [ci] * 7
        lib.ckda_backward_workspace_bytes.restype = sz
        lib.ckda_backward.argtypes = [vp] * 7 + [ci] * 7 + [vp] * 8 + [vp, sz, vp]
        lib.ckda_backward.restype = ci
        lib.kda_backward.argtypes = [vp] * 7 + [ci] * 7 + [vp] * 8 + [vp, sz, vp]
        lib.kda_backward.restype = ci
        lib.ckda_backward_ex.argtypes = [vp] * 7 + [ci] * 8 + [vp] * 8 + [vp, sz, vp]
        lib.ckda_backward_ex.restype = ci
        lib.ckda_decode_step.argtypes = [vp] * 7 + [ci] * 5 + [vp]
        lib.ckda_decode_step.restype = ci
        ll, fl = ctypes.c_longlong, ctypes.c_float
        lib.gdr_forward_workspace_bytes.argtypes = [ci] * 8
        lib.gdr_forward_workspace_bytes.restype = sz
        lib.gdr_forward.argtypes = [vp] * 7 + [ci] * 8 + [vp, vp, vp, sz, vp]
        lib.gdr_forward.restype = ci
        lib.gdr_backward_workspace_bytes.argtypes = [ci] * 8
        lib.gdr_backward_workspace_bytes.restype = sz
        lib.gdr_backward.argtypes = [vp] * 7 + [ci] * 8 + [vp] * 8 + [vp, sz, vp]
        lib.gdr_backward.restype = ci
        lib.gdr_decode_step.argtypes = [vp] * 7 + [ci, vp] + [ci] * 6 + [vp]
        lib.gdr_decode_step.restype = ci
        lib.qk_norm_rotary.argtypes = ([vp] * 6 + [ci] * 5 + [ll] * 2 + [ci] * 2 + [fl] * 3
                                       + [ci, vp, vp, ll, ll, vp])
        lib.qk_norm_rotary.restype = ci
        lib.qk_norm_rotary_backward_workspace_bytes.argtypes = [ci] * 2
        lib.qk_norm_rotary_backward_workspace_bytes.restype = sz
        lib.qk_norm_rotary_backward.argtypes = ([vp] * 8 + [ci] * 5 + [ll] * 4 + [ci] * 2
                                                + [fl] * 3 + [ci, vp, vp, ll, ll]
                                                + [vp] * 3 + [sz, vp])
        lib.qk_norm_rotary_backward.restype = ci
        lib.ckda_rotary.argtypes = ([vp] * 3 + [ci] * 4 + [ll, ci, fl, ci, ci, vp, ll, vp])
        lib.ckda_rotary.restype = ci
        _lib = lib
    return _lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return CKDA_BF16
    if t.dtype == torch.float32:
        return CKDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status: int, what: str):
    if status != 0:
        msg = library().ckda_status_string(status).decode()
        raise CkdaError(f"{what} failed with status {status}: {msg}")


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def forward_workspace_bytes(B, T, H, dk, dv, N, dtype, options=0) -> int:
    code = dtype if isinstance(dtype, int) else (CKDA_BF16 if dtype == torch.bfloat16 else CKDA_F32)
    if options:
        return int(library().ckda_forward_ex_workspace_bytes(B, T, H, dk, dv, N, code, options))
    return int(library().ckda_forward_workspace_bytes(B, T, H, dk, dv, N, code))


def _need(t, name, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


OPT_KDA, OPT_QK_L2NORM, OPT_O_BF16, OPT_SPLIT = 1, 2, 4, 8   # CKDA_OPT_* in include/ckda.h


def forward(q, k, v, g, beta, S0=None, cu_seqlens=None, *, out=None, final_state=None,
            workspace=None, output_final_state=True, normalize_qk=False,
            out_dtype=torch.float32, kda=False, no_alloc=False, split=False):
    """CKDA chunkwise forward.  Returns ``(o, S_T)`` (``S_T`` is None when
    ``output_final_state`` is False).  See ``ckda_forward`` in include/ckda.h
    for shapes; ``final_state`` may be ``S0`` itself to advance it in place.

    ``normalize_qk`` (L2-normalise q and k rows in the kernel), ``out_dtype``
    (``torch.bfloat16`` for a bf16 ``o``) and ``kda`` (gate signs ignored) map
    to the options of ``ckda_forward_ex``; with none of them set the call goes
    to ``ckda_forward``.  ``no_alloc=True`` calls ``ckda_forward_noalloc``,
    which uses the library's fixed scratch instead of a workspace (pass
    ``out``, and ``final_state`` or ``output_final_state=False``, so that
    nothing is allocated here either).  ``split=True`` runs the two-kernel
    hand-off (``CKDA_OPT_SPLIT``) in place of the fused kernel."""
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    opts = ((OPT_KDA if kda else 0) | (OPT_QK_L2NORM if normalize_qk else 0)
            | (OPT_O_BF16 if out_dtype == torch.bfloat16 else 0) | (OPT_SPLIT if split else 0))
    entry = "ckda_forward_noalloc" if no_alloc else (
        "ckda_forward_ex" if opts else "ckda_forward")
    return _forward(entry, q, k, v, g, beta, S0, cu_seqlens, out, final_state, workspace,
                    output_final_state, opts)


def kda_forward(q, k, v, g, beta, S0=None, cu_seqlens=None, *, out=None, final_state=None,
                workspace=None, output_final_state=True):
    """KDA mode of the forward (gate signs ignored, |g| used); same arguments and
    results as :func:`forward`.  See ``kda_forward`` in include/ckda.h."""
    return _forward("kda_forward", q, k, v, g, beta, S0, cu_seqlens, out, final_state,
                    workspace, output_final_state)


def _forward(entry, q, k, v, g, beta, S0, cu_seqlens, out, final_state, workspace,
             output_final_state, opts=0):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(k, "k", shape=(B, T, H, dk))
    _need(v, "v", shape=(B, T, H, dv))
    _need(g, "g", torch.float32, (B, T, H, dk))
    _need(beta, "beta", torch.float32, (B, T, H))
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if S0 is not None:
        _need(S0, "S0", torch.float32, (N, H, dk, dv))
    dev = q.device
    o_dt = torch.bfloat16 if opts & OPT_O_BF16 else torch.float32
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=o_dt, device=dev)
    _need(o, "out", o_dt, (B, T, H, dv))
    S_T = None
    if output_final_state:
        S_T = final_state if final_state is not None else torch.empty(
            (N, H, dk, dv), dtype=torch.float32, device=dev)
        _need(S_T, "final_state", torch.float32, (N, H, dk, dv))
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
            B, T, H, dk, dv, N, code)
    if entry == "ckda_forward_noalloc":
        st = library().ckda_forward_noalloc(*head, opts, _ptr(o), _ptr(S_T), _stream(dev))
        _check(st, entry)
        return o, S_T
    ws_bytes = forward_workspace_bytes(B, T, H, dk, dv, N, code, opts)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    tail = (_ptr(o), _ptr(S_T), _ptr(workspace), ws_bytes, _stream(dev))
    fn = getattr(library(), entry)
    st = fn(*head, opts, *tail) if entry == "ckda_forward_ex" else fn(*head, *tail)
    _check(st, entry)
    return o, S_T


def backward_workspace_bytes(B, T, H, dk, dv, N, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (CKDA_BF16 if dtype == torch.bfloat16 else CKDA_F32)
    return int(library().ckda_backward_workspace_bytes(B, T, H, dk, dv, N, code))


def backward(q, k, v, g, beta, do, S0=None, dS_T=None, cu_seqlens=None, *, workspace=None,
             need_dS0=True, kda=False, normalize_qk=False):
    """Gradients of ``sum(do * o) + sum(dS_T * S_T)`` for the forward's inputs:
    returns ``(dq, dk, dv, dg, dbeta, dS0)`` as fp32 tensors (``dS0`` is None
    when ``need_dS0`` is False).  See ``ckda_backward`` in include/ckda.h;
    ``kda=True`` calls ``kda_backward`` (the backward of :func:`kda_forward`);
    ``normalize_qk=True`` is the backward of ``forward(..., normalize_qk=True)``
    (``ckda_backward_ex``)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(k, "k", shape=(B, T, H, dk))
    _need(v, "v", shape=(B, T, H, dv))
    _need(g, "g", torch.float32, (B, T, H, dk))
    _need(beta, "beta", torch.float32, (B, T, H))
    _need(do, "do", torch.float32, (B, T, H, dv))
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        N = cu_seqlens.numel() - 1
    else:
        N = B
    for t, n in ((S0, "S0"), (dS_T, "dS_T")):
        if t is not None:
            _need(t, n, torch.float32, (N, H, dk, dv))
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, T, H, dk), **f32)
    dk_ = torch.empty((B, T, H, dk), **f32)
    dv_ = torch.empty((B, T, H, dv), **f32)
    dg = torch.empty((B, T, H, dk), **f32)
    db = torch.empty((B, T, H), **f32)
    dS0 = torch.empty((N, H, dk, dv), **f32) if need_dS0 else None
    ws_bytes = backward_workspace_bytes(B, T, H, dk, dv, N, code)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
            B, T, H, dk, dv, N, code)
    tail = (_ptr(do), _ptr(dS_T), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db),
            _ptr(dS0), _ptr(workspace), ws_bytes, _stream(dev))
    if normalize_qk:
        entry = "ckda_backward_ex"
        st = library().ckda_backward_ex(*head, OPT_QK_L2NORM | (OPT_KDA if kda else 0), *tail)
    else:
        entry = "kda_backward" if kda else "ckda_backward"
        st = getattr(library(), entry)(*head, *tail)
    _check(st, entry)
    return dq, dk_, dv_, dg, db, dS0


def decode_step(q, k, v, g, beta, S, *, out=None):
    """One decode step; ``S`` ([N, H, dk, dv] fp32) is updated in place.
    Returns o ``[N, H, dv]`` fp32."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(k, "k", shape=(N, H, dk))
    _need(v, "v", shape=(N, H, dv))
    _need(g, "g", torch.float32, (N, H, dk))
    _need(beta, "beta", torch.float32, (N, H))
    _need(S, "S", torch.float32, (N, H, dk, dv))
    o = out if out is not None else torch.empty((N, H, dv), dtype=torch.float32, device=q.device)
    _need(o, "out", torch.float32, (N, H, dv))
    st = library().ckda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
                                    _ptr(o), N, H, dk, dv, code, _stream(q.device))
    _check(st, "ckda_decode_step")
    return o


# ------------------------------------------------------------------ gated delta rule

def gdr_forward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (CKDA_BF16 if dtype == torch.bfloat16 else CKDA_F32)
    return int(library().gdr_forward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, code))


def _gdr_sizes(q, k, v, g, beta, cu_seqlens):
    """Checks the inputs shared by the forward and the backward; their sizes."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have 4 dimensions [B, T, heads, channels]")
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[-2:]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(k, "k", shape=(B, T, Hk, dk))
    _need(v, "v", shape=(B, T, Hv, dv))
    _need(g, "g", torch.float32, (B, T, Hv))
    _need(beta, "beta", torch.float32, (B, T, Hv))
    if cu_seqlens is None:
        return B, T, Hk, Hv, dk, dv, B
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    return B, T, Hk, Hv, dk, dv, cu_seqlens.numel() - 1


def _same_device(dev, *tensors):
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on {dev}, got one on {t.device}")


def gdr_forward(q, k, v, g, beta, S0=None, cu_seqlens=None, *, out=None, final_state=None,
                workspace=None, output_final_state=True):
    """Gated delta rule over a batch of sequences: one log-gate ``g`` per token
    and head, value heads sharing query/key heads in groups.  Returns
    ``(o, S_T)``, ``o`` in the type of ``q`` (``S_T`` is None when
    ``output_final_state`` is False).  See ``gdr_forward`` in include/ckda.h for
    shapes; ``final_state`` may be ``S0`` itself."""
    code = _dtype_code(q)
    B, T, Hk, Hv, dk, dv, N = _gdr_sizes(q, k, v, g, beta, cu_seqlens)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (N, Hv, dk, dv))
    dev = q.device
    o = out if out is not None else torch.empty((B, T, Hv, dv), dtype=q.dtype, device=dev)
    _need(o, "out", q.dtype, (B, T, Hv, dv))
    S_T = None
    if output_final_state:
        S_T = final_state if final_state is not None else torch.empty(
            (N, Hv, dk, dv), dtype=torch.float32, device=dev)
        _need(S_T, "final_state", torch.float32, (N, Hv, dk, dv))
    ws_bytes = gdr_forward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, code)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _same_device(dev, k, v, g, beta, S0, cu_seqlens, o, S_T, workspace)
    with torch.cuda.device(dev):
        st = library().gdr_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
                                   _ptr(cu_seqlens), B, T, Hk, Hv, dk, dv, N, code, _ptr(o),
                                   _ptr(S_T), _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "gdr_forward")
    return o, S_T


def gdr_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (CKDA_BF16 if dtype == torch.bfloat16 else CKDA_F32)
    return int(library().gdr_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, code))


def gdr_backward(q, k, v, g, beta, do, S0=None, dS_T=None, cu_seqlens=None, *, workspace=None,
                 need_dS0=True):
    """Gradients of ``sum(do * o) + sum(dS_T * S_T)`` of :func:`gdr_forward`:
    ``(dq, dk, dv, dg, dbeta, dS0)``, the first three in the type of ``q``, the
    others fp32 (``dS0`` is None when ``need_dS0`` is False).  See
    ``gdr_backward`` in include/ckda.h."""
    code = _dtype_code(q)
    B, T, Hk, Hv, dk, dv, N = _gdr_sizes(q, k, v, g, beta, cu_seqlens)
    _need(do, "do", q.dtype, (B, T, Hv, dv))
    for t, n in ((S0, "S0"), (dS_T, "dS_T")):
        if t is not None:
            _need(t, n, torch.float32, (N, Hv, dk, dv))
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty((B, T, Hv), **f32), torch.empty((B, T, Hv), **f32)
    dS0 = torch.empty((N, Hv, dk, dv), **f32) if need_dS0 else None
    ws_bytes = gdr_backward_workspace_bytes(B, T, Hk, Hv, dk, dv, N, code)
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _same_device(dev, k, v, g, beta, do, S0, dS_T, cu_seqlens, workspace)
    with torch.cuda.device(dev):
        st = library().gdr_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
                                    _ptr(cu_seqlens), B, T, Hk, Hv, dk, dv, N, code, _ptr(do),
                                    _ptr(dS_T), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg),
                                    _ptr(db), _ptr(dS0), _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "gdr_backward")
    return dq, dk_, dv_, dg, db, dS0


def gdr_decode_step(q, k, v, g, beta, S, slots=None, *, out=None):
    """One token of the gated delta rule for N rows; row n's state is
    ``S[slots[n]]`` (``S[n]`` without ``slots``), updated in place.  Rows whose
    slot is outside the pool, or named by an earlier row, are padding: their
    ``o`` is zero.  Returns o ``[N, Hv, dv]`` in the type of ``q``."""
    if q.dim() != 3 or v.dim() != 3 or S.dim() != 4:
        raise ValueError("q, k and v must have 3 dimensions [N, heads, channels], S 4")
    N, Hk, dk = q.shape
    Hv, dv = v.shape[-2:]
    code = _dtype_code(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(k, "k", shape=(N, Hk, dk))
    _need(v, "v", shape=(N, Hv, dv))
    _need(g, "g", torch.float32, (N, Hv))
    _need(beta, "beta", torch.float32, (N, Hv))
    pool = S.shape[0]
    _need(S, "S", torch.float32, (pool, Hv, dk, dv))
    if slots is not None:
        _need(slots, "slots", torch.int32, (N,))
    dev = q.device
    o = out if out is not None else torch.empty((N, Hv, dv), dtype=q.dtype, device=dev)
    _need(o, "out", q.dtype, (N, Hv, dv))
    _same_device(dev, k, v, g, beta, S, slots, o)
    with torch.cuda.device(dev):
        st = library().gdr_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
                                       _ptr(slots), pool, _ptr(o), N, Hk, Hv, dk, dv, code,
                                       _stream(dev))
    _check(st, "gdr_decode_step")
    return o


# ------------------------------------------------------------------ norm and rotation

_NORMS = {"none": 0, "l2": 1, "rms": 2}              # CKDA_NORM_* in include/ckda.h
_LAYOUTS = {"half": 0, "interleaved": 1}             # CKDA_ROTARY_*


def rotary_frequencies(rotary_dim, base=10000.0, *, scaling=None, factor=1.0,
                       original_length=None, beta_fast=32.0, beta_slow=1.0, device=None):
    """Angles per position of the ``rotary_dim / 2`` pairs (fp64, radians), and
    the scale of the rotated channels that goes with them.

    ``scaling`` stretches the context ``factor``-fold: ``"linear"`` divides all
    angles; ``"base"`` raises the base so that the slowest pair turns ``factor``
    times slower and the fastest one is unchanged; ``"ramp"`` divides the angles
    of pairs that turn less than ``beta_slow`` times within ``original_length``
    positions, keeps those that turn more than ``beta_fast`` times, blends in
    between, and scales by ``0.1 ln(factor) + 1``."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if factor < 1.0 or base <= 1.0:
        raise ValueError("factor must be at least 1 and base above 1")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling='base' needs rotary_dim of at least 4")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freqs = base ** (-i / rotary_dim)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "ramp":
        if original_length is None or original_length < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("scaling='ramp' needs original_length and beta_fast > beta_slow > 0")
        # index of the pair that turns n times within the original length
        def pair(n):
            return (rotary_dim * math.log(original_length / (n * 2 * math.pi))
                    / (2 * math.log(base)))
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rotary_dim - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freqs = freqs / factor * ramp + freqs * (1 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freqs.to(device), scale


def _rows(t, name, dtype=None, lead=None, d=None):
    """Rows [..., heads, d] whose heads are dense and whose tokens are one
    distance apart; (heads, tokens, distance in elements)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() < 3:
        raise ValueError(f"{name} must have at least 3 dimensions [..., heads, channels]")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if lead is not None and tuple(t.shape[:-2]) != tuple(lead):
        raise ValueError(f"{name} must have leading dimensions {tuple(lead)}, got {tuple(t.shape)}")
    if d is not None and t.shape[-1] != d:
        raise ValueError(f"{name} must have {d} channels, got {t.shape[-1]}")
    heads, width = t.shape[-2:]
    tokens = t.shape[:-2].numel()
    if t.numel() == 0:
        return heads, tokens, heads * width
    if (width > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != width):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    ld = None
    span = 1                            # tokens that the dimensions so far cover
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * span:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        span *= n
    ld = heads * width if ld is None else ld
    if ld < heads * width:
        raise ValueError(f"{name}: tokens must not overlap")
    return heads, tokens, ld


def _angles(positions, freqs, lead, d):
    if freqs is None:
        return 0, None
    if positions is None:
        raise ValueError("positions are needed with freqs")
    _need(positions, "positions", torch.int32, lead)
    _need(freqs, "freqs", torch.float64)
    if freqs.dim() != 1 or not 0 < 2 * freqs.numel() <= d:
        raise ValueError(f"freqs must have 1 to {d // 2} entries, got {tuple(freqs.shape)}")
    return 2 * freqs.numel(), positions


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def qk_norm_rotary(q, k, positions=None, freqs=None, *, norm="rms", q_weight=None, k_weight=None,
                   eps=1e-6, layout="half", q_scale=1.0, rotary_scale=1.0, q_out=None,
                   k_out=None):
    """Normalises every head of ``q`` [..., Hq, d] and ``k`` [..., Hk, d]
    (``norm`` is "rms", "l2" or "none", with an optional weight each), rotates
    the first ``2 len(freqs)`` channels by ``positions * freqs`` and multiplies
    ``q`` by ``q_scale``, in one pass.  ``q`` and ``k`` may be slices of one
    projection; results are dense unless ``q_out`` / ``k_out`` (which may be
    ``q`` / ``k``) are given.  See ``qk_norm_rotary`` in include/ckda.h and
    :func:`rotary_frequencies`."""
    code = _dtype_code(q)
    Hq, tokens, ldq = _rows(q, "q")
    lead, d = tuple(q.shape[:-2]), q.shape[-1]
    Hk, _, ldk = _rows(k, "k", q.dtype, lead, d)
    rd, positions = _angles(positions, freqs, lead, d)
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _need(t, n, torch.float32, (d,))
    dev = q.device
    qo = q_out if q_out is not None else torch.empty(q.shape, dtype=q.dtype, device=dev)
    ko = k_out if k_out is not None else torch.empty(k.shape, dtype=q.dtype, device=dev)
    hq, _, ldqo = _rows(qo, "q_out", q.dtype, lead, d)
    hk, _, ldko = _rows(ko, "k_out", q.dtype, lead, d)
    if (hq, hk) != (Hq, Hk):
        raise ValueError("q_out and k_out must have the heads of q and k")
    _same_device(dev, k, positions, freqs, q_weight, k_weight, qo, ko)
    with torch.cuda.device(dev):
        st = library().qk_norm_rotary(
            _ptr(q), _ptr(k), _ptr(positions), _ptr(freqs), _ptr(q_weight), _ptr(k_weight),
            tokens, Hq, Hk, d, rd, ldq, ldk, _choice(_NORMS, norm, "norm"),
            _choice(_LAYOUTS, layout, "layout"), eps, q_scale, rotary_scale, code, _ptr(qo),
            _ptr(ko), ldqo, ldko, _stream(dev))
    _check(st, "qk_norm_rotary")
    return qo, ko


def qk_norm_rotary_backward(dq_out, dk_out, q, k, positions=None, freqs=None, *, norm="rms",
                            q_weight=None, k_weight=None, eps=1e-6, layout="half", q_scale=1.0,
                            rotary_scale=1.0, dq=None, dk=None, workspace=None):
    """Gradients of :func:`qk_norm_rotary` for the gradients ``dq_out``,
    ``dk_out`` of its results: ``(dq, dk, dq_weight, dk_weight)``, the weights'
    fp32 (None where there is no weight).  ``dq`` / ``dk`` may be slices of the
    projection's gradient."""
    code = _dtype_code(q)
    Hq, tokens, ldq = _rows(q, "q")
    lead, d = tuple(q.shape[:-2]), q.shape[-1]
    Hk, _, ldk = _rows(k, "k", q.dtype, lead, d)
    uq, _, lddq = _rows(dq_out, "dq_out", q.dtype, lead, d)
    uk, _, lddk = _rows(dk_out, "dk_out", q.dtype, lead, d)
    rd, positions = _angles(positions, freqs, lead, d)
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _need(t, n, torch.float32, (d,))
    dev = q.device
    gq = dq if dq is not None else torch.empty(q.shape, dtype=q.dtype, device=dev)
    gk = dk if dk is not None else torch.empty(k.shape, dtype=q.dtype, device=dev)
    oq, _, ldgq = _rows(gq, "dq", q.dtype, lead, d)
    ok, _, ldgk = _rows(gk, "dk", q.dtype, lead, d)
    if (uq, uk) != (Hq, Hk) or (oq, ok) != (Hq, Hk):
        raise ValueError("gradients must have the heads of q and k")
    dwq = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    dwk = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    ws_bytes = 0
    if q_weight is not None or k_weight is not None:
        ws_bytes = int(library().qk_norm_rotary_backward_workspace_bytes(tokens, d))
        if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _same_device(dev, k, dq_out, dk_out, positions, freqs, q_weight, k_weight, gq, gk, workspace)
    with torch.cuda.device(dev):
        st = library().qk_norm_rotary_backward(
            _ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(positions), _ptr(freqs),
            _ptr(q_weight), _ptr(k_weight), tokens, Hq, Hk, d, rd, lddq, lddk, ldq, ldk,
            _choice(_NORMS, norm, "norm"), _choice(_LAYOUTS, layout, "layout"), eps, q_scale,
            rotary_scale, code, _ptr(gq), _ptr(gk), ldgq, ldgk, _ptr(dwq), _ptr(dwk),
            _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "qk_norm_rotary_backward")
    return gq, gk, dwq, dwk


def rotary(x, positions, freqs, *, layout="half", rotary_scale=1.0, inverse=False, out=None):
    """Rotates the first ``2 len(freqs)`` channels of every head of ``x``
    [..., H, d] by ``positions * freqs``; ``inverse`` by the opposite angle (the
    backward).  ``out`` may be ``x``.  See ``ckda_rotary`` in include/ckda.h."""
    code = _dtype_code(x)
    H, tokens, ldx = _rows(x, "x")
    lead, d = tuple(x.shape[:-2]), x.shape[-1]
    if freqs is None:
        raise ValueError("freqs are needed")
    rd, positions = _angles(positions, freqs, lead, d)
    dev = x.device
    o = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    ho, _, ldo = _rows(o, "out", x.dtype, lead, d)
    if ho != H:
        raise ValueError("out must have the heads of x")
    _same_device(dev, positions, freqs, o)
    with torch.cuda.device(dev):
        st = library().ckda_rotary(_ptr(x), _ptr(positions), _ptr(freqs), tokens, H, d, rd, ldx,
                                   _choice(_LAYOUTS, layout, "layout"), rotary_scale,
                                   int(inverse), code, _ptr(o), ldo, _stream(dev))
    _check(st, "ckda_rotary")
    return o
