"""A gated linear recurrence over channels (argument marshalling only).

As in ``linear``: torch CUDA (HIP) tensors are checked and their device
pointers go to ``libgdn2.so`` with torch's current stream of their device.
There is no CPU or torch fallback.
"""
from __future__ import annotations

import ctypes

from .binding import GDN2_BF16, GDN2_F32, _check
from .linear import _bytes, _dtype_code, _like, _need, _ptr, _register, _run, _space

SCAN_MARK = 128  # tokens from mark to mark


class Gdn2ScanDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("gate_dtype", ctypes.c_int32), ("gate_logits", ctypes.c_int32), ("complement", ctypes.c_int32),
    ]


_vp, _sz, _sd, _szp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Gdn2ScanDesc), ctypes.POINTER(ctypes.c_size_t)
_register(("gdn2_scan_fwd_workspace", [_sd, _szp]), ("gdn2_scan_fwd", [_sd] + [_vp] * 7 + [_sz, _vp]),
          ("gdn2_scan_fwd_varlen_workspace", [_sd, _szp]), ("gdn2_scan_fwd_varlen", [_sd] + [_vp] * 8 + [_sz, _vp]),
          ("gdn2_scan_bwd_workspace", [_sd, _szp]), ("gdn2_scan_bwd", [_sd] + [_vp] * 10 + [_sz, _vp]),
          ("gdn2_scan_bwd_varlen_workspace", [_sd, _szp]), ("gdn2_scan_bwd_varlen", [_sd] + [_vp] * 11 + [_sz, _vp]),
          ("gdn2_scan_step", [_sd] + [_vp] * 5))


def make_scan_desc(batch, seqlen, dim, dtype=GDN2_BF16, gate_dtype=GDN2_F32, gate_logits=0, complement=0) -> Gdn2ScanDesc:
    return Gdn2ScanDesc(batch, seqlen, dim, dtype, gate_dtype, gate_logits, complement)


def gated_scan_fwd_workspace(desc: Gdn2ScanDesc) -> int:
    return _bytes("gdn2_scan_fwd_workspace", desc)


def gated_scan_fwd_varlen_workspace(desc: Gdn2ScanDesc) -> int:
    return _bytes("gdn2_scan_fwd_varlen_workspace", desc)


def gated_scan_bwd_workspace(desc: Gdn2ScanDesc) -> int:
    return _bytes("gdn2_scan_bwd_workspace", desc)


def gated_scan_bwd_varlen_workspace(desc: Gdn2ScanDesc) -> int:
    return _bytes("gdn2_scan_bwd_varlen_workspace", desc)


def _sizes(x, log_decay, cu_seqlens, gate_logits, complement, step=False):
    """(the token axes, what make_scan_desc takes) of checked inputs."""
    import torch
    if step:
        if x.dim() != 2:
            raise ValueError("x is [N,D]")
        tok, N, T = tuple(x.shape[:1]), x.shape[0], 1
    elif cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x is [B,T,D]")
        tok, N, T = tuple(x.shape[:2]), x.shape[0], x.shape[1]
    else:
        if x.dim() not in (2, 3) or (x.dim() == 3 and x.shape[0] != 1):
            raise ValueError("packed tensors are [T,D] or [1,T,D]")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a 1-D tensor of N+1 offsets")
        _check(cu_seqlens, "cu_seqlens", tuple(cu_seqlens.shape), (torch.int32,), x.device)
        tok, N, T = tuple(x.shape[:-1]), cu_seqlens.numel() - 1, x.shape[-2]
    D = x.shape[-1]
    if D < 1:
        raise ValueError("x needs at least one channel")
    code = _dtype_code(x, "x")
    _like(x, "x", x.shape, x.dtype, x.device)
    gcode = _dtype_code(log_decay, "log_decay")
    _like(log_decay, "log_decay", x.shape, log_decay.dtype, x.device)
    return tok, (N, T, D, code, gcode, int(bool(gate_logits)), int(bool(complement)))


def _marks_shape(x, cu_seqlens, T):
    n = (T + SCAN_MARK - 1) // SCAN_MARK
    return (n, x.shape[-1]) if cu_seqlens is not None else (x.shape[0], n, x.shape[-1])


def _fwd(x, log_decay, cu_seqlens, state0, gate_logits, complement, out, state_out, return_state, return_marks, workspace):
    import torch
    tok, sizes = _sizes(x, log_decay, cu_seqlens, gate_logits, complement)
    N, T, D = sizes[:3]
    dev, f32 = x.device, torch.float32
    if state0 is not None:
        _like(state0, "state0", (N, D), f32, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", x.shape, x.dtype, dev)
    if state_out is not None:
        _like(state_out, "state_out", (N, D), f32, dev)
    elif return_state:
        state_out = torch.empty((N, D), dtype=f32, device=dev)
    marks = torch.empty(_marks_shape(x, cu_seqlens, T), dtype=f32, device=dev) if return_marks else None
    name = "gdn2_scan_fwd" if cu_seqlens is None else "gdn2_scan_fwd_varlen"
    ws, n = _space(workspace, _need(name + "_workspace", make_scan_desc, *sizes), dev)
    _run(name, dev, make_scan_desc(*sizes), *([] if cu_seqlens is None else [_ptr(cu_seqlens)]), _ptr(x), _ptr(log_decay), _ptr(state0),
         _ptr(out), _ptr(state_out), _ptr(marks), _ptr(ws), n)
    return out, state_out, marks


def gated_scan_fwd(x, log_decay, state0=None, gate_logits=False, complement=False, out=None, state_out=None,
                   return_state=True, return_marks=False, workspace=None):
    """h_t = a_t h_{t-1} + w_t x_t for every channel, a = exp(log_decay), y = h.

    x [B,T,D], log_decay [B,T,D] (bf16 or fp32 each); ``gate_logits``: log_decay
    holds logits g, log a = -softplus(g).  w = 1, or 1 - a with ``complement``.
    state0 [B,D] fp32 or None; state_out may be state0.  ``return_marks``: also
    the state that enters every 128th token, which ``gated_scan_bwd`` takes.
    ``workspace``: None allocates what the call needs, or a uint8 device tensor
    of at least gated_scan_fwd_workspace() bytes.
    Returns (y like x, final state [B,D] fp32 or None, marks
    [B,ceil(T/128),D] fp32 or None).
    """
    return _fwd(x, log_decay, None, state0, gate_logits, complement, out, state_out, return_state, return_marks, workspace)


def gated_scan_fwd_varlen(x, log_decay, cu_seqlens, state0=None, gate_logits=False, complement=False, out=None,
                          state_out=None, return_state=True, return_marks=False, workspace=None):
    """``gated_scan_fwd`` over N sequences packed along one token axis.

    x, log_decay [T,D] (or with a leading 1); cu_seqlens int32 [N+1] on the
    device; states [N,D]; marks [ceil(T/128),D].  Tokens outside every sequence
    are not written: a given ``out`` keeps them, a new one has any value there.
    """
    return _fwd(x, log_decay, cu_seqlens, state0, gate_logits, complement, out, state_out, return_state, return_marks, workspace)


def _bwd(dy, x, log_decay, marks, cu_seqlens, state0, d_state, gate_logits, complement, want_state0, workspace):
    import torch
    tok, sizes = _sizes(x, log_decay, cu_seqlens, gate_logits, complement)
    N, T, D = sizes[:3]
    dev, f32 = x.device, torch.float32
    _like(dy, "dy", x.shape, x.dtype, dev)
    _like(marks, "marks", _marks_shape(x, cu_seqlens, T), f32, dev)
    for t, n in ((state0, "state0"), (d_state, "d_state")):
        if t is not None:
            _like(t, n, (N, D), f32, dev)
    if want_state0 is None:
        want_state0 = state0 is not None
    dx, dg = torch.empty_like(x), torch.empty_like(log_decay)
    ds0 = torch.empty((N, D), dtype=f32, device=dev) if want_state0 else None
    name = "gdn2_scan_bwd" if cu_seqlens is None else "gdn2_scan_bwd_varlen"
    ws, n = _space(workspace, _need(name + "_workspace", make_scan_desc, *sizes), dev)
    _run(name, dev, make_scan_desc(*sizes), *([] if cu_seqlens is None else [_ptr(cu_seqlens)]), _ptr(dy), _ptr(x), _ptr(log_decay),
         _ptr(marks), _ptr(state0), _ptr(d_state), _ptr(dx), _ptr(dg), _ptr(ds0), _ptr(ws), n)
    return dict(dx=dx, d_log_decay=dg, d_state0=ds0)


def gated_scan_bwd(dy, x, log_decay, marks, state0=None, d_state=None, gate_logits=False, complement=False,
                   want_state0=None, workspace=None):
    """Gradients of <dy, y> + <d_state, h_T> for ``gated_scan_fwd``, whose inputs and marks these are.

    d_state [B,D] fp32 or None (zeros).  Returns a dict: dx like x, d_log_decay
    like log_decay (of the logits with ``gate_logits``), d_state0 [B,D] fp32
    (``want_state0``: by default where state0 is given, else None).
    ``workspace``: None allocates it, or a uint8 device tensor of at least
    gated_scan_bwd_workspace() bytes.
    """
    return _bwd(dy, x, log_decay, marks, None, state0, d_state, gate_logits, complement, want_state0, workspace)


def gated_scan_bwd_varlen(dy, x, log_decay, marks, cu_seqlens, state0=None, d_state=None, gate_logits=False,
                          complement=False, want_state0=None, workspace=None):
    """``gated_scan_bwd`` for ``gated_scan_fwd_varlen``: packed tensors, states [N,D].

    Gradients of tokens outside every sequence are not written (any value).
    """
    return _bwd(dy, x, log_decay, marks, cu_seqlens, state0, d_state, gate_logits, complement, want_state0, workspace)


def gated_scan_step(x, log_decay, state, gate_logits=False, complement=False, out=None):
    """One decode step for N sequences; updates ``state`` [N,D] fp32 in place.

    x, log_decay [N,D] as for ``gated_scan_fwd``.  Returns y like x.
    """
    import torch
    tok, sizes = _sizes(x, log_decay, None, gate_logits, complement, step=True)
    _like(state, "state", x.shape, torch.float32, x.device)
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", x.shape, x.dtype, x.device)
    _run("gdn2_scan_step", x.device, make_scan_desc(*sizes), _ptr(x), _ptr(log_decay), _ptr(state), _ptr(out))
    return out
