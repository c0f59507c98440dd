"""A gated linear recurrence over channels (argument marshalling only).

As in ``linear``: torch CUDA (HIP) tensors are checked and their device
pointers go to ``libgdn2.so`` with torch's current stream of their device.
There is no CPU or torch fallback.
"""
from __future__ import annotations

import ctypes
import functools

from .binding import GDN2_BF16, GDN2_F32
from .facts import facts, like, needed, new_like
from .linear import _bytes, _ptr, _register, _run, _space
from .rotary import _type_code

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


@functools.lru_cache(maxsize=1024)
def _request(kind, x, log_decay, cu_seqlens, gate_logits, complement, states, *tokens):
    """(the descriptor, workspace bytes, N, marks' shape) of checked facts.

    kind: "fwd", "bwd" or "step"; states and tokens: (name, facts) pairs of
    tensors [N,D] fp32 and of tensors like x, None among the facts skipped.
    """
    import torch
    needed(x, "x")
    needed(log_decay, "log_decay")
    shape, _, dtype, dev = x
    packed = cu_seqlens is not None
    if kind == "step":
        if len(shape) != 2:
            raise ValueError("x is [N,D]")
        N, T = shape[0], 1
    elif not packed:
        if len(shape) != 3:
            raise ValueError("x is [B,T,D]")
        N, T = shape[0], shape[1]
    else:
        if len(shape) not in (2, 3) or (len(shape) == 3 and shape[0] != 1):
            raise ValueError("packed tensors are [T,D] or [1,T,D]")
        if len(cu_seqlens[0]) != 1 or cu_seqlens[0][0] < 1:
            raise ValueError("cu_seqlens must be a 1-D tensor of N+1 offsets")
        like(cu_seqlens, "cu_seqlens", cu_seqlens[0], (torch.int32,), dev)
        N, T = cu_seqlens[0][0] - 1, shape[-2]
    D = shape[-1]
    if D < 1:
        raise ValueError("x needs at least one channel")
    code, gcode = _type_code(dtype, "x"), _type_code(log_decay[2], "log_decay")
    like(x, "x", shape, (dtype,), dev)
    like(log_decay, "log_decay", shape, (log_decay[2],), dev)
    for name, f in states:
        if f is not None:
            like(f, name, (N, D), (torch.float32,), dev)
    for name, f in tokens:
        if f is not None:
            like(f, name, shape, (dtype,), dev)
    desc = make_scan_desc(N, T, D, code, gcode, int(gate_logits), int(complement))
    n = (T + SCAN_MARK - 1) // SCAN_MARK
    need = 0 if kind == "step" else _bytes(f"gdn2_scan_{kind}{'_varlen' if packed else ''}_workspace", desc)
    return desc, need, N, (n, D) if packed else (shape[0], n, D)


def _offsets(cu_seqlens):
    if cu_seqlens is None:  # which stands for whole sequences within
        raise ValueError("cu_seqlens is missing")


def _fwd(x, log_decay, cu_seqlens, state0, gate_logits, complement, out, state_out, return_state, return_marks, workspace):
    import torch
    desc, need, N, mshape = _request("fwd", facts(x), facts(log_decay), facts(cu_seqlens), bool(gate_logits), bool(complement),
                                     (("state0", facts(state0)), ("state_out", facts(state_out))), ("out", facts(out)))
    dev, f32 = x.device, torch.float32
    if out is None:
        out = new_like(x)
    if state_out is None and return_state:
        state_out = torch.empty((N, x.shape[-1]), dtype=f32, device=dev) if state0 is None else new_like(state0)
    marks = torch.empty(mshape, dtype=f32, device=dev) if return_marks else None
    ws, n = _space(workspace, need, dev)
    if cu_seqlens is None:
        _run("gdn2_scan_fwd", dev, desc, _ptr(x), _ptr(log_decay), _ptr(state0), _ptr(out), _ptr(state_out), _ptr(marks), _ptr(ws), n)
    else:
        _run("gdn2_scan_fwd_varlen", dev, desc, _ptr(cu_seqlens), _ptr(x), _ptr(log_decay), _ptr(state0), _ptr(out), _ptr(state_out),
             _ptr(marks), _ptr(ws), n)
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
    _offsets(cu_seqlens)
    return _fwd(x, log_decay, cu_seqlens, state0, gate_logits, complement, out, state_out, return_state, return_marks, workspace)


def _bwd(dy, x, log_decay, marks, cu_seqlens, state0, d_state, gate_logits, complement, want_state0, workspace):
    import torch
    needed(dy, "dy")
    desc, need, N, mshape = _request("bwd", facts(x), facts(log_decay), facts(cu_seqlens), bool(gate_logits), bool(complement),
                                     (("state0", facts(state0)), ("d_state", facts(d_state))), ("dy", facts(dy)))
    dev, f32 = x.device, torch.float32
    fm = facts(marks)
    needed(fm, "marks")
    like(fm, "marks", mshape, (f32,), dev)
    if want_state0 is None:
        want_state0 = state0 is not None
    dx, dg = new_like(x), new_like(log_decay)
    ds0 = torch.empty((N, x.shape[-1]), dtype=f32, device=dev) if want_state0 else None
    ws, n = _space(workspace, need, dev)
    if cu_seqlens is None:
        _run("gdn2_scan_bwd", dev, desc, _ptr(dy), _ptr(x), _ptr(log_decay), _ptr(marks), _ptr(state0), _ptr(d_state), _ptr(dx), _ptr(dg),
             _ptr(ds0), _ptr(ws), n)
    else:
        _run("gdn2_scan_bwd_varlen", dev, desc, _ptr(cu_seqlens), _ptr(dy), _ptr(x), _ptr(log_decay), _ptr(marks), _ptr(state0),
             _ptr(d_state), _ptr(dx), _ptr(dg), _ptr(ds0), _ptr(ws), n)
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
    _offsets(cu_seqlens)
    return _bwd(dy, x, log_decay, marks, cu_seqlens, state0, d_state, gate_logits, complement, want_state0, workspace)


def gated_scan_step(x, log_decay, state, gate_logits=False, complement=False, out=None):
    """One decode step for N sequences; updates ``state`` [N,D] fp32 in place.

    x, log_decay [N,D] as for ``gated_scan_fwd``.  Returns y like x.
    """
    needed(state, "state")
    desc, _, _, _ = _request("step", facts(x), facts(log_decay), None, bool(gate_logits), bool(complement),
                             (("state", facts(state)),), ("out", facts(out)))
    if out is None:
        out = new_like(x)
    _run("gdn2_scan_step", x.device, desc, _ptr(x), _ptr(log_decay), _ptr(state), _ptr(out))
    return out
