"""Linear attention with a decay for each head, and layer norm (argument marshalling only).

As in ``binding``: torch CUDA (HIP) tensors are checked for type, dtype,
shape, device and contiguity, and their device pointers go to ``libgdn2.so``
with torch's current stream of their device.  There is no CPU or torch
fallback.
"""
from __future__ import annotations

import ctypes
import functools

from .binding import GDN2_BF16, GDN2_F32, Gdn2Error, _check, load_library

GDN2_DECAY_TOKEN, GDN2_DECAY_HEAD = 0, 1


class Gdn2LinearDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
        ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("decay_kind", ctypes.c_int32), ("q_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


class Gdn2NormDesc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("dim", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


_signatures = []  # (entry point, argument types)
_calls = {}  # entry point -> ctypes function


def _register(*signatures):
    _signatures.extend(signatures)


def _lib():
    lib = load_library()
    if len(_calls) != len(_signatures):
        ready = {}
        for name, args in _signatures:
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ctypes.c_int, args
            ready[name] = fn
        _calls.update(ready)
    return lib


_vp, _sz, _szp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
_ld, _nd = ctypes.POINTER(Gdn2LinearDesc), ctypes.POINTER(Gdn2NormDesc)
_register(("gdn2_linear_fwd_workspace", [_ld, _szp]), ("gdn2_linear_fwd", [_ld] + [_vp] * 8 + [_sz, _vp]),
          ("gdn2_linear_fwd_varlen_workspace", [_ld, _szp]), ("gdn2_linear_fwd_varlen", [_ld] + [_vp] * 9 + [_sz, _vp]),
          ("gdn2_linear_bwd_workspace", [_ld, _szp]), ("gdn2_linear_bwd", [_ld] + [_vp] * 13 + [_sz, _vp]),
          ("gdn2_linear_bwd_varlen_workspace", [_ld, _szp]), ("gdn2_linear_bwd_varlen", [_ld] + [_vp] * 14 + [_sz, _vp]),
          ("gdn2_linear_step", [_ld] + [_vp] * 7),
          ("gdn2_layer_norm_fwd", [_nd] + [_vp] * 7), ("gdn2_layer_norm_bwd_workspace", [_nd, _szp]),
          ("gdn2_layer_norm_bwd", [_nd] + [_vp] * 9 + [_sz, _vp]))


def _call(name):
    if name not in _calls:
        _lib()
    return _calls[name]


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1)
def _torch_calls():
    """The current device's index, and torch's current stream of a device as a hipStream_t."""
    import torch
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
            stream or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _like(t, name, shape, dtype, dev):
    """`_check` for one dtype, its four questions asked at once where all hold."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check(t, name, shape, (dtype,), dev)


def _run(name, dev, desc, *args):
    """Call an entry point on `dev`'s current stream; raises on a bad status."""
    fn = _calls.get(name) or _call(name)
    if dev.type != "cuda":
        raise ValueError(f"{name}: tensors must be on a GPU, not on {dev}")
    device, stream = _torch_calls()
    index = dev.index
    if device() == index:
        st = fn(desc, *args, stream(index))
    else:
        import torch
        with torch.cuda.device(dev):
            st = fn(desc, *args, stream(index))
    if st != 0:
        raise Gdn2Error(st, name)


def _bytes(name, desc):
    n = ctypes.c_size_t(0)
    st = _call(name)(desc, ctypes.byref(n))
    if st != 0:
        raise Gdn2Error(st, name)
    return int(n.value)


@functools.lru_cache(maxsize=256)
def _need(name, make, *sizes):
    """Workspace bytes of a request, which depend on its sizes alone."""
    return _bytes(name, make(*sizes))


def _dtype_code(t, name):
    import torch
    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    if t.dtype == torch.float32:
        return GDN2_F32
    raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def make_linear_desc(batch, seqlen, heads, dk, dv, dtype=GDN2_BF16, decay_kind=GDN2_DECAY_TOKEN,
                     q_scale=1.0) -> Gdn2LinearDesc:
    return Gdn2LinearDesc(batch, seqlen, heads, dk, dv, dtype, decay_kind, q_scale, 0)


def make_norm_desc(rows, groups, dim, dtype=GDN2_BF16, weight_dtype=GDN2_F32, eps=1e-5) -> Gdn2NormDesc:
    return Gdn2NormDesc(rows, groups, dim, dtype, weight_dtype, eps, 0)


def _sizes(q, k, v, log_decay, tok, batch, seqlen, q_scale):
    """What make_linear_desc takes, of checked inputs."""
    import torch
    H, dk, dv, dev = tok[-1], k.shape[-1], v.shape[-1], k.device
    code = _dtype_code(k, "q/k/v")
    for t, n, d in ((q, "q", dk), (k, "k", dk), (v, "v", dv)):
        _like(t, n, tok + (d,), k.dtype, dev)
    # [H]: one value per head; a per-token decay has all of tok's axes
    kind = GDN2_DECAY_HEAD if log_decay.dim() == 1 else GDN2_DECAY_TOKEN
    _like(log_decay, "log_decay", (H,) if kind == GDN2_DECAY_HEAD else tok, torch.float32, dev)
    return batch, seqlen, H, dk, dv, code, kind, q_scale


def _packed(k, cu_seqlens):
    import torch
    lead = k.shape[:-3]
    if k.dim() < 3 or len(lead) > 1 or (len(lead) == 1 and lead[0] != 1):
        raise ValueError("packed tensors are [T,H,d] or [1,T,H,d]")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of N+1 offsets")
    _check(cu_seqlens, "cu_seqlens", tuple(cu_seqlens.shape), (torch.int32,), k.device)
    return tuple(k.shape[:-1]), cu_seqlens.numel() - 1, k.shape[-3]


def _space(workspace, need, dev):
    """The scratch to use and its bytes: `workspace` when given, else a new one."""
    import torch
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need else (None, 0)
    _check(workspace, "workspace", tuple(workspace.shape), (torch.uint8,), dev)
    return workspace, workspace.numel()


def linear_chunk_fwd_workspace(desc: Gdn2LinearDesc) -> int:
    return _bytes("gdn2_linear_fwd_workspace", desc)


def linear_chunk_fwd_varlen_workspace(desc: Gdn2LinearDesc) -> int:
    return _bytes("gdn2_linear_fwd_varlen_workspace", desc)


def linear_chunk_bwd_workspace(desc: Gdn2LinearDesc) -> int:
    return _bytes("gdn2_linear_bwd_workspace", desc)


def linear_chunk_bwd_varlen_workspace(desc: Gdn2LinearDesc) -> int:
    return _bytes("gdn2_linear_bwd_varlen_workspace", desc)


def layer_norm_bwd_workspace(desc: Gdn2NormDesc) -> int:
    return _bytes("gdn2_layer_norm_bwd_workspace", desc)


def _fwd(q, k, v, log_decay, cu_seqlens, state0, q_scale, out, state_out, return_state, workspace):
    import torch
    if cu_seqlens is None:
        if k.dim() != 4:
            raise ValueError("k is [B,T,H,dk]")
        tok, N, T = tuple(k.shape[:-1]), k.shape[0], k.shape[1]
    else:
        tok, N, T = _packed(k, cu_seqlens)
    sizes = _sizes(q, k, v, log_decay, tok, N, T, q_scale)
    dev, sshape, f32 = k.device, (N, tok[-1], k.shape[-1], v.shape[-1]), torch.float32
    if state0 is not None:
        _like(state0, "state0", sshape, f32, dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _like(out, "out", v.shape, v.dtype, dev)
    if state_out is not None:
        _like(state_out, "state_out", sshape, f32, dev)
    elif return_state:
        state_out = torch.empty(sshape, dtype=torch.float32, device=dev)
    name = "gdn2_linear_fwd" if cu_seqlens is None else "gdn2_linear_fwd_varlen"
    ws, n = (None, 0) if workspace is False else _space(None if workspace is True else workspace,
                                                        _need(name + "_workspace", make_linear_desc, *sizes[:-1]), dev)
    _run(name, dev, make_linear_desc(*sizes), *([] if cu_seqlens is None else [_ptr(cu_seqlens)]), _ptr(q), _ptr(k), _ptr(v),
         _ptr(log_decay), _ptr(state0), _ptr(out), _ptr(state_out), _ptr(ws), n)
    return out, state_out


def linear_chunk_fwd(q, k, v, log_decay, state0=None, q_scale=1.0, out=None, state_out=None, return_state=True,
                     workspace=True):
    """Chunked linear attention: S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T, o_t = q_scale S_t^T q_t.

    q, k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32, one dtype); log_decay fp32
    [B,T,H], or [H] for one value per head; state0 [B,H,dk,dv] fp32 or None.
    ``workspace``: True (or None) allocates the scratch that long sequences on
    few chains run in parallel segments with, False runs without, or a uint8
    device tensor of at least linear_chunk_fwd_workspace() bytes.
    Returns (o like v, final state [B,H,dk,dv] fp32 or None).
    """
    return _fwd(q, k, v, log_decay, None, state0, q_scale, out, state_out, return_state, workspace)


def linear_chunk_fwd_varlen(q, k, v, log_decay, cu_seqlens, state0=None, q_scale=1.0, out=None, state_out=None,
                            return_state=True, workspace=True):
    """``linear_chunk_fwd`` over N sequences packed along one token axis.

    q, k [T,H,dk], v [T,H,dv], log_decay [T,H] or [H] (or all but [H] with a
    leading 1); cu_seqlens int32 [N+1] on the device; states [N,H,dk,dv].
    Tokens outside every sequence are not written: a given ``out`` keeps
    them, a new one has any value there.
    """
    return _fwd(q, k, v, log_decay, cu_seqlens, state0, q_scale, out, state_out, return_state, workspace)


def _bwd(q, k, v, log_decay, cu_seqlens, state0, d_o, d_state, q_scale, want_state0, workspace):
    import torch
    if cu_seqlens is None:
        if k.dim() != 4:
            raise ValueError("k is [B,T,H,dk]")
        tok, N, T = tuple(k.shape[:-1]), k.shape[0], k.shape[1]
    else:
        tok, N, T = _packed(k, cu_seqlens)
    sizes = _sizes(q, k, v, log_decay, tok, N, T, q_scale)
    dev, sshape, f32 = k.device, (N, tok[-1], k.shape[-1], v.shape[-1]), torch.float32
    _like(d_o, "d_o", v.shape, v.dtype, dev)
    for t, n in ((state0, "state0"), (d_state, "d_state")):
        if t is not None:
            _like(t, n, sshape, f32, dev)
    if want_state0 is None:
        want_state0 = state0 is not None
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
             d_log_decay=torch.empty_like(log_decay),
             d_state0=torch.empty(sshape, dtype=torch.float32, device=dev) if want_state0 else None)
    name = "gdn2_linear_bwd" if cu_seqlens is None else "gdn2_linear_bwd_varlen"
    ws, n = _space(workspace, _need(name + "_workspace", make_linear_desc, *sizes[:-1]), dev)
    _run(name, dev, make_linear_desc(*sizes), *([] if cu_seqlens is None else [_ptr(cu_seqlens)]), _ptr(q), _ptr(k), _ptr(v),
         _ptr(log_decay), _ptr(state0), _ptr(d_o), _ptr(d_state), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
         _ptr(g["d_log_decay"]), _ptr(g["d_state0"]), _ptr(ws), n)
    return g


def linear_chunk_bwd(q, k, v, log_decay, state0, d_o, d_state=None, q_scale=1.0, want_state0=None, workspace=None):
    """Gradients of <d_o, o> + <d_state, S_T> for ``linear_chunk_fwd``.

    d_o like v; d_state [B,H,dk,dv] fp32 or None (zeros).  Returns a dict: dq,
    dk, dv in the type of q, k, v; d_log_decay fp32 like log_decay; d_state0
    fp32 (``want_state0``: by default where state0 is given, else None).
    ``workspace``: None allocates it, or a uint8 device tensor of at least
    linear_chunk_bwd_workspace() bytes.
    """
    return _bwd(q, k, v, log_decay, None, state0, d_o, d_state, q_scale, want_state0, workspace)


def linear_chunk_bwd_varlen(q, k, v, log_decay, cu_seqlens, state0, d_o, d_state=None, q_scale=1.0, want_state0=None,
                            workspace=None):
    """``linear_chunk_bwd`` for ``linear_chunk_fwd_varlen``: packed tensors, states [N,H,dk,dv].

    Gradients of tokens outside every sequence are not written (any value).
    """
    return _bwd(q, k, v, log_decay, cu_seqlens, state0, d_o, d_state, q_scale, want_state0, workspace)


def linear_recurrent_step(q, k, v, log_decay, state, q_scale=1.0, out=None):
    """One decode step for N sequences; updates ``state`` [N,H,dk,dv] fp32 in place.

    q, k [N,H,dk], v [N,H,dv]; log_decay fp32 [N,H] or [H].  Returns o like v.
    """
    import torch
    if k.dim() != 3:
        raise ValueError("k is [N,H,dk]")
    tok = tuple(k.shape[:-1])
    sizes = _sizes(q, k, v, log_decay, tok, tok[0], 1, q_scale)
    _like(state, "state", tok + (k.shape[-1], v.shape[-1]), torch.float32, k.device)
    if out is None:
        out = torch.empty_like(v)
    else:
        _like(out, "out", v.shape, v.dtype, k.device)
    _run("gdn2_linear_step", k.device, make_linear_desc(*sizes), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(state), _ptr(out))
    return out


def _norm_sizes(x, weight, bias, eps):
    """What make_norm_desc takes, of checked inputs."""
    if x.dim() < 1:
        raise ValueError("x needs an axis to normalise")
    D = x.shape[-1]
    code = _dtype_code(x, "x")
    _like(x, "x", x.shape, x.dtype, x.device)
    groups, wd = 1, GDN2_F32
    first = weight if weight is not None else bias
    if first is not None:
        wd = _dtype_code(first, "weight")
        if first.dim() == 2 and x.dim() >= 2:
            groups = x.shape[-2]
        shape = (D,) if first.dim() == 1 else (groups, D)
        for t, n in ((weight, "weight"), (bias, "bias")):
            if t is not None:
                _like(t, n, shape, first.dtype, x.device)
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return rows, max(groups, 1), D, code, wd, eps


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None):
    """Layer norm over the last axis of x (bf16 or fp32).

    weight, bias: [D], or [x.shape[-2], D] for a row of them per head; fp32 or
    bf16, None for ones / zeros.  Returns (y like x, mean, rstd), the last two
    fp32 of x's shape without its last axis.
    """
    import torch
    sizes = _norm_sizes(x, weight, bias, eps)
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", x.shape, x.dtype, x.device)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _run("gdn2_layer_norm_fwd", x.device, make_norm_desc(*sizes), _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), _ptr(mean), _ptr(rstd))
    return out, mean, rstd


def layer_norm_bwd(dy, x, weight, mean, rstd, want_weight=None, want_bias=False, workspace=None, bias=None):
    """Gradients of <dy, y> for ``layer_norm_fwd``: (dx, d_weight, d_bias).

    ``weight`` None: ones.  d_weight (``want_weight``: by default where weight
    is given) and d_bias (``want_bias``) have the weight's shape and type
    (without one those of ``bias``, the forward's, which is not read; [D] fp32
    without either), None where not wanted.  ``workspace``: None allocates it,
    or a uint8 device tensor of at least layer_norm_bwd_workspace() bytes.
    """
    import torch
    sizes = _norm_sizes(x, weight, bias, 0.0)
    dev, stat, first = x.device, x.shape[:-1], weight if weight is not None else bias
    _like(dy, "dy", x.shape, x.dtype, dev)
    _like(mean, "mean", stat, torch.float32, dev)
    _like(rstd, "rstd", stat, torch.float32, dev)
    if want_weight is None:
        want_weight = weight is not None

    def like():
        return torch.empty(x.shape[-1:], dtype=torch.float32, device=dev) if first is None else torch.empty_like(first)

    dx = torch.empty_like(x)
    dw, db = like() if want_weight else None, like() if want_bias else None
    ws, n = None, 0
    if want_weight or want_bias or workspace is not None:
        ws, n = _space(workspace, _need("gdn2_layer_norm_bwd_workspace", make_norm_desc, *sizes[:-1]), dev)
    _run("gdn2_layer_norm_bwd", dev, make_norm_desc(*sizes), _ptr(dy), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw),
         _ptr(db), _ptr(ws), n)
    return dx, dw, db
