"""Rotary positions and norms of queries and keys (argument marshalling only).

As in ``linear``: torch CUDA (HIP) tensors are checked and their device
pointers go to ``libgdn2.so`` with torch's current stream of their device.
There is no CPU or torch fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math

from .binding import GDN2_BF16, GDN2_F32
from .facts import contiguous, facts, like, needed, new_like
from .linear import _bytes, _ptr, _register, _run, _space

GDN2_ROTARY_HALF, GDN2_ROTARY_INTERLEAVED = 0, 1
GDN2_QK_NONE, GDN2_QK_RMS, GDN2_QK_L2 = 0, 1, 2


class Gdn2RotaryDesc(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("period", ctypes.c_int64), ("q_heads", ctypes.c_int64),
        ("k_heads", ctypes.c_int64), ("dim", ctypes.c_int64), ("rotary", ctypes.c_int64),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("offset", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("magnitude", ctypes.c_float),
    ]


_vp, _sz, _rd = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Gdn2RotaryDesc)
_register(("gdn2_rotary_fwd", [_rd] + [_vp] * 7), ("gdn2_rotary_bwd", [_rd] + [_vp] * 7),
          ("gdn2_qk_norm_fwd", [_rd] + [_vp] * 9),
          ("gdn2_qk_norm_bwd_workspace", [_rd, ctypes.POINTER(ctypes.c_size_t)]),
          ("gdn2_qk_norm_bwd", [_rd] + [_vp] * 13 + [_sz, _vp]))


def make_rotary_desc(tokens, q_heads, k_heads, dim, rotary, period=None, q_stride=None, k_stride=None, offset=0,
                     dtype=GDN2_BF16, weight_dtype=GDN2_F32, layout=GDN2_ROTARY_HALF, norm=GDN2_QK_NONE, eps=0.0,
                     magnitude=1.0) -> Gdn2RotaryDesc:
    return Gdn2RotaryDesc(tokens, max(tokens, 1) if period is None else period, q_heads, k_heads, dim, rotary,
                          q_heads * dim if q_stride is None else q_stride, k_heads * dim if k_stride is None else k_stride,
                          offset, dtype, weight_dtype, layout, norm, eps, magnitude)


def rotary_frequencies(rotary, base=10000.0, scaling=None, factor=1.0, original_length=None, slow=1.0, fast=32.0,
                       device="cuda"):
    """Radians a position of the rotary/2 pairs, fp64 [rotary/2]: base^(-2j/rotary), scaled for long contexts.

    ``scaling``: None; "linear" divides every frequency by ``factor``; "base"
    raises the base by factor^(rotary/(rotary-2)), which leaves the fastest pair
    and divides the slowest by ``factor``; "parts" keeps pairs that turn more
    than ``fast`` times over ``original_length`` positions, divides those that
    turn less than ``slow`` times by ``factor`` and mixes linearly between (the
    rotation's magnitude then usually is 0.1 ln(factor) + 1).
    """
    import torch
    if rotary < 2 or rotary % 2:
        raise ValueError("rotary must be even and positive")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        base = base * factor ** (rotary / max(rotary - 2, 1))
    f = torch.tensor([base ** (-2.0 * j / rotary) for j in range(rotary // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_length is None or not fast > slow:
            raise ValueError("scaling by parts needs original_length and fast > slow")
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = keep * f + (1 - keep) * (f / factor)
    return f.to(device)


def _strided(f, name, tok, dtype, dev):
    """Heads, channels and the elements between tokens of [*tok, H, d]: tokens evenly spaced, a token contiguous."""
    shape, st, dt, on = f
    if dt != dtype:
        raise TypeError(f"{name} must be {dtype}, not {dt}")
    if on != dev:
        raise ValueError(f"{name} must be on {dev}, not on {on}")
    if len(shape) != len(tok) + 2 or tuple(shape[:-2]) != tok:
        raise ValueError(f"{name} has shape {tuple(shape)}, its tokens must be {tok}")
    H, d = shape[-2:]
    if contiguous(shape, st):
        return H, d, H * d
    ok = (d == 1 or st[-1] == 1) and (H == 1 or st[-2] == d)
    step, span = None, 1  # of the innermost token axis that has more than one token
    for n, s in zip(reversed(tok), reversed(st[:-2])):
        if n != 1:
            if step is None:
                step = s
            ok = ok and s == step * span
            span *= n
    step = H * d if step is None else step
    if not ok or step < H * d:
        raise ValueError(f"{name} must hold each token's heads contiguously and its tokens at one distance")
    return H, d, step


def _type_code(dtype, name):
    import torch
    if dtype == torch.bfloat16:
        return GDN2_BF16
    if dtype == torch.float32:
        return GDN2_F32
    raise TypeError(f"{name} must be bfloat16 or float32, not {dtype}")


@functools.lru_cache(maxsize=1024)
def _request(names, q, k, freq, positions, q_weight, k_weight, interleaved, magnitude, norm, eps):
    """The descriptor (offset 0) of checked facts."""
    import torch
    needed(q, names[0])
    shape, _, dtype, dev = q
    if len(shape) < 3:
        raise ValueError(f"{names[0]} is [..., H, d] with at least one token axis")
    tok = tuple(shape[:-2])
    code = _type_code(dtype, names[0])
    Hq, d, qs = _strided(q, names[0], tok, dtype, dev)
    Hk, ks = 0, 0
    if k is not None:
        Hk, dk, ks = _strided(k, names[1], tok, dtype, dev)
        if dk != d:
            raise ValueError(f"{names[1]} has {dk} channels, {names[0]} has {d}")
    rot = 0
    if freq is not None:
        if len(freq[0]) != 1:
            raise ValueError("freq is [rotary/2]")
        like(freq, "freq", freq[0], (torch.float64,), dev)
        rot = 2 * freq[0][0]
        if rot > d:
            raise ValueError(f"freq turns {rot} channels of {d}")
    period = max(tok[-1], 1)  # positions count along the last token axis
    if positions is not None:
        n = len(positions[0])
        if n < 1 or tuple(positions[0]) != tok[max(len(tok) - n, 0):]:
            raise ValueError(f"positions have shape {tuple(positions[0])}, not {tok} or its last axes")
        like(positions, "positions", positions[0], (torch.int32,), dev)
        period = max(math.prod(positions[0]), 1)
    wd, first = GDN2_F32, q_weight if q_weight is not None else k_weight
    if first is not None:
        wd = _type_code(first[2], "weight")
        for w, n in ((q_weight, names[0]), (k_weight, names[1])):
            if w is not None:
                like(w, f"{n}_weight", (d,), (first[2],), dev)
    return make_rotary_desc(math.prod(tok), Hq, Hk, d, rot, period, qs, ks, 0, code, wd,
                            GDN2_ROTARY_INTERLEAVED if interleaved else GDN2_ROTARY_HALF, norm, eps, magnitude)


def _plan(q, k, freq, positions, offset, interleaved, magnitude, norm=GDN2_QK_NONE, eps=0.0, q_weight=None, k_weight=None,
          names=("q", "k")):
    """The descriptor of a checked request."""
    desc = _request(names, facts(q), facts(k), facts(freq), facts(positions), facts(q_weight), facts(k_weight),
                    bool(interleaved), float(magnitude), norm, float(eps))
    if offset:  # the shared one stays as it is
        desc = Gdn2RotaryDesc.from_buffer_copy(desc)
        desc.offset = offset
        if desc.offset != offset:  # ctypes keeps the low 64 bits
            raise ValueError("offset is out of range")
    return desc


def _out(given, name, x):
    if given is None:
        return None if x is None else new_like(x)
    if x is None:
        raise ValueError(f"{name} has nothing to hold")
    like(facts(given), name, x.shape, (x.dtype,), x.device)
    return given


_NORMS = {"rms": GDN2_QK_RMS, "l2": GDN2_QK_L2}


def _norm_code(norm):
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'rms' or 'l2', not {norm!r}")
    return _NORMS[norm]


def rotary_fwd(q, k, freq, positions=None, offset=0, interleaved=False, magnitude=1.0, q_out=None, k_out=None):
    """Turn the first 2 * len(freq) channels of every head by position * freq.

    q [..., Hq, d], k [..., Hk, d] or None (bf16 or fp32, one dtype, at least
    one token axis): contiguous, or slices that hold each token's heads together
    with the tokens at one distance.  freq: fp64 [rotary/2], see
    ``rotary_frequencies``.  positions: int32 of the tokens' shape or its last
    axes; None counts along the last token axis.  ``offset`` is added to either.
    Pairs are channels (j, j + rotary/2), or (2j, 2j + 1) with ``interleaved``.
    q_out, k_out: contiguous outputs, which may be q and k themselves where
    these are contiguous.  Returns (q_out, k_out).
    """
    desc = _plan(q, k, freq, positions, offset, interleaved, magnitude)
    q_out, k_out = _out(q_out, "q_out", q), _out(k_out, "k_out", k)
    _run("gdn2_rotary_fwd", q.device, desc, _ptr(q), _ptr(k), _ptr(freq), _ptr(positions), _ptr(q_out), _ptr(k_out))
    return q_out, k_out


def rotary_bwd(d_q_out, d_k_out, freq, positions=None, offset=0, interleaved=False, magnitude=1.0, dq=None, dk=None):
    """Gradients (dq, dk) of <d_q_out, q_out> + <d_k_out, k_out> for ``rotary_fwd``, arguments as there."""
    desc = _plan(d_q_out, d_k_out, freq, positions, offset, interleaved, magnitude, names=("d_q_out", "d_k_out"))
    dq, dk = _out(dq, "dq", d_q_out), _out(dk, "dk", d_k_out)
    _run("gdn2_rotary_bwd", d_q_out.device, desc, _ptr(d_q_out), _ptr(d_k_out), _ptr(freq), _ptr(positions),
         _ptr(dq), _ptr(dk))
    return dq, dk


def qk_norm_rotary_fwd(q, k, q_weight=None, k_weight=None, freq=None, positions=None, offset=0, interleaved=False,
                       magnitude=1.0, norm="rms", eps=1e-6, q_out=None, k_out=None):
    """Norm of every head of q and k, a weight, and the rotation of ``rotary_fwd``, in one pass.

    norm "rms": x / sqrt(mean x^2 + eps); "l2": x / |x| (eps takes no part; zero
    rows stay zero).  q_weight, k_weight: [d], fp32 or bf16 (one type), None for ones.
    freq None: no rotation.  Other arguments as for ``rotary_fwd``.  Returns
    (q_out, k_out).
    """
    desc = _plan(q, k, freq, positions, offset, interleaved, magnitude, _norm_code(norm), eps, q_weight, k_weight)
    q_out, k_out = _out(q_out, "q_out", q), _out(k_out, "k_out", k)
    _run("gdn2_qk_norm_fwd", q.device, desc, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(freq),
         _ptr(positions), _ptr(q_out), _ptr(k_out))
    return q_out, k_out


def qk_norm_rotary_bwd_workspace(desc: Gdn2RotaryDesc) -> int:
    return _bytes("gdn2_qk_norm_bwd_workspace", desc)


@functools.lru_cache(maxsize=256)
def _sum_bytes(tokens, q_heads, k_heads, dim, rotary, dtype):
    return qk_norm_rotary_bwd_workspace(make_rotary_desc(tokens, q_heads, k_heads, dim, rotary, dtype=dtype, norm=GDN2_QK_RMS))


def qk_norm_rotary_bwd(d_q_out, d_k_out, q, k, q_weight=None, k_weight=None, freq=None, positions=None, offset=0,
                       interleaved=False, magnitude=1.0, norm="rms", eps=1e-6, workspace=None):
    """Gradients of <d_q_out, q_out> + <d_k_out, k_out> for ``qk_norm_rotary_fwd``.

    d_q_out, d_k_out are contiguous, q and k the forward's inputs.  Returns a
    dict: dq, dk like q, k; d_q_weight, d_k_weight like the weights, None where
    there is none.  ``workspace``: None allocates it, or a uint8 device tensor
    of at least qk_norm_rotary_bwd_workspace() bytes.
    """
    desc = _plan(q, k, freq, positions, offset, interleaved, magnitude, _norm_code(norm), eps, q_weight, k_weight)
    dev = q.device
    for g, x, n in ((d_q_out, q, "d_q_out"), (d_k_out, k, "d_k_out")):
        if (x is None) != (g is None):
            raise ValueError(f"{n} is missing" if g is None else f"{n} has no input")
        if x is not None:
            like(facts(g), n, x.shape, (q.dtype,), dev)
    dq, dk = _out(None, "dq", q), _out(None, "dk", k)
    dqw = None if q_weight is None else new_like(q_weight)
    dkw = None if k_weight is None else new_like(k_weight)
    ws, n = None, 0
    if dqw is not None or dkw is not None or workspace is not None:
        ws, n = _space(workspace, _sum_bytes(desc.tokens, desc.q_heads, desc.k_heads, desc.dim, desc.rotary, desc.dtype), dev)
    _run("gdn2_qk_norm_bwd", dev, desc, _ptr(d_q_out), _ptr(d_k_out), _ptr(q), _ptr(k), _ptr(q_weight),
         _ptr(k_weight), _ptr(freq), _ptr(positions), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), _ptr(ws), n)
    return dict(dq=dq, dk=dk, d_q_weight=dqw, d_k_weight=dkw)
