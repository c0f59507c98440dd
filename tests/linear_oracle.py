"""fp64 reference of linear attention with a decay for each head and of layer
norm, token by token and row by row on the CPU, and the error bounds that the
parity tests hold the kernels to.

Bounds.  u = 2^-8 is the largest relative error of one rounding to bf16,
e = 2^-24 that of one to fp32.  Elementwise, with |.| the same recurrence on
absolute values (every term positive), the forward's output differs by at most

    u |o|  (the output's rounding)  +  u |.|  (the state's, as it is read)
    +  2^-15 |.|  (the scores in two bf16 parts)  +  n e |.|  (fp32 sums)

with n the sums' length plus the exponents' size, and without the terms in u
and 2^-15 for fp32 inputs.  As a relative L2 norm over many elements, whose
rounding errors are spread evenly over half a step, one rounding is at most
2^-8 / sqrt(3) = 2.26e-3 and two are 3.2e-3; fp32 results are held to 1e-5.
"""
from __future__ import annotations

import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24
ONE, TWO, F32 = U / math.sqrt(3) + 1e-5, U * math.sqrt(2 / 3) + 1e-5, 1e-5


def _f64(x):
    return None if x is None else x.detach().double().cpu()


def linear_forward(q, k, v, la, s0, scale):
    """[B,T,H,*] tensors, la [B,T,H] or [H]: (o, final state), fp64."""
    q, k, v, la, s0 = map(_f64, (q, k, v, la, s0))
    B, T, H, dk = k.shape
    a = (la.expand(B, T, H) if la.dim() == 1 else la).exp()
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64) if s0 is None else s0.clone()
    o = torch.empty(v.shape, dtype=torch.float64)
    for t in range(T):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, :, None] * S).sum(2)
    return o, S


def linear_backward(q, k, v, la, s0, scale, d_o, d_s):
    """Gradients of <d_o, o> + <d_s, S_T>: dq, dk, dv, d_log_decay, d_state0."""
    q, k, v, la, s0, d_o, d_s = map(_f64, (q, k, v, la, s0, d_o, d_s))
    B, T, H, dk = k.shape
    a = (la.expand(B, T, H) if la.dim() == 1 else la).exp()
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64) if s0 is None else s0.clone()
    before = []
    dq = torch.empty_like(q)
    for t in range(T):
        before.append(S)
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * (S * d_o[:, t, :, None, :]).sum(3)
    dS = torch.zeros_like(S) if d_s is None else d_s.clone()
    dk_, dv, dla = torch.empty_like(k), torch.empty_like(v), torch.empty(B, T, H, dtype=torch.float64)
    for t in range(T - 1, -1, -1):
        dS = dS + scale * q[:, t, :, :, None] * d_o[:, t, :, None, :]
        dk_[:, t] = (dS * v[:, t, :, None, :]).sum(3)
        dv[:, t] = (dS * k[:, t, :, :, None]).sum(2)
        dla[:, t] = a[:, t] * (dS * before[t]).sum((2, 3))
        dS = a[:, t, :, None, None] * dS
    return dict(dq=dq, dk=dk_, dv=dv, d_log_decay=dla.sum((0, 1)) if la.dim() == 1 else dla, d_state0=dS)


def rel_l2(x, ref):
    d = (x.double().cpu() - ref).norm()
    n = ref.norm()
    return float(d / n) if n > 0 else float(d)


def check(name, x, ref, tol, bound=None):
    """Finite, within `tol` in relative L2 (tensors of 4096 elements or more, or all for fp32 tolerances), and
    elementwise within `bound`."""
    y = x.double().cpu()
    assert y.shape == ref.shape, f"{name}: shape {tuple(y.shape)} for {tuple(ref.shape)}"
    assert torch.isfinite(y).all(), f"{name}: non-finite values"
    r = rel_l2(x, ref)
    if tol <= F32 or ref.numel() >= 4096:
        assert r <= tol, f"{name}: rel_l2 {r:.3e} > {tol:.2e}"
    if bound is not None:
        over = ((y - ref).abs() - bound).max() if y.numel() else torch.tensor(0.0)
        assert over <= 0, f"{name}: an element is {float(over):.3e} past its bound"


def layer_norm(x, w, b, eps):
    x, w, b = map(_f64, (x, w, b))
    mean = x.mean(-1)
    rstd = 1.0 / ((x - mean[..., None]).square().mean(-1) + eps).sqrt()
    y = (x - mean[..., None]) * rstd[..., None]
    y = y if w is None else y * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """dx, and the gradients of a weight and bias [D] or [G, D] (w None: [D])."""
    dy, x, w, mean, rstd = map(_f64, (dy, x, w, mean, rstd))
    h = (x - mean[..., None]) * rstd[..., None]
    e = dy if w is None else dy * w
    dx = rstd[..., None] * (e - e.mean(-1, keepdim=True) - h * (e * h).mean(-1, keepdim=True))
    keep = 1 if w is None else w.dim()
    axes = tuple(range(x.dim() - keep))
    return dx, (dy * h).sum(axes), dy.sum(axes)
