"""fp64 reference (CPU) of rotary positions and of the query and key norms, row
by row, with the error bounds that the parity tests hold the kernels to.

Bounds, elementwise, with e = 2^-24 (half a step of fp32, relative).  A cosine
or sine of the kernel: the reduced angle is at most pi/4 and rounded twice (1.6
e), the series adds at most 3 e and the magnitude's product 1 e, together below
6 e m.  A turned element sums two products of it: 2 more roundings of each
product, so it is off by at most 9 e m (|u| + |v|), T below.

The norm's sum of squares: a lane adds at most 16 squares in four sums (4
products and 4 sums each) and joins them (2), then come at most 6 joins over
lanes, the mean's product and eps: 18 e of it, 9 e of r = 1 / sqrt.  The root's
approximation (2 e) is refined by a step of three products, a difference and a
product: 3.5 e.  With h = x r that makes 13.5 e of h, 15 e of w h, and 24 e m (|wh|
+ |wh'|) behind the turn.  (Rows summed in 64 bits have less.)

Backward: w g is off by 10 e; a term w g h of the channel sum by 25 e, and the
sum is added up by lanes of at most 16 terms, then over at most 64 lanes (6
joins), each rounding its partial sum: 22 e more; h n sum is off by 13.5 + 48 + 2
e; with the difference and r's product dx is off by at most 80 e r (w T + |h| n
sum w T |h|).  A weight's gradient is a sum over rows of g h, each off by 24 e: a
lane adds at most 40 in fp32, then come at most 8 joins: 72 e sum T |h|.  A bf16
result is rounded once more, by at most 2^-8 of it.
"""
from __future__ import annotations

import torch

E = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _d(x):
    return None if x is None else x.detach().to("cpu", F64)


def angles(tok, freq, positions, offset):
    if positions is None:
        p = torch.arange(tok[-1])
    else:
        p = positions.detach().cpu()
    p = (p.to(torch.int64) + offset).to(F64).expand(tok)
    return p[..., None, None] * _d(freq)


def rotate(x, theta, m, inter, back=False):
    """x [..., H, d] fp64, theta [..., 1, rot/2]: (the turned x, m (|u| + |v|) in the places of u and v)."""
    rot = 2 * theta.shape[-1]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    c, s = m * theta.cos(), m * theta.sin() * (-1 if back else 1)
    y, size = x.clone(), x.abs()
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = c * u - s * v, s * u + c * v
    size[..., a] = size[..., b] = abs(m) * (u.abs() + v.abs())
    return y, size


def turn_only(x, freq, positions, offset, inter, m, back=False):
    x = _d(x)
    y, size = rotate(x, angles(tuple(x.shape[:-2]), freq, positions, offset), m, inter, back)
    return y, 9 * E * size


def _inverse(x, norm, eps):
    ss = x.square().sum(-1, keepdim=True)
    s = ss / x.shape[-1] + eps if norm == "rms" else ss
    return torch.where(s > 0, 1.0 / s.sqrt(), torch.zeros_like(s))


def norm_turn(x, w, freq, positions, offset, inter, m, norm, eps):
    x = _d(x)
    y = x * _inverse(x, norm, eps)
    y = y if w is None else y * _d(w)
    if freq is None:
        return y, 15 * E * y.abs()
    y, size = rotate(y, angles(tuple(x.shape[:-2]), freq, positions, offset), m, inter)
    return y, 24 * E * size


def norm_turn_backward(dy, x, w, freq, positions, offset, inter, m, norm, eps):
    """dx, dw [d] and their bounds."""
    x, dy = _d(x), _d(dy)
    r = _inverse(x, norm, eps)
    h, n = x * r, (1.0 / x.shape[-1] if norm == "rms" else 1.0)
    w = torch.ones(x.shape[-1], dtype=F64) if w is None else _d(w)
    if freq is None:
        g, size = dy, dy.abs()
    else:
        g, size = rotate(dy, angles(tuple(x.shape[:-2]), freq, positions, offset), m, inter, back=True)
    dx = r * (w * g - h * n * (w * g * h).sum(-1, keepdim=True))
    t = w.abs() * size
    bound = 80 * E * r * (t + h.abs() * n * (t * h.abs()).sum(-1, keepdim=True))
    axes = tuple(range(x.dim() - 1))
    return dx, (g * h).sum(axes), bound, 72 * E * (size * h.abs()).sum(axes)


def check(name, got, want, bound):
    """Right shape, finite, and every element within its bound and its own rounding."""
    y = got.detach().cpu().double()
    assert y.shape == want.shape, f"{name}: shape {tuple(y.shape)} for {tuple(want.shape)}"
    assert torch.isfinite(y).all(), f"{name}: non-finite values"
    limit = bound + 1e-40
    if got.dtype != torch.float32:
        limit = limit + half_step(got.dtype) * (want.abs() + bound)
    over = ((y - want).abs() - limit).max() if y.numel() else torch.tensor(0.0)
    assert over <= 0, f"{name}: an element is {float(over):.3e} past its bound (largest value {float(want.abs().max()):.3e})"
