"""fp64 reference (CPU) of the gated scan, token by token, with the error
bounds that the parity tests hold the kernels to.

Bounds, elementwise, with e = 2^-24.  A decay a is off by at most (6 + 2 |g|) e
of itself, g the stored gate: its exponent's product with log2(e) is rounded to
2 |g| e, and the exponential, the reciprocal and the difference from 1 add at
most 6 roundings; so is w = 1 - a.  A term of a state that has passed n tokens
has been multiplied by n decays and joined at most n + 20 times (n times within
its lane, and over lanes, groups and tiles in between), each joint one product
and one sum: its error is the sum of those of its decays and of 2 (n + 20)
roundings, which the recurrence on absolute values carries along:

    E_t = a_t (E_{t-1} + (8 + 2 |g_t|) e H_{t-1}) + (6 + 2 |g_t|) e |u_t|,
    H_t = a_t H_{t-1} + |u_t|,     error of h_t <= E_t + 40 e H_t

and the same backward for r.  A bf16 result is rounded once more, by 2^-8.
"""
from __future__ import annotations

import torch

from tests.rotary_oracle import E, F64, check, half_step  # noqa: F401


def _d(x):
    return None if x is None else x.detach().to("cpu", F64)


def decays(gate, logits):
    g = _d(gate)
    log_a = -torch.nn.functional.softplus(g) if logits else g
    size = torch.where(torch.isfinite(g), g.abs(), torch.zeros_like(g)).clamp_max(200.0)
    return log_a.exp(), -torch.expm1(log_a), 6 + 2 * size


def forward(x, gate, s0, logits, comp):
    """[T, D] of one sequence, s0 [D] or None: h, its bound, the states entering each token and their bound."""
    x = _d(x)
    a, w, k = decays(gate, logits)
    T, D = x.shape
    u = w * x if comp else x
    h = torch.zeros(D, dtype=F64) if s0 is None else _d(s0).clone()
    H, err = h.abs(), torch.zeros(D, dtype=F64)
    hs, bs, before, bbefore = (torch.empty(T, D, dtype=F64) for _ in range(4))
    for t in range(T):
        before[t], bbefore[t] = h, err + 40 * E * H
        err = a[t] * (err + (k[t] + 2) * E * H) + k[t] * E * u[t].abs()
        H = a[t] * H + u[t].abs()
        h = a[t] * h + u[t]
        hs[t], bs[t] = h, err + 40 * E * H
    return hs, bs, before, bbefore, (h, err + 40 * E * H)


def backward(dy, x, gate, s0, ds, logits, comp):
    """Gradients of <dy, h> + <ds, h_T>: dict of (value, bound) dx, d_gate, d_state0."""
    x, dy = _d(x), _d(dy)
    a, w, k = decays(gate, logits)
    T, D = x.shape
    _, _, before, bbefore, _ = forward(x, gate, s0, logits, comp)
    r = torch.zeros(D, dtype=F64) if ds is None else _d(ds).clone()
    R, err = r.abs(), torch.zeros(D, dtype=F64)
    out = {n: (torch.empty(T, D, dtype=F64), torch.empty(T, D, dtype=F64)) for n in ("dx", "d_gate")}
    for t in range(T - 1, -1, -1):
        s, S, serr = dy[t] + r, dy[t].abs() + R, err
        sb = serr + 42 * E * S
        ww = w[t] if comp else torch.ones_like(r)
        out["dx"][0][t] = ww * s
        out["dx"][1][t] = ww * (sb + k[t] * E * S)
        err = a[t] * (serr + (k[t] + 2) * E * S)
        r, R = a[t] * s, a[t] * S
        rb = err + 40 * E * R
        z = before[t] - (x[t] if comp else 0)
        zb = bbefore[t] + 2 * E * (before[t].abs() + x[t].abs())
        d, b = r * z, rb * z.abs() + R * zb + rb * zb + 2 * E * R * z.abs()
        if logits:
            d, b = -w[t] * d, w[t] * (b + (k[t] + 2) * E * (d.abs() + b))
        out["d_gate"][0][t], out["d_gate"][1][t] = d, b
    out["d_state0"] = (r, err + 40 * E * R)
    return out
