"""The fp64 references of the rotary, norm and scan tests (CPU): their gradients
against autograd of the definitions and against central differences."""
import pytest
import torch

from tests import rotary_oracle as ro
from tests import scan_oracle as so

F64 = torch.float64


def rn(*s, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed), dtype=F64)


def differences(f, x, d, step=1e-6):
    """<grad f, d> by central differences."""
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation(inter):
    x, f = rn(2, 5, 3, 12), 0.3 ** torch.arange(4, dtype=F64)
    y, _ = ro.turn_only(x, f, None, 3, inter, 1.5)
    # as complex numbers
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if inter else (slice(0, 4), slice(4, 8))
    z = torch.complex(x[..., a], x[..., b]) * 1.5 * torch.exp(1j * (torch.arange(5) + 3.0)[:, None, None] * f)
    assert torch.allclose(y[..., a], z.real) and torch.allclose(y[..., b], z.imag) and torch.equal(y[..., 8:], x[..., 8:])
    # back is the transpose, and the inverse where the magnitude is 1
    t, _ = ro.turn_only(y, f, None, 3, inter, 1 / 1.5, back=True)
    assert torch.allclose(t, x)


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norm_gradients(norm):
    x, w, dy, f = rn(4, 3, 10), 1 + 0.3 * rn(10, seed=1), rn(4, 3, 10, seed=2), 0.3 ** torch.arange(3, dtype=F64)
    p = torch.tensor([5, 1, 900, 0], dtype=torch.int32)
    args = (f, p, 7, False, 0.8)

    def loss(x, w):
        return (ro.norm_turn(x, w, *args, norm, 1e-3)[0] * dy).sum()

    dx, dw, bx, bw = ro.norm_turn_backward(dy, x, w, *args, norm, 1e-3)
    d, e = rn(4, 3, 10, seed=3), rn(10, seed=4)
    assert abs(differences(lambda t: loss(t, w), x, d) - (dx * d).sum()) < 1e-7
    assert abs(differences(lambda t: loss(x, t), w, e) - (dw * e).sum()) < 1e-7
    assert (bx >= 0).all() and (bw >= 0).all() and float(bx.max()) < 1e-4


@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("comp", [False, True])
def test_scan_gradients(comp, logits):
    T, D = 9, 4
    x, gate, s0, dy, ds = rn(T, D), rn(T, D, seed=1), rn(D, seed=2), rn(T, D, seed=3), rn(D, seed=4)
    if not logits:
        gate = -gate.abs() - 0.05

    def loss(x, gate, s0):
        h, _, _, _, (last, _) = so.forward(x, gate, s0, logits, comp)
        return (h * dy).sum() + (last * ds).sum()

    out = so.backward(dy, x, gate, s0, ds, logits, comp)
    ins = [x, gate, s0]
    for i, n in enumerate(("dx", "d_gate", "d_state0")):
        d = rn(*ins[i].shape, seed=10 + i)
        num = differences(lambda t: loss(*(t if j == i else ins[j] for j in range(3))), ins[i], d)
        assert abs(num - (out[n][0] * d).sum()) < 1e-7, n
    # the definition written with plain tensors, through autograd
    leaf = [t.clone().requires_grad_() for t in ins]
    a = torch.sigmoid(-leaf[1]) if logits else leaf[1].exp()
    u = (1 - a) * leaf[0] if comp else leaf[0]
    h, total = leaf[2], 0.0
    for t in range(T):
        h = a[t] * h + u[t]
        total = total + (h * dy[t]).sum()
    for got, n in zip(torch.autograd.grad(total + (h * ds).sum(), leaf), ("dx", "d_gate", "d_state0")):
        assert torch.allclose(got, out[n][0], atol=1e-12), n


def test_scan_states():
    x, gate, s0 = rn(300, 3), -rn(300, 3, seed=1).abs(), rn(3, seed=2)
    h, _, before, _, (last, _) = so.forward(x, gate, s0, False, False)
    assert torch.equal(before[0], s0) and torch.equal(before[1:], h[:-1]) and torch.equal(last, h[-1])
    a = gate.exp()
    assert torch.allclose(h[1], a[1] * (a[0] * s0 + x[0]) + x[1])
