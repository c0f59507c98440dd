"""Every compiled form of the norms with rotary positions: types, layouts, norms,
weights, whole vectors and single elements."""
import pytest
import torch

from tests import rotary_oracle as ref
from tests.test_gpu_rotary import BF, F32, freqs, rn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


@pytest.mark.parametrize("weight", [None, F32, BF])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 32), (256, 256), (96, 24), (80, 20), (42, 22)])
def test_norm_in_both_layouts(g, d, rot, inter, dtype, norm, weight):
    q, k = 2 * rn(2, 19, 3, d, dtype=dtype), 0.3 * rn(2, 19, 1, d, dtype=dtype, seed=1)
    dq, dk = rn(2, 19, 3, d, dtype=dtype, seed=2), rn(2, 19, 1, d, dtype=dtype, seed=3)
    ws = [None if weight is None else (1 + 0.2 * rn(d, seed=4 + i)).to(weight) for i in range(2)]
    f = freqs(g, rot)
    kw = dict(offset=70, interleaved=inter, magnitude=1.1, norm=norm, eps=1e-4)
    outs = g.qk_norm_rotary_fwd(q, k, *ws, f, **kw)
    grads = g.qk_norm_rotary_bwd(dq, dk, q, k, *ws, f, **kw)
    for n, x, dy, w, y in (("q", q, dq, ws[0], outs[0]), ("k", k, dk, ws[1], outs[1])):
        ref.check(n, y, *ref.norm_turn(x, w, f, None, 70, inter, 1.1, norm, 1e-4))
        dx, dw, bx, bw = ref.norm_turn_backward(dy, x, w, f, None, 70, inter, 1.1, norm, 1e-4)
        ref.check("d" + n, grads["d" + n], dx, bx)
        if w is None:
            assert grads[f"d_{n}_weight"] is None
        else:
            ref.check(f"d_{n}_weight", grads[f"d_{n}_weight"], dw, bw)
