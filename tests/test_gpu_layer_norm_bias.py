"""Layer norm with a bias and no weight: the bias' gradient has the bias' own
shape and type, a row for each head among them."""
import pytest
import torch

from tests import linear_oracle as ref
from tests.test_gpu_layer_norm import BF, F32, compare, gpu, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


@pytest.mark.parametrize("bias_type", [F32, BF])
@pytest.mark.parametrize("shape,heads", [((3, 7, 4, 96), True), ((50, 3, 33), True), ((40, 200), False), ((0, 5, 16), True)])
def test_bias_without_weight(g, shape, heads, bias_type):
    x, _, b, dy = make(shape, F32, shape[-2:] if heads else shape[-1:], bias_type, seed=7)
    X, B, DY = gpu(x, b, dy)
    y, mean, rstd = g.layer_norm_fwd(X, None, B)
    y_r, mean_r, rstd_r = ref.layer_norm(x, None, b, 1e-5)
    # x - mean and the variance are off by 2^-24 of the row's values each, times rstd
    xd, r = x.double(), rstd_r[..., None]
    h = ((xd - mean_r[..., None]) * r).abs()
    compare("y", y, y_r, h + r * xd.abs().amax(-1, keepdim=True) * (1 + h) + b.double().abs(), F32)
    dx, dw, db = g.layer_norm_bwd(DY, X, None, mean, rstd, want_bias=True, bias=B)
    assert dw is None and db.shape == b.shape and db.dtype == bias_type
    # per-head rows: each the sum over its own rows of dy
    axes = tuple(range(x.dim() - b.dim()))
    compare("d_bias", db, dy.double().sum(axes), dy.double().abs().sum(axes), bias_type)
    dx2, _, _ = g.layer_norm_bwd(DY, X, None, mean, rstd)
    assert torch.equal(dx, dx2)


def test_bias_is_checked(g):
    x, _, _, dy = make((6, 4, 32), F32, None, None)
    X, DY = gpu(x, dy)
    _, mean, rstd = g.layer_norm_fwd(X)
    with pytest.raises(ValueError, match="bias"):
        g.layer_norm_bwd(DY, X, None, mean, rstd, want_bias=True, bias=torch.zeros(3, 32, device="cuda"))
    with pytest.raises(TypeError):
        g.layer_norm_bwd(DY, X, torch.ones(32, device="cuda"), mean, rstd, want_bias=True, bias=torch.zeros(32, device="cuda", dtype=BF))
