"""Every compiled form of the gated scan: types, gate types, forms, packed or not,
whole vectors and single elements, over one tile and over several."""
import pytest
import torch

from tests import scan_oracle as ref
from tests.test_gpu_scan import BF, F32, both, check_backward, check_forward, dev, make

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (BF, F32), (F32, BF), (F32, F32)]
FORMS = [(logits, comp) for logits in (False, True) for comp in (False, True)]


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def ids(x):
    return "-".join(str(v).replace("torch.", "") for v in x)


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("D", [72, 13])
@pytest.mark.parametrize("lens", [[100], [3, 0, 70, 1, 200, 129, 400]], ids=["one tile", "several"])
def test_packed(g, lens, D, form, types):
    d = make(len(lens), sum(lens), D, *types, form[0], packed=True, seed=D + len(lens))
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    y, S, marks, r = both(g, d, *form, cu)
    assert y.dtype == types[0] and r["d_log_decay"].dtype == types[1]
    check_forward(d, y, S, marks, *form, lens)
    check_backward(d, r, *form, lens)
    # without states: the same sequences from zeros, and no gradient behind them
    d = {n: None if n in ("s0", "ds") else v for n, v in d.items()}
    y, S, marks, r = both(g, d, *form, cu)
    assert r["d_state0"] is None
    check_forward(d, y, S, marks, *form, lens)
    check_backward(d, r, *form, lens)


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("D", [72, 13])
def test_over_runs_of_tiles(g, D, form, types):
    # enough tiles for the map of a run, and the last one partial
    d = make(2, 128 * 18 + 37, D, *types, form[0], seed=D)
    y, S, marks, r = both(g, d, *form)
    check_forward(d, y, S, marks, *form)
    check_backward(d, r, *form)


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("form", FORMS, ids=ids)
@pytest.mark.parametrize("N,D", [(9, 64), (3, 21)])
def test_step(g, N, D, form, types):
    d = make(N, 1, D, *types, form[0], seed=D)
    x = dev(d)
    state = x["s0"].clone()
    y = g.gated_scan_step(x["x"][:, 0].contiguous(), x["gate"][:, 0].contiguous(), state, gate_logits=form[0], complement=form[1])
    assert y.dtype == types[0]
    check_forward(d, y[:, None], state, None, *form)


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("packed", [False, True])
def test_tensors_from_odd_addresses(g, packed, types):
    # rows of whole vectors that stand on no vector's address: single elements
    lens = [130, 40]
    d = make(2, 170 if packed else 140, 64, *types, True, packed=packed, seed=3)
    shifted = {}
    for n, v in d.items():
        hold = torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda")
        shifted[n] = hold[1:].view(v.shape).copy_(v)
    x = shifted
    cu = torch.tensor([0, 130, 170], dtype=torch.int32, device="cuda")
    if packed:
        y, S, marks = g.gated_scan_fwd_varlen(x["x"], x["gate"], cu, x["s0"], True, True, return_marks=True)
        r = g.gated_scan_bwd_varlen(x["dy"], x["x"], x["gate"], marks, cu, x["s0"], x["ds"], True, True)
    else:
        y, S, marks = g.gated_scan_fwd(x["x"], x["gate"], x["s0"], True, True, return_marks=True)
        r = g.gated_scan_bwd(x["dy"], x["x"], x["gate"], marks, x["s0"], x["ds"], True, True)
    check_forward(d, y, S, marks, True, True, lens if packed else None)
    check_backward(d, r, True, True, lens if packed else None)
