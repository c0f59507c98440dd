"""Linear attention, bf16: o and dv are fp32-like results rounded once.

Elementwise, with u = 2^-8 the largest relative error of one rounding to bf16
and |.| the same recurrence on absolute values (every term positive), an
element may be off by

    (1 + u) ((3 2^-16 + n 2^-24) |.|)  +  u |o|

where the three operands made on the way (scores, state as it is read, values
that update a state) each go into the matrix products as two bf16 parts, which
leave at most u^2 = 2^-16 of the operand, n = 2 d + T + 200 counts the fp32
sums and the exponents' size, and the last rounding is the result's own.  A
state that is read as one bf16 part adds u |.|, which this bound does not hold.
"""
import pytest
import torch

from tests import linear_oracle as ref
from tests.test_gpu_linear import BF, dev, make, split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def hold(name, x, want, size, d, T):
    n = 2 * d + T + 200
    bound = (1 + ref.U) * (3 * 2.0 ** -16 + n * ref.E) * size + ref.U * want.abs()
    ref.check(name, x, want, ref.ONE, bound)


def positive(s):
    return {n: x if x is None or n == "la" else x.double().abs() for n, x in s.items()}


def hold_forward(o, s, scale):
    o_ref, _ = ref.linear_forward(s["q"], s["k"], s["v"], s["la"], s["s0"], scale)
    p = positive(s)
    size, _ = ref.linear_forward(p["q"], p["k"], p["v"], p["la"], p["s0"], scale)
    hold("o", o, o_ref, size, s["k"].shape[-1], s["k"].shape[1])


def hold_dv(dv, s, scale):
    want = ref.linear_backward(s["q"], s["k"], s["v"], s["la"], s["s0"], scale, s["d_o"], s["d_s"])["dv"]
    p = positive(s)
    size = ref.linear_backward(p["q"], p["k"], p["v"], p["la"], p["s0"], scale, p["d_o"], p["d_s"])["dv"]
    hold("dv", dv, want, size, s["k"].shape[-1], s["k"].shape[1])


# whole chains: half heads, one wave a column tile up to 64 columns, whole
# heads above 128 chains; the second line in segments, on both sides of 64
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,T,H,dk,dv", [(2, 201, 3, 128, 128), (1, 64, 4, 100, 127), (2, 130, 3, 72, 56), (3, 90, 43, 64, 80), (3, 90, 43, 72, 80),
                                         (1, 700, 3, 128, 128), (1, 1100, 2, 66, 75), (2, 700, 3, 128, 64)])
def test_forward(g, B, T, H, dk, dv, decay):
    s = make(B, T, H, dk, dv, BF, decay=decay, seed=T + dv)
    x = dev(s)
    o, _ = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], q_scale=0.7)
    hold_forward(o, s, 0.7)


@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 300, 2, 128, 128), (1, 300, 2, 64, 64), (1, 200, 3, 128, 56), (1, 200, 3, 40, 128)])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_dv(g, B, T, H, dk, dv, decay):
    s = make(B, T, H, dk, dv, BF, decay=decay, seed=T + dv)
    x = dev(s)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.7)
    hold_dv(got["dv"], s, 0.7)


@pytest.mark.parametrize("dk,dv", [(128, 128), (48, 75)])
def test_packed(g, dk, dv):
    lens, H = [130, 1, 600, 0, 64], 2
    d = make(len(lens), sum(lens), H, dk, dv, BF, decay="head", packed=True, seed=dv)
    x = dev(d)
    cu = torch.tensor([0, 130, 131, 731, 731, 795], dtype=torch.int32, device="cuda")
    o, _ = g.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], q_scale=0.7)
    gr = g.linear_chunk_bwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], x["d_o"], x["d_s"], q_scale=0.7)
    for _, at, n, s in split(d, lens, H):
        if n:
            hold_forward(o[at:at + n][None], s, 0.7)
            hold_dv(gr["dv"][at:at + n][None], s, 0.7)
