"""The norms with rotary positions where arithmetic is at its limits: an eps below
fp32's normal numbers, weight gradients over very many rows, positions far out."""
import pytest
import torch

from tests import rotary_oracle as ref

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def rn(*shape, dtype=F32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(100 + seed)).to(dtype).cuda()


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F32), (33, F32)])
@pytest.mark.parametrize("eps", [1e-40, 1e-45, 2e-38])
def test_eps_below_normal_numbers(g, eps, d, dtype):
    # lanes behind the last row hold rows of zeros, whose mean is eps alone; so do rows of zeros
    f, w = g.rotary_frequencies(16), 1 + 0.1 * rn(d, seed=4)
    for T in (1, 37, 300):
        q, dq = rn(T, 3, d, dtype=dtype), rn(T, 3, d, dtype=dtype, seed=1)
        for zeros in (False, True):
            if zeros:
                q[T // 2, 1] = 0
                dq[T // 2, 1] = 0  # 1 / sqrt(eps) of anything else is past fp32
            y = g.qk_norm_rotary_fwd(q, None, w, None, f, eps=eps)[0]
            r = g.qk_norm_rotary_bwd(dq, None, q, None, w, None, f, eps=eps)
            ref.check("q", y, *ref.norm_turn(q, w, f, None, 0, False, 1.0, "rms", eps))
            dx, dw, bx, bw = ref.norm_turn_backward(dq, q, w, f, None, 0, False, 1.0, "rms", eps)
            ref.check("dq", r["dq"], dx, bx)
            ref.check("d_q_weight", r["d_q_weight"], dw, bw)
