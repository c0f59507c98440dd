"""Linear attention at the edges of what its launches take."""
import pytest
import torch

from tests import linear_oracle as ref
from tests.test_gpu_linear import BF, dev, make
from tests.test_gpu_linear_precision import hold_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def test_many_packed_states_of_odd_size(g):
    # 127 x 127 states are scanned element by element, 64 workgroups of 256
    # lanes each: 2^18 of them are 2^32 lanes.  Nearly all sequences are empty.
    N, D, T = (1 << 18) + 7, 127, 600
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    d = dev(make(1, T, 1, D, D, BF, state=False, packed=True))
    at = [0, 1, N // 2, N - 1]
    lens = [64, 1, 400, 135]
    ends = torch.zeros(N, dtype=torch.int64)
    ends[at] = torch.tensor(lens)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), ends.cumsum(0)]).to(torch.int32).cuda()
    o, S = g.linear_chunk_fwd_varlen(d["q"], d["k"], d["v"], d["la"], cu)
    lo = 0
    for i, n in zip(at, lens):
        s = {x: None if d[x] is None else d[x][None, lo:lo + n].cpu() for x in ("q", "k", "v", "la", "s0")}
        hold_forward(o[lo:lo + n][None], s, 1.0)
        ref.check(f"state {i}", S[i:i + 1], ref.linear_forward(s["q"], s["k"], s["v"], s["la"], None, 1.0)[1], ref.F32)
        lo += n
    S[at] = 0.0
    for part in S.split(1 << 16):
        assert not part.any()
