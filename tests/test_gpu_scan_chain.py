"""The gated scan over chains of many tiles, whose states pass between
workgroups."""
import math

import pytest
import torch

from tests import scan_oracle as ref
from tests.test_gpu_scan import BF, F32, both, check_backward, check_forward, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


# 1 to 3 tiles, the 15th to 17th (the map of a run is left behind the 16th), and the 33rd
@pytest.mark.parametrize("tiles", [2, 3, 15, 16, 17, 32, 33, 50])
@pytest.mark.parametrize("D", [64, 72, 3])
def test_tiles(g, tiles, D):
    for T in (128 * tiles, 128 * tiles - 127, 128 * tiles - 5):
        d = make(1, T, D, seed=tiles, state=T % 2 == 1)
        y, S, marks, r = both(g, d, False, False)
        check_forward(d, y, S, marks, False, False)
        check_backward(d, r, False, False)


# a state is left behind every 256th tile
@pytest.mark.parametrize("tiles,D", [(256, 8), (257, 3), (258, 8), (273, 8), (513, 8)])
def test_tiles_behind_a_state(g, tiles, D):
    d = make(1, 128 * tiles - tiles % 3, D, BF, seed=tiles)
    y, S, marks, r = both(g, d, False, True)
    check_forward(d, y, S, marks, False, True)
    check_backward(d, r, False, True)


def test_sequences_over_a_state(g):
    # packed: the axis is one chain, sequences end on both sides of its 256th tile
    lens = [32767, 1, 700, 33500]
    d = make(len(lens), sum(lens), 8, F32, packed=True, seed=8)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    y, S, marks, r = both(g, d, True, True, cu)
    check_forward(d, y, S, marks, True, True, lens)
    check_backward(d, r, True, True, lens)


@pytest.mark.parametrize("N,D", [(1, 1), (7, 64), (9, 64), (3, 200), (20, 130), (33, 64), (11, 230)])
def test_chains(g, N, D):
    # fewer chains than counters, and numbers that leave them unequal shares
    d = make(N, 2500, D, BF, BF, True, seed=N)
    y, S, marks, r = both(g, d, True, True)
    check_forward(d, y, S, marks, True, True)
    check_backward(d, r, True, True)


def test_long_memories_across_tiles(g):
    # decays next to 1: every tile's state reaches the end
    for comp in (False, True):
        d = make(1, 5000, 16, seed=1)
        d["gate"] = -torch.rand(d["gate"].shape, generator=torch.Generator().manual_seed(1)) * 2e-4
        y, S, marks, r = both(g, d, False, comp)
        check_forward(d, y, S, marks, False, comp)
        check_backward(d, r, False, comp)


def test_many_sequences_over_many_tiles(g):
    gen = torch.Generator().manual_seed(2)
    lens = [int(n) for n in torch.randint(0, 300, (30,), generator=gen)] + [2500, 1, 1, 700]
    d = make(len(lens), sum(lens), 72, BF, packed=True, seed=3)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    y, S, marks, r = both(g, d, False, True, cu)
    check_forward(d, y, S, marks, False, True, lens)
    check_backward(d, r, False, True, lens)


@pytest.mark.parametrize("packed", [False, True])
def test_state_in_place_over_many_tiles(g, packed):
    lens = [3000, 0, 1500, 7, 900]
    N, T = (len(lens), sum(lens)) if packed else (3, 2600)
    d = dev(make(N, T, 64, BF, packed=packed, seed=4))
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    call = (lambda st, out: g.gated_scan_fwd_varlen(d["x"], d["gate"], cu, st, state_out=out, return_marks=True)) if packed else (
        lambda st, out: g.gated_scan_fwd(d["x"], d["gate"], st, state_out=out, return_marks=True))
    y, S, m = call(d["s0"], None)
    for _ in range(5):
        st = d["s0"].clone()
        y2, _, m2 = call(st, st)
        assert torch.equal(y, y2) and torch.equal(S, st) and torch.equal(m, m2)


def test_same_bits_every_time(g):
    d = make(2, 6000, 256, F32, seed=5)
    first = both(g, d, False, False)
    for _ in range(5):
        again = both(g, d, False, False)
        assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))
        assert all(torch.equal(first[3][n], again[3][n]) for n in first[3])


def test_two_streams_with_their_own_workspaces(g):
    ds = [dev(make(2, 4000, 512, BF, seed=i)) for i in range(2)]
    want = [g.gated_scan_fwd(d["x"], d["gate"], d["s0"])[0] for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(4):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(g.gated_scan_fwd(d["x"], d["gate"], d["s0"])[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_workspace_for_many_calls(g):
    from gated_delta_rule_decay_amd.scan import make_scan_desc
    n = max(g.gated_scan_fwd_workspace(make_scan_desc(2, 3000, 128)), g.gated_scan_bwd_workspace(make_scan_desc(1, 5000, 64)))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for N, T, D in ((2, 3000, 128), (1, 5000, 64), (2, 300, 16), (2, 3000, 128)):
        d = dev(make(N, T, D, BF, seed=T))
        y, S, m = g.gated_scan_fwd(d["x"], d["gate"], d["s0"], return_marks=True, workspace=ws)
        r = g.gated_scan_bwd(d["dy"], d["x"], d["gate"], m, d["s0"], d["ds"], workspace=ws)
        y2, S2, m2 = g.gated_scan_fwd(d["x"], d["gate"], d["s0"], return_marks=True)
        r2 = g.gated_scan_bwd(d["dy"], d["x"], d["gate"], m2, d["s0"], d["ds"])
        assert torch.equal(y, y2) and torch.equal(S, S2) and torch.equal(m, m2) and all(torch.equal(r[k], r2[k]) for k in r)


@pytest.mark.parametrize("D", [64, 11])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_packed_sequences_keep_apart(g, D, bad):
    # what one sequence holds reaches no other, within a tile or over many
    lens = [50, 300, 2500, 60, 1, 4000, 7]
    d = make(len(lens), sum(lens), D, F32, packed=True, seed=11)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int()
    want = both(g, d, False, True, cu.cuda())
    for q in (2, 5):
        a, b = int(cu[q]), int(cu[q + 1])
        spoilt = {n: v.clone() for n, v in d.items()}
        for t in (a, a + 700, b - 1):
            spoilt["x"][t] = bad
            spoilt["dy"][t] = bad
        spoilt["gate"][a + 5, ::2] = float("nan")
        spoilt["gate"][b - 2, ::2] = float("nan")
        spoilt["s0"][q] = bad
        spoilt["ds"][q] = bad
        got = both(g, spoilt, False, True, cu.cuda())
        rows = torch.ones(sum(lens), dtype=torch.bool)
        rows[a:b] = False
        others = [i for i in range(len(lens)) if i != q]
        assert torch.equal(got[0].cpu()[rows], want[0].cpu()[rows]) and torch.equal(got[1][others], want[1][others])
        for n in ("dx", "d_log_decay"):
            assert torch.equal(got[3][n].cpu()[rows], want[3][n].cpu()[rows]), n
        assert torch.equal(got[3]["d_state0"][others], want[3]["d_state0"][others])
        assert not got[0].cpu()[a:b].isfinite().all()


@pytest.mark.parametrize("D", [64, 11])
def test_marks_of_rows_outside_every_sequence_are_not_used(g, D):
    T = 1400
    d = make(2, T, D, F32, packed=True, seed=12)
    cu = torch.tensor([200, 300, 900], dtype=torch.int32).cuda()
    x = dev(d)
    y, S, marks = g.gated_scan_fwd_varlen(x["x"], x["gate"], cu, x["s0"], return_marks=True)
    outside = [j for j in range(11) if not 200 <= 128 * j < 900]
    for v in (0.0, float("nan"), float("inf")):
        marks[outside] = v
        r = g.gated_scan_bwd_varlen(x["dy"], x["x"], x["gate"], marks, cu, x["s0"], x["ds"])
        cut = {n: w[200:900] if n in ("x", "gate", "dy") else w for n, w in d.items()}
        check_backward(cut, {"dx": r["dx"][200:900], "d_log_decay": r["d_log_decay"][200:900], "d_state0": r["d_state0"]},
                       False, False, [100, 600])


def test_offsets_past_32_bits(g):
    # more than 2^31 elements a tensor; a cleared state makes the last tokens a sequence of their own
    D, last = 2048, 300
    T = (1 << 31) // D + last
    x = torch.randn(1, T, D, dtype=BF, device="cuda")
    gate = -torch.rand(1, T, D, dtype=BF, device="cuda")
    gate[0, -last] = -math.inf
    y, S, marks = g.gated_scan_fwd(x, gate, return_marks=True)
    head, tail = slice(0, 150), slice(T - last, T)
    for sl in (head, tail):
        h, b, _, _, _ = ref.forward(x[0, sl], gate[0, sl], None, False, False)
        ref.check("y", y[0, sl], h, b)
    r = g.gated_scan_bwd(y, x, gate, marks)
    want = ref.backward(y[0, tail], x[0, tail], gate[0, tail], None, None, False, False)
    for n, k in (("dx", "dx"), ("d_log_decay", "d_gate")):
        ref.check(n, r[n][0, tail][1:], want[k][0][1:], want[k][1][1:])


def test_many_short_sequences(g):
    # as many workgroups as sequences, of the larger kind
    N, T, D = 70000, 3, 5
    d = dev(make(N, T, D, F32, seed=13))
    y, S, m = g.gated_scan_fwd(d["x"], d["gate"], d["s0"], return_marks=True)
    r = g.gated_scan_bwd(d["dy"], d["x"], d["gate"], m, d["s0"], d["ds"])
    h, a = d["s0"].double(), d["gate"].double().exp()
    for t in range(T):
        h = a[:, t] * h + d["x"][:, t].double()
        assert ((y[:, t].double() - h).abs() <= 2.0 ** -18 * (h.abs() + 20)).all()
    assert torch.equal(S, y[:, -1])
    q = d["ds"].double()
    for t in range(T - 1, -1, -1):
        q = d["dy"][:, t].double() + q
        assert ((r["dx"][:, t].double() - q).abs() <= 2.0 ** -18 * (q.abs() + 20)).all()
        q = a[:, t] * q
    assert ((r["d_state0"].double() - q).abs() <= 2.0 ** -18 * (q.abs() + 20)).all()
