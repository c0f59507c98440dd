"""Linear attention with a decay for each head on the GPU: forward, packed
forward, backward and decode step against the fp64 recurrence."""
import math

import pytest
import torch

from tests import linear_oracle as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def make(B, T, H, dk, dv, dtype, decay="token", state=True, seed=0, packed=False):
    gen = torch.Generator().manual_seed(1000 + seed)
    tok = (T, H) if packed else (B, T, H)
    rn = lambda *s: torch.randn(s, generator=gen)
    unit = lambda *s: torch.nn.functional.normalize(rn(*s), dim=-1)
    d = dict(q=unit(*tok, dk).to(dtype), k=unit(*tok, dk).to(dtype), v=rn(*tok, dv).to(dtype), d_o=rn(*tok, dv).to(dtype),
             s0=0.1 * rn(B, H, dk, dv) if state else None, d_s=0.1 * rn(B, H, dk, dv) if state else None)
    if decay == "token":
        d["la"] = -torch.nn.functional.softplus(rn(*tok) - 2)
    elif decay == "head":
        d["la"] = torch.log1p(-torch.exp2(-(3 + 7 * torch.rand(H, generator=gen))))
    elif decay == "none":
        d["la"] = torch.zeros(tok)
    else:  # "resets": ordinary decays with zeros, far ones and minus infinity among them
        d["la"] = -torch.nn.functional.softplus(rn(*tok) - 2)
        at = torch.rand(tok, generator=gen)
        d["la"][at < 0.1] = 0.0
        d["la"][(at > 0.80) & (at < 0.85)] = -900.0
        d["la"][at > 0.98] = -math.inf
    return d


def dev(d):
    return {n: None if x is None else x.cuda() for n, x in d.items()}


def bound_o(d, o, scale, dtype, T):
    pos = lambda x: None if x is None else x.double().abs()
    A, _ = ref.linear_forward(pos(d["q"]), pos(d["k"]), pos(d["v"]), d["la"], pos(d["s0"]), scale)
    n = ref.E * (2 * d["q"].shape[-1] + T + 200)
    return n * A + ((ref.U * o.abs() + (ref.U + 2.0 ** -15) * A) if dtype == BF else 0.0)


def run_forward(g, d, scale, dtype, **kw):
    x = dev(d)
    o, S = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], q_scale=scale, **kw)
    torch.cuda.synchronize()
    assert o.dtype == dtype and S.dtype == F32
    return o, S


HEADS = [(128, 128), (64, 64), (72, 56), (1, 1), (33, 100), (128, 17), (5, 128), (65, 64), (40, 128), (66, 70), (127, 127)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", HEADS)
@pytest.mark.parametrize("T", [1, 64, 201])
def test_forward(g, T, dk, dv, dtype):
    d = make(2, T, 3, dk, dv, dtype, seed=T)
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.7)
    o, S = run_forward(g, d, 0.7, dtype)
    ref.check("o", o, o_ref, ref.TWO if dtype == BF else ref.F32, bound_o(d, o_ref, 0.7, dtype, T))
    ref.check("state", S, S_ref, ref.F32)


@pytest.mark.parametrize("T", [2, 31, 32, 33, 63, 65, 127, 128, 129])
def test_forward_lengths(g, T):
    for dtype in (BF, F32):
        d = make(1, T, 2, 64, 128, dtype, seed=T)
        o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 1.0)
        o, S = run_forward(g, d, 1.0, dtype)
        ref.check("o", o, o_ref, ref.TWO if dtype == BF else ref.F32, bound_o(d, o_ref, 1.0, dtype, T))
        ref.check("state", S, S_ref, ref.F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["token", "head", "none", "resets"])
@pytest.mark.parametrize("workspace", [True, False])
def test_forward_segments_and_decays(g, workspace, decay, dtype):
    # 700 tokens on 6 chains: three segments with a workspace, one pass without
    d = make(2, 700, 3, 128, 64, dtype, decay=decay, state=decay != "head")
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.5)
    if workspace:
        from gated_delta_rule_decay_amd.linear import make_linear_desc
        assert g.linear_chunk_fwd_workspace(make_linear_desc(2, 700, 3, 128, 64)) > 0
    o, S = run_forward(g, d, 0.5, dtype, workspace=workspace)
    ref.check("o", o, o_ref, ref.TWO if dtype == BF else ref.F32, bound_o(d, o_ref, 0.5, dtype, 700))
    ref.check("state", S, S_ref, ref.F32)


def test_forward_state_in_place_and_given_outputs(g):
    d = dev(make(2, 300, 2, 128, 128, BF))
    want_o, want_S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"])
    st, out = d["s0"].clone(), torch.empty_like(d["v"])
    o, S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], st, out=out, state_out=st)
    assert o is out and S is st
    assert torch.equal(o, want_o) and torch.equal(S, want_S)
    o, S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"], return_state=False)
    assert S is None and torch.equal(o, want_o)


def test_forward_without_tokens_or_sequences(g):
    d = dev(make(2, 0, 3, 16, 8, BF))
    o, S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"])
    assert o.shape == (2, 0, 3, 8) and torch.equal(S, d["s0"])
    o, S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"])
    assert torch.equal(S, torch.zeros_like(S))
    gr = g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["d_o"], d["d_s"])
    assert torch.equal(gr["d_state0"], d["d_s"])
    d = dev(make(0, 5, 3, 16, 8, BF, decay="head", state=False))
    o, S = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"])
    gr = g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], None, d["d_o"])
    assert o.numel() == 0 and torch.equal(gr["d_log_decay"], torch.zeros_like(d["la"]))


def test_forward_large_values(g):
    # bf16 has fp32's range: nothing here is rescaled or clipped
    d = make(1, 130, 2, 128, 128, BF)
    d["k"], d["v"] = d["k"] * 2.0 ** 40, d["v"] * 2.0 ** 30
    d["q"] = d["q"] * 2.0 ** -50
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 1.0)
    o, S = run_forward(g, d, 1.0, BF)
    ref.check("o", o, o_ref, ref.TWO, bound_o(d, o_ref, 1.0, BF, 130))
    ref.check("state", S, S_ref, ref.F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_rows(g, dtype):
    # contiguous tensors that start off a 16-byte border
    d = make(1, 70, 2, 64, 64, dtype)
    want_o, want_S = run_forward(g, d, 1.0, dtype)

    def off(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return y.copy_(x)

    x = dev(d)
    o, S = g.linear_chunk_fwd(off(x["q"]), off(x["k"]), off(x["v"]), off(x["la"]), off(x["s0"]), out=off(x["v"]),
                              state_out=off(x["s0"]))
    assert torch.equal(o, want_o) and torch.equal(S, want_S)


PACKS = [[5], [1, 0, 64, 65, 0, 130], [300, 1, 2, 700], [0, 0], [64] * 5]


def split(d, lens, H):
    """The padded-free batch of one sequence each."""
    at = 0
    for i, n in enumerate(lens):
        la = d["la"] if d["la"].dim() == 1 else d["la"][None, at:at + n]
        pick = lambda x: x[None, at:at + n]
        yield i, at, n, dict(q=pick(d["q"]), k=pick(d["k"]), v=pick(d["v"]), d_o=pick(d["d_o"]), la=la,
                             s0=None if d["s0"] is None else d["s0"][i:i + 1],
                             d_s=None if d["d_s"] is None else d["d_s"][i:i + 1])
        at += n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("lens", PACKS)
def test_packed(g, lens, decay, dtype):
    N, T, H, dk, dv, tail = len(lens), sum(lens), 3, 72, 64, 7
    d = make(N, T + tail, H, dk, dv, dtype, decay=decay, state=decay == "token", packed=True, seed=T)
    x = dev(d)
    offs = [0]
    for n in lens:
        offs.append(offs[-1] + n)
    cu = torch.tensor(offs, dtype=torch.int32, device="cuda")
    # tokens behind the last sequence: left as they are
    mark = torch.full_like(x["v"], 77.0)
    o, S = g.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], q_scale=0.6, out=mark)
    gr = g.linear_chunk_bwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], x["d_o"], x["d_s"], q_scale=0.6)
    torch.cuda.synchronize()
    assert (o[T:] == 77).all()
    tot = torch.zeros(H, dtype=torch.float64)
    want = dict(o=[], dq=[], dk=[], dv=[], d_log_decay=[])
    for i, at, n, s in split(d, lens, H):
        o_ref, S_ref = ref.linear_forward(s["q"], s["k"], s["v"], s["la"], s["s0"], 0.6)
        ref.check(f"o {i}", o[at:at + n][None], o_ref, ref.TWO if dtype == BF else ref.F32, bound_o(s, o_ref, 0.6, dtype, n))
        ref.check(f"state {i}", S[i:i + 1], S_ref, ref.F32)
        b = ref.linear_backward(s["q"], s["k"], s["v"], s["la"], s["s0"], 0.6, s["d_o"], s["d_s"])
        for name in ("dq", "dk", "dv"):
            want[name].append(b[name][0])
        if decay == "head":
            tot += b["d_log_decay"]
        else:
            want["d_log_decay"].append(b["d_log_decay"][0])
            ref.check(f"d_state0 {i}", gr["d_state0"][i:i + 1], b["d_state0"], ref.F32)
    for name in ("dq", "dk", "dv"):
        ref.check(name, gr[name][:T], torch.cat(want[name]), (ref.TWO if name == "dv" else ref.ONE) if dtype == BF else ref.F32)
    if decay == "head":
        ref.check("d_log_decay", gr["d_log_decay"], tot, ref.F32)
        assert gr["d_state0"] is None
    else:
        ref.check("d_log_decay", gr["d_log_decay"][:T], torch.cat(want["d_log_decay"]), ref.F32)


@pytest.mark.parametrize("offsets", [[0, 9, 4, 20], [-5, 3, 400, 2 ** 30], [50, 40, 30, 20], [2 ** 31 - 1, -2 ** 31, 0, 0]])
def test_packed_bad_offsets_stay_inside(g, offsets):
    # unspecified values, but nothing outside the tensors is touched: the
    # outputs lie inside larger buffers whose borders are checked
    d = dev(make(3, 20, 2, 64, 64, BF, packed=True))
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    big = torch.full((20 * 2 * 64 + 256,), 5.0, dtype=BF, device="cuda")
    out = big[128:-128].view(20, 2, 64)
    g.linear_chunk_fwd_varlen(d["q"], d["k"], d["v"], d["la"], cu, d["s0"], out=out)
    g.linear_chunk_bwd_varlen(d["q"], d["k"], d["v"], d["la"], cu, d["s0"], d["d_o"], d["d_s"])
    torch.cuda.synchronize()
    assert (big[:128] == 5).all() and (big[-128:] == 5).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (72, 56), (1, 1), (33, 100), (128, 17), (17, 128), (66, 70), (126, 102)])
@pytest.mark.parametrize("T", [1, 65, 300])
def test_backward(g, T, dk, dv, dtype):
    d = make(2, T, 2, dk, dv, dtype, seed=T)
    want = ref.linear_backward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.7, d["d_o"], d["d_s"])
    x = dev(d)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.7)
    torch.cuda.synchronize()
    for n in want:
        assert got[n].dtype == (dtype if n in ("dq", "dk", "dv") else F32)
        tol = ref.F32 if dtype == F32 or n in ("d_log_decay", "d_state0") else ref.TWO if n == "dv" else ref.ONE
        ref.check(n, got[n], want[n], tol)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["head", "none", "resets"])
def test_backward_segments_and_decays(g, decay, dtype):
    d = make(1, 1500, 2, 64, 128, dtype, decay=decay, state=decay == "resets")
    want = ref.linear_backward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.3, d["d_o"], d["d_s"])
    x = dev(d)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.3, want_state0=True)
    again = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.3, want_state0=True)
    torch.cuda.synchronize()
    for n in want:
        tol = ref.F32 if dtype == F32 or n in ("d_log_decay", "d_state0") else ref.TWO if n == "dv" else ref.ONE
        ref.check(n, got[n], want[n], tol)
        assert torch.equal(got[n], again[n]), n  # the same on every run


def test_backward_zero_scale(g):
    d = dev(make(1, 70, 2, 64, 64, F32))
    got = g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["d_o"], d["d_s"], q_scale=0.0)
    c = {n: x.cpu() for n, x in d.items()}
    want = ref.linear_backward(c["q"], c["k"], c["v"], c["la"], c["s0"], 0.0, c["d_o"], c["d_s"])
    for n in want:
        ref.check(n, got[n], want[n], ref.F32)


def test_backward_against_differences(g):
    # central differences of the fp64 forward along one random direction for
    # each input: step 1e-4, so the difference's own error is about 1e-8
    d = make(2, 90, 2, 24, 40, F32, seed=5)
    x = dev(d)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.9)
    gen = torch.Generator().manual_seed(9)

    def loss(c):
        o, S = ref.linear_forward(c["q"], c["k"], c["v"], c["la"], c["s0"], 0.9)
        return float((o * d["d_o"].double()).sum() + (S * d["d_s"].double()).sum())

    for n, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("la", "d_log_decay"), ("s0", "d_state0")):
        step = torch.randn(d[n].shape, generator=gen).double()
        up, down = (dict(d, **{n: d[n].double() + s * 1e-4 * step}) for s in (1, -1))
        want = (loss(up) - loss(down)) / 2e-4
        have = float((got[name].double().cpu() * step).sum())
        size = float((got[name].double().cpu().abs() * step.abs()).sum())
        assert abs(have - want) <= 2e-6 * size, (name, have, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (72, 56), (1, 1), (33, 101), (128, 20)])
@pytest.mark.parametrize("N,H,decay", [(3, 5, "token"), (1, 1, "head"), (70, 16, "token")])
def test_step(g, N, H, decay, dk, dv, dtype):
    d = make(N, 1, H, dk, dv, dtype, decay=decay)
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.7)
    x = dev(d)
    la = x["la"] if decay == "head" else x["la"][:, 0]
    st = x["s0"].clone()
    o = g.linear_recurrent_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], la, st, q_scale=0.7)
    torch.cuda.synchronize()
    pos = lambda t: t.double().abs()
    A, _ = ref.linear_forward(pos(d["q"]), pos(d["k"]), pos(d["v"]), d["la"], pos(d["s0"]), 0.7)
    # fp32 sums of dk terms, one rounding of the output
    bound = ref.E * (dk + 20) * A[:, 0] + (ref.U * o_ref[:, 0].abs() if dtype == BF else 0.0)
    ref.check("o", o, o_ref[:, 0], ref.ONE if dtype == BF else ref.F32, bound)
    ref.check("state", st, S_ref, ref.F32)


def test_chunks_then_steps_are_the_recurrence(g):
    # a prompt in two calls, then decoding, as a server runs them
    d = make(2, 200, 4, 128, 128, BF)
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.09)
    x = dev(d)
    cut = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "la")]
    o1, st = g.linear_chunk_fwd(*cut(0, 97), x["s0"], q_scale=0.09)
    o2, st = g.linear_chunk_fwd(*cut(97, 190), st, q_scale=0.09, state_out=st)
    outs = [o1, o2]
    for t in range(190, 200):
        q, k, v, la = (x[n][:, t].contiguous() for n in ("q", "k", "v", "la"))
        outs.append(g.linear_recurrent_step(q, k, v, la, st, q_scale=0.09)[:, None])
    ref.check("o", torch.cat(outs, 1), o_ref, ref.TWO)
    ref.check("state", st, S_ref, ref.F32)


def test_against_the_delta_rule_without_erase(g):
    # b = 0, w = 1: the gated delta rule is this recurrence
    d = dev(make(1, 130, 2, 128, 128, F32))
    zero = torch.zeros_like(d["la"])
    o1, S1 = g.chunk_fwd(d["q"], d["k"], d["v"], d["la"], zero, zero + 1, d["s0"])
    o2, S2 = g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"])
    assert ref.rel_l2(o2, o1.double().cpu()) <= 2e-5 and ref.rel_l2(S2, S1.double().cpu()) <= 2e-5


def test_graph_replays(g):
    d = dev(make(1, 600, 2, 128, 128, BF))
    dec = dev(make(2, 1, 3, 128, 128, BF, seed=3))
    from gated_delta_rule_decay_amd.linear import make_linear_desc
    out, st = torch.empty_like(d["v"]), torch.empty_like(d["s0"])
    ws = torch.empty(g.linear_chunk_fwd_workspace(make_linear_desc(1, 600, 2, 128, 128)), dtype=torch.uint8, device="cuda")
    step = [dec[n][:, 0].contiguous() for n in ("q", "k", "v", "la")]
    dst = dec["s0"].clone()

    def work():
        g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"], out=out, state_out=st, workspace=ws)
        o = g.linear_recurrent_step(*step, dst)
        return o, g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["d_o"], d["d_s"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, gr = work()
    for i in range(4):
        d["v"].copy_(torch.randn_like(d["v"]))  # new inputs, eager work and a wait between the replays
        dst.copy_(dec["s0"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in gr.items()}
        got.update(o=out.clone(), S=st.clone(), step=o.clone(), dst=dst.clone())
        dst.copy_(dec["s0"])
        o2, g2 = work()
        want = dict(g2, o=out, S=st, step=o2, dst=dst)
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


def test_two_streams(g):
    a, b = dev(make(1, 500, 2, 128, 128, BF, seed=1)), dev(make(1, 500, 2, 128, 128, BF, seed=2))
    want = [g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"]) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, x in zip(streams, (a, b)):
        with torch.cuda.stream(s):
            got.append(g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"]))
    torch.cuda.synchronize()
    for (o, S), (o2, S2) in zip(got, want):
        assert torch.equal(o, o2) and torch.equal(S, S2)


# where the launch chooses: segments below 128 chains, halves of heads from
# 128, whole heads from 256; one head more or less on each side
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H", [(1, 127), (1, 128), (51, 5), (16, 16)])
def test_forward_many_chains(g, B, H, dtype):
    d = make(B, 260, H, 72, 80, dtype, seed=H)
    o_ref, S_ref = ref.linear_forward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.4)
    o, S = run_forward(g, d, 0.4, dtype)
    ref.check("o", o, o_ref, ref.TWO if dtype == BF else ref.F32, bound_o(d, o_ref, 0.4, dtype, 260))
    ref.check("state", S, S_ref, ref.F32)


# enough chains that a segment is longer than 512 tokens: the widest sums of
# the decay's gradient, over one segment and a part of a second
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,decay", [(1100, "token"), (1024, "head"), (577, "resets")])
def test_backward_many_chains(g, T, decay, dtype):
    d = make(3, T, 171, 16, 24, dtype, decay=decay, seed=T)
    want = ref.linear_backward(d["q"], d["k"], d["v"], d["la"], d["s0"], 0.7, d["d_o"], d["d_s"])
    x = dev(d)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.7)
    torch.cuda.synchronize()
    for n in want:
        tol = ref.F32 if dtype == F32 or n in ("d_log_decay", "d_state0") else ref.TWO if n == "dv" else ref.ONE
        ref.check(n, got[n], want[n], tol)


def test_packed_many_heads(g):
    # whole sequences, one workgroup each: an empty one among them
    lens, H = [70, 0, 1, 300], 130
    d = make(4, sum(lens), H, 32, 48, BF, packed=True)
    x = dev(d)
    cu = torch.tensor([0, 70, 70, 71, 371], dtype=torch.int32, device="cuda")
    o, S = g.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"])
    for i, at, n, s in split(d, lens, H):
        o_ref, S_ref = ref.linear_forward(s["q"], s["k"], s["v"], s["la"], s["s0"], 1.0)
        if n:
            ref.check(f"o {i}", o[at:at + n][None], o_ref, ref.TWO, bound_o(s, o_ref, 1.0, BF, n))
        ref.check(f"state {i}", S[i:i + 1], S_ref, ref.F32)


def test_packed_many_sequences(g):
    # over 1024 sequences: the plan's other form
    N, H = 1500, 2
    lens = [(7 * i) % 5 for i in range(N)]
    offs = [0]
    for n in lens:
        offs.append(offs[-1] + n)
    d = make(N, offs[-1], H, 16, 24, BF, packed=True)
    x = dev(d)
    cu = torch.tensor(offs, dtype=torch.int32, device="cuda")
    o, S = g.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"])
    gr = g.linear_chunk_bwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], x["d_o"], x["d_s"])
    # the same sequences as a padded batch: no decay and no key behind an end
    pad = lambda t: torch.stack([torch.cat([t[a:b], t.new_zeros((4 - (b - a), *t.shape[1:]))]) for a, b in zip(offs, offs[1:])])
    args = [pad(d[n]) for n in ("q", "k", "v", "la")]
    o_ref, S_ref = ref.linear_forward(*args, d["s0"], 1.0)
    b = ref.linear_backward(*args, d["s0"], 1.0, pad(d["d_o"]), d["d_s"])
    take = lambda t: torch.cat([t[i, :n] for i, n in enumerate(lens)])
    ref.check("o", o, take(o_ref), ref.TWO)
    ref.check("state", S, S_ref, ref.F32)
    for n in ("dq", "dk", "dv", "d_log_decay"):
        ref.check(n, gr[n], take(b[n]), ref.F32 if n == "d_log_decay" else ref.TWO if n == "dv" else ref.ONE)
    ref.check("d_state0", gr["d_state0"], b["d_state0"], ref.F32)


def test_packed_neighbours_do_not_mix(g):
    # one sequence of NaN, and NaN behind the last one
    lens, H = [65, 70, 130], 2
    d = dev(make(3, sum(lens) + 9, H, 64, 64, BF, packed=True))
    cu = torch.tensor([0, 65, 135, 265], dtype=torch.int32, device="cuda")
    run = lambda: (g.linear_chunk_fwd_varlen(d["q"], d["k"], d["v"], d["la"], cu, d["s0"]),
                   g.linear_chunk_bwd_varlen(d["q"], d["k"], d["v"], d["la"], cu, d["s0"], d["d_o"], d["d_s"]))
    (o1, S1), g1 = run()
    for n in ("q", "k", "v", "d_o"):
        d[n][65:135] = float("nan")
        d[n][265:] = float("nan")
    (o2, S2), g2 = run()
    keep = torch.cat([torch.arange(65), torch.arange(135, 265)]).cuda()
    assert torch.equal(o1[keep], o2[keep]) and torch.equal(S1[[0, 2]], S2[[0, 2]])
    for n in ("dq", "dk", "dv", "d_log_decay"):
        assert torch.equal(g1[n][keep], g2[n][keep]), n
    assert torch.equal(g1["d_state0"][[0, 2]], g2["d_state0"][[0, 2]])


def test_outputs_stay_inside_their_tensors(g):
    # borders of the outputs, at head sizes whose rows end inside a unit
    for dtype, dk, dv in ((BF, 66, 33), (F32, 33, 70), (BF, 128, 127)):
        d = dev(make(1, 75, 3, dk, dv, dtype))
        big = torch.full((75 * 3 * dv + 64,), 9.0, dtype=dtype, device="cuda")
        st = torch.full((3 * dk * dv + 64,), 9.0, device="cuda")
        g.linear_chunk_fwd(d["q"], d["k"], d["v"], d["la"], d["s0"], out=big[32:-32].view(1, 75, 3, dv),
                           state_out=st[32:-32].view(1, 3, dk, dv))
        for x in (big, st):
            assert (x[:32] == 9).all() and (x[-32:] == 9).all()
        step = torch.full((3 * dv + 64,), 9.0, dtype=dtype, device="cuda")
        g.linear_recurrent_step(d["q"][:, 0].contiguous(), d["k"][:, 0].contiguous(), d["v"][:, 0].contiguous(),
                                d["la"][:, 0].contiguous(), d["s0"], out=step[32:-32].view(1, 3, dv))
        assert (step[:32] == 9).all() and (step[-32:] == 9).all()


def test_two_graphs_with_workspaces_of_their_own(g):
    d = dev(make(1, 500, 2, 128, 64, BF))
    want = g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["d_o"], d["d_s"])
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(g.linear_chunk_bwd(d["q"], d["k"], d["v"], d["la"], d["s0"], d["d_o"], d["d_s"]))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            for n in want:
                assert torch.equal(o[n], want[n]), n
