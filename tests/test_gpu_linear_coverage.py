"""Linear attention on the GPU where the other tests compare nothing element by
element, or only a kernel with itself: gradients of few tokens, segments of
more than 64 value channels, the launch's choices on both sides, scratch on
two streams, bad offsets with bordered outputs.

Elementwise bounds: with u = 2^-8 one rounding to bf16, |.| the same recurrence
on absolute values and n = 2 d + T + 200 (fp32 sums and the exponents' size),

    bf16:  (1 + u) ((3 2^-16 + n 2^-24) |.|) + u |x|      fp32:  n 2^-24 |.|

(two bf16 parts of the scores, of the state and of its update leave 2^-16 each).
"""
import ctypes

import pytest
import torch

from tests import linear_oracle as ref
from tests.test_gpu_linear import BF, F32, dev, make, split
from tests.test_gpu_linear_precision import positive

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def hold(name, x, want, size, s):
    dtype = s["v"].dtype
    assert x.dtype == dtype
    n = s["k"].shape[-1] + s["v"].shape[-1] + s["k"].shape[1] + 200
    bound = n * ref.E * size
    if dtype == BF:
        bound = (1 + ref.U) * (bound + 3 * 2.0 ** -16 * size) + ref.U * want.abs()
    ref.check(name, x, want, ref.ONE if dtype == BF else ref.F32, bound)


def hold_forward(o, S, s, scale):
    o_ref, S_ref = ref.linear_forward(s["q"], s["k"], s["v"], s["la"], s["s0"], scale)
    p = positive(s)
    size, _ = ref.linear_forward(p["q"], p["k"], p["v"], p["la"], p["s0"], scale)
    hold("o", o, o_ref, size, s)
    ref.check("state", S, S_ref, ref.F32)


def hold_backward(got, s, scale, pick=lambda x: x):
    want = ref.linear_backward(s["q"], s["k"], s["v"], s["la"], s["s0"], scale, s["d_o"], s["d_s"])
    p = positive(s)
    size = ref.linear_backward(p["q"], p["k"], p["v"], p["la"], p["s0"], scale, p["d_o"], p["d_s"])
    for n in ("dq", "dk", "dv"):
        hold(n, pick(got[n]), want[n], size[n], s)
    return want


HEADS = [(128, 128), (64, 64), (72, 56), (1, 1), (33, 100), (128, 17), (17, 128), (66, 70), (126, 102)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", HEADS)
@pytest.mark.parametrize("T", [1, 2, 33, 65])
def test_gradients_of_few_tokens(g, T, dk, dv, dtype):
    s = make(2, T, 2, dk, dv, dtype, seed=T)
    x = dev(s)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.7)
    want = hold_backward(got, s, 0.7)
    for n in ("d_log_decay", "d_state0"):
        ref.check(n, got[n], want[n], ref.F32)


# 600 tokens and more on few chains: segments, whose states are scanned
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,dk,dv", [(700, 128, 128), (1100, 40, 75), (1500, 128, 127)])
def test_segments_of_wide_heads(g, T, dk, dv, dtype):
    from gated_delta_rule_decay_amd.linear import make_linear_desc
    assert g.linear_chunk_fwd_workspace(make_linear_desc(1, T, 2, dk, dv, 1 if dtype == BF else 0)) > 0
    s = make(1, T, 2, dk, dv, dtype, seed=T)
    x = dev(s)
    o, S = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], q_scale=0.5)
    hold_forward(o, S, s, 0.5)
    got = g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"], q_scale=0.5)
    hold_backward(got, s, 0.5)
    # the state in place through the scan, and segments that begin with a state and end nowhere
    st = x["s0"].clone()
    o2, S2 = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], st, q_scale=0.5, state_out=st)
    assert S2 is st and torch.equal(S2, S) and torch.equal(o2, o)
    o3, none = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], q_scale=0.5, return_state=False)
    assert none is None and torch.equal(o3, o)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (72, 75)])
def test_packed_segments_of_wide_heads(g, dk, dv, dtype):
    lens, H = [1, 0, 640, 65, 700], 2
    d = make(len(lens), sum(lens), H, dk, dv, dtype, packed=True, seed=dv)
    x = dev(d)
    cu = torch.tensor([0, 1, 1, 641, 706, 1406], dtype=torch.int32, device="cuda")
    st = x["s0"].clone()
    o, S = g.linear_chunk_fwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, st, q_scale=0.5, state_out=st)
    got = g.linear_chunk_bwd_varlen(x["q"], x["k"], x["v"], x["la"], cu, x["s0"], x["d_o"], x["d_s"], q_scale=0.5)
    for i, at, n, s in split(d, lens, H):
        if n:
            hold_forward(o[at:at + n][None], S[i:i + 1], s, 0.5)
            hold_backward(got, s, 0.5, lambda t: t[at:at + n][None])
        else:
            assert torch.equal(S[i], x["s0"][i])


# Where the forward chooses: up to 111 chains segments, from 112 on whole
# chains, in half heads up to 128 chains and whole heads above; and one pass
# up to 512 tokens (fp32: 256) on any number of chains.
@pytest.mark.parametrize("B,H,T,dv,cut", [(1, 111, 520, 80, True), (1, 112, 520, 80, False), (2, 64, 200, 80, False), (3, 43, 200, 80, False),
                                          (1, 3, 512, 100, False), (1, 3, 513, 100, True)])
def test_both_sides_of_the_forward_choices(g, B, H, T, dv, cut):
    from gated_delta_rule_decay_amd.linear import make_linear_desc
    assert (g.linear_chunk_fwd_workspace(make_linear_desc(B, T, H, 24, dv)) > 0) == cut
    s = make(B, T, H, 24, dv, BF, seed=H)
    x = dev(s)
    o, S = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"], q_scale=0.4)
    hold_forward(o, S, s, 0.4)


def test_scratch_on_two_streams(g):
    # segments in both directions: each call has a table, sums and a scan of its own
    xs = [dev(make(1, 900, 2, 128, 128, BF, seed=i)) for i in (1, 2)]

    def work(x):
        o, S = g.linear_chunk_fwd(x["q"], x["k"], x["v"], x["la"], x["s0"])
        return dict(g.linear_chunk_bwd(x["q"], x["k"], x["v"], x["la"], x["s0"], x["d_o"], x["d_s"]), o=o, S=S)

    want = [work(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for st, x in zip(streams, xs):
            with torch.cuda.stream(st):
                got.append(work(x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for n in b:
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("offsets", [[0, 900, 400, 600], [-5, 3, 400, 2 ** 30], [500, 40, 30, 600], [2 ** 31 - 1, -2 ** 31, 0, 0],
                                     [0, 600, 0, 600]])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_bad_offsets_with_bordered_outputs(g, offsets, decay):
    """Unspecified values, but neither outputs nor scratch are left: each lies
    between borders that are looked at, the workspace of exactly its size."""
    from gated_delta_rule_decay_amd import linear as ln
    T, H, D, N = 600, 2, 64, 3
    d = dev(make(N, T, H, D, D, BF, decay=decay, packed=True))
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    desc = ln.make_linear_desc(N, T, H, D, D, decay_kind=ln.GDN2_DECAY_HEAD if decay == "head" else ln.GDN2_DECAY_TOKEN)
    kept = []

    def bordered(numel, dtype):
        t = torch.full((numel + 512,), 5, dtype=dtype, device="cuda")  # 256 elements on each side keep 256-byte alignment
        kept.append((t, numel))
        return t[256:256 + numel]

    def look():
        torch.cuda.synchronize()
        for t, n in kept:
            assert (t[:256] == 5).all() and (t[256 + n:] == 5).all()

    p = lambda t: t.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    q, k, v, la, s0, d_o, d_s = (d[n] for n in ("q", "k", "v", "la", "s0", "d_o", "d_s"))
    ins = [p(cu), p(q), p(k), p(v), p(la)]
    need = g.linear_chunk_fwd_varlen_workspace(desc)
    assert need > 0  # a plan, segments and a scan
    st = ln._call("gdn2_linear_fwd_varlen")(ctypes.byref(desc), *ins, p(s0), p(bordered(v.numel(), BF)), p(bordered(s0.numel(), F32)),
                                            p(bordered(need, torch.uint8)), need, stream)
    assert st == 0
    look()
    need = g.linear_chunk_bwd_varlen_workspace(desc)
    st = ln._call("gdn2_linear_bwd_varlen")(ctypes.byref(desc), *ins, p(s0), p(d_o), p(d_s), p(bordered(q.numel(), BF)),
                                            p(bordered(k.numel(), BF)), p(bordered(v.numel(), BF)), p(bordered(la.numel(), F32)),
                                            p(bordered(s0.numel(), F32)), p(bordered(need, torch.uint8)), need, stream)
    assert st == 0
    look()
