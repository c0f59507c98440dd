"""Rotary positions and the query and key norms on the GPU, forward and
backward, against the fp64 definition."""
import pytest
import torch

from tests import rotary_oracle as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def rn(*shape, dtype=F32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(100 + seed)).to(dtype).cuda()


def freqs(g, rot):
    return g.rotary_frequencies(rot) if rot else None


# whole heads, parts of them, sizes that are no vectors
DIMS = [(128, 128), (128, 64), (64, 64), (256, 256), (96, 32), (80, 80), (40, 24), (75, 50), (254, 254), (17, 2), (2, 2), (255, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", DIMS)
def test_rotary(g, d, rot, inter, dtype):
    q, k, f = rn(2, 37, 5, d, dtype=dtype), rn(2, 37, 2, d, dtype=dtype, seed=1), freqs(g, rot)
    for fn, back in ((g.rotary_fwd, False), (g.rotary_bwd, True)):
        a, b = fn(q, k, f, offset=1000, interleaved=inter, magnitude=1.2)
        for n, x, y in (("q", q, a), ("k", k, b)):
            assert y.dtype == dtype and y.is_contiguous()
            ref.check(n, y, *ref.turn_only(x, f, None, 1000, inter, 1.2, back))


def positions_of(kind, B, T):
    gen = torch.Generator().manual_seed(5)
    if kind == "none":
        return None
    if kind == "shared":
        return torch.randint(0, 70000, (T,), generator=gen, dtype=torch.int32)
    if kind == "own":
        return torch.randint(0, 1 << 20, (B, T), generator=gen, dtype=torch.int32)
    return torch.randint(-500, 500, (B, T), generator=gen, dtype=torch.int32)


@pytest.mark.parametrize("kind", ["none", "shared", "own", "negative"])
@pytest.mark.parametrize("offset", [0, 123457, -77])
def test_positions(g, kind, offset):
    B, T, d = 3, 21, 64
    q, k, f, p = rn(B, T, 4, d), rn(B, T, 4, d, seed=1), freqs(g, d), positions_of(kind, B, T)
    a, b = g.rotary_fwd(q, k, f, positions=None if p is None else p.cuda(), offset=offset)
    ref.check("q", a, *ref.turn_only(q, f, p, offset, False, 1.0))
    ref.check("k", b, *ref.turn_only(k, f, p, offset, False, 1.0))


def test_far_positions(g):
    # 2^31 - 1 turns of the fastest pair: 64-bit angles are off by 3 2^-53 of 2^31, 2^-20 of a radian at most
    q, f = rn(4, 2, 32), freqs(g, 32)
    p = torch.tensor([2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1], dtype=torch.int32)
    a, _ = g.rotary_fwd(q, None, f, positions=p.cuda())
    want, bound = ref.turn_only(q, f, p, 0, False, 1.0)
    ref.check("q", a, want, bound + 2.0 ** -20 * (want.abs() + q.double().cpu().abs().sum(-1, keepdim=True)))


@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_frequencies(g, scaling):
    f = g.rotary_frequencies(64, base=500.0, scaling=scaling, factor=4.0, original_length=2048)
    j = torch.arange(32, dtype=torch.float64)
    want = 500.0 ** (-j / 32)
    if scaling == "linear":
        want = want / 4
    elif scaling == "base":
        want = (500.0 * 4.0 ** (64 / 62)) ** (-j / 32)
        assert abs(float(f[-1].cpu() * 4 / 500.0 ** (-31 / 32)) - 1) < 1e-12 and float(f[0]) == 1.0
    elif scaling == "parts":
        keep = ((2048 * want / (2 * torch.pi) - 1) / 31).clamp(0, 1)
        want = keep * want + (1 - keep) * want / 4
        assert float(f[0]) == 1.0 and abs(float(f[-1].cpu() / (500.0 ** (-31 / 32) / 4)) - 1) < 1e-12
    assert f.dtype == torch.float64 and f.is_cuda
    assert ((f.cpu() - want).abs() <= 1e-13 * want).all()
    q = rn(1, 300, 3, 64)
    a, _ = g.rotary_fwd(q, None, f, offset=30000)
    ref.check("q", a, *ref.turn_only(q, f, None, 30000, False, 1.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 33])
def test_slices_of_a_projection(g, d, dtype):
    qkv = rn(2, 19, 4 + 2 * 2, d, dtype=dtype)
    q, k = qkv[..., :4, :], qkv[..., 4:6, :]
    f = freqs(g, d - d % 2)
    want = g.rotary_fwd(q.contiguous(), k.contiguous(), f)
    kept = qkv.clone()
    got = g.rotary_fwd(q, k, f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(qkv, kept)
    got = g.qk_norm_rotary_fwd(q, k, freq=f)
    want = g.qk_norm_rotary_fwd(q.contiguous(), k.contiguous(), freq=f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dy = [rn(2, 19, 4, d, dtype=dtype, seed=2), rn(2, 19, 2, d, dtype=dtype, seed=3)]
    w = rn(d, seed=4)
    got = g.qk_norm_rotary_bwd(*dy, q, k, w, w, f)
    want = g.qk_norm_rotary_bwd(*dy, q.contiguous(), k.contiguous(), w, w, f)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    # a batch entry's slice: one token axis of the two
    got = g.rotary_fwd(q[1], k[1], f)
    assert torch.equal(got[0], g.rotary_fwd(q[1].contiguous(), None, f)[0])


def test_unaligned_tensors(g):
    f = freqs(g, 64)
    for dtype in (BF, F32):
        q = rn(3, 11, 2, 64, dtype=dtype)
        hold = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
        u = hold[1:].view(q.shape)
        u.copy_(q)
        a, _ = g.rotary_fwd(u, None, f)
        ref.check("q", a, *ref.turn_only(q, f, None, 0, False, 1.0))
        out = torch.full((q.numel() + 2,), 7.0, dtype=dtype, device="cuda")
        g.qk_norm_rotary_fwd(q, None, freq=f, q_out=out[1:-1].view(q.shape))
        assert out[0] == 7 and out[-1] == 7
        ref.check("q", out[1:-1].view(q.shape), *ref.norm_turn(q, None, f, None, 0, False, 1.0, "rms", 1e-6))


def test_in_place(g):
    q, k, f = rn(2, 9, 4, 64, dtype=BF), rn(2, 9, 1, 64, dtype=BF, seed=1), freqs(g, 64)
    for fn in (g.rotary_fwd, g.rotary_bwd):
        a, b = fn(q, k, f, interleaved=True)
        x, y = q.clone(), k.clone()
        r = fn(x, y, f, None, 0, True, 1.0, x, y)
        assert r[0] is x and torch.equal(x, a) and torch.equal(y, b)
    a, b = g.qk_norm_rotary_fwd(q, k, freq=f)
    x, y = q.clone(), k.clone()
    g.qk_norm_rotary_fwd(x, y, freq=f, q_out=x, k_out=y)
    assert torch.equal(x, a) and torch.equal(y, b)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (300, 3), (65, 64), (2, 0)])
def test_heads(g, Hq, Hk):
    f = freqs(g, 16)
    q, k = rn(5, Hq, 16), rn(5, Hk, 16, seed=1) if Hk else None
    a, b = g.rotary_fwd(q, k, f)
    ref.check("q", a, *ref.turn_only(q, f, None, 0, False, 1.0))
    if Hk:
        ref.check("k", b, *ref.turn_only(k, f, None, 0, False, 1.0))
    else:
        assert b is None
    dq = rn(5, Hq, 16, seed=2)
    dk = rn(5, Hk, 16, seed=3) if Hk else None
    w = 1 + 0.1 * rn(16, seed=4)
    r = g.qk_norm_rotary_bwd(dq, dk, q, k, w, w if Hk else None, f)
    dx, dw, bx, bw = ref.norm_turn_backward(dq, q, w, f, None, 0, False, 1.0, "rms", 1e-6)
    ref.check("dq", r["dq"], dx, bx)
    ref.check("d_q_weight", r["d_q_weight"], dw, bw)
    if Hk:
        dx, dw, bx, bw = ref.norm_turn_backward(dk, k, w, f, None, 0, False, 1.0, "rms", 1e-6)
        ref.check("dk", r["dk"], dx, bx)
        ref.check("d_k_weight", r["d_k_weight"], dw, bw)


@pytest.mark.parametrize("weight", [None, F32, BF])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot", DIMS + [(128, 0), (7, 0), (1, 0)])
def test_norm(g, d, rot, dtype, norm, weight):
    inter = rot % 4 == 2
    q, k = 3 * rn(2, 13, 6, d, dtype=dtype), 0.2 * rn(2, 13, 2, d, dtype=dtype, seed=1)
    dq, dk = rn(2, 13, 6, d, dtype=dtype, seed=2), rn(2, 13, 2, d, dtype=dtype, seed=3)
    ws = [None if weight is None else (1 + 0.2 * rn(d, seed=4 + i)).to(weight) for i in range(2)]
    f = freqs(g, rot)
    kw = dict(offset=50, interleaved=inter, magnitude=0.9, norm=norm, eps=1e-3)
    m = 0.9
    outs = g.qk_norm_rotary_fwd(q, k, *ws, f, **kw)
    grads = g.qk_norm_rotary_bwd(dq, dk, q, k, *ws, f, **kw)
    for n, x, dy, w, y in (("q", q, dq, ws[0], outs[0]), ("k", k, dk, ws[1], outs[1])):
        assert y.dtype == dtype
        ref.check(n, y, *ref.norm_turn(x, w, f, None, 50, inter, m, norm, 1e-3))
        dx, dw, bx, bw = ref.norm_turn_backward(dy, x, w, f, None, 50, inter, m, norm, 1e-3)
        ref.check("d" + n, grads["d" + n], dx, bx)
        if w is None:
            assert grads[f"d_{n}_weight"] is None
        else:
            assert grads[f"d_{n}_weight"].dtype == weight
            ref.check(f"d_{n}_weight", grads[f"d_{n}_weight"], dw, bw)


@pytest.mark.parametrize("norm,eps", [("rms", 1e-6), ("rms", 0.0), ("l2", 0.0)])
def test_rows_of_any_size(g, norm, eps):
    # rows of zeros, and rows whose squares overflow or vanish in fp32
    q = rn(8, 3, 64)
    scale = torch.tensor([0.0, 1.0, 1e30, 1e-30, 3e37, 1e-37, 1e-3, 0.0], device="cuda")
    q = q * scale[:, None, None]
    f = freqs(g, 32)
    y, _ = g.qk_norm_rotary_fwd(q, None, freq=f, norm=norm, eps=eps)
    ref.check("q", y, *ref.norm_turn(q, None, f, None, 0, False, 1.0, norm, eps))
    assert (y[0] == 0).all() and (y[7] == 0).all()
    dy = rn(8, 3, 64, seed=1)
    dy[scale.log10().abs() > 20] *= 1e-4  # keeps the gradients of tiny rows below fp32's largest value
    r = g.qk_norm_rotary_bwd(dy, None, q, None, freq=f, norm=norm, eps=eps)
    dx, _, bx, _ = ref.norm_turn_backward(dy, q, None, f, None, 0, False, 1.0, norm, eps)
    keep = dx.abs().amax((1, 2)) < 1e37
    ref.check("dq", r["dq"][keep.cuda()], dx[keep], bx[keep])
    if norm == "l2" or eps == 0:
        assert (r["dq"][0] == 0).all()


@pytest.mark.parametrize("d", [8, 64])
def test_weight_sums_over_many_rows(g, d):
    # more tiles than the launch has workgroups, the last one partial
    T = 1024 * 16 * 2 + 77
    q, dq, w = rn(T, 1, d, dtype=BF), rn(T, 1, d, dtype=BF, seed=1), 1 + 0.1 * rn(d, seed=2)
    f = freqs(g, d)
    r = g.qk_norm_rotary_bwd(dq, None, q, None, w, None, f)
    dx, dw, bx, bw = ref.norm_turn_backward(dq, q, w, f, None, 0, False, 1.0, "rms", 1e-6)
    ref.check("dq", r["dq"], dx, bx)
    ref.check("d_q_weight", r["d_q_weight"], dw, bw)
    again = g.qk_norm_rotary_bwd(dq, None, q, None, w, None, f)
    for n in r:
        assert r[n] is None or torch.equal(r[n], again[n]), n


def test_without_tokens(g):
    f, w = freqs(g, 8), torch.ones(8, device="cuda")
    q = rn(0, 2, 8)
    a, b = g.rotary_fwd(q, q, f)
    assert a.shape == (0, 2, 8) and b.shape == (0, 2, 8)
    r = g.qk_norm_rotary_bwd(q, q, q, q, w, w, f)
    assert torch.equal(r["d_q_weight"], torch.zeros(8, device="cuda")) and torch.equal(r["d_k_weight"], torch.zeros(8, device="cuda"))
    q = rn(2, 0, 2, 8)
    assert g.qk_norm_rotary_fwd(q, q, w, w, f)[0].shape == (2, 0, 2, 8)


def test_given_workspace_and_refusals(g):
    from gated_delta_rule_decay_amd.rotary import GDN2_QK_RMS, make_rotary_desc
    q, w, f = rn(4, 6, 2, 64), torch.ones(64, device="cuda"), freqs(g, 64)
    n = g.qk_norm_rotary_bwd_workspace(make_rotary_desc(24, 2, 2, 64, 64, dtype=0, norm=GDN2_QK_RMS))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    a = g.qk_norm_rotary_bwd(q, q, q, q, w, w, f, workspace=ws)
    b = g.qk_norm_rotary_bwd(q, q, q, q, w, w, f)
    assert all(torch.equal(a[k], b[k]) for k in a)
    with pytest.raises(RuntimeError):
        g.qk_norm_rotary_bwd(q, q, q, q, w, w, f, workspace=ws[:n - 256])
    with pytest.raises(RuntimeError):
        qkv = rn(4, 6, 4, 64)
        g.rotary_fwd(qkv[..., :2, :], None, f, q_out=qkv.view(-1)[:4 * 6 * 2 * 64].view(4, 6, 2, 64))


def test_captured_and_on_another_stream(g):
    q, k, w, f = rn(2, 50, 4, 64, dtype=BF), rn(2, 50, 4, 64, dtype=BF, seed=1), 1 + 0.1 * rn(64, seed=2), freqs(g, 64)
    dq, dk = rn(2, 50, 4, 64, dtype=BF, seed=3), rn(2, 50, 4, 64, dtype=BF, seed=4)

    def both():
        a, b = g.qk_norm_rotary_fwd(q, k, w, w, f)
        r = g.qk_norm_rotary_bwd(dq, dk, q, k, w, w, f)
        return [a, b, *r.values()]

    want = [x.clone() for x in both()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        q.copy_(rn(2, 50, 4, 64, dtype=BF, seed=10 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, both())), i


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F32), (33, F32)])
@pytest.mark.parametrize("norm,eps", [("rms", 1e-6), ("l2", 0.0)])
def test_rows_that_hold_no_numbers(g, norm, eps, d, dtype):
    # they show it, and their neighbours in the wave are as they were
    q, k, f = rn(2, 40, 3, d, dtype=dtype), rn(2, 40, 1, d, dtype=dtype, seed=1), freqs(g, 16)
    dy, dk = rn(2, 40, 3, d, dtype=dtype, seed=2), rn(2, 40, 1, d, dtype=dtype, seed=3)
    want = g.qk_norm_rotary_fwd(q, k, freq=f, norm=norm, eps=eps)[0]
    back = g.qk_norm_rotary_bwd(dy, dk, q, k, freq=f, norm=norm, eps=eps)["dq"]
    x = q.clone()
    x[0, 3, 1, 5] = float("nan")
    x[1, 7, 2, 20] = float("inf")
    keep = torch.ones(x.shape[:-1], dtype=torch.bool, device="cuda")
    keep[0, 3, 1] = keep[1, 7, 2] = False
    y = g.qk_norm_rotary_fwd(x, k, freq=f, norm=norm, eps=eps)[0]
    dx = g.qk_norm_rotary_bwd(dy, dk, x, k, freq=f, norm=norm, eps=eps)["dq"]
    assert torch.equal(y[keep], want[keep]) and torch.equal(dx[keep], back[keep])
    assert y[0, 3, 1].isnan().all() and dx[0, 3, 1].isnan().all() and dx[1, 7, 2].isnan().all()
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[20] = False  # inf / inf; the others are divided by it
    assert y[1, 7, 2, 20].isnan() and (y[1, 7, 2][rest] == 0).all()


def test_offsets_past_32_bits(g):
    # more than 2^31 elements a tensor
    H, d, last = 16, 128, 37
    T = (1 << 31) // (H * d) + last
    q, f, w = torch.randn(1, T, H, d, dtype=BF, device="cuda"), freqs(g, d), 1 + 0.1 * rn(d, seed=1)
    y = g.qk_norm_rotary_fwd(q, None, w, freq=f)[0]
    turned = g.rotary_fwd(q, None, f)[0]
    dq = g.qk_norm_rotary_bwd(y, None, q, None, w, freq=f)["dq"]
    for first in (0, T - last):
        sl = (slice(None), slice(first, first + last))
        ref.check("q", y[sl], *ref.norm_turn(q[sl], w, f, None, first, False, 1.0, "rms", 1e-6))
        ref.check("turned", turned[sl], *ref.turn_only(q[sl], f, None, first, False, 1.0))
        dx, _, b, _ = ref.norm_turn_backward(y[sl], q[sl], w, f, None, first, False, 1.0, "rms", 1e-6)
        ref.check("dq", dq[sl], dx, b)
