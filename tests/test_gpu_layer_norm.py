"""Layer norm on the GPU, forward and backward, against fp64; and the mixer
with its norm as a layer runs them together.

Tolerances: one rounding to bf16 is 2^-8 / sqrt(3) of the result in relative
L2 (ONE); fp32 results are held to 1e-5 elementwise of the sizes summed.
"""
import pytest
import torch

from tests import linear_oracle as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def make(shape, dtype, wshape, wdtype, seed=0, shift=0.3):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)
    x = (rn(*shape) * (0.5 + rn(*shape[:-1], 1).abs()) + shift * rn(*shape[:-1], 1)).to(dtype)
    w = None if wshape is None else (1 + 0.1 * rn(*wshape)).to(wdtype)
    b = None if wshape is None else (0.1 * rn(*wshape)).to(wdtype)
    return x, w, b, rn(*shape).to(dtype)


def gpu(*xs):
    return [None if x is None else x.cuda() for x in xs]


def compare(name, x, want, size, dtype):
    """Elementwise: one rounding of the result to its type, plus fp32 errors of `size`, what was added up."""
    y = x.double().cpu()
    assert y.shape == want.shape, name
    assert torch.isfinite(y).all(), name
    over = (y - want).abs() - (1e-6 * size + (ref.U * want.abs() if dtype == BF else 0.0) + 1e-30)
    assert over.numel() == 0 or over.max() <= 0, f"{name}: {float(over.max()):.3e} past its bound"


def check_all(g, x, w, b, dy, eps=1e-5):
    X, W, B, DY = gpu(x, w, b, dy)
    y, mean, rstd = g.layer_norm_fwd(X, W, B, eps=eps)
    dx, dw, db = g.layer_norm_bwd(DY, X, W, mean, rstd, want_weight=True, want_bias=True)
    torch.cuda.synchronize()
    y_r, mean_r, rstd_r = ref.layer_norm(x, w, b, eps)
    xd = x.double()
    compare("mean", mean, mean_r, xd.abs().mean(-1), F32)
    # the variance is taken about the fp32 mean, which is off by 2^-24 of the
    # values' size; x - mean is exact to 2^-24 of that size again
    size = xd.abs().amax(-1)
    compare("rstd", rstd, rstd_r, rstd_r * (1 + rstd_r * size), F32)
    wa = torch.ones(x.shape[-1]).double() if w is None else w.double().abs()
    h = (xd - mean_r[..., None]) * rstd_r[..., None]
    spread = h.abs() + (rstd_r * size)[..., None] * (1 + h.abs())
    compare("y", y, y_r, spread * wa + (0 if b is None else b.double().abs()), x.dtype)
    # the backward from the statistics that the forward stored
    dx_r, dw_r, db_r = ref.layer_norm_backward(dy, x, w, mean.cpu(), rstd.cpu())
    e = dy.double().abs() * wa
    r = rstd_r[..., None]
    spread2 = r * (e + e.mean(-1, keepdim=True) + spread * (e * spread).mean(-1, keepdim=True))
    compare("dx", dx, dx_r, spread2 * 2, x.dtype)
    axes = tuple(range(x.dim() - (1 if w is None else w.dim())))
    wt = F32 if w is None else w.dtype
    assert dw.dtype == wt and db.dtype == wt
    compare("d_weight", dw, dw_r, (dy.double().abs() * spread).sum(axes), wt)
    compare("d_bias", db, db_r, dy.double().abs().sum(axes), wt)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 31, 64, 65, 128, 200, 511, 1000, 1023, 1024, 1025, 2047, 2048, 2056, 4100,
                               8191, 8192, 8193, 12345, 16384])
def test_widths(g, D, dtype):
    rows = 37 if D < 4000 else 5
    check_all(g, *make((rows, D), dtype, (D,), F32, seed=D))


@pytest.mark.parametrize("rows", [0, 1, 2, 15, 16, 17, 64, 1000, 5003])
def test_rows(g, rows):
    x, w, b, dy = make((rows, 96), BF, (96,), BF, seed=rows)
    _, _, _, _, dw, db = check_all(g, x, w, b, dy)
    if rows == 0:
        assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,D", [(2, 50, 3, 128), (1, 1, 16, 64), (3, 7, 16, 128), (2, 9, 24, 33), (1, 5, 1, 16),
                                     (1, 40, 1000, 8), (2, 3, 5, 2048)])
def test_weights_of_each_head(g, B, T, H, D, dtype):
    check_all(g, *make((B, T, H, D), dtype, (H, D), F32, seed=H))


def test_without_weight_and_choices(g):
    x, _, _, dy = make((3, 5, 80), BF, None, None)
    check_all(g, x, None, None, dy)
    X, DY = gpu(x, dy)
    y, mean, rstd = g.layer_norm_fwd(X)
    dx, dw, db = g.layer_norm_bwd(DY, X, None, mean, rstd)
    assert dw is None and db is None and mean.shape == (3, 5)
    W = torch.ones(80, device="cuda")
    dx2, dw2, db2 = g.layer_norm_bwd(DY, X, W, mean, rstd)
    assert torch.equal(dx, dx2) and dw2.shape == (80,) and db2 is None


def test_large_mean(g):
    # a mean of 100 spreads: the variance must not cancel
    gen = torch.Generator().manual_seed(0)
    x = 100 + torch.randn(9, 513, generator=gen)
    check_all(g, x, torch.ones(513), None, torch.randn(9, 513, generator=gen))


def test_constant_rows(g):
    x = torch.full((4, 256), 3.0)
    y, mean, rstd = g.layer_norm_fwd(x.cuda(), eps=1e-5)
    assert (y == 0).all() and (mean == 3).all()
    assert torch.allclose(rstd.cpu(), torch.full((4,), 1e-5).rsqrt(), rtol=1e-6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned(g, dtype):
    x, w, b, dy = make((33, 64), dtype, (64,), F32)
    X, W, B, DY = gpu(x, w, b, dy)

    def off(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    y, mean, rstd = g.layer_norm_fwd(off(X), off(W), off(B))
    y_r, _, _ = ref.layer_norm(x, w, b, 1e-5)
    ref.check("y", y, y_r, ref.ONE if dtype == BF else ref.F32, 2 * ref.U * (1 + y_r.abs()))
    dx, dw, db = g.layer_norm_bwd(off(DY), off(X), off(W), off(mean), off(rstd), want_bias=True)
    dx_r, dw_r, db_r = ref.layer_norm_backward(dy, x, w, mean, rstd)
    ref.check("dw", dw, dw_r, ref.F32)
    ref.check("db", db, db_r, ref.F32)
    ref.check("dx", dx, dx_r, ref.ONE if dtype == BF else ref.F32, 2 * ref.U * (1 + dx_r.abs()))


def test_same_on_every_run(g):
    x, w, b, dy = gpu(*make((4096, 4, 128), BF, (4, 128), F32))
    y, mean, rstd = g.layer_norm_fwd(x, w, b)
    one = g.layer_norm_bwd(dy, x, w, mean, rstd, want_bias=True)
    two = g.layer_norm_bwd(dy, x, w, mean, rstd, want_bias=True)
    for p, q in zip(one, two):
        assert torch.equal(p, q)


def test_backward_against_differences(g):
    x, w, b, dy = make((6, 50), F32, (50,), F32, seed=4)
    X, W, B, DY = gpu(x, w, b, dy)
    _, mean, rstd = g.layer_norm_fwd(X, W, B)
    got = dict(zip("xwb", g.layer_norm_bwd(DY, X, W, mean, rstd, want_bias=True)))
    c, gen = dict(x=x.double(), w=w.double(), b=b.double()), torch.Generator().manual_seed(1)
    loss = lambda c: float((ref.layer_norm(c["x"], c["w"], c["b"], 1e-5)[0] * dy.double()).sum())
    for n in c:
        step = torch.randn(c[n].shape, generator=gen).double()
        up, down = (dict(c, **{n: c[n] + s * 1e-4 * step}) for s in (1, -1))
        want, grad = (loss(up) - loss(down)) / 2e-4, got[n].double().cpu()
        # the difference's own error is of the order of its step squared, 1e-8 times third derivatives
        assert abs(float((grad * step).sum()) - want) <= 2e-6 * float((grad.abs() * step.abs()).sum()), n


def test_layer_of_mixer_and_norm(g):
    """Block norm, linear attention, norm of each head: a layer's forward and
    backward as one run, captured in a graph and replayed."""
    B, T, H, D = 2, 150, 4, 64
    gen = torch.Generator().manual_seed(8)
    rn = lambda *s: torch.randn(s, generator=gen)
    x, w1, b1 = rn(B, T, H * D), 1 + 0.1 * rn(H * D), 0.1 * rn(H * D)
    w2, dz = 1 + 0.1 * rn(H, D), rn(B, T, H, D)
    la = -torch.nn.functional.softplus(rn(B, T, H) - 2)
    X, W1, B1, W2, DZ, LA = gpu(x, w1, b1, w2, dz, la)

    def layer():
        y, m1, r1 = g.layer_norm_fwd(X, W1, B1)
        h = y.view(B, T, H, D)
        o, S = g.linear_chunk_fwd(h, h, h, LA, q_scale=D ** -0.5)
        z, m2, r2 = g.layer_norm_fwd(o, W2)
        do, dw2, _ = g.layer_norm_bwd(DZ, o, W2, m2, r2)
        gr = g.linear_chunk_bwd(h, h, h, LA, None, do, q_scale=D ** -0.5)
        dh = (gr["dq"] + gr["dk"] + gr["dv"]).view(B, T, H * D)
        dx, dw1, db1 = g.layer_norm_bwd(dh, X, W1, m1, r1, want_bias=True)
        return dict(z=z, dx=dx, dw1=dw1, db1=db1, dw2=dw2, dla=gr["d_log_decay"])

    got = layer()
    # fp64 autograd of the same layer
    c = [t.double().requires_grad_() for t in (x, w1, b1, w2, la)]
    m = c[0].mean(-1, keepdim=True)
    h = (c[0] - m) / ((c[0] - m).square().mean(-1, keepdim=True) + 1e-5).sqrt() * c[1] + c[2]
    h = h.view(B, T, H, D)
    S, os = torch.zeros(B, H, D, D).double(), []
    for t in range(T):
        S = c[4][:, t].exp()[..., None, None] * S + h[:, t, :, :, None] * h[:, t, :, None, :]
        os.append(D ** -0.5 * (h[:, t, :, :, None] * S).sum(2))
    o = torch.stack(os, 1)
    m = o.mean(-1, keepdim=True)
    z = (o - m) / ((o - m).square().mean(-1, keepdim=True) + 1e-5).sqrt() * c[3]
    z.backward(dz.double())
    want = dict(z=z.detach(), dx=c[0].grad, dw1=c[1].grad, db1=c[2].grad, dw2=c[3].grad, dla=c[4].grad)
    for n in want:  # each operator is held to 1e-5; a layer of six in a row to 6e-5
        assert ref.rel_l2(got[n], want[n]) <= 6e-5, (n, ref.rel_l2(got[n], want[n]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer()
    for _ in range(3):
        X.copy_(torch.randn_like(X))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        snap = {n: t.clone() for n, t in kept.items()}
        for n, t in layer().items():
            assert torch.equal(snap[n], t), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape,heads", [((2300, 16, 128), True), ((9000, 512), False), ((1300, 4096), False), ((5000, 33), False),
                                        ((700, 10000), False)])
def test_many_rounds(g, shape, heads, dtype):
    # more rows than one round of the launch takes
    check_all(g, *make(shape, dtype, shape[-2:] if heads else shape[-1:], F32, seed=3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape,heads", [((700, 8192), False), ((130, 5, 5000), True), ((4200, 1536), False), ((290, 8193), False)])
def test_many_rounds_of_wide_rows(g, shape, heads, dtype):
    check_all(g, *make(shape, dtype, shape[-2:] if heads else shape[-1:], F32, seed=shape[-1]))


def test_bad_rows_stay_alone(g):
    x, w, b, dy = gpu(*make((40, 3, 72), BF, (3, 72), F32))
    one = g.layer_norm_fwd(x, w, b)
    grads = g.layer_norm_bwd(dy, x, w, one[1], one[2], want_bias=True)
    x2, dy2 = x.clone(), dy.clone()
    x2[0, 1], dy2[0, 1] = float("nan"), float("inf")
    two = g.layer_norm_fwd(x2, w, b)
    grads2 = g.layer_norm_bwd(dy2, x2, w, two[1], two[2], want_bias=True)
    keep = torch.ones(40, 3, dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    for p, q in zip(one, two):
        assert torch.equal(p[keep], q[keep])
    assert torch.equal(grads[0][keep], grads2[0][keep])
    for p, q in zip(grads[1:], grads2[1:]):  # the other heads' weights
        assert torch.equal(p[[0, 2]], q[[0, 2]])


def test_outputs_stay_inside_their_tensors(g):
    for D in (33, 64, 8200):
        x, w, b, dy = gpu(*make((5, D), BF, (D,), F32))
        big = torch.full((5 * D + 64,), 9.0, dtype=BF, device="cuda")
        g.layer_norm_fwd(x, w, b, out=big[32:-32].view(5, D))
        assert (big[:32] == 9).all() and (big[-32:] == 9).all()
