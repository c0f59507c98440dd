"""The gated scan, the query and key norms with rotary positions, and linear
attention one behind the other, as a layer uses them: training, packed
sequences, and a prompt followed by single tokens.  Every stage is held to its
own fp64 reference on the inputs that it got from the stage before it."""
import pytest
import torch

from tests import linear_oracle as lin, rotary_oracle as rot, scan_oracle as scan
from tests.test_gpu_linear import bound_o

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H, d = 3, 64


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def rn(*shape, dtype=F32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(700 + seed)).to(dtype).cuda()


def inputs(tok, dtype):
    return dict(x=rn(*tok, 3 * H * d, dtype=dtype), gate=rn(*tok, 3 * H * d, dtype=dtype, seed=1) - 1,
                la=-torch.nn.functional.softplus(rn(*tok, H, seed=2) - 2), qw=1 + 0.1 * rn(d, seed=3), kw=1 + 0.1 * rn(d, seed=4))


def heads(u):
    """q, k [..., H, d] as slices of the scan's rows, v copied."""
    q, k, v = u.view(*u.shape[:-1], 3, H, d).unbind(-3)
    return q, k, v.contiguous()


def check_scan(i, y, h0=None, x=None, gate=None):
    h, b, _, _, last = scan.forward(x, gate, h0, True, True)
    scan.check(f"scan {i}", y, h, b)
    return last


def check_turn(name, y, x, w, f, positions, offset):
    rot.check(name, y, *rot.norm_turn(x, w, f, positions, offset, False, 1.0, "rms", 1e-6))


def check_linear(dtype, q, k, v, la, o, S):
    """[B,T,H,*]"""
    o_ref, S_ref = lin.linear_forward(q, k, v, la, None, 0.125)
    tensors = dict(q=q.cpu(), k=k.cpu(), v=v.cpu(), la=la.cpu(), s0=None)
    lin.check("o", o, o_ref, lin.TWO if dtype == BF else lin.F32, bound_o(tensors, o_ref, 0.125, dtype, q.shape[1]))
    lin.check("state", S, S_ref, lin.F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_training(g, dtype):
    B, T = 2, 201
    i, f = inputs((B, T), dtype), g.rotary_frequencies(d)
    u, _, marks = g.gated_scan_fwd(i["x"], i["gate"], gate_logits=True, complement=True, return_marks=True)
    q, k, v = heads(u)
    q1, k1 = g.qk_norm_rotary_fwd(q, k, i["qw"], i["kw"], f)
    o, S = g.linear_chunk_fwd(q1, k1, v, i["la"], q_scale=0.125)
    for b in range(B):
        check_scan(b, u[b], x=i["x"][b], gate=i["gate"][b])
    check_turn("q", q1, q, i["qw"], f, None, 0)
    check_turn("k", k1, k, i["kw"], f, None, 0)
    check_linear(dtype, q1, k1, v, i["la"], o, S)

    d_o = rn(B, T, H, d, dtype=dtype, seed=5)
    l = g.linear_chunk_bwd(q1, k1, v, i["la"], None, d_o, q_scale=0.125)
    n = g.qk_norm_rotary_bwd(l["dq"], l["dk"], q, k, i["qw"], i["kw"], f)
    du = torch.stack([n["dq"], n["dk"], l["dv"]], dim=2).view(u.shape)
    r = g.gated_scan_bwd(du, i["x"], i["gate"], marks, gate_logits=True, complement=True)
    for name, x, dy, w in (("q", q, l["dq"], i["qw"]), ("k", k, l["dk"], i["kw"])):
        dx, dw, bx, bw = rot.norm_turn_backward(dy, x, w, f, None, 0, False, 1.0, "rms", 1e-6)
        rot.check("d" + name, n["d" + name], dx, bx)
        rot.check(f"d_{name}_weight", n[f"d_{name}_weight"], dw, bw)
    for b in range(B):
        want = scan.backward(du[b], i["x"][b], i["gate"][b], None, None, True, True)
        scan.check("dx", r["dx"][b], *want["dx"])
        scan.check("d_gate", r["d_log_decay"][b], *want["d_gate"])
    # the gradient of the whole run against a difference of its fp64 formula along one direction
    if dtype == F32:
        loss = lambda x: float((run64(x, i, f.cpu()) * d_o.double().cpu()).sum())
        x, e = i["x"].double().cpu(), 1e-5
        way = torch.randn(x.shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        diff = (loss(x + e * way) - loss(x - e * way)) / (2 * e)
        dot = r["dx"].double().cpu() * way
        # fp32 stages leave dx within 1e-5 of its length, and a sum of products with `way`
        # is off by at most that times the length of `way`
        assert abs(float(dot.sum()) - diff) <= 1e-5 * float(r["dx"].double().norm().cpu() * way.norm())


def run64(x, i, f):
    a, w, _ = scan.decays(i["gate"], True)
    h, u = torch.zeros(x.shape[0], x.shape[2], dtype=torch.float64), []
    for t in range(x.shape[1]):
        h = a[:, t] * h + w[:, t] * x[:, t]
        u.append(h)
    q, k, v = torch.stack(u, 1).view(*x.shape[:2], 3, H, d).unbind(2)
    q1 = rot.norm_turn(q, i["qw"], f, None, 0, False, 1.0, "rms", 1e-6)[0]
    k1 = rot.norm_turn(k, i["kw"], f, None, 0, False, 1.0, "rms", 1e-6)[0]
    return lin.linear_forward(q1, k1, v, i["la"], None, 0.125)[0]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_sequences(g, dtype):
    lens = [70, 0, 1, 140, 30]
    T = sum(lens)
    i, f = inputs((T,), dtype), g.rotary_frequencies(d)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    positions = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    u, _, _ = g.gated_scan_fwd_varlen(i["x"], i["gate"], cu, gate_logits=True, complement=True)
    q, k, v = heads(u)
    q1, k1 = g.qk_norm_rotary_fwd(q, k, i["qw"], i["kw"], f, positions)
    o, S = g.linear_chunk_fwd_varlen(q1, k1, v, i["la"], cu, q_scale=0.125)
    at = 0
    for n, m in enumerate(lens):
        sl = slice(at, at + m)
        if m:
            check_scan(n, u[sl], x=i["x"][sl], gate=i["gate"][sl])
            check_turn("q", q1[sl], q[sl], i["qw"], f, None, 0)
            check_turn("k", k1[sl], k[sl], i["kw"], f, None, 0)
            check_linear(dtype, q1[None, sl], k1[None, sl], v[None, sl], i["la"][None, sl], o[None, sl], S[n:n + 1])
        at += m


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_and_single_tokens(g, dtype):
    N, T, more = 3, 130, 9
    i, f = inputs((N, T + more), dtype), g.rotary_frequencies(d)
    x, gate, la = i["x"], i["gate"], i["la"]
    form = dict(gate_logits=True, complement=True)
    u, state, _ = g.gated_scan_fwd(x[:, :T].contiguous(), gate[:, :T].contiguous(), **form)
    q, k, v = heads(u)
    q1, k1 = g.qk_norm_rotary_fwd(q, k, i["qw"], i["kw"], f)
    o, S = g.linear_chunk_fwd(q1, k1, v, la[:, :T].contiguous(), q_scale=0.125)
    us, qs, ks, vs, os_ = [u], [q1], [k1], [v], [o]
    for t in range(T, T + more):
        u = g.gated_scan_step(x[:, t].contiguous(), gate[:, t].contiguous(), state, **form)[:, None]
        q, k, v = heads(u)
        q1, k1 = g.qk_norm_rotary_fwd(q, k, i["qw"], i["kw"], f, offset=t)
        check_turn("q", q1, q, i["qw"], f, None, t)
        o = g.linear_recurrent_step(q1[:, 0], k1[:, 0], v[:, 0], la[:, t].contiguous(), S, q_scale=0.125)
        for a, b in ((us, u), (qs, q1), (ks, k1), (vs, v), (os_, o[:, None])):
            a.append(b)
    u, q1, k1, v, o = (torch.cat(a, 1) for a in (us, qs, ks, vs, os_))
    for n in range(N):
        last, bound = check_scan(n, u[n], x=x[n], gate=gate[n])
        scan.check("state", state[n], last, bound)
    check_linear(dtype, q1, k1, v, la, o, S)
