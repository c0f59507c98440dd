"""The gated scan where memories are long and gates do not change: roundings
that have the same sign on every token must not add up over a memory.

A channel's decay is a = 1 - w on every token, with w = (n + 0.47) 2^-24, so
that a rounded to fp32 is off by 0.47 2^-24 on each.  Bounds, with e = 2^-24
and k = 6 + 2 |g| (g the stored gate): the kernel knows w to k e of itself, and u
to (k + 1) e.  Between two states that pass over (one every 2^15 tokens) a
token's map is joined at most J = 104 times: with 16 tokens in its lane, 24
groups of tokens and their parts, and 2 x 32 tiles, runs and their parts.  Every
joint multiplies by one factor that is rounded twice, and adds:

- the complement of a joined factor, a sum of complements times such factors, is
  off by at most (k + 3 J) e of itself, and since complements times what is
  behind them sum to at most 1, a state by (k + 3 J) e max |h|;
- a state's own terms by (k + 1 + 3 J) e for each span of 2^15 tokens.

So |error of h| <= (2 k + 1 + 3 J (1 + spans)) e max |h|, whatever the length of
the memory; the same holds of r.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

E, J, F64 = 2.0 ** -24, 104, torch.float64
T = 40000
STEPS = (3, 20, 101, 400, 2001, 7000, 30000, 100000)


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def limits(k):
    return (2 * k + 1 + 3 * J * (1 + T / 2 ** 15 + 1)) * E


def most(x):
    return x.abs().amax(0)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D", [8, 5])
@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("logits", [False, True])
def test_constant_gates(g, logits, comp, D, packed):
    w = (torch.tensor(STEPS[-D:], dtype=F64) + 0.47) * E
    gate = (w.log() - torch.log1p(-w) if logits else torch.log1p(-w)).float()
    stored = gate.to(F64)
    a, w = (torch.sigmoid(-stored), torch.sigmoid(stored)) if logits else (stored.exp(), -torch.expm1(stored))
    k = 6 + 2 * stored.abs()
    s0, ds = torch.full((D,), 0.75, dtype=F64), torch.full((D,), -1.5, dtype=F64)
    x, dy = torch.ones(D, dtype=F64), torch.full((D,), 0.5, dtype=F64)
    # h_t = a^t s0 + (1 - a^t) u / w, and r from the end likewise
    p = torch.exp(torch.arange(1, T + 1, dtype=F64)[:, None] * torch.log1p(-w))
    before_p = torch.cat([torch.ones(1, D, dtype=F64), p[:-1]])
    u = w * x if comp else x
    h, before = p * s0 + (1 - p) * (u / w), before_p * s0 + (1 - before_p) * (u / w)
    back = before_p.flip(0)  # of the tokens behind each
    behind = back * ds + (1 - back) * (a * dy / w)  # r_{t+1}, from r = a (dy + r); at the end ds
    s = dy + behind
    r = a * s

    N = 2 if packed else 1
    tok = lambda v: v.float().expand(N * T if packed else T, D).contiguous().cuda() if packed else v.float().expand(1, T, D).contiguous().cuda()
    st = lambda v: v.float().expand(N, D).contiguous().cuda()
    args = tok(x), tok(gate)
    form = dict(gate_logits=logits, complement=comp)
    if packed:
        cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
        y, S, marks = g.gated_scan_fwd_varlen(*args, cu, st(s0), return_marks=True, **form)
        got = g.gated_scan_bwd_varlen(tok(dy), *args, marks, cu, st(s0), st(ds), **form)
    else:
        y, S, marks = g.gated_scan_fwd(*args, st(s0), return_marks=True, **form)
        got = g.gated_scan_bwd(tok(dy), *args, marks, st(s0), st(ds), **form)
    rows = lambda v: v.cpu().to(F64).view(N, T, D)

    def near(name, value, want, bound):
        over = ((value - want).abs() / bound).amax(tuple(range(value.dim() - 1)))
        assert (over <= 1).all(), f"{name}: {[f'{v:.2f}' for v in over.tolist()]} of the bounds for w = {w.tolist()}"

    bh, bs = limits(k) * most(h), limits(k) * (most(s) + 0.5)
    near("y", rows(y), h, bh)
    near("state", S.cpu().to(F64), h[-1], bh)
    near("dx", rows(got["dx"]), w * s if comp else s, (w * (bs + k * E * most(s)) if comp else bs))
    z = before - x if comp else before
    d = r * z
    bz = bh + 2 * E * (most(before) + 1)
    bd = bs * most(z) + most(r) * bz + bs * bz
    if logits:
        d, bd = -w * d, w * (bd + (k + 2) * E * (most(d) + bd))
    near("d_log_decay", rows(got["d_log_decay"]), d, bd + 2 * E * most(d))
    near("d_state0", got["d_state0"].cpu().to(F64), r[0], bs)
