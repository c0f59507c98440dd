"""Timed cases of the rotary positions, the query and key norms and the gated scan, with their plain forms.

Rotary positions turn the pairs (u, v) of a head's first ``rot`` channels by
theta = position * frequency, both scaled by a magnitude m:

    u' = m (cos(theta) u - sin(theta) v),      v' = m (sin(theta) u + cos(theta) v)

with u = x[j], v = x[j + rot/2] (half layout) or u = x[2j], v = x[2j + 1]
(interleaved).  The norms divide every head's query and key by its root mean
square (or its length) and multiply by a weight before the rotation.  The gated
scan is, for each channel,

    h_t = a_t h_{t-1} + w_t x_t,     a = exp(log_decay) or sigmoid(-logit),     w = 1 or 1 - a

and leaves the state that enters every 128th token for its backward pass.
``own`` chooses between the framework's kernels and the plain form.
"""
import math

import torch

own = False

EPS = 1e-6
MARK = 128


def listed():
    return [
        # decoding with many sequences, each at a far position of its own, inside a fused q, k, v projection
        dict(name="rotary fwd, 256 sequences", op="rotary_fwd", B=256, T=1, Hq=16, Hk=16, d=128, rot=128, inter=False,
             dtype="bf16", pos="decode", scaling="none", fused=True),
        # the training step on a long document: frequencies scaled by parts, half of the head turned
        dict(name="rotary bwd, long document", op="rotary_bwd", B=1, T=65536, Hq=16, Hk=16, d=128, rot=64, inter=True,
             dtype="bf16", pos="count", scaling="parts", fused=False),
        # decoding one sequence: latency
        dict(name="qk norm fwd, one sequence", op="norm_fwd", B=1, T=1, Hq=16, Hk=16, d=128, rot=128, inter=False,
             dtype="bf16", pos="decode", scaling="none", fused=False, norm="rms", weight="f32"),
        # a training or prefill batch of the repository's main workload, read from a fused projection
        dict(name="qk norm fwd, batch", op="norm_fwd", B=8, T=4096, Hq=16, Hk=16, d=128, rot=128, inter=False,
             dtype="bf16", pos="count", scaling="none", fused=True, norm="rms", weight="f32"),
        # the training step of the same layer
        dict(name="qk norm bwd, batch", op="norm_bwd", B=8, T=4096, Hq=16, Hk=16, d=128, rot=128, inter=False,
             dtype="bf16", pos="count", scaling="none", fused=False, norm="rms", weight="f32"),
        # fine-tuning in full precision on packed positions: few key heads, odd sizes, unit lengths
        dict(name="qk norm bwd, odd fp32", op="norm_bwd", B=1, T=1001, Hq=6, Hk=2, d=75, rot=50, inter=False,
             dtype="f32", pos="packed", scaling="linear", fused=False, norm="l2", weight="f32"),
        # one short prompt: what a request costs at least
        dict(name="scan fwd, short prompt", op="scan_fwd", B=1, T=64, D=2048, dtype="bf16", gate="f32", logits=False,
             comp=False, state=True, marks=False, lens=""),
        # the training forward of a batch, gates as logits
        dict(name="scan fwd, batch", op="scan_fwd", B=8, T=4096, D=2048, dtype="bf16", gate="bf16", logits=True,
             comp=True, state=True, marks=True, lens=""),
        # the training step of the same layer
        dict(name="scan bwd, batch", op="scan_bwd", B=8, T=4096, D=2048, dtype="bf16", gate="bf16", logits=True,
             comp=True, state=True, marks=True, lens=""),
        # one long document, decays in full precision
        dict(name="scan fwd, long document", op="scan_fwd", B=1, T=65536, D=2048, dtype="bf16", gate="f32", logits=False,
             comp=False, state=False, marks=False, lens=""),
        # training on packed documents in full precision, an odd width
        dict(name="scan bwd, packed fp32", op="scan_bwd", B=6, T=7777, D=515, dtype="f32", gate="f32", logits=False,
             comp=False, state=True, marks=True, lens="1,0,515,4096,64,3101"),
        # decoding with many sequences
        dict(name="scan step, 256 sequences", op="scan_step", B=256, T=1, D=2048, dtype="bf16", gate="bf16", logits=True,
             comp=True, state=True, marks=False, lens=""),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "norm_fwd", "norm_bwd", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd",
                     "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if not op.startswith("scan"):
        d = rng.choice([64, 128, 128, 256, rng.randint(2, 256), 8 * rng.randint(1, 32)])
        rot = rng.choice([d, d, d // 2, rng.randint(2, d)])
        rot = max(2, rot - rot % 2)
        Hq = rng.choice([1, 2, 3, 5, 8, 16, 24, 32])
        Hk = rng.choice([Hq, Hq, 1, max(1, Hq // 4)])
        tokens = _log_int(rng, 1, (1 << 26) // ((Hq + Hk) * d))
        B = rng.choice([1, 1, 2, 3, 8])
        T = max(1, min(65536, tokens // B))
        pos = rng.choice(["count", "packed", "decode"])
        if pos == "decode":
            B, T = min(B * T, 4096), 1
        case = dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, inter=rng.random() < 0.5, dtype=dtype, pos=pos,
                    scaling=rng.choice(["none", "linear", "base", "parts"]), fused=rng.random() < 0.5 and op.endswith("fwd"))
        if op.startswith("norm"):
            case.update(norm=rng.choice(["rms", "rms", "l2"]), weight=rng.choice(["f32", "f32", "bf16", "none"]))
        return case
    D = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128), 8 * _log_int(rng, 1, 1024)])
    case = dict(op=op, D=D, dtype=dtype, gate=rng.choice(["f32", dtype]), logits=rng.random() < 0.5, comp=rng.random() < 0.5,
                state=rng.random() < 0.6, marks=False, lens="")
    if op == "scan_step":
        return dict(case, B=_log_int(rng, 1, min(4096, (1 << 23) // D)), T=1, state=True)
    case["marks"] = op == "scan_bwd" or rng.random() < 0.5
    most = (1 << (26 if op == "scan_fwd" else 25)) // D  # tokens
    least = 1 if op == "scan_fwd" else 2  # the first token of a zero state has no gradient of its decay
    if rng.random() < 0.35:  # packed sequences
        n = rng.randint(1, 9)
        top = max(2, min(16384, most // n))
        lens = [rng.choice([0, 1, _log_int(rng, 1, top), _log_int(rng, 1, top)]) if i else _log_int(rng, least, top)
                for i in range(n)]
        return dict(case, B=n, T=sum(lens), lens=",".join(map(str, lens)))
    B = rng.choice([1, 1, 2, 3, 8])
    return dict(case, B=B, T=_log_int(rng, least, max(2, min(65536, most // B))))


def _frequencies(rot, scaling):
    """Radians a position of the rot/2 pairs, in 64 bits, and the magnitude of the rotation."""
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base, s = 10000.0, 8.0
    if scaling == "base":
        base *= s ** (rot / max(rot - 2, 1))
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        return f / s, 1.0
    if scaling == "parts":  # fast pairs stay, slow ones are divided by s, a ramp between
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        return keep * f + (1 - keep) * f / s, 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    f32 = torch.float32

    def normal(*shape, dtype=f32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=f32).to(dtype)

    st = {"case": case}
    op, B, T = case["op"], case["B"], case["T"]
    if not op.startswith("scan"):
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        if case["pos"] == "decode":
            tok = (B,)
            st["positions"] = torch.randint(0, 131072, (B,), generator=gen, device="cuda", dtype=torch.int32)
        elif case["pos"] == "packed":  # documents of drawn lengths, each counted from 0
            tok = (B * T,)
            start = (torch.rand(B * T, generator=gen, device="cuda") < 0.004).long()
            start[0] = 1
            at = torch.arange(B * T, device="cuda")
            st["positions"] = (at - (at * start).cummax(0).values).int()
        else:
            tok = (B, T)
            st["positions"] = None
        if case["fused"]:  # [.., 3 projections, H, d] with as many value heads as key heads
            qkv = normal(*tok, Hq + 2 * Hk, d, dtype=dt)
            st["q"], st["k"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hk, :]
        else:
            st["q"], st["k"] = normal(*tok, Hq, d, dtype=dt), normal(*tok, Hk, d, dtype=dt)
        st["freq"], st["magnitude"] = _frequencies(case["rot"], case["scaling"])
        if op.startswith("norm"):
            wt = case["weight"]
            for n in ("wq", "wk"):
                st[n] = None if wt == "none" else (1.0 + 0.1 * normal(d)).to(torch.bfloat16 if wt == "bf16" else f32)
        if op.endswith("bwd"):
            st["dq"], st["dk"] = normal(*tok, Hq, d, dtype=dt), normal(*tok, Hk, d, dtype=dt)
        return st

    D = case["D"]
    lens = [int(n) for n in case["lens"].split(",")] if case["lens"] else []
    tok = (T,) if lens else (B,) if op == "scan_step" else (B, T)
    st["x"] = normal(*tok, D, dtype=dt)
    # memories of a few to some thousand tokens, a length for each channel
    logit = normal(*tok, D) - 8.0 * torch.rand(D, generator=gen, device="cuda")
    st["gate"] = (logit if case["logits"] else -torch.nn.functional.softplus(logit)).to(
        torch.bfloat16 if case["gate"] == "bf16" else f32)
    st["state"] = normal(B, D) if case["state"] else None
    if lens:
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        st["cu"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        st["live"] = [i for i, n in enumerate(lens) if n]
        st["first"] = torch.tensor([offs[i] for i in st["live"]], device="cuda")
        st["last"] = torch.tensor([offs[i + 1] - 1 for i in st["live"]], device="cuda")
        st["live"] = torch.tensor(st["live"], device="cuda")
    if op == "scan_bwd":
        st["dy"] = normal(*tok, D, dtype=dt)
        st["ds"] = normal(B, D)
        st["marks"] = _forward(st, torch.float64)[2].float()
    return st


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import gated_delta_rule_decay_amd as g

    c = s["case"]
    op = c["op"]
    if not op.startswith("scan"):
        turn = dict(positions=s["positions"], interleaved=c["inter"], magnitude=s["magnitude"])
        if op == "rotary_fwd":
            return g.rotary_fwd(s["q"], s["k"], s["freq"], **turn)
        if op == "rotary_bwd":
            return g.rotary_bwd(s["dq"], s["dk"], s["freq"], **turn)
        if op == "norm_fwd":
            return g.qk_norm_rotary_fwd(s["q"], s["k"], s["wq"], s["wk"], s["freq"], norm=c["norm"], eps=EPS, **turn)
        return g.qk_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["freq"], norm=c["norm"], eps=EPS,
                                    **turn)
    form = dict(gate_logits=c["logits"], complement=c["comp"])
    if op == "scan_step":
        return {"y": g.gated_scan_step(s["x"], s["gate"], s["state"], **form), "state": s["state"]}
    if op == "scan_fwd":
        if "cu" in s:
            y, S, marks = g.gated_scan_fwd_varlen(s["x"], s["gate"], s["cu"], s["state"], return_marks=c["marks"], **form)
        else:
            y, S, marks = g.gated_scan_fwd(s["x"], s["gate"], s["state"], return_marks=c["marks"], **form)
        return {"y": y, "state": S, "marks": marks}
    if "cu" in s:
        return g.gated_scan_bwd_varlen(s["dy"], s["x"], s["gate"], s["marks"], s["cu"], s["state"], s["ds"], **form)
    return g.gated_scan_bwd(s["dy"], s["x"], s["gate"], s["marks"], s["state"], s["ds"], **form)


def _angles(s):
    """cos and sin of every token's angles [.., 1, rot/2], times the magnitude; angles in 64 bits."""
    c, p = s["case"], s["positions"]
    if p is None:
        p = torch.arange(c["T"], device="cuda")
    theta = (p.double()[..., None] * s["freq"])[..., None, :]
    return (s["magnitude"] * theta.cos()).float(), (s["magnitude"] * theta.sin()).float()


def _turn(s, x, back=False):
    c = s["case"]
    rot = c["rot"]
    cos, sin = _angles(s)
    if back:
        sin = -sin
    if c["inter"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([cos * u - sin * v, sin * u + cos * v], -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([cos * u - sin * v, sin * u + cos * v], -1)
    return torch.cat([y, x[..., rot:]], -1) if rot < c["d"] else y


def _inverse_size(s, x):
    if s["case"]["norm"] == "rms":
        return (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x.square().sum(-1, keepdim=True).rsqrt()


def _compose(a, b, s0=None):
    """h_t = a_t h_{t-1} + b_t along axis -2, from h = s0, by doubling."""
    if s0 is not None:
        b = torch.cat([torch.addcmul(b[..., :1, :], a[..., :1, :], s0[..., None, :]), b[..., 1:, :]], -2)
    n, T = 1, a.shape[-2]
    while n < T:
        b = torch.cat([b[..., :n, :], torch.addcmul(b[..., n:, :], a[..., n:, :], b[..., :-n, :])], -2)
        if 2 * n < T:
            a = torch.cat([a[..., :n, :], a[..., n:, :] * a[..., :-n, :]], -2)
        n *= 2
    return b


def _gates(s, ft):
    """a and 1 - a; the smaller one directly, so that neither is a difference of near numbers."""
    if s["case"]["logits"]:
        x = s["gate"].to(ft)
        return torch.sigmoid(-x), torch.sigmoid(x)
    x = s["gate"].to(ft)
    return x.exp(), -x.expm1()


def _forward(s, ft):
    """h, the last states, and the states that enter every 128th token."""
    c = s["case"]
    a, w = _gates(s, ft)
    u = s["x"].to(ft)
    if c["comp"]:
        u = w * u
    s0 = None if s["state"] is None else s["state"].to(ft)
    if "cu" not in s:
        h = _compose(a, u, s0)
        first = h.new_zeros(c["B"], 1, c["D"]) if s0 is None else s0[:, None]
        return h, h[:, -1], torch.cat([first, h[:, MARK - 1:-1:MARK]], 1)
    at, live = s["first"], s["live"]
    if s0 is not None:
        u = u.index_copy(0, at, u[at] + a[at] * s0[live])
    h = _compose(a.index_fill(0, at, 0.0), u)
    S = h.new_zeros(c["B"], c["D"]) if s0 is None else s0
    S = S.index_copy(0, live, h[s["last"]])
    before = torch.cat([h.new_zeros(1, c["D"]), h[:-1]])
    before = before.index_copy(0, at, h.new_zeros(len(at), c["D"]) if s0 is None else s0[live])
    return h, S, before[::MARK]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if not op.startswith("scan"):
        dt = s["q"].dtype
        if op == "rotary_fwd":
            return tuple(_turn(s, s[n].float()).to(dt) for n in ("q", "k"))
        if op == "rotary_bwd":
            return tuple(_turn(s, s[n].float(), back=True).to(dt) for n in ("dq", "dk"))
        if op == "norm_fwd":
            out = []
            for n, w in (("q", s["wq"]), ("k", s["wk"])):
                x = s[n].float()
                x = x * _inverse_size(s, x)
                out.append(_turn(s, x if w is None else x * w.float()).to(dt))
            return tuple(out)
        out = {}
        for n, w in (("q", s["wq"]), ("k", s["wk"])):
            x, g = s[n].float(), _turn(s, s["d" + n].float(), back=True)
            r = _inverse_size(s, x)
            h = x * r
            dw = None if w is None else (g * h).flatten(0, -2).double().sum(0).to(w.dtype)
            g = g if w is None else g * w.float()
            e = (g * h).sum(-1, keepdim=True)
            out["d" + n] = (r * (g - h * (e / c["d"] if c["norm"] == "rms" else e))).to(dt)
            out["d_%s_weight" % n] = dw
        return out
    x, dt = s["x"], s["x"].dtype
    if op == "scan_step":
        a, w = _gates(s, torch.float32)
        h = a * s["state"] + (w * x.float() if c["comp"] else x.float())
        s["state"].copy_(h)
        return {"y": h.to(dt), "state": s["state"]}
    h, S, marks = _forward(s, torch.float32)
    if op == "scan_fwd":
        return {"y": h.to(dt), "state": S, "marks": marks if c["marks"] else None}
    a, w = _gates(s, torch.float32)
    g, x = s["dy"].float(), x.float()
    s0, ds = s["state"], s["ds"]
    if "cu" in s:
        at, live = s["first"], s["live"]
        g = g.index_copy(0, s["last"], g[s["last"]] + ds[live])
        before = torch.cat([h.new_zeros(1, c["D"]), h[:-1]])
        before = before.index_copy(0, at, h.new_zeros(len(at), c["D"]) if s0 is None else s0[live])
        # g_t = dy_t + a_{t+1} g_{t+1}, not over a sequence's end
        after = torch.cat([a[1:], a.new_zeros(1, c["D"])]).index_fill(0, s["last"], 0.0)
        g = _compose(after.flip(-2), g.flip(-2)).flip(-2)
        d0 = None if s0 is None else ds.index_copy(0, live, a[at] * g[at])
    else:
        g = torch.cat([g[:, :-1], g[:, -1:] + ds[:, None]], 1)
        first = h.new_zeros(c["B"], 1, c["D"]) if s0 is None else s0[:, None]
        before = torch.cat([first, h[:, :-1]], 1)
        after = torch.cat([a[:, 1:], a.new_zeros(c["B"], 1, c["D"])], 1)
        g = _compose(after.flip(-2), g.flip(-2)).flip(-2)
        d0 = None if s0 is None else a[:, 0] * g[:, 0]
    dl = a * g * (before - x if c["comp"] else before)
    if c["logits"]:
        dl = -w * dl
    return {"dx": (w * g if c["comp"] else g).to(dt), "d_log_decay": dl.to(s["gate"].dtype), "d_state0": d0}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if not op.startswith("scan"):
        rot, half = case["rot"], case["rot"] // 2
        p = torch.arange(case["T"], device="cuda") if s["positions"] is None else s["positions"]
        z = torch.polar(torch.full((), s["magnitude"], dtype=f, device="cuda").expand(*p.shape, half),
                        p.to(f).unsqueeze(-1) * s["freq"]).unsqueeze(-2)

        def turned(x, z):  # pairs as complex numbers
            y = x.clone()
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, half), slice(half, rot))
            t = torch.complex(x[..., a], x[..., b]) * z
            y[..., a], y[..., b] = t.real, t.imag
            return y

        if op == "rotary_fwd":
            return turned(s["q"].to(f), z), turned(s["k"].to(f), z)
        if op == "rotary_bwd":
            return turned(s["dq"].to(f), z.conj()), turned(s["dk"].to(f), z.conj())
        outs, grads = [], {}
        for n in ("q", "k"):
            x, w = s[n].to(f), s["w" + n]
            w = torch.ones(case["d"], dtype=f, device="cuda") if w is None else w.to(f)
            size = (x * x).sum(-1, keepdim=True)
            many = case["d"] if case["norm"] == "rms" else 1
            r = 1.0 / torch.sqrt(size / many + (EPS if case["norm"] == "rms" else 0.0))
            if op == "norm_fwd":
                outs.append(turned(x * r * w, z))
                continue
            e = turned(s["d" + n].to(f), z.conj())
            # d r / d x = -r^3 x / many
            grads["d" + n] = e * w * r - x * r ** 3 / many * (e * w * x).sum(-1, keepdim=True)
            grads["d_%s_weight" % n] = None if s["w" + n] is None else (e * x * r).flatten(0, -2).sum(0)
        return tuple(outs) if outs else grads

    B, T, D = case["B"], case["T"], case["D"]
    x, l = s["x"].to(f), s["gate"].to(f)
    if case["logits"]:
        l = -torch.nn.functional.softplus(l)
    a, w = torch.exp(l), -torch.expm1(l)
    u = w * x if case["comp"] else x
    if op == "scan_step":
        h = a * s["state"].to(f) + u
        return {"y": h, "state": h}
    packed = "cu" in s
    offs = s["cu"].tolist() if packed else None
    seqs = [(i, offs[i], offs[i + 1]) for i in range(B)] if packed else [(slice(None), 0, T)]
    time = (lambda v, t: v[t]) if packed else (lambda v, t: v[:, t])
    S = torch.zeros(B, D, dtype=f, device="cuda") if s["state"] is None else s["state"].to(f)
    before = torch.empty_like(x)
    h, last = torch.empty_like(x), S.clone()
    for i, lo, hi in seqs:
        now = S[i]
        for t in range(lo, hi):
            time(before, t).copy_(now)
            now = torch.addcmul(time(u, t), time(a, t), now)
            time(h, t).copy_(now)
        last[i] = now
    if op == "scan_fwd":
        marks = before[::MARK] if packed else before[:, ::MARK]
        return {"y": h, "state": last, "marks": marks if case["marks"] else None}
    dy, ds = s["dy"].to(f), s["ds"].to(f)
    g, d0 = torch.empty_like(x), ds.clone()
    for i, lo, hi in seqs:
        r = ds[i]
        for t in range(hi - 1, lo - 1, -1):
            r = r + time(dy, t)
            time(g, t).copy_(r)
            r = r * time(a, t)
        d0[i] = r
    dl = a * g * before
    if case["comp"]:
        dl = dl - a * g * x
    if case["logits"]:
        dl = -dl * torch.sigmoid(s["gate"].to(f))
    return {"dx": w * g if case["comp"] else g, "d_log_decay": dl, "d_state0": None if s["state"] is None else d0}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if not op.startswith("scan"):
        tokens, heads, d, rot = case["B"] * case["T"], case["Hq"] + case["Hk"], case["d"], case["rot"]
        n = tokens * heads * d
        small = 4 * rot + (0 if case["pos"] == "count" else 4 * tokens)
        turn = 3 * tokens * heads * rot
        if op.startswith("rotary"):
            return {"bytes": 2 * n * e + small, "flops": turn}
        weights = {"none": 0, "f32": 8 * d, "bf16": 4 * d}[case["weight"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + small + weights, "flops": turn + 4 * n}
        return {"bytes": 3 * n * e + small + 2 * weights, "flops": turn + 11 * n}
    n = (case["T"] if case["lens"] else case["B"] * case["T"]) * case["D"]
    eg = 2 if case["gate"] == "bf16" else 4
    states = 4 * case["B"] * case["D"]
    marks = 4 * (n // MARK) if case["marks"] else 0
    if op == "scan_step":
        return {"bytes": n * (2 * e + eg) + 2 * states, "flops": 6 * n}
    if op == "scan_fwd":
        return {"bytes": n * (2 * e + eg) + marks + states * (2 if case["state"] else 1), "flops": 6 * n}
    return {"bytes": n * (3 * e + 2 * eg) + marks + states * (3 if case["state"] else 1), "flops": 14 * n}
