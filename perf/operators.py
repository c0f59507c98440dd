"""Timed cases of the linear-attention and layer-norm operators, with their plain forms.

Linear attention with a decay for each head, per (batch, head) with a state S [dk, dv]:

    S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T,      o_t = q_scale S_t^T q_t

``log_decay`` has one value per token and head, or one per head.  Layer norm
over the last axis, the weight and bias shared by all rows or one row of them
per head.  ``own`` chooses between the framework's kernels and the plain form.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-5


def listed():
    return [
        # one prompt of a single token-sized chunk: what a request costs at least
        dict(name="linear fwd, short prompt", op="fwd", B=1, H=16, T=64, dk=128, dv=128, dtype="bf16",
             decay="token", lens="", state0=True),
        # a training or prefill batch of the repository's main workload
        dict(name="linear fwd, batch", op="fwd", B=8, H=16, T=4096, dk=128, dv=128, dtype="bf16",
             decay="token", lens="", state0=True),
        # a long document on few chains, retention's fixed decays
        dict(name="linear fwd, long document", op="fwd", B=1, H=16, T=65536, dk=128, dv=128, dtype="bf16",
             decay="head", lens="", state0=False),
        # prompts of mixed lengths packed on one axis, odd head sizes, full precision
        dict(name="linear fwd, packed fp32", op="fwd", B=6, H=5, T=7777, dk=96, dv=75, dtype="f32",
             decay="token", lens="1,0,515,4096,64,3101", state0=True),
        # the training step of a layer
        dict(name="linear bwd, batch", op="bwd", B=4, H=16, T=4096, dk=128, dv=128, dtype="bf16",
             decay="token", lens="", state0=True),
        # training on packed documents, learned decays per head, smaller heads
        dict(name="linear bwd, packed", op="bwd", B=5, H=24, T=8192, dk=64, dv=64, dtype="bf16",
             decay="head", lens="2048,1,4095,640,1408", state0=False),
        # fine-tuning in full precision, odd sizes
        dict(name="linear bwd, odd fp32", op="bwd", B=2, H=3, T=1001, dk=72, dv=56, dtype="f32",
             decay="token", lens="", state0=True),
        # decoding with many sequences: the state is read and written once
        dict(name="linear step, 256 sequences", op="step", B=256, H=16, T=1, dk=128, dv=128, dtype="bf16",
             decay="token", lens="", state0=True),
        # decoding one sequence: latency
        dict(name="linear step, one sequence", op="step", B=1, H=16, T=1, dk=128, dv=128, dtype="bf16",
             decay="head", lens="", state0=True),
        # the mixer's output, normalised per head with a weight per head
        dict(name="norm fwd, heads", op="norm_fwd", rows=8 * 4096 * 16, D=128, G=16, dtype="bf16", bias=False),
        # the block's norm in training
        dict(name="norm bwd, width 2048", op="norm_bwd", rows=8 * 4096, D=2048, G=1, dtype="bf16", bias=True),
        # few rows of an odd width, full precision
        dict(name="norm bwd, odd fp32", op="norm_bwd", rows=1001, D=1023, G=1, dtype="f32", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        G = rng.choice([1, 1, 1, _log_int(rng, 2, 32)])
        D = _log_int(rng, 16, 8192 if G == 1 else 256)
        if rng.random() < 0.5:
            D -= D % 8
        rows = G * _log_int(rng, 1, max(1, (1 << 25) // (G * D)))
        return dict(op=op, rows=rows, D=D, G=G, dtype=dtype, bias=rng.random() < 0.5)
    dk, dv = (rng.choice([64, 128, 128, rng.randint(1, 128)]) for _ in range(2))
    H = rng.choice([1, 2, 3, 5, 8, 16, 24, 32])
    decay = rng.choice(["token", "token", "head"])
    state0 = rng.random() < 0.6
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 4096 // H), H=H, T=1, dk=dk, dv=dv, dtype=dtype, decay=decay, lens="",
                    state0=True)
    most = 1 << (19 if op == "fwd" else 18)  # token-heads
    least = 1 if op == "fwd" else 2  # the first token of a zero state has no gradient of its decay
    if rng.random() < 0.35:  # packed sequences
        n = rng.randint(1, 9)
        top = min(16384, most // (H * n))
        lens = [rng.choice([0, 1, _log_int(rng, 1, top), _log_int(rng, 1, top)]) if i else _log_int(rng, least, top)
                for i in range(n)]
        return dict(op=op, B=n, H=H, T=sum(lens), dk=dk, dv=dv, dtype=dtype, decay=decay,
                    lens=",".join(map(str, lens)), state0=state0)
    B = rng.choice([1, 1, 2, 3, 8])
    return dict(op=op, B=B, H=H, T=_log_int(rng, least, min(16384, most // (B * H))), dk=dk, dv=dv, dtype=dtype, decay=decay,
                lens="", state0=state0)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else []


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    f32 = torch.float32

    def normal(*shape, dtype=f32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=f32).to(dtype)

    st = {"case": case}
    if case["op"].startswith("norm"):
        rows, D, G = case["rows"], case["D"], case["G"]
        # activations with a mean and a scale of their own per row
        st["x"] = (normal(rows, D) * (0.5 + normal(rows, 1).abs()) + 0.3 * normal(rows, 1)).to(dt)
        st["x"] = st["x"].view(rows // G, G, D) if G > 1 else st["x"]
        wshape = (G, D) if G > 1 else (D,)
        st["weight"] = 1.0 + 0.1 * normal(*wshape)
        st["bias"] = 0.1 * normal(*wshape) if case["bias"] else None
        if case["op"] == "norm_bwd":
            st["dy"] = normal(*st["x"].shape, dtype=dt)
            x = st["x"].float()
            st["mean"] = x.mean(-1)
            st["rstd"] = (x.var(-1, unbiased=False) + EPS).rsqrt()
        return st

    B, H, T, dk, dv, op = (case[n] for n in ("B", "H", "T", "dk", "dv", "op"))
    lens = _lens(case)
    tok = (T, H) if lens else (B, H) if op == "step" else (B, T, H)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)).to(dt)

    st["q"], st["k"], st["v"] = unit(*tok, dk), unit(*tok, dk), normal(*tok, dv, dtype=dt)
    if case["decay"] == "token":  # log a = -softplus(x), x ~ N(-2, 1)
        st["la"] = -torch.nn.functional.softplus(normal(*tok) - 2.0)
    else:  # one fixed rate per head, memories of 16 to some thousand tokens
        st["la"] = torch.log1p(-torch.exp2(-(4.0 + 7.0 * torch.rand(H, generator=gen, device="cuda"))))
    st["state"] = 0.1 * normal(B, H, dk, dv) if case["state0"] else None
    st["scale"] = 1.0 / math.sqrt(dk)
    if lens:
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        st["cu"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        # where each packed token stands in a padded [B, longest] batch
        most = max(max(lens), 1)
        st["at"] = torch.cat([torch.arange(n, device="cuda") + i * most for i, n in enumerate(lens)])
        st["longest"] = most
    if op == "bwd":
        st["do"] = normal(*tok, dv, dtype=dt)
        st["ds"] = 0.1 * normal(B, H, dk, dv)
    return st


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import gated_delta_rule_decay_amd as g

    op = s["case"]["op"]
    if op == "norm_fwd":
        y, mean, rstd = g.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = g.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], want_bias=s["bias"] is not None)
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "step":
        o = g.linear_recurrent_step(s["q"], s["k"], s["v"], s["la"], s["state"], q_scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "fwd":
        if "cu" in s:
            o, S = g.linear_chunk_fwd_varlen(s["q"], s["k"], s["v"], s["la"], s["cu"], s["state"], q_scale=s["scale"])
        else:
            o, S = g.linear_chunk_fwd(s["q"], s["k"], s["v"], s["la"], s["state"], q_scale=s["scale"])
        return {"o": o, "state": S}
    if "cu" in s:
        return g.linear_chunk_bwd_varlen(s["q"], s["k"], s["v"], s["la"], s["cu"], s["state"], s["do"], s["ds"],
                                         q_scale=s["scale"])
    return g.linear_chunk_bwd(s["q"], s["k"], s["v"], s["la"], s["state"], s["do"], s["ds"], q_scale=s["scale"])


def _padded(s, x):
    """Packed [T, ...] -> [B, longest, ...] with zeros behind each sequence."""
    n = s["case"]["B"] * s["longest"]
    return x.new_zeros((n, *x.shape[1:])).index_copy(0, s["at"], x).view(s["case"]["B"], s["longest"], *x.shape[1:])


def _chunked(q, k, v, la, s0, scale):
    """The chunked form in 32 bits: q, k, v [B,T,H,d], la [B,T,H] in 64 bits (sums of decays lose in 32)."""
    B, T, H, dk = k.shape
    dv = v.shape[-1]
    n = -(-T // CHUNK)

    def cut(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - T))
        x = x.view(B, n, CHUNK, *x.shape[2:])
        return x.movedim(3, 1).contiguous()  # [B, H, n, CHUNK, ...]

    q, k, v, la = cut(q), cut(k), cut(v), cut(la)
    g = la.cumsum(-1)
    total = g[..., -1]
    upper = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).triu(1)
    decay = (g[..., :, None] - g[..., None, :]).masked_fill(upper, -math.inf).float().exp()
    o = ((q @ k.transpose(-1, -2).contiguous()) * decay) @ v
    # what each chunk adds to the state, and the state before each chunk
    add = (k * (total[..., None] - g).float().exp()[..., None]).transpose(-1, -2).contiguous() @ v
    end = total.cumsum(-1)  # [B, H, n]
    start = torch.cat([torch.zeros_like(end[..., :1]), end], -1)
    later = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).triu(0)
    mix = (start[..., :, None] - end[..., None, :]).masked_fill(later, -math.inf).float().exp()
    states = (mix @ add.view(B, H, n, dk * dv)).view(B, H, n + 1, dk, dv)
    if s0 is not None:
        states = states + start.float().exp()[..., None, None] * s0[:, :, None]
    o = o + (q * g.float().exp()[..., None]) @ states[:, :, :n]
    return scale * o.movedim(1, 3).reshape(B, n * CHUNK, H, dv)[:, :T], states[:, :, n]


def _plain_forward(s, q, k, v, la, s0):
    packed = "cu" in s
    B, H = s["case"]["B"], s["case"]["H"]
    if packed:
        q, k, v = _padded(s, q), _padded(s, k), _padded(s, v)
        if la.dim() == 1:
            # no decay behind a sequence's end, so its state stays
            la = _padded(s, la.expand(s["case"]["T"], H))
        else:
            la = _padded(s, la)
    elif la.dim() == 1:
        la = la.expand(B, s["case"]["T"], H)
    o, S = _chunked(q, k, v, la, s0, s["scale"])
    return (o.reshape(-1, H, o.shape[-1])[s["at"]] if packed else o), S


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(-1, keepdim=True) + EPS).rsqrt()
        y = xc * rstd * s["weight"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(s["x"].dtype), "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if op == "norm_bwd":
        x, dy = s["x"].float(), s["dy"].float()
        rstd = s["rstd"][..., None]
        xh = (x - s["mean"][..., None]) * rstd
        wdy = dy * s["weight"]
        dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if s["bias"] is not None else None}
    if op == "step":
        q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
        S.mul_(s["la"].exp()[..., None, None]).add_(k[..., :, None] * v[..., None, :])
        o = s["scale"] * (q[..., None, :] @ S)[..., 0, :]
        return {"o": o.to(s["q"].dtype), "state": S}
    dt = s["q"].dtype
    q, k, v, la, s0 = s["q"].float(), s["k"].float(), s["v"].float(), s["la"].double(), s["state"]
    if op == "fwd":
        o, S = _plain_forward(s, q, k, v, la, s0)
        return {"o": o.to(dt), "state": S}
    with torch.enable_grad():
        ins = [x.detach().requires_grad_() for x in (q, k, v, la)]
        st = None if s0 is None else s0.detach().requires_grad_()
        o, S = _plain_forward(s, *ins, st)
        g = torch.autograd.grad([o, S], ins + ([] if st is None else [st]), [s["do"].float(), s["ds"]])
    return {"dq": g[0].to(dt), "dk": g[1].to(dt), "dv": g[2].to(dt), "d_log_decay": g[3].float(),
            "d_state0": g[4] if st is not None else None}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"].startswith("norm"):
        x, w = s["x"].to(f), s["weight"].to(f)
        if case["op"] == "norm_fwd":
            mu = x.sum(-1, keepdim=True) / x.shape[-1]
            r = 1.0 / torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
            y = (x - mu) * r * w + (0.0 if s["bias"] is None else s["bias"].to(f))
            return {"y": y, "mean": mu[..., 0], "rstd": r[..., 0]}
        dy, D = s["dy"].to(f), x.shape[-1]
        r = s["rstd"].to(f).unsqueeze(-1)
        h = (x - s["mean"].to(f).unsqueeze(-1)) * r
        e = dy * w
        dx = r * (e - e.sum(-1, keepdim=True) / D - h * (e * h).sum(-1, keepdim=True) / D)
        return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": None if s["bias"] is None else dy.sum(0)}

    # token by token, every sequence of a packed batch in step
    op, H = case["op"], case["H"]
    q, k, v, la = (s[n].to(f) for n in ("q", "k", "v", "la"))
    packed, step = "cu" in s, op == "step"
    if packed:
        B, L = case["B"], s["longest"]

        def lay(x):
            y = torch.zeros(B * L, *x.shape[1:], dtype=f, device=x.device)
            y[s["at"]] = x
            return y.view(B, L, *x.shape[1:])
    else:
        B, L = case["B"], case["T"]
        lay = (lambda x: x[:, None]) if step else (lambda x: x)
    a = la.exp()
    if case["decay"] == "head":
        a = a.expand(case["T"], H) if packed else a.expand(B, H) if step else a.expand(B, L, H)
    live = torch.ones(B, L, H, dtype=f, device=q.device)
    if packed:
        live = lay(torch.ones(case["T"], H, dtype=f, device=q.device))
    q, k, v, a = lay(q) * s["scale"], lay(k), lay(v), lay(a) + (1.0 - live)
    q, k, v, a = (x.transpose(0, 1).contiguous() for x in (q, k, v, a))  # [L, B, H, ...]
    S = torch.zeros(B, H, case["dk"], case["dv"], dtype=f, device=q.device)
    if s["state"] is not None:
        S += s["state"]

    def back(x):
        x = x.transpose(0, 1)
        return x.reshape(B * L, *x.shape[2:])[s["at"]] if packed else x[:, 0] if step else x

    if op != "bwd":
        o = torch.empty_like(v)
        for t in range(L):
            S.mul_(a[t, :, :, None, None]).add_(k[t, :, :, :, None] * v[t, :, :, None, :])
            torch.sum(q[t, :, :, :, None] * S, 2, out=o[t])
        return {"o": back(o), "state": S}
    do = lay(s["do"].to(f)).transpose(0, 1).contiguous()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S.mul_(a[t, :, :, None, None]).add_(k[t, :, :, :, None] * v[t, :, :, None, :])
        torch.sum(S * do[t, :, :, None, :], 3, out=dq[t])
    dS = s["ds"].to(f)
    last = (S * dS).sum((2, 3))
    for t in range(L - 1, -1, -1):
        dS = dS + q[t, :, :, :, None] * do[t, :, :, None, :]
        torch.sum(dS * k[t, :, :, :, None], 2, out=dv[t])
        torch.sum(dS * v[t, :, :, None, :], 3, out=dk[t])
        dS = dS * a[t, :, :, None, None]
    each = ((q * dq).sum(-1) - (k * dk).sum(-1)) * live.transpose(0, 1)
    dla = (each.flip(0).cumsum(0).flip(0) + last) * live.transpose(0, 1)
    dla = dla.sum((0, 1)) if case["decay"] == "head" else back(dla)
    return {"dq": back(dq) * s["scale"], "dk": back(dk), "dv": back(dv), "d_log_decay": dla,
            "d_state0": dS if s["state"] is not None else None}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, w = case["rows"] * case["D"], 4 * case["G"] * case["D"]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + w * (2 if case["bias"] else 1), "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + w * (3 if case["bias"] else 2), "flops": 14 * n}
    H, dk, dv = case["H"], case["dk"], case["dv"]
    tok = (case["T"] if case["lens"] else case["B"] * case["T"]) * H
    decay = 4 * (tok if case["decay"] == "token" else H)
    state = 4 * case["B"] * H * dk * dv
    if case["op"] == "bwd":
        given = 2 if case["state0"] else 0  # state0 in, its gradient out
        return {"bytes": tok * e * (4 * dk + 3 * dv) + 2 * decay + (1 + given) * state, "flops": 10 * tok * dk * dv}
    return {"bytes": tok * e * (2 * dk + 2 * dv) + decay + (2 if case["state0"] else 1) * state, "flops": 4 * tok * dk * dv}
