"""The norms with rotary positions where arithmetic is at its limits: an eps below
fp32's normal numbers, weight gradients over very many rows, positions far out."""
import pytest
import torch

from tests import rotary_oracle as ref

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_decay_amd as pkg
    return pkg


def rn(*shape, dtype=F32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(100 + seed)).to(dtype).cuda()


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F32), (33, F32)])
@pytest.mark.parametrize("eps", [1e-40, 1e-45, 2e-38])
def test_eps_below_normal_numbers(g, eps, d, dtype):
    # lanes behind the last row hold rows of zeros, whose mean is eps alone; so do rows of zeros
    f, w = g.rotary_frequencies(16), 1 + 0.1 * rn(d, seed=4)
    for T in (1, 37, 300):
        q, dq = rn(T, 3, d, dtype=dtype), rn(T, 3, d, dtype=dtype, seed=1)
        for zeros in (False, True):
            if zeros:
                q[T // 2, 1] = 0
                dq[T // 2, 1] = 0  # 1 / sqrt(eps) of anything else is past fp32
            y = g.qk_norm_rotary_fwd(q, None, w, None, f, eps=eps)[0]
            r = g.qk_norm_rotary_bwd(dq, None, q, None, w, None, f, eps=eps)
            ref.check("q", y, *ref.norm_turn(q, w, f, None, 0, False, 1.0, "rms", eps))
            dx, dw, bx, bw = ref.norm_turn_backward(dq, q, w, f, None, 0, False, 1.0, "rms", eps)
            ref.check("dq", r["dq"], dx, bx)
            ref.check("d_q_weight", r["d_q_weight"], dw, bw)


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_weight_sums_over_very_many_rows(g, norm):
    # a thousand rows for each lane of the launch, and terms that do not change, so that
    # roundings of one lane's sum would all go to the same side
    T, d = 4 * 1024 * 1000 + 3, 255
    q, dq = 1 + rn(d).abs(), 1 + rn(d, seed=1).abs()
    w = 1 + 0.1 * rn(d, seed=2)
    f = torch.zeros(1, dtype=F64, device="cuda")
    r = g.qk_norm_rotary_bwd(dq.expand(T, 1, d).contiguous(), None, q.expand(T, 1, d).contiguous(), None, w, None, f, norm=norm)
    dx, dw, bx, bw = ref.norm_turn_backward(dq.expand(1, 1, d), q.expand(1, 1, d), w, f, None, 0, False, 1.0, norm, 1e-6)
    ref.check("d_q_weight", r["d_q_weight"], T * dw, T * bw)
    for first in (0, T - 5):
        ref.check("dq", r["dq"][first:first + 5], dx.expand(5, 1, d), bx.expand(5, 1, d))


def test_weight_sums_of_k_and_of_wide_vectors(g):
    # some hundred rows a lane, eight bf16 channels a vector, q and k apart; the sums over rows in parts
    T, Hq, Hk, d = 200000, 24, 8, 64
    q, dq = torch.randn(T, Hq, d, dtype=BF, device="cuda") + 1, torch.randn(T, Hq, d, dtype=BF, device="cuda") + 1
    k, dk = torch.randn(T, Hk, d, dtype=BF, device="cuda") - 1, torch.randn(T, Hk, d, dtype=BF, device="cuda") + 1
    w = 1 + 0.1 * rn(d, seed=2)
    r = g.qk_norm_rotary_bwd(dq, dk, q, k, w, w, norm="l2")
    for n, x, dy in (("q", q, dq), ("k", k, dk)):
        want, bound = torch.zeros(d, dtype=F64, device="cuda"), torch.zeros(d, dtype=F64, device="cuda")
        for a, b in zip(x.split(20000), dy.split(20000)):
            a, b = a.double(), b.double()
            t = b * (a / a.norm(dim=-1, keepdim=True))
            want += t.sum((0, 1))
            bound += 72 * ref.E * t.abs().sum((0, 1))
        ref.check(f"d_{n}_weight", r[f"d_{n}_weight"], want.cpu(), bound.cpu())


def far_angles(positions, freq):
    """cos and sin of position * freq, the product reduced in integers."""
    bits = 300

    def arctan_of_inverse(n):
        term = total = (1 << bits) // n
        k, sign = 1, 1
        while term:
            term //= n * n
            k, sign = k + 2, -sign
            total += sign * (term // k)
        return total

    two_pi = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))  # Machin's formula, times 2^bits
    c, s = (torch.empty(len(positions), 1, len(freq), dtype=F64) for _ in range(2))
    for i, p in enumerate(positions):
        for j, f in enumerate(freq):
            top, bottom = f.as_integer_ratio()  # a power of 2 below
            rest = ((p * top << bits) // bottom) % two_pi  # radians times 2^bits
            t = torch.tensor(rest / (1 << bits), dtype=F64)
            c[i, 0, j], s[i, 0, j] = t.cos(), t.sin()
    return c, s


@pytest.mark.parametrize("offset", [0, -(1 << 40), (1 << 40) - 3, 123456789012, 1 << 24])
@pytest.mark.parametrize("inter", [False, True])
def test_angles_of_far_positions(g, inter, offset):
    # the bounds are those of near positions: angles lose nothing on the way
    d, positions = 16, [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 77777777]
    f = torch.tensor([0.7499, 1.0, 1 / 3, 0.1 ** 0.5, 1e-3, 2.5, 1e-9, 3.999], dtype=F64)
    q, k = rn(len(positions), 2, d), rn(len(positions), 1, d, seed=1)
    pos = torch.tensor(positions, dtype=torch.int32).cuda()
    c, s = far_angles([offset + p for p in positions], f.tolist())
    a, b = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    for back, fn in ((1, g.rotary_fwd), (-1, g.rotary_bwd)):
        for x, y in zip((q, k), fn(q, k, f.cuda(), positions=pos, offset=offset, interleaved=inter)):
            x = x.cpu().double()
            want, size = torch.empty_like(x), torch.empty_like(x)
            u, v = x[..., a], x[..., b]
            want[..., a], want[..., b] = c * u - back * s * v, back * s * u + c * v
            size[..., a] = size[..., b] = u.abs() + v.abs()
            ref.check("x", y, want, 9 * ref.E * size)
    y = g.qk_norm_rotary_fwd(q, None, freq=f.cuda(), positions=pos, offset=offset, interleaved=inter)[0]
    h = q.cpu().double()
    h = h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    u, v = h[..., a], h[..., b]
    want, size = torch.empty_like(h), torch.empty_like(h)
    want[..., a], want[..., b] = c * u - s * v, s * u + c * v
    size[..., a] = size[..., b] = u.abs() + v.abs()
    ref.check("normed", y, want, 24 * ref.E * size)
