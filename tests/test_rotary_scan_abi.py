"""Refusals of the rotary, query/key norm and gated scan calls (CPU): host-side
validation answers before any HIP call, so the fake addresses are never
dereferenced."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_decay_amd as g
from gated_delta_rule_decay_amd import binding as bd
from gated_delta_rule_decay_amd import linear as ln
from gated_delta_rule_decay_amd import rotary as ro
from gated_delta_rule_decay_amd import scan as sc

OK, NULL, SHAPE, DTYPE, UNSUPPORTED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5, 6
BASE, SLOT = 1 << 40, 1 << 33


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.library_path()):
        from gated_delta_rule_decay_amd.build import build_library
        build_library()
    return ln._lib()


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * SLOT + off)


def ref(d):
    return None if d is None else ctypes.byref(d)


def rd(norm=ro.GDN2_QK_NONE, **kw):
    base = dict(tokens=24, q_heads=4, k_heads=2, dim=64, rotary=64, norm=norm)
    base.update(kw)
    return ro.make_rotary_desc(**base)


def turn(lib, d, back=False, **kw):
    a = dict(q=P(0), k=P(1), f=P(2), p=P(3), qo=P(4), ko=P(5))
    a.update(kw)
    f = lib.gdn2_rotary_bwd if back else lib.gdn2_rotary_fwd
    return f(ref(d), a["q"], a["k"], a["f"], a["p"], a["qo"], a["ko"], None)


def nfwd(lib, d, **kw):
    a = dict(q=P(0), k=P(1), f=P(2), p=P(3), qo=P(4), ko=P(5), qw=P(6), kw=P(7))
    a.update(kw)
    return lib.gdn2_qk_norm_fwd(ref(d), a["q"], a["k"], a["qw"], a["kw"], a["f"], a["p"], a["qo"], a["ko"], None)


def nbwd(lib, d, **kw):
    a = dict(q=P(0), k=P(1), f=P(2), p=P(3), dqo=P(4), dko=P(5), qw=P(6), kw=P(7), dq=P(8), dk=P(9), dqw=P(10), dkw=P(11),
             ws=P(12), n=1 << 30)
    a.update(kw)
    return lib.gdn2_qk_norm_bwd(ref(d), a["dqo"], a["dko"], a["q"], a["k"], a["qw"], a["kw"], a["f"], a["p"], a["dq"], a["dk"],
                                a["dqw"], a["dkw"], a["ws"], a["n"], None)


BAD_ROTARY = [
    (dict(tokens=-1, period=1), SHAPE), (dict(period=0), SHAPE), (dict(period=7), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(k_heads=-1), SHAPE), (dict(dim=0, rotary=0), SHAPE), (dict(rotary=63), SHAPE), (dict(rotary=66), SHAPE), (dict(rotary=-2), SHAPE),
    (dict(dtype=2), DTYPE), (dict(weight_dtype=-1), DTYPE), (dict(layout=2), SHAPE), (dict(layout=-1), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(magnitude=float("inf")), SHAPE),
    (dict(magnitude=float("nan")), SHAPE), (dict(offset=(1 << 40) + 1), SHAPE), (dict(offset=-(1 << 41)), SHAPE),
    (dict(dim=257), UNSUPPORTED), (dict(q_heads=65536), UNSUPPORTED), (dict(k_heads=65536), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(q_stride=255), SHAPE), (dict(k_stride=127), SHAPE), (dict(q_stride=1 << 60), SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_ROTARY)
def test_bad_rotary_descriptors(lib, kw, status):
    n = ctypes.c_size_t(7)
    assert turn(lib, rd(**kw)) == status and turn(lib, rd(**kw), back=True) == status
    d = rd(norm=ro.GDN2_QK_RMS, **kw)
    assert nfwd(lib, d) == status and nbwd(lib, d) == status
    assert lib.gdn2_qk_norm_bwd_workspace(ref(d), ctypes.byref(n)) == status and n.value == 7


def test_norm_kinds(lib):
    for k in (ro.GDN2_QK_RMS, ro.GDN2_QK_L2, 3, -1):
        assert turn(lib, rd(norm=k)) == SHAPE
    for k in (ro.GDN2_QK_NONE, 3, -1):
        assert nfwd(lib, rd(norm=k)) == SHAPE and nbwd(lib, rd(norm=k)) == SHAPE


def test_rotary_null_arguments(lib):
    assert turn(lib, None) == NULL and nfwd(lib, None) == NULL and nbwd(lib, None) == NULL
    for n in ("q", "k", "f", "qo", "ko"):
        assert turn(lib, rd(), **{n: None}) == NULL and nfwd(lib, rd(norm=1), **{n: None}) == NULL, n
    for n in ("q", "k", "f", "dqo", "dko", "dq", "dk"):
        assert nbwd(lib, rd(norm=2), **{n: None}) == NULL, n
    assert lib.gdn2_qk_norm_bwd_workspace(ref(rd(norm=1)), None) == NULL
    # nothing to do: no tokens
    assert turn(lib, rd(tokens=0), q=None, k=None, f=None, qo=None, ko=None) == OK
    assert nbwd(lib, rd(norm=1, tokens=0), q=None, dq=None, dqw=None, dkw=None, ws=None, n=0) == OK


def test_rotary_aliasing(lib):
    q_bytes = 24 * 4 * 64 * 2
    for i in (1, 2, 3):
        assert turn(lib, rd(), qo=P(i)) == ALIAS, i
    assert turn(lib, rd(), ko=P(0)) == ALIAS and turn(lib, rd(), ko=P(4)) == ALIAS and turn(lib, rd(), qo=P(0, 16)) == ALIAS
    # exactly in place, but not where the input is a slice of something wider
    assert turn(lib, rd(q_stride=512), qo=P(0)) == ALIAS
    assert turn(lib, rd(), qo=P(0, q_bytes - 2)) == ALIAS
    assert turn(lib, rd(q_stride=512), qo=P(0, q_bytes)) == ALIAS  # between the first and the last token's rows
    for i in (6, 7):
        assert nfwd(lib, rd(norm=1), qo=P(i)) == ALIAS, i
    for i in range(8):
        assert nbwd(lib, rd(norm=1), dq=P(i)) == ALIAS, i
    for i in (9, 10, 11, 12):
        assert nbwd(lib, rd(norm=1), dq=P(i)) == ALIAS, i
    assert nbwd(lib, rd(norm=1), dqw=P(11)) == ALIAS


def test_rotary_workspaces(lib):
    d, n = rd(norm=1), ctypes.c_size_t(0)
    assert lib.gdn2_qk_norm_bwd_workspace(ref(d), ctypes.byref(n)) == OK and n.value > 0
    assert nbwd(lib, d, ws=None, n=0) == WORKSPACE and nbwd(lib, d, n=n.value - 1) == WORKSPACE
    assert nbwd(lib, d, ws=P(12, 128), n=n.value) == WORKSPACE
    d = rd(norm=1, tokens=0)
    assert lib.gdn2_qk_norm_bwd_workspace(ref(d), ctypes.byref(n)) == OK and n.value == 0


def sd(**kw):
    base = dict(batch=3, seqlen=256, dim=64)
    base.update(kw)
    return sc.make_scan_desc(**base)


def sfwd(lib, d, packed=False, **kw):
    a = dict(cu=P(20), x=P(0), g=P(1), s0=P(2), y=P(3), so=P(4), m=P(5), ws=P(12), n=1 << 32)
    a.update(kw)
    f = lib.gdn2_scan_fwd_varlen if packed else lib.gdn2_scan_fwd
    return f(ref(d), *([a["cu"]] if packed else []), a["x"], a["g"], a["s0"], a["y"], a["so"], a["m"], a["ws"], a["n"], None)


def sbwd(lib, d, packed=False, **kw):
    a = dict(cu=P(20), dy=P(0), x=P(1), g=P(2), m=P(3), s0=P(4), ds=P(5), dx=P(6), dg=P(7), ds0=P(8), ws=P(12), n=1 << 32)
    a.update(kw)
    f = lib.gdn2_scan_bwd_varlen if packed else lib.gdn2_scan_bwd
    return f(ref(d), *([a["cu"]] if packed else []), a["dy"], a["x"], a["g"], a["m"], a["s0"], a["ds"], a["dx"], a["dg"], a["ds0"],
             a["ws"], a["n"], None)


def sstep(lib, d, **kw):
    a = dict(x=P(0), g=P(1), s=P(2), y=P(3))
    a.update(kw)
    return lib.gdn2_scan_step(ref(d), a["x"], a["g"], a["s"], a["y"], None)


BAD_SCAN = [(dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
            (dict(gate_dtype=7), DTYPE), (dict(batch=1 << 40, dim=1 << 30), SHAPE), (dict(batch=1 << 24), UNSUPPORTED), (dict(batch=(1 << 22) - 32, dim=3), UNSUPPORTED),
            (dict(dim=1 << 30), UNSUPPORTED), (dict(dim=1 << 32, batch=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_SCAN)
def test_bad_scan_descriptors(lib, kw, status):
    n = ctypes.c_size_t(7)
    assert sfwd(lib, sd(**kw)) == status and sbwd(lib, sd(**kw)) == status
    assert lib.gdn2_scan_fwd_workspace(ref(sd(**kw)), ctypes.byref(n)) == status
    assert lib.gdn2_scan_bwd_workspace(ref(sd(**kw)), ctypes.byref(n)) == status and n.value == 7
    kw1 = dict(kw)
    kw1.setdefault("seqlen", 1)
    assert sstep(lib, sd(**kw1)) == status


def test_scan_lengths(lib):
    assert sfwd(lib, sd(seqlen=1 << 31), packed=True) == SHAPE and sbwd(lib, sd(seqlen=1 << 31), packed=True) == SHAPE
    assert sfwd(lib, sd(batch=(1 << 31) - 1), packed=True) == SHAPE
    assert sfwd(lib, sd(batch=1, seqlen=1 << 31)) == UNSUPPORTED
    assert sfwd(lib, sd(batch=1 << 12, seqlen=1 << 30, dim=64)) == UNSUPPORTED  # tiles
    assert sstep(lib, sd(seqlen=2)) == SHAPE


def test_scan_null_arguments(lib):
    assert sfwd(lib, None) == NULL and sbwd(lib, None) == NULL and sstep(lib, None) == NULL
    for n in ("x", "g", "y"):
        assert sfwd(lib, sd(), **{n: None}) == NULL and sfwd(lib, sd(), packed=True, **{n: None}) == NULL, n
    for n in ("dy", "x", "g", "m", "dx", "dg"):
        assert sbwd(lib, sd(), **{n: None}) == NULL and sbwd(lib, sd(), packed=True, **{n: None}) == NULL, n
    for n in ("x", "g", "s", "y"):
        assert sstep(lib, sd(seqlen=1), **{n: None}) == NULL, n
    assert sfwd(lib, sd(), packed=True, cu=None) == NULL and sbwd(lib, sd(), packed=True, cu=None) == NULL
    assert lib.gdn2_scan_fwd_workspace(ref(sd()), None) == NULL
    assert sfwd(lib, sd(batch=0), x=None, g=None, y=None) == OK
    assert sstep(lib, sd(batch=0, seqlen=1), x=None, g=None, y=None, s=None) == OK


def test_scan_aliasing(lib):
    for i in (0, 1, 2, 4, 5):
        assert sfwd(lib, sd(), y=P(i)) == ALIAS, i
    assert sfwd(lib, sd(), so=P(2, 4)) == ALIAS and sfwd(lib, sd(), so=P(0)) == ALIAS and sfwd(lib, sd(), m=P(2)) == ALIAS
    assert sfwd(lib, sd(), packed=True, y=P(20)) == ALIAS
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 12):
        assert sbwd(lib, sd(), dx=P(i)) == ALIAS, i
    assert sbwd(lib, sd(), packed=True, dg=P(20)) == ALIAS
    assert sstep(lib, sd(seqlen=1), y=P(2)) == ALIAS and sstep(lib, sd(seqlen=1), s=P(0)) == ALIAS


def test_scan_workspaces(lib):
    d, n = sd(), ctypes.c_size_t(0)
    for size, call in ((lib.gdn2_scan_fwd_varlen_workspace, sfwd), (lib.gdn2_scan_bwd_varlen_workspace, sbwd)):
        assert size(ref(d), ctypes.byref(n)) == OK and n.value > 0
        assert call(lib, d, packed=True, ws=None, n=0) == WORKSPACE and call(lib, d, packed=True, n=n.value - 1) == WORKSPACE
        assert call(lib, d, packed=True, ws=P(12, 16), n=n.value) == WORKSPACE
        assert call(lib, d, packed=True, ws=P(0), n=n.value) == ALIAS


def test_descriptor_layouts(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines, want = [], []
    for cls, name in ((ro.Gdn2RotaryDesc, "gdn2_rotary_desc"), (sc.Gdn2ScanDesc, "gdn2_scan_desc")):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn2.h"\nint main(void) {\n' + "\n".join(lines)
                   + "\nreturn 0;\n}\n")
    subprocess.run([cc, "-I", inc, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want


# the binding's own checks, before the library is called
def test_rotary_binding_refusals():
    q, k, f = torch.zeros(2, 8, 3, 16), torch.zeros(2, 8, 1, 16), torch.zeros(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="GPU"):
        g.rotary_fwd(q, k, f)
    with pytest.raises(TypeError):
        g.rotary_fwd(q, k, f.float())
    with pytest.raises(TypeError):
        g.rotary_fwd(q, k.bfloat16(), f)
    with pytest.raises(TypeError):
        g.rotary_fwd(q.half(), None, f)
    with pytest.raises(ValueError, match="turns"):
        g.rotary_fwd(q, k, torch.zeros(9, dtype=torch.float64))
    with pytest.raises(ValueError, match="channels"):
        g.rotary_fwd(q, k[..., :8], f)
    with pytest.raises(ValueError, match="tokens"):
        g.rotary_fwd(q, k[:, :4], f)
    with pytest.raises(ValueError, match="positions"):
        g.rotary_fwd(q, k, f, positions=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        g.rotary_fwd(q, k, f, positions=torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguously"):
        g.rotary_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, f)
    with pytest.raises(ValueError, match="contiguously"):
        g.rotary_fwd(q[..., ::2], None, f[:4])
    with pytest.raises(ValueError, match="contiguously"):
        g.rotary_fwd(q[:, ::2][:, :, :, :].expand(2, 4, 3, 16)[:, :3], None, f)
    with pytest.raises(ValueError, match="token axis"):
        g.rotary_fwd(q[0, 0], None, f)
    with pytest.raises(ValueError, match="q_out"):
        g.rotary_fwd(q, k, f, q_out=q[:, :4])
    with pytest.raises(ValueError, match="norm"):
        g.qk_norm_rotary_fwd(q, k, norm="max")
    with pytest.raises(ValueError, match="weight"):
        g.qk_norm_rotary_fwd(q, k, torch.ones(8))
    with pytest.raises(TypeError):
        g.qk_norm_rotary_fwd(q, k, torch.ones(16), torch.ones(16).bfloat16())
    with pytest.raises(ValueError, match="d_q_out"):
        g.qk_norm_rotary_bwd(q[:, :4], k, q, k)
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=8, base=0.0), dict(rotary=8, scaling="other"),
                dict(rotary=8, scaling="parts"), dict(rotary=8, factor=-1.0)):
        with pytest.raises(ValueError):
            g.rotary_frequencies(device="cpu", **bad)


def test_scan_binding_refusals():
    x = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="GPU"):
        g.gated_scan_fwd(x, x)
    with pytest.raises(TypeError):
        g.gated_scan_fwd(x.half(), x)
    with pytest.raises(TypeError):
        g.gated_scan_fwd(x, x.double())
    with pytest.raises(ValueError, match="log_decay"):
        g.gated_scan_fwd(x, x[:, :4])
    with pytest.raises(ValueError, match="contiguous"):
        g.gated_scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), x)
    with pytest.raises(ValueError, match="state0"):
        g.gated_scan_fwd(x, x, torch.zeros(2, 8))
    with pytest.raises(ValueError, match="packed"):
        g.gated_scan_fwd_varlen(x, x, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        g.gated_scan_fwd_varlen(x[0], x[0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="marks"):
        g.gated_scan_bwd(x, x, x, torch.zeros(2, 2, 16))
    with pytest.raises(ValueError, match="dy"):
        g.gated_scan_bwd(x[:, :4], x, x, torch.zeros(2, 1, 16))
    with pytest.raises(ValueError, match=r"\[N,D\]"):
        g.gated_scan_step(x, x, x)
    with pytest.raises(ValueError, match="state"):
        g.gated_scan_step(x[0], x[0], torch.zeros(8, 8))
