"""Refusals of the linear-attention and layer-norm calls (CPU): host-side
validation answers before any HIP call, so the fake addresses are never
dereferenced."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_decay_amd as g
from gated_delta_rule_decay_amd import binding as bd
from gated_delta_rule_decay_amd import linear as ln

NULL, SHAPE, DTYPE, UNSUPPORTED, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6
BASE, SLOT = 1 << 40, 1 << 32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.library_path()):
        from gated_delta_rule_decay_amd.build import build_library
        build_library()
    return ln._lib()


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * SLOT + off)


def desc(**kw):
    base = dict(batch=2, seqlen=128, heads=4, dk=128, dv=128)
    base.update(kw)
    return ln.make_linear_desc(**base)


def fwd(lib, d, packed=False, **kw):
    a = dict(cu=P(20), q=P(0), k=P(1), v=P(2), la=P(3), s0=P(4), o=P(5), so=P(6), ws=None, n=0)
    a.update(kw)
    f = lib.gdn2_linear_fwd_varlen if packed else lib.gdn2_linear_fwd
    return f(None if d is None else ctypes.byref(d), *([a["cu"]] if packed else []), a["q"], a["k"], a["v"], a["la"],
             a["s0"], a["o"], a["so"], a["ws"], a["n"], None)


def bwd(lib, d, packed=False, **kw):
    a = dict(cu=P(20), q=P(0), k=P(1), v=P(2), la=P(3), s0=P(4), do=P(5), ds=P(6), dq=P(7), dk=P(8), dv=P(9), dla=P(10),
             ds0=P(11), ws=P(12), n=1 << 31)
    a.update(kw)
    f = lib.gdn2_linear_bwd_varlen if packed else lib.gdn2_linear_bwd
    return f(None if d is None else ctypes.byref(d), *([a["cu"]] if packed else []), a["q"], a["k"], a["v"], a["la"],
             a["s0"], a["do"], a["ds"], a["dq"], a["dk"], a["dv"], a["dla"], a["ds0"], a["ws"], a["n"], None)


def step(lib, d, **kw):
    a = dict(q=P(0), k=P(1), v=P(2), la=P(3), st=P(4), o=P(5))
    a.update(kw)
    return lib.gdn2_linear_step(None if d is None else ctypes.byref(d), a["q"], a["k"], a["v"], a["la"], a["st"], a["o"], None)


BAD = [(dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(heads=0), SHAPE), (dict(dk=0), SHAPE), (dict(dv=0), SHAPE),
       (dict(dk=129), UNSUPPORTED), (dict(dv=200), UNSUPPORTED), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
       (dict(decay_kind=2), SHAPE), (dict(batch=1 << 40, seqlen=1 << 30), SHAPE), (dict(batch=1 << 26), UNSUPPORTED),
       (dict(heads=1 << 26), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_linear_descriptors(lib, kw, status):
    d = desc(**kw)
    n = ctypes.c_size_t(7)
    assert fwd(lib, d) == status and bwd(lib, d) == status
    assert lib.gdn2_linear_fwd_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    assert lib.gdn2_linear_bwd_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    assert n.value == 7
    kw1 = dict(kw)
    kw1.setdefault("seqlen", 1)
    assert step(lib, desc(**kw1)) == status


def test_long_sequences(lib):
    assert fwd(lib, desc(seqlen=1 << 31), packed=True) == SHAPE
    assert fwd(lib, desc(batch=1, heads=1, seqlen=1 << 31)) == UNSUPPORTED
    r = desc()
    r.reserved = 1
    assert fwd(lib, r) == SHAPE


def test_null_arguments(lib):
    assert fwd(lib, None) == NULL and bwd(lib, None) == NULL and step(lib, None) == NULL
    for n in ("q", "k", "v", "la", "o"):
        assert fwd(lib, desc(), **{n: None}) == NULL, n
        assert fwd(lib, desc(), packed=True, **{n: None}) == NULL, n
    assert fwd(lib, desc(), packed=True, cu=None) == NULL
    for n in ("q", "k", "v", "la", "do", "dq", "dk", "dv", "dla"):
        assert bwd(lib, desc(), **{n: None}) == NULL, n
    for n in ("q", "k", "v", "la", "st", "o"):
        assert step(lib, desc(seqlen=1), **{n: None}) == NULL, n
    assert lib.gdn2_linear_fwd_workspace(ctypes.byref(desc()), None) == NULL
    assert step(lib, desc(seqlen=2)) == SHAPE


def test_aliasing(lib):
    one = 2 * 128 * 4 * 128 * 2
    for n in ("q", "k", "v", "la", "s0"):
        assert fwd(lib, desc(), o=P(("q", "k", "v", "la", "s0").index(n))) == ALIAS, n
    assert fwd(lib, desc(), so=P(4, 64)) == ALIAS       # overlaps state0, not exactly it
    assert fwd(lib, desc(), so=P(5)) == ALIAS and fwd(lib, desc(), so=P(0)) == ALIAS
    assert fwd(lib, desc(), o=P(0, one - 2)) == ALIAS
    assert fwd(lib, desc(), packed=True, o=P(20)) == ALIAS
    for i in range(7):
        assert bwd(lib, desc(), dv=P(i)) == ALIAS, i
    for i in (7, 8, 10, 11):
        assert bwd(lib, desc(), dv=P(i)) == ALIAS, i
    assert bwd(lib, desc(), ds0=P(12)) == ALIAS
    assert step(lib, desc(seqlen=1), o=P(4)) == ALIAS and step(lib, desc(seqlen=1), st=P(2)) == ALIAS


def test_workspaces(lib):
    d = desc(batch=1, heads=2, seqlen=4096)
    n = ctypes.c_size_t(0)
    assert lib.gdn2_linear_fwd_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(lib, d, ws=P(12), n=n.value - 1) == WORKSPACE
    assert fwd(lib, d, ws=P(12, 16), n=n.value) == WORKSPACE
    assert fwd(lib, d, ws=P(0), n=n.value) == ALIAS
    assert lib.gdn2_linear_bwd_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(lib, d, ws=None, n=0) == WORKSPACE and bwd(lib, d, n=n.value - 1) == WORKSPACE
    assert bwd(lib, d, ws=P(12, 128), n=n.value) == WORKSPACE
    # whole chains fill the GPU: no scratch
    big = desc(batch=16, heads=16, seqlen=4096)
    assert lib.gdn2_linear_fwd_workspace(ctypes.byref(big), ctypes.byref(n)) == 0 and n.value == 0


def nd(**kw):
    base = dict(rows=64, groups=4, dim=128)
    base.update(kw)
    return ln.make_norm_desc(**base)


def nfwd(lib, d, **kw):
    a = dict(x=P(0), w=P(1), b=P(2), y=P(3), m=P(4), r=P(5))
    a.update(kw)
    return lib.gdn2_layer_norm_fwd(None if d is None else ctypes.byref(d), a["x"], a["w"], a["b"], a["y"], a["m"], a["r"], None)


def nbwd(lib, d, **kw):
    a = dict(dy=P(0), x=P(1), w=P(2), m=P(3), r=P(4), dx=P(5), dw=P(6), db=P(7), ws=P(8), n=1 << 31)
    a.update(kw)
    return lib.gdn2_layer_norm_bwd(None if d is None else ctypes.byref(d), a["dy"], a["x"], a["w"], a["m"], a["r"], a["dx"],
                                   a["dw"], a["db"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-4), SHAPE), (dict(groups=0), SHAPE), (dict(dim=0), SHAPE), (dict(rows=63), SHAPE), (dict(dtype=5), DTYPE),
    (dict(weight_dtype=-1), DTYPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(dim=16385), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=1 << 60), SHAPE), (dict(rows=0, groups=1 << 50), UNSUPPORTED)])
def test_bad_norm_descriptors(lib, kw, status):
    d, n = nd(**kw), ctypes.c_size_t(0)
    assert nfwd(lib, d) == status and nbwd(lib, d) == status
    assert lib.gdn2_layer_norm_bwd_workspace(ctypes.byref(d), ctypes.byref(n)) == status


def test_norm_arguments(lib):
    assert nfwd(lib, None) == NULL and nbwd(lib, None) == NULL
    assert nfwd(lib, nd(), x=None) == NULL and nfwd(lib, nd(), y=None) == NULL
    for n in ("dy", "x", "m", "r", "dx"):
        assert nbwd(lib, nd(), **{n: None}) == NULL, n
    for i in range(3):
        assert nfwd(lib, nd(), y=P(i)) == ALIAS
    assert nfwd(lib, nd(), m=P(5)) == ALIAS
    for i in range(5):
        assert nbwd(lib, nd(), dx=P(i)) == ALIAS
    assert nbwd(lib, nd(), dw=P(7)) == ALIAS
    assert nbwd(lib, nd(), ws=None, n=0) == WORKSPACE and nbwd(lib, nd(), ws=P(8, 8)) == WORKSPACE
    assert nbwd(lib, nd(), n=4) == WORKSPACE
    assert nfwd(lib, nd(rows=0), x=None, y=None) == 0


def test_descriptor_layouts(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines, want = [], []
    for cls, name in ((ln.Gdn2LinearDesc, "gdn2_linear_desc"), (ln.Gdn2NormDesc, "gdn2_norm_desc")):
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
def test_binding_refusals():
    q = torch.zeros(2, 8, 3, 16)
    la = torch.zeros(2, 8, 3)
    with pytest.raises(ValueError, match="GPU"):
        g.linear_chunk_fwd(q, q, q, la, workspace=False)
    with pytest.raises(ValueError, match="contiguous"):
        g.linear_chunk_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, la)
    with pytest.raises(ValueError, match="shape"):
        g.linear_chunk_fwd(q, q, q, la[:, :4])
    with pytest.raises(TypeError):
        g.linear_chunk_fwd(q, q, q.bfloat16(), la)
    with pytest.raises(TypeError):
        g.linear_chunk_fwd(q.half(), q.half(), q.half(), la)
    with pytest.raises(TypeError):
        g.linear_chunk_fwd(q, q, q, la.bfloat16())
    with pytest.raises(ValueError, match="state0"):
        g.linear_chunk_fwd(q, q, q, la, torch.zeros(2, 3, 16, 8))
    with pytest.raises(ValueError, match="d_o"):
        g.linear_chunk_bwd(q, q, q, la, None, q[:, :4])
    with pytest.raises(ValueError, match="packed"):
        g.linear_chunk_fwd_varlen(q, q, q, la, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        g.linear_chunk_fwd_varlen(q[0], q[0], q[0], la[0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="state"):
        g.linear_recurrent_step(q[:, 0].contiguous(), q[:, 0].contiguous(), q[:, 0].contiguous(), la[:, 0].contiguous(),
                                torch.zeros(2, 3, 16, 8))
    x = torch.zeros(4, 5, 16)
    with pytest.raises(ValueError, match="weight"):
        g.layer_norm_fwd(x, torch.ones(8))
    with pytest.raises(ValueError, match="weight"):
        g.layer_norm_fwd(x, torch.ones(4, 16))
    with pytest.raises(TypeError):
        g.layer_norm_fwd(x, torch.ones(16), torch.ones(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="mean"):
        g.layer_norm_bwd(x, x, None, torch.zeros(4), torch.zeros(4, 5))
    with pytest.raises(ValueError, match="GPU"):
        g.layer_norm_fwd(x)
