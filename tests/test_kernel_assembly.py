"""What the compiler makes of the kernels' branches (CPU: compiles, runs nothing).

Where registers are short, the compiler moves live values to accumulation
registers or to scratch memory.  Such a move is wrong where a branch of single
lanes has the other lanes off: they lose theirs.  It has put moves between the
end of a branch and the instruction that turns the lanes back on.
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from gated_delta_rule_decay_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="needs hipcc")


def functions(assembly):
    """(name, lines) of each function."""
    name, lines = None, []
    for line in assembly.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            if name:
                yield name, lines
            name, lines = m.group(1), []
        elif name:
            lines.append(line)
    if name:
        yield name, lines


def mask_writes(lines):
    """Instructions that write the lanes' mask."""
    return [x for x in (line.split(";")[0].strip() for line in lines) if re.match(r"(s_\w*(save|wr)exec|s_\w+ exec\b|v_cmpx)", x)]


def moves_of_some_lanes(lines):
    """Moves of registers away between the start of a block and the instruction that turns lanes back on in it."""
    found, block = [], None
    for line in lines:
        x = line.split(";")[0].strip()
        if re.match(r"^\.LBB", line) or line.startswith("; %bb"):
            block = []
        elif block is None or not x:
            continue
        elif re.match(r"s_or_(b64 exec|saveexec)", x):
            found += [y for y in block if re.match(r"(v_accvgpr_write|scratch_store|buffer_store\w+ .* s32)", y)]
            block = None
        elif x.startswith(("s_cbranch", "s_branch")) or mask_writes([x]):
            block = None
        else:
            block.append(x)
    return found


def spills(assembly):
    """Registers of each kernel that do not fit: (in scratch memory, moved to accumulation registers)."""
    kernel = r"\.agpr_count: +(\d+).*?\.name: +(\w+).*?\.vgpr_spill_count: +(\d+)"
    return {m[1]: (int(m[2]), int(m[0])) for m in re.findall(kernel, assembly, re.S)}


@pytest.fixture(scope="module")
def assembly():
    def one(src):
        cmd = [build.HIPCC, *build.FLAGS, "-S", "--cuda-device-only", src, "-o", "-"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        return os.path.basename(src), (dict(functions(r.stdout)), spills(r.stdout))

    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        return dict(ex.map(one, build.sources()))


def test_the_reading_of_assembly():
    body = ["\tv_accvgpr_write_b32 a0, v1 ; 4-byte spill", "\ts_or_b64 exec, exec, s[0:1]", "\tv_accvgpr_write_b32 a1, v2"]
    assert moves_of_some_lanes([".LBB0_1: ; %x", *body]) == ["v_accvgpr_write_b32 a0, v1"]
    assert moves_of_some_lanes(["; %bb.3:", "\tscratch_store_dword off, v1, off", "\ts_or_saveexec_b64 s[4:5], s[4:5]"])
    assert not moves_of_some_lanes([".LBB0_1:", *body[1:]]) and not moves_of_some_lanes(body[2:])
    assert mask_writes(["\ts_and_saveexec_b64 s[0:1], vcc", "\ts_and_b64 vcc, exec, s[0:1]", "\ts_xor_b64 exec, exec, s[2:3]"]) == [
        "s_and_saveexec_b64 s[0:1], vcc", "s_xor_b64 exec, exec, s[2:3]"]
    assert [n for n, _ in functions("_Za:\n x\n_Zb:\n y\n")] == ["_Za", "_Zb"]


def test_no_register_is_moved_away_for_some_lanes(assembly):
    bad = {f"{src}: {name}": m[0] for src, (fs, _) in assembly.items() for name, lines in fs.items() if (m := moves_of_some_lanes(lines))}
    assert not bad, bad


@pytest.mark.parametrize("source", ["scan_fwd.hip", "scan_bwd.hip"])
def test_no_lane_of_the_scan_branches_by_itself(assembly, source):
    kernels = {n: lines for n, lines in assembly[source][0].items() if "_kernel" in n}
    assert len(kernels) == 40  # 4 combinations of types, packed or not, 1 channel a lane or 8 in four forms
    bad = {n: m[0] for n, lines in kernels.items() if (m := mask_writes(lines))}
    assert not bad, bad


@pytest.mark.parametrize("source", ["scan_fwd.hip", "scan_bwd.hip", "scan.hip", "rotary.hip"])
def test_registers_suffice(assembly, source):
    kernels, counts = {n for n in assembly[source][0] if "_kernel" in n}, assembly[source][1]
    assert kernels == set(counts)
    assert not {n: c for n, c in counts.items() if c != (0, 0)}
